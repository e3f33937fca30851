"""The operators at a model's two ends on the CPU: the oracle against hand numbers and differences, and
every refusal of the C ABI and of the binding that needs no GPU."""
import ctypes
import math
import types

import numpy as np
import pytest

import oracle
from rollout_logprob_consistency_gb300 import binding

OFF = (1.0, 0, 1.0, 0.0)


# ----------------------------------------------------------------------------- the oracle

def test_verify_oracle_by_hand():
    p, q = np.log([0.5, 0.3, 0.2]), np.log([0.2, 0.7, 0.1])
    row = np.stack([p, p])
    # token 1: u 0.7 < 0.3 accepts up to u = 3/7
    for u, ok in ((0.42, True), (0.44, False)):
        r = oracle.ends.verify_sequence(row, q[None], [1], [u], 0.1, OFF)
        assert r["accepted"] == int(ok)
    # refused: max(p - q, 0) = (0.3, 0, 0.1), three quarters of it token 0's
    for draw, y in ((0.0, 0), (0.74, 0), (0.76, 2)):
        r = oracle.ends.verify_sequence(row, q[None], [1], [0.9], draw, OFF)
        assert r["ids"] == [y, -1] and r["logprob"][0] == pytest.approx(p[y])
    # a certain drafter leaves p without its token: (0.5, 0.2) of 0.7
    for draw, y in ((0.71, 0), (0.72, 2)):
        assert oracle.ends.verify_sequence(row, None, [1], [0.31], draw, OFF)["ids"] == [y, -1]
    # accepted: the next from p itself; no draft at all: the first
    assert oracle.ends.verify_sequence(row, q[None], [0], [0.9], 0.81, OFF)["ids"] == [0, 2]
    assert oracle.ends.verify_sequence(row, q[None], [-1], [0.9], 0.6, OFF)["ids"] == [1, -1]
    # temperature 0: the largest is accepted, everything else refused in its favour
    assert oracle.ends.verify_sequence(row, q[None], [0], [0.99], 0.5, (0.0, 0, 1.0, 0.0))["ids"] == [0, 0]
    assert oracle.ends.verify_sequence(row, q[None], [1], [0.01], 0.5, (0.0, 0, 1.0, 0.0))["ids"] == [0, -1]


def test_verify_oracle_yields_the_target():
    """Over all drafts, weighed by q, and a grid of uniform numbers, the first token is distributed as p."""
    rng = np.random.default_rng(1)
    zp, zq = rng.normal(size=5), rng.normal(size=5)
    for settings in (OFF, (0.7, 3, 1.0, 0.0)):
        p, q = oracle.ends.processed(zp, *settings)[0], oracle.ends.processed(zq, *settings)[0]
        grid = (np.arange(200) + 0.5) / 200
        f = np.zeros(5)
        for x in np.nonzero(q)[0]:
            for u in grid:
                ys = [oracle.ends.verify_sequence(np.stack([zp, zp]), zq[None], [x], [u], d, settings)["ids"][0]
                      for d in (grid[::10] if u * q[x] >= p[x] else [0.5])]
                f += q[x] / len(grid) * np.bincount(ys, minlength=5) / len(ys)
        # each border of u is met within half a step of its grid, each of the draw within one of 20
        assert np.all(np.abs(f - p) < 0.5 / 200 * 5 + 1.0 / 20 * np.maximum(q - p, 0).sum())


def test_verify_oracle_uses_the_samplers_distribution():
    rng = np.random.default_rng(2)
    for _ in range(30):
        z, u = rng.normal(size=40) * 2, float(rng.random())
        s = (0.8, 12, 0.9, 0.05)
        a = oracle.sample_row(z, u, *s)
        r = oracle.ends.verify_sequence(z[None], None, [], [], u, s)
        assert r["ids"] == [a["id"]] and r["logprob"][0] == pytest.approx(a["logprob"], abs=1e-12)


def test_embed_oracle_by_hand():
    table = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    assert np.array_equal(oracle.ends.embed(table, [2, -1, 0, 2], 2.0), [[10, 12], [0, 0], [2, 4], [10, 12]])
    grad, size, n = oracle.ends.embed_backward([[1.0], [2.0], [-4.0], [8.0]], [1, -1, 1, 0], 3, 0.5)
    assert np.array_equal(grad, [[4.0], [-1.5], [0.0]]) and np.array_equal(size, [[4.0], [2.5], [0.0]])
    assert n.tolist() == [1, 2, 0]


def test_residual_norm_oracle_by_hand():
    h, step = oracle.ends.residual_norm([[1.0, 1.0]], [[3.0, 4.0]], None, np.array([1.0, 2.0]),
                                        np.array([[0.5]]), 2.0, 0.0)
    rms = math.sqrt(12.5)
    np.testing.assert_allclose(step, [[3 / rms, 8 / rms]])
    np.testing.assert_allclose(h, 1 + step)
    np.testing.assert_allclose(oracle.ends.norm_rows([[3.0, 4.0]], np.array([1.0, 2.0]), 0.0), [[3 / rms, 8 / rms]])


@pytest.mark.parametrize("gate", [None, "channel", "token", "element"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("pre", [False, True])
def test_residual_norm_oracle_gradient_by_differences(gate, post, pre):
    rng = np.random.default_rng(3)
    T, d, s, eps = 3, 4, 0.7, 1e-3
    shape = {None: None, "channel": (d,), "token": (T, 1), "element": (T, d)}[gate]
    a = dict(h=rng.normal(size=(T, d)), x=rng.normal(size=(T, d)), gamma=rng.normal(size=d) if pre else None,
             gamma_post=rng.normal(size=d) if post else None, gate=None if shape is None else rng.normal(size=shape))
    dh, dy = rng.normal(size=(T, d)), rng.normal(size=(T, d))

    def loss(**kw):
        b = {**a, **kw}
        h, _ = oracle.ends.residual_norm(b["h"], b["x"], None, b["gamma_post"], b["gate"], s, eps)
        return np.sum(h * dh) + (np.sum(oracle.ends.norm_rows(h, b["gamma"], eps) * dy) if pre else 0.0)

    h, _ = oracle.ends.residual_norm(a["h"], a["x"], None, a["gamma_post"], a["gate"], s, eps)
    got = oracle.ends.residual_norm_backward(h, a["x"], dh, dy if pre else None, a["gamma"], a["gamma_post"],
                                             a["gate"], s, eps)
    names = dict(h="dresidual", x="dblock", gamma="dgamma", gamma_post="dgamma_post", gate="dgate")
    assert set(got) == {names[k] for k in a if a[k] is not None}
    for k, name in names.items():
        if a[k] is None:
            continue
        for at in np.ndindex(a[k].shape):
            e = np.zeros_like(a[k])
            e[at] = 1e-5
            diff = (loss(**{k: a[k] + e}) - loss(**{k: a[k] - e})) / 2e-5
            assert diff == pytest.approx(got[name][0][at], abs=1e-7), (k, at)


# ----------------------------------------------------------------------------- refusals

@pytest.fixture(scope="module")
def tim():
    import __graft_entry__
    __graft_entry__.build()
    import rollout_logprob_consistency_gb300 as tim
    return tim


P = 1 << 30  # stands for a device address: nothing here gets as far as using it
FAR = [P * n for n in range(1, 20)]
SHAPE, ARG, WORKSPACE = 2, 1, 7


def _verify(tim, **kw):
    a = dict(target=FAR[0], ts=256, tp=64, draft=FAR[1], ds=192, dp=64, dtype=1, B=4, N=3, V=64, ids=FAR[2],
             u=FAR[3], ud=FAR[4], s=OFF, rows=(None,) * 4, q=None, no_params=False, out=FAR[5], lp=FAR[6], n=FAR[7],
             ws=FAR[8], nbytes=1 << 20)
    a.update(kw)
    p = binding._SampleParams(*a["s"], *a["rows"])
    q = None if a["q"] is None else ctypes.byref(binding._SampleParams(*a["q"], None, None, None, None))
    return tim.lib().tim_verify(a["target"], a["ts"], a["tp"], a["draft"], a["ds"], a["dp"], a["dtype"], a["B"],
                                a["N"], a["V"], a["ids"], a["u"], a["ud"],
                                None if a["no_params"] else ctypes.byref(p), q, a["out"], a["lp"], a["n"],
                                a["ws"], a["nbytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(target=None), ARG), (dict(target=P + 1), ARG), (dict(draft=P + 1), ARG), (dict(dtype=3), ARG),
    (dict(dtype=0, target=P + 2), ARG), (dict(ts=-1), SHAPE), (dict(tp=(1 << 40) + 1), SHAPE), (dict(ds=-64), SHAPE),
    (dict(dp=1 << 41), SHAPE), (dict(B=0), SHAPE), (dict(N=0), SHAPE), (dict(N=1025), SHAPE), (dict(N=-1), SHAPE),
    (dict(B=1 << 28), SHAPE), (dict(V=0), SHAPE), (dict(V=393217), SHAPE), (dict(ids=None), ARG),
    (dict(ids=P + 2), ARG), (dict(u=None), ARG), (dict(u=P + 2), ARG), (dict(ud=None), ARG), (dict(ud=P + 1), ARG),
    (dict(no_params=True), ARG), (dict(s=(-1.0, 0, 1.0, 0.0)), ARG), (dict(s=(math.nan, 0, 1.0, 0.0)), ARG),
    (dict(s=(1.0, 0, 0.0, 0.0)), ARG), (dict(s=(1.0, 0, 1.0, 1.5)), ARG), (dict(q=(1e7, 0, 1.0, 0.0)), ARG),
    (dict(q=(1.0, 0, 1.0, -1.0)), ARG), (dict(rows=(P + 1, None, None, None)), ARG), (dict(out=None), ARG),
    (dict(lp=None), ARG), (dict(n=None), ARG), (dict(n=P + 2), ARG), (dict(out=FAR[2] + 44), ARG),
    (dict(lp=FAR[2] - 60), ARG), (dict(n=FAR[2]), ARG), (dict(out=FAR[3] - 4), ARG), (dict(lp=FAR[3] + 44), ARG),
    (dict(n=FAR[4] + 12), ARG), (dict(out=FAR[4]), ARG), (dict(lp=FAR[5] + 60), ARG), (dict(n=FAR[6] - 12), ARG), (dict(ws=None), WORKSPACE), (dict(ws=P + 8), WORKSPACE),
    (dict(nbytes=1024 + 4 * 7 * 32), WORKSPACE)])
def test_verify_refusals(tim, kw, code):
    assert _verify(tim, **kw) == code


def _embed(tim, **kw):
    a = dict(table=FAR[0], dtype=1, ld=64, ids=FAR[1], T=8, V=100, d=64, scale=1.0, out=FAR[2], ldo=64, ws=FAR[3],
             nbytes=1024)
    a.update(kw)
    return tim.lib().tim_embed(a["table"], a["dtype"], a["ld"], a["ids"], a["T"], a["V"], a["d"], a["scale"],
                               a["out"], a["ldo"], a["ws"], a["nbytes"], None)


EMBED_BAD = [(dict(dtype=5), ARG), (dict(ids=None), ARG), (dict(ids=P + 2), ARG), (dict(T=0), SHAPE),
             (dict(T=1 << 31), SHAPE), (dict(V=0), SHAPE), (dict(V=2 ** 31 - 255), SHAPE), (dict(d=0), SHAPE),
             (dict(d=65537), SHAPE), (dict(scale=math.nan), ARG), (dict(scale=math.inf), ARG),
             (dict(ws=None), WORKSPACE), (dict(ws=P + 128), WORKSPACE), (dict(nbytes=1023), WORKSPACE)]


@pytest.mark.parametrize("kw,code", EMBED_BAD + [
    (dict(table=None), ARG), (dict(table=P + 1), ARG), (dict(ld=63), SHAPE), (dict(ld=(1 << 31) + 1), SHAPE),
    (dict(out=None), ARG), (dict(ldo=63), SHAPE), (dict(out=FAR[0] + 2 * 100 * 64 - 2), ARG),
    (dict(out=FAR[0] - 2 * 8 * 64 + 2), ARG), (dict(out=FAR[1]), ARG)])
def test_embed_refusals(tim, kw, code):
    assert _embed(tim, **kw) == code


def _embed_backward(tim, **kw):
    a = dict(dy=FAR[0], dtype=1, ldy=64, ids=FAR[1], T=8, V=100, d=64, scale=1.0, out=FAR[2], out_dtype=0, acc=0,
             ws=FAR[3], nbytes=1 << 20)
    a.update(kw)
    return tim.lib().tim_embed_backward(a["dy"], a["dtype"], a["ldy"], a["ids"], a["T"], a["V"], a["d"], a["scale"],
                                        a["out"], a["out_dtype"], a["acc"], a["ws"], a["nbytes"], None)


@pytest.mark.parametrize("kw,code", EMBED_BAD + [
    (dict(dy=None), ARG), (dict(dy=P + 1), ARG), (dict(ldy=63), SHAPE), (dict(out=None), ARG),
    (dict(out=P + 2), ARG), (dict(out_dtype=2), ARG), (dict(out_dtype=3), ARG), (dict(acc=2), ARG),
    (dict(out=FAR[0] + 1024 - 4), ARG), (dict(out=FAR[1] - 100), ARG)])
def test_embed_backward_refusals(tim, kw, code):
    assert _embed_backward(tim, **kw) == code


def _block(**kw):
    a = dict(T=8, d=64, dtype=1, block=FAR[0], ld=64, gamma_post=FAR[1], gate=FAR[2], ld_gate=64, kind=3, scale=1.0,
             gamma=FAR[3], eps=1e-6)
    a.update({k: v for k, v in kw.items() if k in a})
    return binding._Block(a["T"], a["d"], a["dtype"], a["block"], a["ld"], a["gamma_post"], a["gate"], a["ld_gate"],
                          a["kind"], a["scale"], a["gamma"], a["eps"], 0)


def _norm(tim, **kw):
    a = dict(no_block=False, h=FAR[4], ldr=64, out_h=FAR[5], ldh=64, out_y=FAR[6], ldy=64)
    a.update({k: v for k, v in kw.items() if k in a})
    return tim.lib().tim_residual_norm(None if a["no_block"] else ctypes.byref(_block(**kw)), a["h"], a["ldr"],
                                       a["out_h"], a["ldh"], a["out_y"], a["ldy"], None)


BLOCK_BAD = [
    (dict(no_block=True), ARG), (dict(T=0), SHAPE), (dict(T=1 << 31), SHAPE), (dict(d=0), SHAPE), (dict(d=16385), SHAPE),
    (dict(dtype=3), ARG), (dict(block=None), ARG), (dict(block=P + 1), ARG), (dict(ld=63), SHAPE),
    (dict(gamma=P + 1), ARG), (dict(gamma_post=P + 1), ARG), (dict(gate=P + 1), ARG), (dict(gate=None), ARG),
    (dict(kind=0), ARG), (dict(kind=4), ARG), (dict(kind=-1), ARG), (dict(ld_gate=63), SHAPE),
    (dict(kind=1, ld_gate=0), SHAPE), (dict(scale=math.inf), ARG), (dict(eps=-1.0), ARG), (dict(eps=math.nan), ARG)]


@pytest.mark.parametrize("kw,code", BLOCK_BAD + [
    (dict(h=None), ARG), (dict(ldr=63), SHAPE), (dict(out_h=None), ARG), (dict(ldh=1), SHAPE), (dict(out_y=None), ARG),
    (dict(ldy=(1 << 31) + 1), SHAPE), (dict(out_h=FAR[0]), ARG), (dict(out_y=FAR[4]), ARG), (dict(out_h=FAR[4] + 128), ARG),
    (dict(out_h=FAR[4], ldh=65), ARG), (dict(out_y=FAR[0] + 2), ARG), (dict(out_y=FAR[5] + 1022), ARG),
    (dict(out_h=FAR[1] - 2), ARG), (dict(out_h=FAR[2]), ARG), (dict(out_y=FAR[3]), ARG)])
def test_residual_norm_refusals(tim, kw, code):
    assert _norm(tim, **kw) == code


def _norm_backward(tim, **kw):
    a = dict(no_block=False, h=FAR[4], ldh=64, dh=FAR[5], lddh=64, dy=FAR[6], lddy=64, dr=FAR[7], lddr=64, db=FAR[8],
             lddb=64, dgamma=FAR[9], dpost=FAR[10], dgate=FAR[11], lddg=64, acc=0, ws=FAR[12], nbytes=1 << 20)
    a.update({k: v for k, v in kw.items() if k in a})
    return tim.lib().tim_residual_norm_backward(
        None if a["no_block"] else ctypes.byref(_block(**kw)), a["h"], a["ldh"], a["dh"], a["lddh"], a["dy"], a["lddy"],
        a["dr"], a["lddr"], a["db"], a["lddb"], a["dgamma"], a["dpost"], a["dgate"], a["lddg"], a["acc"], a["ws"],
        a["nbytes"], None)


@pytest.mark.parametrize("kw,code", BLOCK_BAD + [
    (dict(gamma=None), ARG), (dict(acc=-1), ARG), (dict(h=None), ARG), (dict(ldh=63), SHAPE), (dict(lddh=63), SHAPE),
    (dict(dh=P + 1), ARG), (dict(dy=P + 1), ARG), (dict(lddy=0), SHAPE), (dict(dr=None), ARG), (dict(lddr=63), SHAPE),
    (dict(db=None), ARG), (dict(lddb=63), SHAPE), (dict(dgamma=None), ARG), (dict(dgamma=P + 2), ARG),
    (dict(dpost=None), ARG), (dict(dgate=None), ARG), (dict(lddg=63), SHAPE), (dict(kind=2, dgate=None), ARG),
    (dict(kind=1, ld_gate=1, dgate=P + 2), ARG), (dict(dr=FAR[4]), ARG), (dict(db=FAR[0]), ARG), (dict(dr=FAR[8]), ARG),
    (dict(dgamma=FAR[10] + 252), ARG), (dict(dgate=FAR[7] + 1022), ARG), (dict(ws=None), WORKSPACE),
    (dict(nbytes=1024 + 8 * 3 * 64 * 4 - 4), WORKSPACE)])
def test_residual_norm_backward_refusals(tim, kw, code):
    assert _norm_backward(tim, **kw) == code


def test_workspace_sizes(tim):
    """None for what is refused; never less for a smaller call, so that a workspace serves those too."""
    assert tim.verify_workspace_size(0, 3) == 0 and tim.verify_workspace_size(4, 0) == 0
    assert tim.verify_workspace_size(4, 3) >= 1024 + 4 * 7 * 32 + 4 * 3 * 8 + 4 * 4 * 4
    assert tim.embed_backward_workspace_size(0, 10, 8) == 0 and tim.embed_backward_workspace_size(5, 10, 0) == 0
    sizes = [tim.embed_backward_workspace_size(T, 1000, 64) for T in
             (1, 2, 100, 8191, 8192, 8193, 32768, 32769, 131072, 131073, 1 << 20)]
    assert sizes == sorted(sizes)
    assert tim.residual_norm_backward_workspace_size(5, 16385) == 0
    sizes = [tim.residual_norm_backward_workspace_size(T, 64) for T in (1, 2, 151, 152, 1000, 1024, 5000)]
    assert sizes == sorted(sizes)


def test_binding_refuses_wrong_tensors(tim):
    torch = pytest.importorskip("torch")
    z, ids = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int32)
    for call in (lambda: tim.embed(z, ids), lambda: tim.embed_backward(z, ids, 10), lambda: tim.embedding(z, ids),
                 lambda: tim.residual_norm(z, z, None, 1e-6), lambda: tim.block_residual(z, z, None, 1e-6),
                 lambda: tim.residual_norm_backward(z, z, z, None, None, 1e-6),
                 lambda: tim.verify(z.view(1, 4, 8), ids[:3].view(1, 3), z[:1, :3], z[0, :1])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        tim.embed(z.double(), ids)


@pytest.mark.parametrize("op", ["verify", "embed", "embed_backward", "residual_norm_backward"])
def test_a_workspace_of_another_device_is_refused(monkeypatch, op):
    """A kernel writes its status there."""
    torch = pytest.importorskip("torch")

    class Lib:
        @staticmethod
        def tim_status_string(*a):
            pytest.fail("launched")

    z, ids, ws = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int32), types.SimpleNamespace(
        ptr=0, nbytes=1 << 20, buf=torch.zeros(1, device="meta"))
    monkeypatch.setattr(binding, "lib", lambda: Lib)
    monkeypatch.setattr(binding, "_type_code", lambda t, name: 0)
    monkeypatch.setattr(binding, "_logits_args", lambda t, name: (*t.shape, 0, t.shape[1]))
    monkeypatch.setattr(binding, "_need", lambda *a, **kw: None)
    monkeypatch.setattr(binding, "_run", lambda dev, stream, call: call(None))
    monkeypatch.setattr(binding, "_DTYPE_CODES", {torch.float32: 0})
    with pytest.raises(ValueError, match="workspace must be on cpu"):
        if op == "verify":
            tim_ids = ids[:3].view(1, 3)
            binding.verify(z.view(1, 4, 8), tim_ids, z[:1, :3], z[0, :1], workspace=ws, check=False)
        elif op == "embed":
            binding.embed(z, ids, workspace=ws, check=False)
        elif op == "embed_backward":
            binding.embed_backward(z, ids, 10, workspace=ws, check=False)
        else:
            binding.residual_norm_backward(z, z, z, None, None, 1e-6, workspace=ws)


def test_one_row_keeps_its_strides(monkeypatch):
    """Whether rows are whole vectors is decided from the strides, and decides the order of a row's sums."""
    torch = pytest.importorskip("torch")
    got = []

    class Lib:
        @staticmethod
        def tim_residual_norm(b, r, ldr, h, ldh, y, ldy, sp):
            got.append((b._obj.ld_block, b._obj.ld_gate, ldr, ldh, ldy))
            return 0

    monkeypatch.setattr(binding, "lib", lambda: Lib)
    monkeypatch.setattr(binding, "_type_code", lambda t, name: 0)
    monkeypatch.setattr(binding, "_vector", lambda t, *a: t.data_ptr())
    monkeypatch.setattr(binding, "_run", lambda dev, stream, call: call(None))
    x, gamma = torch.zeros(4, 11)[:, :8], torch.zeros(8)
    for n in (4, 1):
        out = (torch.zeros(n, 12)[:, :8], torch.zeros(n, 13)[:, :8])
        binding.residual_norm(x[:n], x[:n], gamma, 1e-6, gate=x[:n], out=out)
    binding.residual_norm(*(x.as_strided((1, 8), (s, 1)) for s in (5, 2 ** 31 + 1)), gamma, 1e-6)
    assert got == [(11, 11, 11, 12, 13)] * 2 + [(8, 0, 8, 8, 8)]


FREE = P * 40  # meets nothing of _verify's


@pytest.mark.parametrize("out,size", [("out", 64), ("lp", 64), ("n", 16)])
@pytest.mark.parametrize("what", ["target", "draft", "temperature", "top_k", "top_p", "min_p", "draft's", "workspace"])
def test_verify_refuses_results_over_what_it_still_reads(tim, out, size, what):
    """Other sequences' CTAs read it while one writes.  B = 4, N = 3: 16 ids and logprobs, 4 counts."""
    def call(at):
        if what == "target":
            return _verify(tim, target=FREE, **{out: at})
        if what == "draft":
            return _verify(tim, draft=FREE, **{out: at})
        if what == "workspace":
            return _verify(tim, ws=FREE, **{out: at})
        i = 0 if what == "draft's" else ("temperature", "top_k", "top_p", "min_p").index(what)
        rows = tuple(FREE if j == i else None for j in range(4))
        if what != "draft's":
            return _verify(tim, rows=rows, **{out: at})
        a = dict(out=FAR[5], lp=FAR[6], n=FAR[7])
        a[out] = at
        p, q = binding._SampleParams(*OFF, *(None,) * 4), binding._SampleParams(*OFF, *rows)
        return tim.lib().tim_verify(FAR[0], 256, 64, FAR[1], 192, 64, 1, 4, 3, 64, FAR[2], FAR[3], FAR[4],
                                    ctypes.byref(p), ctypes.byref(q), a["out"], a["lp"], a["n"], FAR[8], 1 << 20, None)

    # bytes: 3 sequence strides of 512 (384 of the draft's) and 3 (2) positions of 128, and the last row's;
    # 4 settings; the workspace's status and its rows
    end = {"target": 3 * 512 + 3 * 128 + 128, "draft": 3 * 384 + 2 * 128 + 128,
           "workspace": tim.verify_workspace_size(4, 3)}.get(what, 16)
    for at in (FREE, FREE + end - 4, FREE - size + 4):
        assert call(at) == ARG, at - FREE


def test_verify_rows_far_apart_do_not_wrap(tim):
    """Strides whose extent is beyond 64 bits: whatever lies above the matrix's address is its."""
    far = 1 << 40
    assert _verify(tim, B=1 << 25, ts=far, tp=far, ds=far, dp=far) == ARG


def test_results_over_the_workspace_are_refused(tim):
    """It holds the status, the sorted tokens and the sums that the launches hand on."""
    assert all(_embed(tim, ws=FREE, out=at) == ARG for at in (FREE, FREE + 1020, FREE - 8 * 64 * 2 + 2))
    end = tim.embed_backward_workspace_size(8, 100, 64)
    assert all(_embed_backward(tim, ws=FREE, out=at) == ARG for at in (FREE, FREE + end - 4, FREE - 100 * 64 * 4 + 4))
    end = tim.residual_norm_backward_workspace_size(8, 64)
    for out, size in (("dr", 1024), ("db", 1024), ("dgate", 1024), ("dgamma", 256), ("dpost", 256)):
        for at in (FREE, FREE + end - 4, FREE - size + 4):
            assert _norm_backward(tim, ws=FREE, **{out: at}) == ARG, (out, at - FREE)


def test_sizes_beyond_32_bits_stay_too_large(tim, monkeypatch):
    """The low 32 bits of 2^32 + 5 are a size that would be served, and the rest of the table left as it was."""
    torch = pytest.importorskip("torch")
    big, most = 2 ** 32 + 5, 2 ** 31 - 1
    assert tim.verify_workspace_size(4, big) == 0 and tim.verify_workspace_size(4, big - 2 ** 33) == 0
    assert tim.embed_backward_workspace_size(8, big, 8) == 0 and tim.embed_backward_workspace_size(8, 100, big) == 0
    assert tim.residual_norm_backward_workspace_size(8, big) == 0
    got = {}

    class Lib:
        def __getattr__(self, name):
            return lambda *a: got.__setitem__(name, a) or 0

    def like(*shape):
        return torch.empty(1).expand(*shape)

    ws = types.SimpleNamespace(ptr=0, nbytes=1 << 20, buf=torch.zeros(1))
    monkeypatch.setattr(binding, "lib", Lib)
    monkeypatch.setattr(binding, "_type_code", lambda t, name: 0)
    monkeypatch.setattr(binding, "_logits_args", lambda t, name: (*t.shape, 0, t.shape[1]))
    monkeypatch.setattr(binding, "_need", lambda *a, **kw: None)
    monkeypatch.setattr(binding, "_run", lambda dev, stream, call: call(None))
    monkeypatch.setattr(binding, "_DTYPE_CODES", {torch.float32: 0})
    kw = dict(workspace=ws, check=False)
    ids = torch.zeros(4, dtype=torch.int32)
    binding.embed_backward(like(4, 8), ids, big, out_dtable=like(big, 8), **kw)
    assert got["tim_embed_backward"][5:7] == (most, 8)
    binding.embed_backward(like(4, big), ids, 8, out_dtable=like(8, big), **kw)
    assert got["tim_embed_backward"][5:7] == (8, most)
    binding.embed(like(big, 8), ids, out=like(4, 8), **kw)
    assert got["tim_embed"][5:7] == (most, 8)
    binding.embed(like(8, big), ids, out=like(4, big), **kw)
    assert got["tim_embed"][5:7] == (8, most)
    monkeypatch.setattr(binding, "_sequence_rows", lambda t, *a: (0, 0, 0))
    binding.verify(like(1, 4, big), ids[:3].view(1, 3), torch.zeros(1, 3), torch.zeros(1), **kw)
    assert got["tim_verify"][7:10] == (1, 3, most)
    binding.residual_norm(like(1, big), like(1, big), None, 1e-6, out=(like(1, big), None))
    assert got["tim_residual_norm"][0]._obj.d == most


def test_a_workspace_that_is_too_small_is_told_so(tim):
    """Also where the bytes that it lacks are an output's."""
    at = FREE + 1024
    assert _verify(tim, ws=FREE, nbytes=1024, out=at) == WORKSPACE
    assert _embed(tim, ws=FREE, nbytes=768, out=FREE + 768) == WORKSPACE
    assert _embed_backward(tim, ws=FREE, nbytes=1024, out=at) == WORKSPACE
    assert _norm_backward(tim, ws=FREE, nbytes=1024, dr=at) == WORKSPACE
