"""tim.residual_norm and its backward on the GPU against the fp64 oracle.

A sum over a row is at most 32 additions in a thread and 10 among threads, so r = 1 / sqrt(mean + eps)
is off by less than 26 x 2^-24 (half of 43, and 4 of its own), scale g n with three products more by 30:
  h:  (32 |step| + |h|) 2^-24 before its rounding u |h| to the type;
  y:  from the h that was returned, 30 x 2^-24 |y|, and u |y|.
The bounds of the gradients stand beside the oracle's formulas (oracle/ends.py), and u of the value where
the result is rounded to a 16-bit type.
"""
import math

import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


@pytest.fixture(scope="module")
def tim():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import rollout_logprob_consistency_gb300 as tim
    return tim


def _dtype(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def _matrix(T, d, dtype, seed, pad=0, offset=0, size=1.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.full((T, offset + d + pad), 77.0, dtype=_dtype(dtype), device="cuda")
    x = buf[:, offset:offset + d]
    x.copy_(size * torch.randn(T, d, generator=g, device="cuda"))
    return x


def _problem(T, d, dtype, gate, post, pre, seed=0, pad=0, offset=0):
    shape = {"none": None, "channel": (1, d), "token": (T, 1), "element": (T, d)}[gate]
    p = dict(h=_matrix(T, d, dtype, seed + 1, pad, offset, 2.0), x=_matrix(T, d, dtype, seed + 2, pad, offset, 0.7),
             gamma=_matrix(1, d, dtype, seed + 3).view(d) if pre else None,
             gamma_post=_matrix(1, d, dtype, seed + 4).view(d) if post else None,
             dh=_matrix(T, d, dtype, seed + 6, pad, offset), dy=_matrix(T, d, dtype, seed + 7, pad, offset),
             gate=None)
    if shape is not None:
        p["gate"] = _matrix(*shape, dtype, seed + 5, pad if gate == "element" else 0)
        if gate == "channel":
            p["gate"] = p["gate"].reshape(d)
    return p


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _half(t):
    """Half a step: relative, and below the normal numbers."""
    import torch
    f = torch.finfo(t.dtype)
    return (f.eps / 2 * (1 + 2.0 ** -6), f.smallest_normal * f.eps / 2) if t.dtype != torch.float32 else (E, 2.0 ** -149)


def _within(got, want, tol, what):
    u, floor = _half(got)
    err = np.abs(_np(got) - want)
    bad = ~(err <= tol + u * np.abs(want) + floor)
    assert not bad.any(), (what, float(err[bad].max()), int(bad.sum()))


def _forward(tim, p, scale, eps, **kw):
    h, y = tim.residual_norm(p["h"], p["x"], p["gamma"], eps, gamma_post=p["gamma_post"], gate=p["gate"],
                             scale=scale, **kw)
    want, step = oracle.ends.residual_norm(_np(p["h"]), _np(p["x"]), _np(p["gamma"]), _np(p["gamma_post"]),
                                           _np(p["gate"]), float(np.float32(scale)), float(np.float32(eps)))
    _within(h, want, (32 * np.abs(step) + np.abs(want)) * E, "h")
    if p["gamma"] is None:
        assert y is None
    else:
        want = oracle.ends.norm_rows(_np(h), _np(p["gamma"]), float(np.float32(eps)))
        _within(y, want, 30 * E * np.abs(want), "y")
    return h, y


NAMES = ("dresidual", "dblock", "dgamma", "dgamma_post", "dgate")


def _backward(tim, p, h, scale, eps, dh=True, dy=True, before=None, **kw):
    dh = p["dh"] if dh else None
    dy = p["dy"] if dy and p["gamma"] is not None else None
    got = tim.residual_norm_backward(h, p["x"], dh, dy, p["gamma"], eps, gamma_post=p["gamma_post"],
                                     gate=p["gate"], scale=scale, **kw)
    want = oracle.ends.residual_norm_backward(
        _np(h), _np(p["x"]), _np(dh), _np(dy), _np(p["gamma"]), _np(p["gamma_post"]), _np(p["gate"]),
        float(np.float32(scale)), float(np.float32(eps)))
    for g, name in zip(got, NAMES):
        assert (g is None) == (name not in want), name
        if g is not None:
            value, size = want[name]
            if before is not None and name in before:
                value = value + before[name]
                size = size + np.abs(value)
            _within(g, value, size * E, name)
    return got


GATES = ["none", "channel", "token", "element"]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("d", [1, 2, 7, 8, 31, 64, 257, 1000, 1001, 2048, 4096])
def test_sizes(tim, dtype, d):
    for n, gate in enumerate(GATES):
        for post in (False, True):
            for pre in (False, True):
                p = _problem(5, d, dtype, gate, post, pre, 100 * d + n)
                h, _ = _forward(tim, p, 0.37, 1e-5)
                _backward(tim, p, h, 0.37, 1e-5)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("d", [4104, 5120, 8192, 8195, 12288, 16384])
@pytest.mark.parametrize("gate", ["channel", "token"])
def test_wide_rows(tim, dtype, d, gate):
    p = _problem(3, d, dtype, gate, True, True, d)
    h, _ = _forward(tim, p, 1.0, 1e-6)
    _backward(tim, p, h, 1.0, 1e-6)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("offset,pad", [(0, 3), (1, 0), (3, 5), (8, 8)])
@pytest.mark.parametrize("gate", GATES)
def test_rows_at_any_address(tim, dtype, offset, pad, gate):
    import torch
    T, d = 6, 264
    p = _problem(T, d, dtype, gate, True, True, 7, pad, offset)
    big = [torch.full((T + 2, offset + d + pad), 7.0, dtype=_dtype(dtype), device="cuda") for _ in range(5)]
    view = [t[:T, offset:offset + d] for t in big]
    h, _ = _forward(tim, p, 0.5, 1e-5, out=(view[0], view[1]))
    sums = [torch.empty(d, device="cuda") for _ in range(2)]
    dgate = {"none": None, "channel": torch.empty(d, device="cuda"), "token": torch.empty(T, 1, device="cuda"),
             "element": view[4]}[gate]
    _backward(tim, p, h, 0.5, 1e-5, out=(view[2], view[3], *sums, dgate))
    for t in big:
        t[:T, offset:offset + d] = 7.0
        assert bool((t == 7.0).all())  # nothing beside the rows is written


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 151, 153, 305, 1000, 3001])
def test_many_rows(tim, dtype, T):
    for d, gate in ((256, "channel"), (2048, "token"), (72, "element")):
        p = _problem(T, d, dtype, gate, True, True, T)
        h, _ = _forward(tim, p, 1.5, 1e-6)
        _backward(tim, p, h, 1.5, 1e-6)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_gradient_alone_and_added_sums(tim, dtype):
    import torch
    T, d = 40, 300
    for gate in GATES:
        p = _problem(T, d, dtype, gate, True, True, 11)
        h, _ = _forward(tim, p, 0.8, 1e-6)
        _backward(tim, p, h, 0.8, 1e-6, dy=False)
        _backward(tim, p, None, 0.8, 1e-6, dy=False)
        _backward(tim, p, h, 0.8, 1e-6, dh=False)
        got = _backward(tim, p, h, 0.8, 1e-6, dh=False, dy=False)
        assert all(not bool(g.any()) for g in got if g is not None)
        base = _matrix(3, d, "f32", 12)
        out = (torch.empty_like(h), torch.empty_like(h), base[0].clone(), base[1].clone(),
               {"none": None, "channel": base[2].clone(), "token": torch.full((T, 1), 7.0, device="cuda"),
                "element": torch.empty_like(h)}[gate])
        before = dict(dgamma=_np(base[0]), dgamma_post=_np(base[1]))
        if gate == "channel":
            before["dgate"] = _np(base[2])
        _backward(tim, p, h, 0.8, 1e-6, out=out, accumulate=True, before=before)


def test_in_place(tim):
    import torch
    p = _problem(9, 512, "bf16", "token", True, True, 13)
    want = _forward(tim, p, 0.5, 1e-6)
    h, x = p["h"].clone(), p["x"].clone()
    got = tim.residual_norm(h, x, p["gamma"], 1e-6, gamma_post=p["gamma_post"], gate=p["gate"], scale=0.5,
                            out=(h, x))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert got[0].data_ptr() == h.data_ptr() and got[1].data_ptr() == x.data_ptr()


def test_rows_do_not_depend_on_the_batch(tim):
    import torch
    p = _problem(700, 1000, "bf16", "channel", True, True, 14)
    h, y = _forward(tim, p, 0.5, 1e-6)
    whole = tim.residual_norm_backward(h, p["x"], p["dh"], p["dy"], p["gamma"], 1e-6, gamma_post=p["gamma_post"],
                                       gate=p["gate"], scale=0.5)
    for i in (0, 333, 699):
        s = slice(i, i + 1)
        one = tim.residual_norm(p["h"][s], p["x"][s], p["gamma"], 1e-6, gamma_post=p["gamma_post"],
                                gate=p["gate"], scale=0.5)
        assert torch.equal(one[0], h[s]) and torch.equal(one[1], y[s])
        part = tim.residual_norm_backward(h[s], p["x"][s], p["dh"][s], p["dy"][s], p["gamma"], 1e-6,
                                          gamma_post=p["gamma_post"], gate=p["gate"], scale=0.5)
        assert torch.equal(part[0], whole[0][s]) and torch.equal(part[1], whole[1][s])
    again = tim.residual_norm_backward(h, p["x"], p["dh"], p["dy"], p["gamma"], 1e-6, gamma_post=p["gamma_post"],
                                       gate=p["gate"], scale=0.5)
    assert all(torch.equal(a, b) for a, b in zip(whole, again))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("offset,pad", [(0, 3), (3, 5), (0, 8), (2, 6)])
def test_rows_of_padded_matrices_do_not_depend_on_the_batch(tim, dtype, offset, pad):
    """A row alone lies at a 16-byte boundary here and there; its strides are still its matrices'."""
    import torch
    for d, gate in ((264, "channel"), (4096, "element")):
        p = _problem(40, d, dtype, gate, True, True, 14, pad, offset)
        kw = dict(gamma_post=p["gamma_post"], scale=0.5)
        h, y = tim.residual_norm(p["h"], p["x"], p["gamma"], 1e-6, gate=p["gate"], **kw)
        whole = tim.residual_norm_backward(p["h"], p["x"], p["dh"], p["dy"], p["gamma"], 1e-6, gate=p["gate"], **kw)
        for i in range(40):
            s = slice(i, i + 1)
            g = p["gate"] if gate == "channel" else p["gate"][s]
            one = tim.residual_norm(p["h"][s], p["x"][s], p["gamma"], 1e-6, gate=g, **kw)
            assert torch.equal(one[0], h[s]) and torch.equal(one[1], y[s]), i
            part = tim.residual_norm_backward(p["h"][s], p["x"][s], p["dh"][s], p["dy"][s], p["gamma"], 1e-6,
                                              gate=g, **kw)
            assert torch.equal(part[0], whole[0][s]) and torch.equal(part[1], whole[1][s]), i


def test_one_row_in_place_by_views_of_other_strides(tim):
    import torch
    p = _problem(1, 264, "bf16", "none", True, True, 23, pad=8)
    want = _forward(tim, p, 0.5, 1e-6)
    h, x = p["h"], p["x"]
    got = tim.residual_norm(h, x, p["gamma"], 1e-6, gamma_post=p["gamma_post"], scale=0.5,
                            out=(h.as_strided((1, 264), (264, 1)), x.as_strided((1, 264), (300, 1))))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert got[0].data_ptr() == h.data_ptr() and got[1].data_ptr() == x.data_ptr()


def test_zero_and_nonfinite_rows(tim):
    """A row of zeros under a norm (eps alone below the root); a NaN or infinite row leaves the others."""
    import torch
    p = _problem(5, 96, "f32", "none", True, True, 15)
    p["x"][1] = 0.0
    p["h"][1] = 0.0
    h, y = _forward(tim, p, 1.0, 1e-6)
    _backward(tim, p, h, 1.0, 1e-6)
    assert not bool(h[1].any()) and not bool(y[1].any())
    x = p["x"].clone()
    x[2, 5] = math.nan
    x[3, 7] = math.inf
    h2, y2 = tim.residual_norm(p["h"], x, p["gamma"], 1e-6, gamma_post=p["gamma_post"])
    for i in (0, 1, 4):
        assert torch.equal(h2[i], h[i]) and torch.equal(y2[i], y[i])
    assert bool(h2[2].isnan().all()) and bool(y2[3].isnan().any())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,pad", [(64, 0), (1000, 3), (4096, 0), (4096, 3), (16384, 0)])
@pytest.mark.parametrize("size", [1e15, 1e-15])
def test_gradients_of_rows_far_from_one(tim, dtype, d, pad, size):
    """The gradient of a row of size s is of size 1 / s, its projection onto the row among it; 1 / s^3 is out
    of fp32's range for these."""
    for gate in GATES:
        p = _problem(3, d, dtype, gate, True, True, d, pad)
        p["h"].mul_(size)
        p["x"].mul_(size)
        _backward(tim, p, p["h"], 0.5, 0.0, dh=False)
        _backward(tim, p, p["h"], 0.5, 0.0)
        for post in (False, True):
            _forward(tim, {**p, "gamma_post": p["gamma_post"] if post else None}, 0.5, 0.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 4096, 16384])
def test_rows_at_the_ends_of_the_range_of_their_squares(tim, dtype, d):
    """Right while the sum of the squares lies below 2^128 and their mean at 2^-126 or above; finite rows
    beyond the one are zeros under the norm and take no part in its gradients."""
    import torch
    p = _problem(4, d, dtype, "none", True, True, 31)
    root = math.sqrt(d)
    signs = torch.where(p["h"] < 0, -1.0, 1.0).to(p["h"].dtype)
    for size in (2.0 ** 63 / root, 2.0 ** -62.5):
        q = {**p, "h": signs * size, "x": signs.flip(0) * size}
        _forward(tim, {**q, "gamma_post": None}, 0.5, 0.0)
        # so that dh and the norm's part of dresidual are of one size, and dblock is within the range
        q["dy"], q["dh"] = p["dy"] * min(size, 1.0), p["dh"] * (min(size, 1.0) / size)
        _backward(tim, q, q["h"], 0.5, 0.0)
    far = {**p, "h": p["h"].clone(), "x": p["x"].clone()}
    far["h"][2] = signs[2] * (2.0 ** 66 / root)
    far["x"][2] = signs[2] * (2.0 ** 66 / root)
    h, y = tim.residual_norm(far["h"], far["x"], p["gamma"], 1e-6, gamma_post=p["gamma_post"])
    assert torch.equal(h[2], far["h"][2]) and not bool(y[2].any())
    got = tim.residual_norm_backward(h, far["x"], p["dh"], p["dy"], p["gamma"], 1e-6, gamma_post=p["gamma_post"])
    assert torch.equal(got[0][2], p["dh"][2]) and not bool(got[1][2].any())
    keep = [0, 1, 3]
    part = {k: v[keep] if v is not None and v.dim() == 2 else v for k, v in p.items()}
    hk, yk = _forward(tim, part, 1.0, 1e-6)
    assert torch.equal(h[keep], hk) and torch.equal(y[keep], yk)
    want = _backward(tim, part, hk, 1.0, 1e-6)
    assert torch.equal(got[0][keep], want[0]) and torch.equal(got[1][keep], want[1])
    # the sums over rows: one row more of zeros, which a CTA of its own leaves
    assert torch.equal(got[2], want[2]) and torch.equal(got[3], want[3])


def test_differences(tim):
    """The gradient in fp32 against central differences of the formula in 64 bits."""
    T, d, scale, eps = 3, 5, 0.7, 1e-3
    for gate in GATES:
        p = _problem(T, d, "f32", gate, True, True, 16)
        h, _ = _forward(tim, p, scale, eps)
        got = tim.residual_norm_backward(h, p["x"], p["dh"], p["dy"], p["gamma"], eps, gamma_post=p["gamma_post"],
                                         gate=p["gate"], scale=scale)
        host = {k: _np(v) for k, v in p.items()}

        def loss(**kw):
            q = {**host, **kw}
            s, _ = oracle.ends.residual_norm(q["h"], q["x"], None, q["gamma_post"], q["gate"],
                                             float(np.float32(scale)), float(np.float32(eps)))
            return np.sum(s * q["dh"]) + np.sum(oracle.ends.norm_rows(s, q["gamma"], float(np.float32(eps))) * q["dy"])

        for g, k in zip(got, ("h", "x", "gamma", "gamma_post", "gate")):
            if host[k] is None:
                continue
            for at in np.ndindex(host[k].shape):
                e = np.zeros_like(host[k])
                e[at] = 1e-5
                diff = (loss(**{k: host[k] + e}) - loss(**{k: host[k] - e})) / 2e-5
                assert abs(diff - float(g[at])) < 2e-5 * (1 + abs(diff)), (gate, k, at)


def test_autograd(tim):
    import torch
    T, d = 30, 136
    for dtype in ("f32", "bf16"):
        for gate in GATES:
            p = _problem(T, d, dtype, gate, True, True, 17)
            leaves = {k: p[k].detach().clone().requires_grad_(True)
                      for k in ("h", "x", "gamma", "gamma_post", "gate") if p[k] is not None}
            ws = tim.Workspace(tim.residual_norm_backward_workspace_size(T, d))
            h, y = tim.block_residual(leaves["h"], leaves["x"], leaves["gamma"], 1e-6,
                                      gamma_post=leaves["gamma_post"], gate=leaves.get("gate"), scale=0.5,
                                      workspace=ws)
            dy = p["dy"].t().contiguous().t()  # columns contiguous
            grads = torch.autograd.grad((h, y), list(leaves.values()), (p["dh"], dy), retain_graph=True)
            want = tim.residual_norm_backward(h.detach(), p["x"], p["dh"], p["dy"], p["gamma"], 1e-6,
                                              gamma_post=p["gamma_post"], gate=p["gate"], scale=0.5)
            for g, w, t in zip(grads, [w for w in want if w is not None], leaves.values()):
                assert g.dtype == t.dtype and torch.equal(g, w.to(t.dtype))
            alone, = torch.autograd.grad(y, leaves["x"], p["dy"], retain_graph=True)
            only = tim.residual_norm_backward(h.detach(), p["x"], None, p["dy"], p["gamma"], 1e-6,
                                              gamma_post=p["gamma_post"], gate=p["gate"], scale=0.5)
            assert torch.equal(alone, only[1])
    h, y = tim.block_residual(leaves["h"], leaves["x"], None, 1e-6)
    assert y is None
    assert torch.equal(torch.autograd.grad(h, leaves["x"], p["dh"])[0], p["dh"])


def test_graph_replay_streams_and_two_calls_at_once(tim):
    import torch
    T, d = 500, 1032
    p = _problem(T, d, "bf16", "channel", True, True, 18)
    kw = dict(gamma_post=p["gamma_post"], gate=p["gate"], scale=0.5)
    ws = tim.Workspace(tim.residual_norm_backward_workspace_size(T, d))
    big = [torch.full((T + 2, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    sums = [torch.empty(d, device="cuda") for _ in range(3)]

    def step():
        h, _ = tim.residual_norm(p["h"], p["x"], p["gamma"], 1e-6, out=(big[0][:T], big[1][:T]), **kw)
        tim.residual_norm_backward(h, p["x"], p["dh"], p["dy"], p["gamma"], 1e-6, workspace=ws,
                                   out=(big[2][:T], big[3][:T], *sums), **kw)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (30, 40):
        q = _problem(T, d, "bf16", "channel", True, True, seed)
        for k in ("h", "x", "dh", "dy"):
            p[k].copy_(q[k])
        graph.replay()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        h, y = tim.residual_norm(p["h"], p["x"], p["gamma"], 1e-6, stream=side, **kw)
        want = tim.residual_norm_backward(h, p["x"], p["dh"], p["dy"], p["gamma"], 1e-6, stream=side, **kw)
        torch.cuda.synchronize()
        assert torch.equal(big[0][:T], h) and torch.equal(big[1][:T], y)
        assert all(torch.equal(a, b) for a, b in zip((big[2][:T], big[3][:T], *sums), want))
    assert all(bool((t[T:] == 7).all()) for t in big)
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [tim.Workspace(ws.nbytes) for _ in range(2)]
    torch.cuda.synchronize()
    got = [[tim.residual_norm_backward(h, p["x"], p["dh"], p["dy"], p["gamma"], 1e-6, workspace=w, stream=s, **kw)
            for s, w in zip(streams, spaces)] for _ in range(6)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for pair in got for g in pair for a, b in zip(g, want))


def test_refusals(tim):
    import torch
    p = _problem(4, 32, "f32", "element", True, True, 19)
    h, x, gamma, gate = p["h"], p["x"], p["gamma"], p["gate"]
    for bad in (lambda: tim.residual_norm(h.t(), x, gamma, 1e-6), lambda: tim.residual_norm(h.half(), x, gamma, 1e-6),
                lambda: tim.residual_norm(h, x, gamma[:31], 1e-6), lambda: tim.residual_norm(h, x, gamma, 1e-6, gate=gate[:3]),
                lambda: tim.residual_norm(h, x, gamma, 1e-6, gate=gate[0, :31]),
                lambda: tim.residual_norm(h, x, gamma, 1e-6, gate=gate.half()),
                lambda: tim.residual_norm_backward(h, x, p["dh"], p["dy"], None, 1e-6),
                lambda: tim.residual_norm_backward(h, x, p["dh"], p["dy"], gamma, 1e-6, accumulate=True)):
        with pytest.raises((ValueError, TypeError)):
            bad()
    for bad in (lambda: tim.residual_norm(h, x, gamma, math.nan), lambda: tim.residual_norm(h, x, gamma, 1e-6, scale=math.inf),
                lambda: tim.residual_norm(h, x, gamma, 1e-6, out=(x, h)),
                lambda: tim.residual_norm(h, x, gamma, 1e-6, out=(h, h)),
                lambda: tim.residual_norm(h[1:], x[1:], gamma, 1e-6, out=(h[:3], x[1:])),
                lambda: tim.residual_norm(h[:0], x[:0], gamma, 1e-6),
                lambda: tim.residual_norm_backward(h, x, p["dh"], p["dy"], gamma, 1e-6, workspace=tim.Workspace(1024))):
        with pytest.raises(tim.TimError):
            bad()
    wide = torch.zeros(1, 16385, device="cuda")
    with pytest.raises(tim.TimError, match="TIM_ERR_SHAPE"):
        tim.residual_norm(wide, wide.clone(), None, 1e-6)


@pytest.mark.slow
def test_beyond_2_31_elements(tim):
    """Matrices of more than 2^31 elements: offsets need 64 bits."""
    import torch
    T, d = 131100, 16384
    h = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    x = torch.ones(T, d, dtype=torch.bfloat16, device="cuda")
    gate = (torch.arange(T, device="cuda") % 128 + 1).to(torch.bfloat16).view(T, 1)
    ones = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    tim.residual_norm(h, x, ones, 0.0, gate=gate, out=(h, x))
    assert torch.equal(h[:, ::4099], gate.expand(T, 4)) and bool((x == 1).all())


@pytest.mark.slow
@pytest.mark.parametrize("T,d", [(262200, 8192), (131100, 16384)])
def test_gradients_beyond_2_31_elements(tim, T, d):
    """With rows on their way to shared memory and without.  Of rows of ones under both norms, with dy = +1, -1,
    +1, ..., dh = c and a gate of g: dresidual = c +- 1, dblock = +-g, dgate = d c."""
    import torch
    h, x, dy = (torch.ones(T, d, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    dy[:, 1::2] = -1
    row = torch.arange(T, device="cuda").view(T, 1)
    c, g = (row % 16).to(torch.bfloat16), (row % 127 + 1).to(torch.bfloat16)
    dh = c.expand(T, d).contiguous()
    ones = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    dres, dblock, dgamma, dpost, dgate = tim.residual_norm_backward(h, x, dh, dy, ones, 0.0, gamma_post=ones, gate=g)
    for i in range(0, T, 1 << 15):
        s = slice(i, i + (1 << 15))
        assert torch.equal(dres[s], dh[s] + dy[s]) and torch.equal(dblock[s], g[s] * dy[s]), i
    # r = 1 is off by four steps at most, a row's sum is one of whole numbers and exact, a sum over rows is
    # that of a CTA's, one on every SM at least, and then of the CTAs'
    assert bool(((dgate - d * c.float()).abs() <= 2.0 ** -20 * d * c.float()).all())
    tol = (T / torch.cuda.get_device_properties(0).multi_processor_count + 70) * 2.0 ** -24
    sign = dy[0].double()
    assert bool(((dgamma.double() - T * sign).abs() <= tol * T).all())
    cd, gd = c.double().view(T), g.double().view(T)
    want, size = (gd * cd).sum() + sign * gd.sum(), (gd * (cd + 1)).sum()
    assert bool(((dpost.double() - want).abs() <= tol * size).all())
