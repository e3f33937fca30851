"""The logits operators on the CPU: the oracle against hand numbers and differences, and every
refusal of the C ABI and of the binding that needs no GPU."""
import ctypes
import math

import numpy as np
import pytest

import oracle


# ----------------------------------------------------------------------------- the oracle

def test_sampler_oracle_top_k_example():
    # k = 2 turns (0.50, 0.30, 0.20) into (0.625, 0.375, 0)
    z = np.log([0.5, 0.3, 0.2])
    for u, want in ((0.0, 0), (0.624, 0), (0.626, 1), (0.99, 1)):
        r = oracle.sample_row(z, u, 1.0, 2, 1.0, 0.0)
        assert r["id"] == want and r["kept"] == 2
        assert r["logprob"] == pytest.approx(math.log((0.625, 0.375)[want]), abs=1e-12)


def test_sampler_oracle_filters_and_order():
    z = np.log([0.1, 0.4, 0.1, 0.4])
    # top-p 0.75 keeps both 0.4 and, mass before it being 0.8, nothing else
    assert oracle.sample_row(z, 0.6, 1.0, 0, 0.75, 0.0)["kept"] == 2
    # 0.85 keeps the lower id of the two equal tokens too
    assert oracle.sample_row(z, 0.0, 1.0, 0, 0.85, 0.0) | {"margin": 0} == pytest.approx(
        dict(id=0, logprob=math.log(0.1 / 0.9), lse=math.log(0.9), kept=3, margin=0), abs=1e-12)
    # the draw goes by id: token 0 holds [0, 0.1), token 1 up to 0.5
    assert [oracle.sample_row(z, u, 1.0, 0, 1.0, 0.0)["id"] for u in (0.05, 0.3, 0.55, 0.9)] == [0, 1, 2, 3]
    # min-p 0.3 > 0.1 / 0.4
    assert oracle.sample_row(z, 0.0, 1.0, 0, 1.0, 0.3)["id"] == 1
    # temperature 0: the first of the largest
    assert oracle.sample_row(z, 0.9, 0.0, 0, 1.0, 0.0) | {"margin": 0} == dict(
        id=1, logprob=0.0, lse=z[1], kept=1, margin=0)


def test_processed_score_is_the_samplers():
    """The sampler's logprob is the processed score of the token it draws."""
    rng = np.random.default_rng(1)
    for _ in range(20):
        z = rng.normal(size=50) * 2
        r = oracle.sample_row(z, float(rng.random()), 0.7, 12, 0.9, 0.0)
        ids, lp = oracle.process_head(z, 0.7, 12, 0.9)
        assert r["logprob"] == pytest.approx(float(lp[list(ids).index(r["id"])]), abs=1e-12)
        assert r["kept"] == int(np.sum(lp > -np.inf))


def test_distill_oracle_whole_head_is_kl():
    """With every token in the head the loss is the KL divergence of the two distributions."""
    rng = np.random.default_rng(2)
    z, t = rng.normal(size=9), rng.normal(size=9)
    p, q = np.exp(z) / np.exp(z).sum(), np.exp(t) / np.exp(t).sum()
    ids = rng.permutation(9)
    for tail in (False, True):
        f = oracle.distill_row(z, ids, np.log(q)[ids], 1.0, "forward", tail)
        assert f[0] == pytest.approx(float(np.sum(q * np.log(q / p))), abs=1e-12)
        np.testing.assert_allclose(f[2], p - q, atol=1e-12)
        r = oracle.distill_row(z, ids, np.log(q)[ids], 1.0, "reverse", tail)
        assert r[0] == pytest.approx(float(np.sum(p * np.log(p / q))), abs=1e-12)


@pytest.mark.parametrize("kind", ["forward", "reverse"])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_oracle_gradient_by_differences(kind, tail):
    rng = np.random.default_rng(3)
    z = rng.normal(size=12)
    ids = np.array([3, -1, 7, 0, 5])
    lp = np.log(np.array([0.4, 0.1, 0.2, 0.15, 0.05]))
    lp[4] = -np.inf
    _, _, g = oracle.distill_row(z, ids, lp, 1.3, kind, tail)
    h = 1e-5
    for v in range(12):
        e = np.zeros(12)
        e[v] = h
        d = (oracle.distill_row(z + e, ids, lp, 1.3, kind, tail)[0]
             - oracle.distill_row(z - e, ids, lp, 1.3, kind, tail)[0]) / (2 * h)
        assert d == pytest.approx(g[v], abs=1e-8)


# ----------------------------------------------------------------------------- refusals

@pytest.fixture(scope="module")
def tim():
    import __graft_entry__
    __graft_entry__.build()
    import rollout_logprob_consistency_gb300 as tim
    return tim


P = 1 << 20  # stands for a device address: nothing here gets as far as using it


def _sample(tim, **kw):
    a = dict(logits=P, dtype=1, ld=64, T=4, V=64, uniform=P, temperature=1.0, top_k=0, top_p=1.0,
             min_p=0.0, rows=(None,) * 4, ids=P, lp=P, lse=P, kept=P, ws=P, nbytes=1024)
    a.update(kw)
    from rollout_logprob_consistency_gb300.binding import _SampleParams
    p = _SampleParams(a["temperature"], a["top_k"], a["top_p"], a["min_p"], *a["rows"])
    return tim.lib().tim_sample(a["logits"], a["dtype"], a["ld"], a["T"], a["V"], a["uniform"],
                                None if kw.get("no_params") else ctypes.byref(p), a["ids"], a["lp"],
                                a["lse"], a["kept"], a["ws"], a["nbytes"], None)


SHAPE, ARG, WORKSPACE = 2, 1, 7


@pytest.mark.parametrize("kw,code", [
    (dict(logits=None), ARG), (dict(logits=P + 1), ARG), (dict(dtype=3), ARG), (dict(dtype=-1), ARG),
    (dict(dtype=0, logits=P + 2), ARG), (dict(T=0), SHAPE), (dict(T=2 ** 31), SHAPE),
    (dict(V=0), SHAPE), (dict(V=393217, ld=393217), SHAPE), (dict(ld=63), SHAPE),
    (dict(ld=2 ** 31 + 1), SHAPE), (dict(uniform=None), ARG), (dict(uniform=P + 2), ARG),
    (dict(ids=None), ARG), (dict(lp=None), ARG), (dict(lse=None), ARG), (dict(kept=None), ARG),
    (dict(kept=P + 1), ARG), (dict(no_params=True), ARG), (dict(temperature=-1.0), ARG),
    (dict(temperature=math.nan), ARG), (dict(temperature=math.inf), ARG),
    (dict(temperature=1e-7), ARG), (dict(top_p=0.0), ARG), (dict(top_p=math.nan), ARG),
    (dict(min_p=-0.1), ARG), (dict(min_p=1.5), ARG), (dict(rows=(P + 1, None, None, None)), ARG),
    (dict(ws=None), WORKSPACE), (dict(ws=P + 8), WORKSPACE), (dict(nbytes=1023), WORKSPACE)])
def test_sample_refusals(tim, kw, code):
    assert _sample(tim, **kw) == code


def _distill(tim, **kw):
    a = dict(logits=P, dtype=1, ld=64, T=4, V=64, ids=P, lp=P, K=8, temperature=1.0, kind=0, tail=0,
             loss=P, lse=P, saved=P, ws=P, nbytes=1024)
    a.update(kw)
    return tim.lib().tim_distill(a["logits"], a["dtype"], a["ld"], a["T"], a["V"], a["ids"], a["lp"],
                                 a["K"], a["temperature"], a["kind"], a["tail"], a["loss"], a["lse"],
                                 a["saved"], a["ws"], a["nbytes"], None)


DISTILL_BAD = [
    (dict(logits=None), ARG), (dict(dtype=7), ARG), (dict(T=0), SHAPE), (dict(V=0), SHAPE),
    (dict(V=393217, ld=400000), SHAPE), (dict(ld=1), SHAPE), (dict(ids=None), ARG),
    (dict(lp=None), ARG), (dict(ids=P + 2), ARG), (dict(K=0), SHAPE), (dict(K=1025), SHAPE),
    (dict(temperature=0.0), ARG), (dict(temperature=math.nan), ARG), (dict(temperature=1e7), ARG),
    (dict(kind=2), ARG)]


@pytest.mark.parametrize("kw,code", DISTILL_BAD + [
    (dict(tail=2), ARG), (dict(loss=None), ARG), (dict(lse=None), ARG), (dict(saved=None), ARG),
    (dict(saved=P + 2), ARG), (dict(ws=None), WORKSPACE), (dict(nbytes=100), WORKSPACE)])
def test_distill_refusals(tim, kw, code):
    assert _distill(tim, **kw) == code


def _backward(tim, **kw):
    a = dict(logits=P, dtype=1, ld=64, T=4, V=64, ids=P, lp=P, K=8, temperature=1.0, kind=0, saved=P,
             grad=P, out=2 * P, ldd=64)
    a.update(kw)
    return tim.lib().tim_distill_backward(a["logits"], a["dtype"], a["ld"], a["T"], a["V"], a["ids"],
                                          a["lp"], a["K"], a["temperature"], a["kind"], a["saved"],
                                          a["grad"], a["out"], a["ldd"], None)


@pytest.mark.parametrize("kw,code", DISTILL_BAD + [
    (dict(saved=None), ARG), (dict(grad=None), ARG), (dict(grad=P + 1), ARG), (dict(out=None), ARG),
    (dict(ldd=63), SHAPE), (dict(out=P), ARG), (dict(out=P + 4 * 64 * 2 - 2), ARG),
    (dict(out=P - 4 * 64 * 2 + 2), ARG)])
def test_distill_backward_refusals(tim, kw, code):
    assert _backward(tim, **kw) == code


def _grad(tim, **kw):
    a = dict(logits=P, dtype=1, ld=64, T=4, V=64, ids=P, lp=P, K=8, temperature=1.0, kind=0, tail=0,
             grad=P, loss=P, out=2 * P, ldd=64, ws=P, nbytes=1024)
    a.update(kw)
    return tim.lib().tim_distill_grad(a["logits"], a["dtype"], a["ld"], a["T"], a["V"], a["ids"],
                                      a["lp"], a["K"], a["temperature"], a["kind"], a["tail"],
                                      a["grad"], a["loss"], a["out"], a["ldd"], a["ws"],
                                      a["nbytes"], None)


@pytest.mark.parametrize("kw,code", DISTILL_BAD + [
    (dict(tail=-1), ARG), (dict(grad=None), ARG), (dict(loss=None), ARG), (dict(loss=P + 1), ARG),
    (dict(out=None), ARG), (dict(ldd=63), SHAPE), (dict(out=P), ARG), (dict(ws=None), WORKSPACE),
    (dict(nbytes=1023), WORKSPACE)])
def test_distill_grad_refusals(tim, kw, code):
    assert _grad(tim, **kw) == code


def test_binding_refuses_wrong_tensors(tim):
    torch = pytest.importorskip("torch")
    z = torch.zeros(2, 8)
    u = torch.zeros(2)
    with pytest.raises(ValueError, match="CUDA"):
        tim.sample(z, u)
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        tim.sample(z.double(), u)
    with pytest.raises(TypeError):
        tim.sample([1.0], u)
    with pytest.raises(ValueError, match="CUDA"):
        tim.distill(z, torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3))
    with pytest.raises(ValueError, match="CUDA"):
        tim.distill_backward(z, torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3),
                             torch.zeros(2, 8), u)
