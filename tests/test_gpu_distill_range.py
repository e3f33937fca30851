"""tim.distill* where the teacher's head and the student's mass lie far apart, and at every
temperature, against the fp64 oracle.

Tolerances, from the arithmetic.  A weight outside the head is 2^x in fp32, x at most 126 octaves
from its reference: two roundings of x and the remainder of its factor, 2.5 x 2^-24 |x| ln2 =
1.3e-5, and the exponential 2^-22.  A thread adds at most 17 of them here (V <= 4099 over 256
threads, a rescaling before each at worst, 2^-22), and 9 joins follow at 2^-22 each: 6.5e-6.  So a
weight, the sum of those outside the head and 1 / S are good to EPS = 2^-15 = 3.1e-5 together, and
ln p_r to EPS absolute.  The head's terms are pairs of floats, far better.  With Q, P the head's
masses, B = sum p (|a| + 1) over the buckets, a = ln p - ln q:
  forward  |dL| <= EPS (Q + q_r)
           |dg|  <= EPS (p Q + q_r P p / p_r) outside, EPS (p (Q + q_r) + q) in the head
  reverse  |dL| <= EPS B
           |dg|  <= EPS p (|a| + 2 + B), a = a_r (or 0) outside
and every result is rounded: the loss and lse 2^-24 relative (the constants in fp32 and the product
2^-22 more for a gradient), the gradient half a step of its type.  What is below 2^-126 may be 0: each
of the K p_k that are takes up to 2^-126 (|a_k| + 1) from B and so from the reverse loss, the rest
2^-126 (|a_r| + 1); a gradient has p_v <= 1 times that and its own p_v (|a_v| + 1).
"""
import math

import numpy as np
import pytest

import oracle
from test_gpu_distill import MODES, _dtype, _half_step, tim  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -15
FLUSH = 2.0 ** -126


def _reference(z, ids, lp, w, tau, kind, tail):
    """loss, lse, gradient, and the tolerances of loss and gradient before any rounding."""
    tau = float(np.float32(tau))
    zh = z.double().cpu().numpy()
    ih, lh, wh = (t.cpu().numpy() for t in (ids, lp, w))
    T, V = zh.shape
    loss, lse, grad = np.zeros(T), np.zeros(T), np.zeros((T, V))
    dloss, dgrad = np.zeros(T), np.zeros((T, V))
    for i in range(T):
        loss[i], lse[i], g = oracle.distill_row(zh[i], ih[i], lh[i], tau, kind, tail)
        hid, lq = ih[i], lh[i].astype(np.float64)
        logp = zh[i] / tau - lse[i]
        p, q = np.exp(logp), np.exp(lq)
        out = np.ones(V, dtype=bool)
        out[hid] = False
        pr, P, Q = p[out].sum(), p[hid].sum(), q.sum()
        qr = 1 - Q if tail and pr > 0 and 1 - Q > 2.0 ** -20 else 0.0
        a = np.abs(logp[hid] - lq)
        tol = np.empty(V)
        if kind == "forward":
            flush = FLUSH
            dloss[i] = EPS * (Q + qr)
            tol[out] = p[out] * Q + (qr * P * (p[out] / pr) if qr else 0.0)
            tol[hid] = p[hid] * (Q + qr) + q
        else:
            ar = abs(math.log(pr) - math.log(qr)) if qr else 0.0
            flush = FLUSH * (2 + ar + (a + 1).sum())
            B = (p[hid] * (a + 1)).sum() + (pr * (ar + 1) if qr else 0.0)
            dloss[i] = EPS * B + flush
            tol[out] = p[out] * (ar + 2 + B)
            tol[hid] = p[hid] * (a + 2 + B)
        scale = abs(wh[i]) / tau
        grad[i] = g * wh[i]
        dgrad[i] = scale * (EPS * tol + 2 * flush)
    return loss, lse, grad, dloss, dgrad


def _close(got, want, tol, what):
    d = np.abs(got.detach().double().cpu().numpy() - want)
    bad = ~(d <= tol)
    at = np.unravel_index(np.argmax(np.where(np.isnan(d), np.inf, d - tol)), d.shape)
    assert not bad.any(), (what, at, float(got[at]), float(want[at]), float(tol[at]), int(bad.sum()))


def _check(tim, z, ids, lp, w, tau, kind, tail):
    """All four calls, none of which may report an error."""
    ref = _reference(z, ids, lp, w, tau, kind, tail)
    rel, least = _half_step(z.dtype)
    tloss = ref[3] + 2.0 ** -23 * np.abs(ref[0])
    tgrad = ref[4] + (rel + 2.0 ** -22) * np.abs(ref[2]) + least
    loss, lse, saved = tim.distill(z, ids, lp, tau, kind=kind, tail=tail)
    _close(loss, ref[0], tloss, "loss")
    _close(lse, ref[1], EPS + 2.0 ** -23 * np.abs(ref[1]), "lse")
    _close(tim.distill_backward(z, ids, lp, saved, w, tau, kind=kind), ref[2], tgrad, "backward")
    loss, grad = tim.distill_grad(z, ids, lp, w, tau, kind=kind, tail=tail)
    _close(loss, ref[0], tloss, "fused loss")
    _close(grad, ref[2], tgrad, "fused gradient")
    leaf = z.detach().clone().requires_grad_(True)
    loss = tim.distill_loss(leaf, ids, lp, tau, kind=kind, tail=tail)
    loss.backward(w)
    _close(loss, ref[0], tloss, "autograd loss")
    _close(leaf.grad, ref[2], tgrad, "autograd gradient")


def _apart(gaps, layout, dtype, tau, weight, V=4099, K=5, held=0.9):
    """Rows whose outside tokens (one of them, the rest far below, or all) lie gaps[i] nats (at tau)
    above the head's largest."""
    import torch
    g = np.random.default_rng(17)
    T = len(gaps)
    ids = np.stack([g.permutation(V)[:K] for _ in range(T)]).astype(np.int32)
    half = np.asarray(gaps)[:, None] * tau / 2
    z = np.repeat(half, V, axis=1)
    if layout == "one":
        z = np.minimum(-half, half) - 100 * tau - g.random((T, V)) * tau
        lone = np.array([next(v for v in g.permutation(V) if v not in ids[i]) for i in range(T)])
        z[np.arange(T), lone] = half[:, 0]
    for i in range(T):
        z[i, ids[i]] = -half[i, 0] - tau * np.arange(K) * 0.5
    t = g.normal(size=(T, K))
    lp = t - np.log(np.exp(t).sum(1, keepdims=True)) + math.log(held)
    to = lambda x, d: torch.from_numpy(np.asarray(x)).to(d).cuda()  # noqa: E731
    return (to(z, torch.float32).to(_dtype(dtype)), to(ids, torch.int32), to(lp, torch.float32),
            torch.full((T,), weight, device="cuda"))


ABOVE = sorted([70 + 0.25 * i for i in range(101)] + [math.log(2) * (126 + 0.1 * i) for i in range(40)])


@pytest.mark.parametrize("kind,tail", MODES)
@pytest.mark.parametrize("layout", ["one", "all"])
@pytest.mark.parametrize("dtype,tau,weight", [("f32", 1.0, 1.0), ("f32", 1.0, 1e-6), ("f32", 0.05, -3.0),
                                              ("bf16", 1.0, 1e-6), ("f16", 0.5, 1.0)])
def test_outside_far_above_the_head(tim, dtype, tau, weight, layout, kind, tail):  # noqa: F811
    """A finite row has a finite loss and a gradient of full precision, whatever the sum outside the
    head is relative to the head's largest."""
    _check(tim, *_apart(ABOVE, layout, dtype, tau, weight), tau, kind, tail)


BELOW = [-x * math.log(2) for x in (20, 39, 41, 53, 60, 90, 99, 101, 104, 115, 120, 125, 127, 140, 160,
                                    300, 700, 1000)]


@pytest.mark.parametrize("kind,tail", MODES)
@pytest.mark.parametrize("layout", ["one", "all"])
@pytest.mark.parametrize("dtype,tau", [("f32", 1.0), ("f32", 0.1), ("f32", 1e-3), ("bf16", 1.0), ("f16", 1.0)])
def test_outside_far_below_the_head(tim, dtype, tau, layout, kind, tail):  # noqa: F811
    """The rest keeps its bucket, loss and gradient, as long as it has any mass."""
    _check(tim, *_apart(BELOW, layout, dtype, tau, 1.0), tau, kind, tail)


def test_rest_of_one_token_by_hand(tim):  # noqa: F811
    """p_r = e^-72, q = (0.9, 0.1): L = 0.9 ln 0.9 + 0.1 (ln 0.1 + 72), gradient 0.1 and -0.1."""
    import torch
    z = torch.full((1, 300), -400.0, device="cuda")
    z[0, 7], z[0, 250] = 20.0, -52.0
    ids = torch.tensor([[7]], dtype=torch.int32, device="cuda")
    lp = torch.tensor([[0.9]], device="cuda").log()
    one = torch.ones(1, device="cuda")
    loss, grad = tim.distill_grad(z, ids, lp, one, tail=True)
    assert float(loss) == pytest.approx(0.9 * math.log(0.9) + 0.1 * (math.log(0.1) + 72), rel=1e-6)
    want = torch.zeros(300)
    want[7], want[250] = 0.1, -0.1
    assert float((grad[0].cpu() - want).abs().max()) <= 1e-6


def test_rest_without_mass(tim):  # noqa: F811
    """-inf, the type's lowest value, and whatever is more than 1074 octaves down: no bucket."""
    import torch
    z, ids, lp, w = _apart([-60.0] * 4, "all", "f32", 1.0, 1.0)
    out = torch.ones_like(z, dtype=torch.bool).scatter_(1, ids.long(), False)
    for i, low in enumerate((-math.inf, torch.finfo(torch.float32).min, -800.0, -750.0)):
        z[i, out[i]] = low
    for kind in ("forward", "reverse"):
        a = tim.distill_grad(z, ids, lp, w, kind=kind, tail=True)
        b = tim.distill_grad(z, ids, lp, w, kind=kind, tail=False)
        assert torch.equal(a[0][:3], b[0][:3]) and torch.equal(a[1][:3], b[1][:3])
        assert bool(a[0].isfinite().all()) and bool(a[1].isfinite().all())


@pytest.mark.parametrize("kind,tail", MODES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tau", [1e-6, 1e-4, 0.05, 0.3, 1.0, 40.0, 1e6])
def test_every_temperature_in_every_call(tim, tau, dtype, kind, tail):  # noqa: F811
    import torch
    g = np.random.default_rng(23)
    T, V, K = 6, 2003, 16
    z = torch.from_numpy((g.normal(size=(T, V)) * 2).astype(np.float32)).cuda().to(_dtype(dtype))
    ids = torch.from_numpy(np.stack([g.permutation(V)[:K] for _ in range(T)]).astype(np.int32)).cuda()
    z[T // 2:].scatter_(1, ids[T // 2:].long(), z[T // 2:].gather(1, ids[T // 2:].long()) + 9)
    t = g.normal(size=(T, K)) * 2
    lp = torch.from_numpy((t - np.log(np.exp(t).sum(1, keepdims=True)) - 0.1).astype(np.float32)).cuda()
    w = torch.from_numpy(g.normal(size=T).astype(np.float32)).cuda()
    _check(tim, z, ids, lp, w, tau, kind, tail)
