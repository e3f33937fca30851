"""tim.distill, its backward, distill_grad and the autograd loss against the fp64 oracle.

Tolerances, from the arithmetic.  A weight outside the head is 2^x in fp32: argument rounding
2 x 2^-24 |x| ln2 (|x| <= 40 octaves where it matters: 3.4e-6 at worst), the exponential 2^-22,
and a thread's fp32 sum of n <= 400 terms n 2^-24 at worst (2.4e-5; rounding errors of both signs
add up to sqrt(n) of that, which is not assumed).  So the sum S and each p_v are good to
EPS = 3e-5 relative; the head's terms are fp64.  Then
  |dL| <= EPS (Q + |c|) + one rounding to fp32,
  |d grad_v| <= |w / tau| (EPS p_v + 2^-126) (|c_rest| + |c_tail| + 1 + |a_v|) + half a step of
                the type (a weight below 2^-126, the smallest normal number, is taken as 0),
with c_tail = q_r P / p_r (forward) or a_r (reverse), which carry the error of p_r.
"""
import math

import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

EPS = 3e-5
FLUSH = 2.0 ** -126


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


def _inputs(T, V, K, dtype, seed, scale=2.0, pad=0, offset=0, held=0.9):
    import torch
    g = np.random.default_rng(seed)
    z = (g.normal(size=(T, V)) * scale).astype(np.float32)
    K = min(K, V)
    ids = np.stack([g.permutation(V)[:K] for _ in range(T)]).astype(np.int32)
    t = g.normal(size=(T, K)) * 2
    lp = (t - np.log(np.exp(t).sum(1, keepdims=True)) + math.log(held)).astype(np.float32)
    buf = torch.full((T, offset + V + pad), 33.0, dtype=_dtype(dtype), device="cuda")
    zt = buf[:, offset:offset + V]
    zt.copy_(torch.from_numpy(z).cuda())
    w = torch.from_numpy(g.normal(size=T).astype(np.float32)).cuda()
    return zt, torch.from_numpy(ids).cuda(), torch.from_numpy(lp).cuda(), w


def _reference(z, ids, lp, w, temperature, kind, tail):
    """loss, lse, grad and their tolerances (without the output's rounding)."""
    zh = z.detach().double().cpu().numpy()
    ih, lh, wh = (t.cpu().numpy() for t in (ids, lp, w))
    tau = float(np.float32(temperature))
    T, V = zh.shape
    out = [np.zeros(T), np.zeros(T), np.zeros((T, V)), np.zeros(T), np.zeros((T, V))]
    for i in range(T):
        loss, lse, g = oracle.distill_row(zh[i], ih[i], lh[i], tau, kind, tail)
        out[0][i], out[1][i], out[2][i] = loss, lse, g * wh[i]
        on = (ih[i] >= 0) & (lh[i] > -np.inf)
        if not on.any():
            continue
        hid, lq = ih[i][on], lh[i][on].astype(np.float64)
        s = zh[i] / tau
        logp = s - lse
        p = np.exp(logp)
        q = np.exp(lq)
        rest = np.ones(V, dtype=bool)
        rest[hid] = False
        pr, P, Q = p[rest].sum(), p[hid].sum(), q.sum()
        qr = max(1 - Q, 0.0) if tail and pr > 0 else 0.0
        with np.errstate(divide="ignore", invalid="ignore"):
            a = np.where(p[hid] > 0, np.abs(logp[hid] - lq), 0.0)
            if kind == "forward":
                c = Q + (qr * P / pr if pr > 0 and qr > 2.0 ** -20 else 0.0) + qr
            else:
                c = (p[hid] * (a + 1)).sum() + (abs(math.log(pr) - math.log(qr)) + 2
                                                 if qr > 2.0 ** -20 else 0.0)
        amp = np.full(V, c + 1.0)
        amp[hid] += a
        out[3][i] = EPS * (c + 1)
        out[4][i] = abs(wh[i]) / tau * (EPS * p + FLUSH) * amp
    return out


def _half_step(t):
    import torch
    return torch.finfo(t).eps / 2, torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2


def _assert_loss(loss, lse, ref, what=""):
    d = np.abs(loss.detach().cpu().numpy().astype(np.float64) - ref[0])
    tol = ref[3] + 2.0 ** -24 * np.abs(ref[0])
    assert np.all(d <= tol), (what, d.max(), int(np.argmax(d - tol)))
    if lse is not None:
        d = np.abs(lse.cpu().numpy().astype(np.float64) - ref[1])
        assert np.all(d <= EPS + 2.0 ** -24 * np.abs(ref[1])), (what, d.max())


def _assert_grad(grad, ref, what=""):
    rel, least = _half_step(grad.dtype)
    d = np.abs(grad.double().cpu().numpy() - ref[2])
    # one more fp32 rounding of the product before the type's own
    tol = ref[4] + (rel + 2.0 ** -23) * np.abs(ref[2]) + least
    assert np.all(d <= tol), (what, float((d - tol).max()), np.unravel_index(np.argmax(d - tol), d.shape))


MODES = [("forward", False), ("forward", True), ("reverse", False), ("reverse", True)]


@pytest.mark.parametrize("kind,tail", MODES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V,K", [(1, 1), (2, 1), (7, 3), (8, 8), (9, 4), (255, 16), (1000, 33),
                                 (4097, 1), (32003, 64), (50257, 1024)])
def test_loss_and_gradient(tim, V, K, dtype, kind, tail):
    import torch
    T = 5
    z, ids, lp, w = _inputs(T, V, K, dtype, V + K)
    ref = _reference(z, ids, lp, w, 1.3, kind, tail)
    loss, lse, saved = tim.distill(z, ids, lp, 1.3, kind=kind, tail=tail)
    _assert_loss(loss, lse, ref)
    grad = tim.distill_backward(z, ids, lp, saved, w, 1.3, kind=kind)
    assert grad.dtype == z.dtype and grad.is_contiguous()
    _assert_grad(grad, ref)
    loss2, grad2 = tim.distill_grad(z, ids, lp, w, 1.3, kind=kind, tail=tail)
    _assert_loss(loss2, None, ref, "grad")
    _assert_grad(grad2, ref, "grad")
    leaf = z.detach().clone().requires_grad_(True)
    loss3 = tim.distill_loss(leaf, ids, lp, 1.3, kind=kind, tail=tail)
    assert torch.equal(loss3.detach(), loss)
    loss3.backward(w)
    _assert_grad(leaf.grad, ref, "autograd")


@pytest.mark.parametrize("kind,tail", MODES)
def test_full_vocabulary(tim, kind, tail):
    z, ids, lp, w = _inputs(3, 151936, 64, "bf16", 5)
    z.scatter_(1, ids[:, :20].long(), z.gather(1, ids[:, :20].long()) + 12)
    ref = _reference(z, ids, lp, w, 1.0, kind, tail)
    loss, lse, saved = tim.distill(z, ids, lp, kind=kind, tail=tail)
    _assert_loss(loss, lse, ref)
    _assert_grad(tim.distill_backward(z, ids, lp, saved, w, kind=kind), ref)
    _assert_grad(tim.distill_grad(z, ids, lp, w, kind=kind, tail=tail)[1], ref)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("offset,pad,oo,op", [(0, 3, 0, 3), (1, 0, 0, 0), (3, 5, 3, 5), (2, 7, 5, 1),
                                              (8, 8, 8, 0)])
def test_rows_at_any_address(tim, dtype, offset, pad, oo, op):
    """Input and output windows of larger buffers; nothing around the output is touched."""
    import torch
    T, V = 4, 1013
    z, ids, lp, w = _inputs(T, V, 9, dtype, 3, pad=pad, offset=offset)
    ref = _reference(z, ids, lp, w, 0.8, "forward", True)
    loss, lse, saved = tim.distill(z, ids, lp, 0.8, tail=True)
    _assert_loss(loss, lse, ref)
    for fused in (False, True):
        buf = torch.full((T, oo + V + op), 5.0, dtype=z.dtype, device="cuda")
        out = buf[:, oo:oo + V]
        if fused:
            tim.distill_grad(z, ids, lp, w, 0.8, tail=True, out_dlogits=out)
        else:
            tim.distill_backward(z, ids, lp, saved, w, 0.8, out_dlogits=out)
        _assert_grad(out, ref, fused)
        assert bool((buf[:, :oo] == 5).all()) and bool((buf[:, oo + V:] == 5).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("offset,pad,oo,op", [(0, 1, 0, 0), (5, 2, 2, 1), (1, 2, 6, 1), (3, 4, 0, 7)])
def test_wide_rows_between_other_addresses(tim, dtype, offset, pad, oo, op):
    """Rows of several slices, each at another distance modulo 16 bytes from its gradient's."""
    import torch
    T, V = 9, 50021
    z, ids, lp, w = _inputs(T, V, 40, dtype, 4, pad=pad, offset=offset)
    ids[2] = -1
    w[5] = 0.0
    ref = _reference(z, ids, lp, w, 1.2, "reverse", True)
    loss, lse, saved = tim.distill(z, ids, lp, 1.2, kind="reverse", tail=True)
    _assert_loss(loss, lse, ref)
    for fused in (False, True):
        buf = torch.full((T, oo + V + op), 5.0, dtype=z.dtype, device="cuda")
        out = buf[:, oo:oo + V]
        if fused:
            tim.distill_grad(z, ids, lp, w, 1.2, kind="reverse", tail=True, out_dlogits=out)
        else:
            tim.distill_backward(z, ids, lp, saved, w, 1.2, kind="reverse", out_dlogits=out)
        _assert_grad(out, ref, fused)
        assert bool((buf[:, :oo] == 5).all()) and bool((buf[:, oo + V:] == 5).all())


@pytest.mark.parametrize("kind,tail", MODES)
def test_masks_and_empty_rows(tim, kind, tail):
    """Entries that are none, rows without entries (whose logits are not read), masked logits."""
    import torch
    z, ids, lp, w = _inputs(8, 3001, 24, "f32", 21, held=0.8)
    ids[1, 5:] = -1
    lp[2, 10:] = -math.inf
    ids[3] = -1
    z[3] = math.nan
    lp[4] = -math.inf
    z[4, 7] = math.inf
    out = torch.ones(3001, dtype=torch.bool, device="cuda")
    out[ids[5].long()] = False
    z[5, out] = -math.inf                      # no mass outside the head
    out[ids[6].long()] = False
    z[6, torch.arange(0, 3001, 2, device="cuda")[out[::2]]] = torch.finfo(torch.float32).min
    w[7] = 0.0
    ref = _reference(torch.nan_to_num(z, nan=0.0, posinf=0.0, neginf=-math.inf), ids, lp, w, 1.0, kind, tail)
    loss, lse, saved = tim.distill(z, ids, lp, kind=kind, tail=tail)
    _assert_loss(loss, lse, ref)
    assert loss[3] == 0 and lse[3] == 0 and loss[4] == 0
    for grad in (tim.distill_backward(z, ids, lp, saved, w, kind=kind),
                 tim.distill_grad(z, ids, lp, w, kind=kind, tail=tail)[1]):
        _assert_grad(grad, ref)
        assert not grad[3].any() and not grad[4].any() and not grad[7].any()


def test_complete_teacher_head_has_no_tail(tim):
    """q_r <= 2^-20 is the rounding of the teacher's own numbers: no bucket."""
    z, ids, lp, w = _inputs(4, 500, 40, "f32", 22, held=1.0)
    for kind in ("forward", "reverse"):
        a = tim.distill(z, ids, lp, kind=kind, tail=True)
        b = tim.distill(z, ids, lp, kind=kind, tail=False)
        assert all((x == y).all() for x, y in zip(a, b))


@pytest.mark.parametrize("tau", [1e-6, 0.05, 1.0, 40.0, 1e6])
def test_temperatures(tim, tau):
    z, ids, lp, w = _inputs(4, 2003, 16, "f32", 23)
    for kind, tail in MODES:
        if tau < 0.01 and kind == "forward":
            continue  # ln p_k of thousands of nats against a bar relative to the sum: see below
        ref = _reference(z, ids, lp, w, tau, kind, tail)
        loss, lse, saved = tim.distill(z, ids, lp, tau, kind=kind, tail=tail)
        d = np.abs(loss.cpu().numpy() - ref[0])
        # the double product z / tau is good to 2^-52 of itself
        assert np.all(d <= ref[3] + 2.0 ** -23 * np.abs(ref[0]) + 1e-9), (kind, tail, d)
        _assert_grad(tim.distill_backward(z, ids, lp, saved, w, tau, kind=kind), ref)


def test_infinite_loss_and_bad_rows_are_reported(tim):
    import torch
    z, ids, lp, w = _inputs(8, 700, 6, "f32", 24)
    good, _, _ = tim.distill(z, ids, lp)
    z[1, ids[1, 2].item()] = -math.inf          # the student gives a teacher's token nothing
    z[2, (ids[2, 0].item() + 1) % 700] = math.nan
    z[3, 5] = math.inf
    ids[4, 3] = 700
    ids[5, 1] = -2
    ids[6, 2] = ids[6, 0]
    lp[7, 0] = math.nan
    ws = tim.Workspace(1024)
    loss, lse, saved = tim.distill(z, ids, lp, workspace=ws, check=False)
    with pytest.raises(tim.TimError):
        ws.check()
    assert loss[0] == good[0] and loss[1] == math.inf
    assert all(math.isnan(loss[i]) for i in range(2, 8))
    w.fill_(1.0)
    w[4] = 0.0
    for grad in (tim.distill_backward(z, ids, lp, saved, w),
                 tim.distill_grad(z, ids, lp, w, workspace=ws, check=False)[1]):
        assert bool(grad[0].isfinite().all()) and bool(grad[1].isfinite().all())
        assert not grad[4].any() and bool(grad[5].isnan().all()) and bool(grad[6].isnan().all())
        assert bool(grad[7].isnan().all()) and bool(grad[2].isnan().any())
    ws.sync_status()
    for i, name in ((4, "TIM_ERR_TOKEN_RANGE"), (5, "TIM_ERR_TOKEN_RANGE"),
                    (6, "TIM_ERR_INVALID_ARG"), (7, "TIM_ERR_INVALID_ARG"), (1, "TIM_ERR_NONFINITE"),
                    (2, "TIM_ERR_NONFINITE"), (3, "TIM_ERR_NONFINITE")):
        with pytest.raises(tim.TimError, match=name):
            tim.distill(z[i:i + 1], ids[i:i + 1], lp[i:i + 1])
        with pytest.raises(tim.TimError, match=name):
            tim.distill_grad(z[i:i + 1], ids[i:i + 1], lp[i:i + 1], w[i:i + 1])
    with pytest.raises(tim.TimError, match="TIM_ERR_INVALID_ARG"):
        tim.distill_backward(z, ids, lp, saved, w, out_dlogits=z)
    with pytest.raises(ValueError):
        tim.distill(z, ids, lp[:, :3])
    with pytest.raises(ValueError):
        tim.distill(z, ids, lp, kind="both")
    with pytest.raises(ValueError):
        tim.distill_backward(z, ids, lp, saved, w, out_dlogits=torch.empty_like(z, dtype=torch.bfloat16))


@pytest.mark.parametrize("kind,tail", MODES)
def test_gradient_by_differences(tim, kind, tail):
    """Central differences of the kernel's own loss.  h = 2^-4: the loss's rounding, below
    2e-6, over 2h is 1.6e-5; the third derivative, below 2 (1 + |L|) p, adds h^2 / 6 of it."""
    import torch
    z, ids, lp, _ = _inputs(1, 40, 8, "f32", 25)
    one = torch.ones(1, device="cuda")
    grad = tim.distill_grad(z, ids, lp, one, kind=kind, tail=tail)[1][0]
    loss0 = float(tim.distill(z, ids, lp, kind=kind, tail=tail)[0])
    p = torch.softmax(z[0].double(), 0)
    h = 2.0 ** -4
    big = z.repeat(80, 1)
    for v in range(40):
        big[2 * v, v] += h
        big[2 * v + 1, v] -= h
    loss = tim.distill(big, ids.repeat(80, 1), lp.repeat(80, 1), kind=kind, tail=tail)[0].double()
    d = (loss[0::2] - loss[1::2]) / (2 * h)
    tol = 2e-5 + h * h / 6 * 8 * (1 + abs(loss0)) * p.clamp(min=0.01)
    assert bool(((d - grad.double()).abs() <= tol).all()), (d - grad).abs().max()


def test_graph_replay_with_a_living_eager_graph(tim):
    """Forward, backward and the fused call captured and replayed on other inputs; an eager
    autograd graph of the same leaf lives meanwhile."""
    import torch
    T, V, K = 7, 20011, 12
    z, ids, lp, w = _inputs(T, V, K, "bf16", 26)
    leaf = z.clone().requires_grad_(True)
    eager = tim.distill_loss(leaf, ids, lp, tail=True)
    ws = tim.Workspace(1024)
    zs = z.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        tim.distill(zs, ids, lp, tail=True, workspace=ws, check=False)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, lse, saved = tim.distill(zs, ids, lp, tail=True, workspace=ws, check=False)
        grad = tim.distill_backward(zs, ids, lp, saved, w)
        loss2, grad2 = tim.distill_grad(zs, ids, lp, w, tail=True, workspace=ws, check=False)
    for seed in (31, 32):
        zs.copy_(_inputs(T, V, K, "bf16", seed)[0])
        graph.replay()
        torch.cuda.synchronize()
        a = tim.distill(zs.clone(), ids, lp, tail=True)
        assert torch.equal(a[0], loss) and torch.equal(a[1], lse)
        assert torch.equal(tim.distill_backward(zs.clone(), ids, lp, a[2], w), grad)
        b = tim.distill_grad(zs.clone(), ids, lp, w, tail=True)
        assert torch.equal(b[0], loss2) and torch.equal(b[1], grad2)
    eager.backward(w)
    ref = _reference(leaf, ids, lp, w, 1.0, "forward", True)
    _assert_grad(leaf.grad, ref)


def test_row_results_do_not_depend_on_the_batch(tim):
    import torch
    z, ids, lp, w = _inputs(30, 151936, 50, "bf16", 27)
    whole = tim.distill(z, ids, lp, tail=True)
    dz = tim.distill_backward(z, ids, lp, whole[2], w)
    lw, gw = tim.distill_grad(z, ids, lp, w, tail=True)
    for i in (0, 13, 29):
        s = slice(i, i + 1)
        one = tim.distill(z[s], ids[s], lp[s], tail=True)
        assert all(torch.equal(a[s], b) for a, b in zip(whole, one))
        assert torch.equal(tim.distill_backward(z[s], ids[s], lp[s], one[2], w[s]), dz[s])
        l1, g1 = tim.distill_grad(z[s], ids[s], lp[s], w[s], tail=True)
        assert torch.equal(l1, lw[s]) and torch.equal(g1, gw[s])


def test_on_policy_distillation_run(tim):
    """The operators as they are used together: sample from the student's logits, score the
    tokens again from the hidden states, take the teacher's top-k head, and the loss with its
    gradient carried on through the student's head."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(5)
    T, d, V, K, tau, eps = 48, 256, 20000, 20, 0.8, 1e-6

    def model(seed):
        h = torch.randn(T, d, generator=g, device="cuda").bfloat16()
        W = (torch.randn(V, d, generator=g, device="cuda") * (2.0 / d ** 0.5)).bfloat16()
        return h, torch.ones(d, device="cuda").bfloat16(), W

    hs, gs, Ws = model(1)
    ht, gt, Wt = model(2)
    hf = hs.float()
    y = ((hf * torch.rsqrt(hf.square().mean(1, keepdim=True) + eps)) * gs.float()).bfloat16()
    W = Ws.clone().requires_grad_(True)
    logits = y.float() @ W.float().t()
    ids, lp_gen, lse_kept, kept = tim.sample(logits.detach(), torch.rand(T, generator=g, device="cuda"),
                                             tau, 50, 0.9)
    lp, lse, n = tim.processed_logprob(hs, gs, Ws, ids, tau, eps, 50, 0.9)
    # the same score from the hidden states: bf16 operands, fp32 sums in another order
    same = n == kept
    assert int(same.sum()) >= T - 2
    assert float((lp - lp_gen)[same].abs().max()) <= 2e-3
    *_, tids, tlp = tim.processed_logprob(ht, gt, Wt, ids, 1.0, eps, K, 0.95, head=True)
    loss = tim.distill_loss(logits, tids, tlp, tau, tail=True)
    loss.sum().backward()
    ref = _reference(logits, tids, tlp, torch.ones(T, device="cuda"), tau, "forward", True)
    _assert_loss(loss, None, ref)
    gz = torch.from_numpy(ref[2]).cuda()
    want = gz.t() @ y.double()
    bound = torch.from_numpy(ref[4]).cuda().t() @ y.double().abs()
    # bf16 gradient of W: half a step, and fp32 products summed over T = 48 rows
    err = (W.grad.double() - want).abs()
    assert bool((err <= bound + 2.0 ** -8 * want.abs() + 48 * 2.0 ** -23 * (gz.abs().t() @ y.double().abs()) + 1e-30).all())
