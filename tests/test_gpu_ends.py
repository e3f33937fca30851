"""The operators at a model's two ends in a run of all together, as a tied-weight model uses them: a decoding
loop that drafts, verifies and looks the accepted tokens up, and a training step whose matrix is embedding
and LM head at once."""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tim():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import rollout_logprob_consistency_gb300 as tim
    return tim


def _model(seed, V=1000, d=128):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*size, s=1.0):
        return (s * torch.randn(*size, generator=g, device="cuda")).to(torch.bfloat16)

    return dict(W=rand(V, d, s=0.2), block=rand(d, d, s=0.1), gamma=rand(d), gamma_post=rand(d), gate=rand(d, s=0.5))


def _hidden(tim, m, ids, scale):
    """A token's hidden state and its norm: lookup, a block of one product, residual update."""
    e = tim.embed(m["W"], ids, scale)
    return tim.residual_norm(e, e @ m["block"], m["gamma"], 1e-6, gamma_post=m["gamma_post"], gate=m["gate"], scale=0.5)


def test_decoding_with_drafts_scores_as_the_trainer(tim):
    """Draft with a smaller model, verify with the larger: the logprobs of the accepted tokens are what
    tim_processed_logprob gives for the hidden states the decoding had, up to the logits' rounding to bf16."""
    import torch
    torch.manual_seed(3)
    B, N, V, scale = 12, 3, 1000, 8.0
    big = _model(1)
    small = {**big, "block": big["block"] + 0.1 * _model(2)["block"]}  # a drafter that nearly agrees
    kw = dict(temperature=0.8, top_k=40, top_p=0.95)
    last = torch.randint(0, V, (B,), device="cuda", dtype=torch.int32)
    accepted = 0
    for _ in range(6):
        ids = torch.empty(B, N, dtype=torch.int32, device="cuda")
        draft = torch.empty(N, B, V, dtype=torch.float32, device="cuda").transpose(0, 1)
        x = last
        for j in range(N):
            draft[:, j] = (_hidden(tim, small, x, scale)[1] @ big["W"].t()).float()
            x = ids[:, j] = tim.sample(draft[:, j], torch.rand(B, device="cuda"), **kw)[0]
        context = torch.cat([last.view(B, 1), ids], 1).contiguous()
        h, y = _hidden(tim, big, context.view(-1), scale)
        logits = (y.float() @ big["W"].float().t()).view(B, N + 1, V)
        out, lp, n = tim.verify(logits, ids, torch.rand(B, N, device="cuda"), torch.rand(B, device="cuda"), draft, **kw)
        score, _, kept = tim.processed_logprob(h, big["gamma"], big["W"], out.view(-1).clamp(min=0).contiguous(),
                                               0.8, 1e-6, 40, 0.95)
        live = (out >= 0).view(-1)
        # Both norms round y to bf16, from sums in different orders: an element in a thousand may come out
        # a step of 2^-7 |y| apart, with |y| up to 6 and |W| up to 0.8 below 2^-4.7 of a logit; the fp32
        # products in different orders are far below that.  A border of top-p that lies within moves a
        # token's share of the mass, so nine in ten rows are compared.
        diff = (score[live] - lp.view(-1)[live]).abs()
        assert float((diff < 2.0 ** -4).float().mean()) > 0.9
        assert bool(((out >= 0).sum(1) == n + 1).all())
        accepted += int(n.sum())
        last = out.gather(1, n.long().view(B, 1)).view(B).contiguous()
        assert bool(((last >= 0) & (last < V)).all())
    assert accepted > 0


def test_training_step_with_a_tied_matrix(tim):
    """Loss of the selected logprobs through head, residual update, block and embedding: the gradient of the
    tied matrix, by the differentiable calls and by the calls themselves, against a chain in 64 bits."""
    import torch
    T, V, d, scale = 60, 300, 64, 4.0
    m = _model(5, V, d)
    g = torch.Generator(device="cuda").manual_seed(6)
    ids = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    ids[5:9] = -1
    target = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    w = torch.rand(T, generator=g, device="cuda")
    W = m["W"].clone().requires_grad_(True)
    post = m["gamma_post"].clone().requires_grad_(True)
    e = tim.embedding(W, ids, scale)
    h, _ = tim.block_residual(e, e @ m["block"], None, 1e-6, gamma_post=post, gate=m["gate"], scale=0.5)
    lp = tim.linear_logprob(h, m["gamma"], W, target, 1.0, 1e-6)
    dW, dpost = torch.autograd.grad((lp * w).sum(), (W, post))

    # the calls themselves, the head's dW and the embedding's in one fp32 matrix
    e = tim.embed(m["W"], ids, scale)
    x = e @ m["block"]
    h, _ = tim.residual_norm(e, x, None, 1e-6, gamma_post=m["gamma_post"], gate=m["gate"], scale=0.5)
    _, lse, _ = tim.logprob(h, m["gamma"], m["W"], target, 1.0, 1e-6)
    dy, total = tim.logprob_backward(h, m["gamma"], m["W"], target, lse, w, 1.0, 1e-6)
    dh, _ = tim.rmsnorm_backward(h, m["gamma"], dy, 1e-6)
    de, dx, _, dpost2, _ = tim.residual_norm_backward(h, x, dh.to(h.dtype), None, None, 1e-6,
                                                      gamma_post=m["gamma_post"], gate=m["gate"], scale=0.5)
    de = de + dx @ m["block"].t()
    tim.embed_backward(de, ids, V, scale, out_dtable=total, accumulate=True)
    assert torch.equal(dpost, dpost2.to(dpost.dtype))
    # autograd rounds the two halves to bf16 and adds them: half a step of each and of the sum
    half = 2.0 ** -8
    head = tim.logprob_backward(h, m["gamma"], m["W"], target, lse, w, 1.0, 1e-6)[1]
    size = head.abs() + (total - head).abs() + total.abs()
    assert bool(((dW.float() - total).abs() <= half * size * 1.01 + 1e-6).all())

    # in 64 bits, every rounding to bf16 passed over: five of 2^-8 of the terms on the way there and back
    # (e, x, h, y, and G, dh, de), each of a vector of which a product takes the root mean square: compared
    # in norm
    W64 = m["W"].double().requires_grad_(True)
    e = torch.where((ids >= 0).view(T, 1), W64[ids.clamp(min=0).long()] * scale, torch.zeros((), dtype=torch.float64, device="cuda"))
    x = e @ m["block"].double()
    n = x / (x.pow(2).mean(1, keepdim=True) + 1e-6).sqrt() * m["gamma_post"].double()
    h = e + 0.5 * m["gate"].double() * n
    y = h / (h.pow(2).mean(1, keepdim=True) + 1e-6).sqrt() * m["gamma"].double()
    lp = torch.log_softmax(y @ W64.t(), 1).gather(1, target.long().view(T, 1)).view(T)
    want, = torch.autograd.grad((lp * w.double()).sum(), W64)
    assert float((total.double() - want).norm() / want.norm()) < 8 * 2.0 ** -8
