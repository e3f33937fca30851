"""The logits operators on a matrix of more than 2^31 elements: its last rows, and some in the middle,
give what they give alone, and no other row's gradient is written."""
import pytest

from test_gpu_distill import tim  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def test_rows_beyond_32_bit_offsets(tim):  # noqa: F811
    import torch
    T, V, K = 14400, 151936, 16
    assert T * V > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(3)
    z = torch.empty(T, V, dtype=torch.bfloat16, device="cuda")
    for i in range(0, T, 1200):
        z[i:i + 1200] = torch.randn(1200, V, generator=g, device="cuda") * 2
    u = torch.rand(T, generator=g, device="cuda")
    ids = torch.randint(0, V // K, (T, K), generator=g, device="cuda")
    ids = (ids + torch.arange(K, device="cuda") * (V // K)).int()
    lp = torch.log_softmax(torch.randn(T, K, generator=g, device="cuda"), 1) - 0.1
    w = torch.rand(T, generator=g, device="cuda")
    rows = [0, 7000, T - 2, T - 1]
    for kw in (dict(), dict(top_k=40, top_p=0.9), dict(top_p=0.9)):
        whole = tim.sample(z, u, **kw)
        for i in rows:
            one = tim.sample(z[i:i + 1], u[i:i + 1], **kw)
            assert one[0][0] == whole[0][i] and one[3][0] == whole[3][i]
            # half a step of each of the two roundings, and the sums' 2^-29 (see the sampler's tests)
            for a, b in ((one[1][0], whole[1][i]), (one[2][0], whole[2][i])):
                assert abs(float(a) - float(b)) <= 2.0 ** -23 * abs(float(b)) + 2.0 ** -28
    loss, lse, saved = tim.distill(z, ids, lp, tail=True)
    grad = tim.distill_backward(z, ids, lp, saved, w)
    fused_loss, fused = tim.distill_grad(z, ids, lp, w, tail=True)
    for i in rows:
        s = slice(i, i + 1)
        a = tim.distill(z[s], ids[s], lp[s], tail=True)
        assert torch.equal(a[0], loss[s]) and torch.equal(a[1], lse[s])
        assert torch.equal(tim.distill_backward(z[s], ids[s], lp[s], a[2], w[s]), grad[s])
        b = tim.distill_grad(z[s], ids[s], lp[s], w[s], tail=True)
        assert torch.equal(b[0], fused_loss[s]) and torch.equal(b[1], fused[s])
