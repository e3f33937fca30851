"""tim.embed and tim.embed_backward on the GPU against the fp64 oracle.

The lookup is an fp32 product rounded once more to the type: |x| (2^-24 + u), u = half a step (in fp32
the product alone).  The gradient of a token with n rows is n - 1 additions in fp32, in whatever
order, and a product: (n + 1) 2^-24 scale sum |dy|, then the type's rounding; an addition to what is there is
one more of the result.  Below the normal numbers the rounding is half the smallest step.
"""
import math

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


def _dtype(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def _round(dtype):
    """Half a step relative to the value, and below the normal numbers."""
    import torch
    f = torch.finfo(dtype)
    return f.eps / 2, f.smallest_normal * f.eps / 2


def _tensor(rows, cols, dtype, seed, pad=0, offset=0, size=1.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.full((rows, offset + cols + pad), 77.0, dtype=_dtype(dtype), device="cuda")
    x = buf[:, offset:offset + cols]
    x.copy_(size * torch.randn(rows, cols, generator=g, device="cuda"))
    return x


def _ids(T, V, seed, kind="zipf"):
    import torch
    g = np.random.default_rng(seed)
    if kind == "zipf":
        ids = np.minimum((g.pareto(0.8, T) * 3).astype(np.int64), V - 1) * 31 % V
    elif kind == "one":
        ids = np.full(T, V // 2)
    elif kind == "distinct":
        ids = g.permutation(max(T, V))[:T] % V
    else:
        ids = g.integers(0, V, T)
    ids = np.where(g.random(T) < 0.1, -1, ids) if kind != "one" else ids
    return torch.from_numpy(ids.astype(np.int32)).cuda()


def _check_lookup(tim, table, ids, scale, **kw):
    got = tim.embed(table, ids, scale, **kw)
    want = oracle.ends.embed(table.double().cpu().numpy(), ids.cpu().numpy(), float(np.float32(scale)))
    u, floor = _round(table.dtype)
    tol = np.abs(want) * (u + (0 if u == 2.0 ** -24 else 2.0 ** -24 * 1.01)) + floor
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol)
    return got


def _check_grad(tim, dy, ids, V, scale, before=None, **kw):
    import torch
    want, size, n = oracle.ends.embed_backward(dy.double().cpu().numpy(), ids.cpu().numpy(), V,
                                               float(np.float32(scale)))
    if before is not None:
        kw.update(out_dtable=before.clone(), accumulate=True)
        want = want + before.double().cpu().numpy()
    got = tim.embed_backward(dy, ids, V, scale, **kw)
    u, floor = _round(got.dtype)
    tol = (n[:, None] + 1) * 2.0 ** -24 * size + u * np.abs(want) * (1 + 2.0 ** -7) + floor
    if got.dtype != torch.float32:
        tol = tol + 2.0 ** -24 * np.abs(want)
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol)
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("d", [1, 3, 8, 20, 63, 64, 513, 1000, 2056, 4096])
@pytest.mark.parametrize("T", [1, 2, 37])
def test_lookup_sizes(tim, dtype, d, T):
    table = _tensor(211, d, dtype, d)
    for scale in (1.0, 0.3, -7.5, 64.0):
        _check_lookup(tim, table, _ids(T, 211, T + d, "any"), scale)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("offset,pad", [(0, 3), (1, 0), (3, 5), (8, 8)])
def test_rows_at_any_address(tim, dtype, offset, pad):
    import torch
    table = _tensor(100, 264, dtype, 1, pad, offset)
    ids = _ids(50, 100, 2, "any")
    _check_lookup(tim, table, ids, 1.7)
    big = torch.full((54, offset + 264 + pad), 7.0, dtype=table.dtype, device="cuda")
    out = big[:50, offset:offset + 264]
    got = _check_lookup(tim, table, ids, 1.7, out=out)
    assert got.data_ptr() == out.data_ptr()
    big[:50, offset:offset + 264] = 7.0
    assert bool((big == 7.0).all())  # nothing beside the rows is written
    _check_grad(tim, _tensor(50, 264, dtype, 3, pad, offset), ids, 100, 0.7)
    _check_grad(tim, _tensor(50, 264, dtype, 3, pad, offset), ids, 100, 0.7, dtype=table.dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 33, 700, 4097])
@pytest.mark.parametrize("kind", ["zipf", "one", "distinct", "any"])
def test_gradient_sizes(tim, dtype, T, kind):
    for V, d in ((1, 8), (300, 24), (511, 7), (513, 16)):
        ids, dy = _ids(T, V, T + V, kind), _tensor(T, d, dtype, T + d)
        _check_grad(tim, dy, ids, V, 1.3)
        _check_grad(tim, dy, ids, V, 1.3, dtype=dy.dtype)


@pytest.mark.parametrize("out", ["f32", "own"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["zipf", "one", "any"])
def test_gradient_added_to_what_is_there(tim, dtype, out, kind):
    before = _tensor(400, 40, "f32" if out == "f32" else dtype, 5).contiguous()
    for T in (3, 900):
        _check_grad(tim, _tensor(T, 40, dtype, T), _ids(T, 400, T, kind), 400, 0.5, before=before)


@pytest.mark.parametrize("T", [4096, 8192, 8193, 20000, 32768, 32769, 131072, 131073, 270001])
def test_long_batches(tim, T):
    """Over every size of the sort's cluster and beyond one sort: small whole numbers add up exactly
    in fp32, so every sum has to be the exact one."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(T)
    for V, kind in ((151936, "zipf"), (700, "any"), (300000, "any")):
        ids = _ids(T, V, T, kind)
        dy = torch.randint(-8, 9, (T, 8), generator=g, device="cuda").to(torch.bfloat16)
        got = tim.embed_backward(dy, ids, V, 2.0)
        live = ids >= 0
        want = torch.zeros(V, 8, dtype=torch.float64, device="cuda")
        want.index_add_(0, ids[live].long(), 2.0 * dy[live].double())
        assert torch.equal(got.double(), want)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T", [131072, 131073, 262144, 270001, 700003])
def test_long_batches_are_rounded_once(tim, dtype, T):
    """Sums of small whole numbers are exact in fp32: in 16 bits too the result is the exact one rounded once,
    whatever sorts a token's rows went through, and so is what is added to a table's own."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(T)
    for V, kind, d in ((151936, "zipf", 8), (90, "any", 3), (5, "one", 16)):
        ids = _ids(T, V, T + d, kind)
        if kind == "one":
            ids = torch.where(torch.arange(T, device="cuda") % 3 == 0, ids, -1)
            ids[T // 2:] = 4
        dy = torch.randint(-8, 9, (T, d), generator=g, device="cuda").to(_dtype(dtype))
        before = torch.randint(-900, 900, (V, d), generator=g, device="cuda").to(_dtype(dtype))
        live = ids >= 0
        want = torch.zeros(V, d, dtype=torch.float64, device="cuda")
        want.index_add_(0, ids[live].long(), 0.5 * dy[live].double())
        for out in {torch.float32, dy.dtype}:
            got = tim.embed_backward(dy, ids, V, 0.5, dtype=out)
            assert torch.equal(got, want.to(out)), (V, kind, out)
            to = before.to(out, copy=True)
            got = tim.embed_backward(dy, ids, V, 0.5, out_dtable=to, accumulate=True)
            assert torch.equal(got, (before.double() + want).to(out)), (V, kind, out)


@pytest.mark.parametrize("T", [140000, 300000])
def test_long_batches_in_any_type_and_address(tim, T):
    for dtype in ("f32", "bf16", "f16"):
        for V, d, pad, offset, kind in ((300, 24, 3, 1, "zipf"), (1000, 264, 0, 0, "any"), (3, 40, 0, 0, "one")):
            if T > 200000 and d > 100:
                continue
            dy, ids = _tensor(T, d, dtype, T + d, pad, offset), _ids(T, V, T, kind)
            _check_grad(tim, dy, ids, V, 0.3)
            _check_grad(tim, dy, ids, V, 0.3, dtype=dy.dtype)


def test_long_batches_are_added_in_the_order_of_their_rows(tim):
    """Rows of one token in every sort: 1, 2^24 and -2^24 add up to 0 in this order alone.  Bad ids of any
    sort are reported."""
    import torch
    T, V = 400000, 1000
    ids = torch.arange(T, device="cuda").int() % (V - 1)
    dy = torch.zeros(T, 8, device="cuda")
    for at, x in ((1000, 1.0), (200000, 2.0 ** 24), (399999, -2.0 ** 24)):
        ids[at] = V - 1
        dy[at] = x
    assert not bool(tim.embed_backward(dy, ids, V).any())
    assert bool((tim.embed_backward(dy.flip(0), ids.flip(0).contiguous(), V)[V - 1] == 1).all())
    dy = _tensor(T, 8, "f32", 6)
    first = tim.embed_backward(dy, ids, V)
    ws = tim.Workspace(tim.embed_backward_workspace_size(T, V, 8))
    for _ in range(3):
        small = tim.embed_backward(dy[:9000], ids[:9000], V, workspace=ws)  # it serves smaller calls between
        assert torch.equal(first, tim.embed_backward(dy, ids, V, workspace=ws))
        assert torch.equal(small, tim.embed_backward(dy[:9000], ids[:9000], V))
    good = ids.clone()
    for at in (5, 131072, 399998):
        good[at], ids[at] = -1, V if at == 5 else -2
    got = tim.embed_backward(dy, ids, V, workspace=ws, check=False)
    with pytest.raises(tim.TimError, match="TIM_ERR_TOKEN_RANGE"):
        ws.check()
    assert torch.equal(got, tim.embed_backward(dy, good, V))


def test_order_is_the_batchs(tim):
    """Equal tokens are added in the order of their rows, so the result does not change with the run,
    and the sum of 1, 2^24, -2^24 in that order is 0."""
    import torch
    dy = torch.tensor([[1.0], [2.0 ** 24], [-2.0 ** 24]], device="cuda")
    ids = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert tim.embed_backward(dy, ids, 1).item() == 0.0
    assert tim.embed_backward(dy.flip(0), ids, 1).item() == 1.0
    dy, ids = _tensor(30000, 64, "f32", 8), _ids(30000, 5000, 9)
    first = tim.embed_backward(dy, ids, 5000)
    for _ in range(3):
        assert torch.equal(first, tim.embed_backward(dy, ids, 5000))


def test_none_and_masked(tim):
    """No token at all; one alone among none; infinities and NaN in rows of none."""
    import torch
    table = _tensor(50, 16, "bf16", 1)
    none = torch.full((40,), -1, dtype=torch.int32, device="cuda")
    assert bool((tim.embed(table, none) == 0).all())
    dy = _tensor(40, 16, "bf16", 2)
    dy[7] = math.nan
    dy[8] = math.inf
    assert bool((tim.embed_backward(dy, none, 50) == 0).all())
    none[20] = 49
    _check_grad(tim, torch.where(torch.arange(40, device="cuda")[:, None] == 20, dy, 0 * torch.nan_to_num(dy)),
                none, 50, 1.0)
    got = tim.embed_backward(dy, none, 50)
    assert torch.equal(got[49], dy[20].float()) and bool((got[:49] == 0).all())


def test_bad_ids_are_reported_and_leave_the_others(tim):
    import torch
    table, ids = _tensor(50, 24, "f32", 1), _ids(30, 50, 2, "any")
    dy = _tensor(30, 24, "f32", 3)
    good = ids.clone()
    good[[3, 9]] = -1
    ids[3], ids[9] = 50, -2
    ws = tim.Workspace(tim.embed_backward_workspace_size(30, 50, 24))
    out = tim.embed(table, ids, workspace=ws, check=False)
    with pytest.raises(tim.TimError, match="TIM_ERR_TOKEN_RANGE"):
        ws.check()
    want = tim.embed(table, good)
    assert bool(out[[3, 9]].isnan().all())
    out[[3, 9]] = 0.0
    assert torch.equal(out, want)
    got = tim.embed_backward(dy, ids, 50, workspace=ws, check=False)
    with pytest.raises(tim.TimError, match="TIM_ERR_TOKEN_RANGE"):
        ws.check()
    assert torch.equal(got, tim.embed_backward(dy, good, 50))
    with pytest.raises(tim.TimError, match="TIM_ERR_TOKEN_RANGE"):
        tim.embed(table, ids)


def test_refusals(tim):
    import torch
    table, ids = _tensor(50, 24, "f32", 1), _ids(30, 50, 2, "any")
    for bad in (lambda: tim.embed(table.t(), ids), lambda: tim.embed(table, ids.long()),
                lambda: tim.embed(table, ids, out=torch.empty(30, 23, device="cuda")),
                lambda: tim.embed(table, ids, out=torch.empty(30, 24, device="cuda").half()),
                lambda: tim.embed_backward(table, ids, 50),
                lambda: tim.embed_backward(table[:30], ids, 50, accumulate=True),
                lambda: tim.embed_backward(table[:30], ids, 50, dtype=torch.float16),
                lambda: tim.embed_backward(table[:30], ids, 50, out_dtable=table[:, :12])):
        with pytest.raises((ValueError, TypeError)):
            bad()
    for bad in (lambda: tim.embed(table, ids, out=table[:30]), lambda: tim.embed(table, ids, math.inf),
                lambda: tim.embed(table, ids[:0]),
                lambda: tim.embed_backward(table[:30], ids, 50, out_dtable=table)):
        with pytest.raises(tim.TimError):
            bad()
    with pytest.raises(tim.TimError, match="TIM_ERR_WORKSPACE"):
        tim.embed_backward(table[:30], ids, 50, workspace=tim.Workspace(1024))


def test_autograd(tim):
    """The gradient in the table's type, of a gradient whose rows are not contiguous, against
    differences: the lookup is linear, so they are exact up to rounding."""
    import torch
    for dtype in ("f32", "bf16"):
        table = _tensor(60, 16, dtype, 1).contiguous().requires_grad_(True)
        ids = _ids(200, 60, 2)
        w = _tensor(16, 200, dtype, 3).t()  # columns contiguous
        out = tim.embedding(table, ids, 4.0)
        (out * w).sum().backward()
        want, size, n = oracle.ends.embed_backward(w.double().cpu().numpy(), ids.cpu().numpy(), 60, 4.0)
        u, _ = _round(table.dtype)
        tol = (n[:, None] + 1) * 2.0 ** -24 * size + (u + 2.0 ** -24) * np.abs(want)
        assert table.grad.dtype == table.dtype
        assert np.all(np.abs(table.grad.double().cpu().numpy() - want) <= tol)
    table = torch.randn(7, 3, device="cuda").requires_grad_(True)
    ids = torch.tensor([0, 2, 2, -1, 6], dtype=torch.int32, device="cuda")
    w = torch.randn(5, 3, device="cuda", dtype=torch.float64)
    grad, = torch.autograd.grad((tim.embedding(table, ids, 0.5).double() * w).sum(), table)
    for v in range(7):
        for i in range(3):
            step = torch.zeros_like(table)
            step[v, i] = 0.5
            with torch.no_grad():
                diff = ((tim.embedding(table + step, ids, 0.5).double() * w).sum()
                        - (tim.embedding(table - step, ids, 0.5).double() * w).sum())
            # two lookups of numbers below 8, each off by 2^-24 of them, times weights below 8 a token
            assert abs(diff.item() - grad[v, i].item()) < 5 * 2 * 8 * 8 * 2.0 ** -24 + 1e-6


def test_graph_replay_streams_and_two_calls_at_once(tim):
    import torch
    T, V, d = 3000, 4000, 72
    table, dy = _tensor(V, d, "bf16", 1).contiguous(), _tensor(T, d, "bf16", 2).contiguous()
    ids = _ids(T, V, 3)
    ws = tim.Workspace(tim.embed_backward_workspace_size(T, V, d))
    out = torch.full((T + 2, d), 7.0, dtype=torch.bfloat16, device="cuda")
    grad = torch.empty(V, d, device="cuda")
    graph = torch.cuda.CUDAGraph()

    def step():
        tim.embed(table, ids, 3.0, out=out[:T], workspace=ws, check=False)
        tim.embed_backward(dy, ids, V, 3.0, out_dtable=grad, workspace=ws, check=False)

    step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        ids.copy_(_ids(T, V, 50 + seed))
        dy.copy_(_tensor(T, d, "bf16", 60 + seed))
        graph.replay()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        assert torch.equal(out[:T], tim.embed(table, ids, 3.0, stream=side))
        assert torch.equal(grad, tim.embed_backward(dy, ids, V, 3.0, stream=side))
    assert bool((out[T:] == 7).all())
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [tim.Workspace(ws.nbytes) for _ in range(2)]
    cases = [(ids, dy), (_ids(T, V, 99), _tensor(T, d, "bf16", 98))]
    want = [tim.embed_backward(g, i, V) for i, g in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(6):
        for n, (i, g) in enumerate(cases):
            got[n].append(tim.embed_backward(g, i, V, workspace=spaces[n], stream=streams[n], check=False))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[n]) for n in range(2) for x in got[n])


def test_long_batch_replayed_and_on_another_stream(tim):
    """Several sorts and their merges in a captured graph, whose inputs change between replays."""
    import torch
    T, V, d = 300000, 4000, 24
    dy, ids, grad = _tensor(T, d, "bf16", 2).contiguous(), _ids(T, V, 3), torch.zeros(V, d, device="cuda")
    ws = tim.Workspace(tim.embed_backward_workspace_size(T, V, d))

    def step():
        tim.embed_backward(dy, ids, V, 3.0, out_dtable=grad, workspace=ws, check=False)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        ids.copy_(_ids(T, V, 50 + seed, "zipf" if seed == 1 else "any"))
        dy.copy_(_tensor(T, d, "bf16", 60 + seed))
        graph.replay()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        assert torch.equal(grad, tim.embed_backward(dy, ids, V, 3.0, stream=side))
    streams = [torch.cuda.Stream() for _ in range(2)]
    cases = [(ids, dy), (_ids(T, V, 99), _tensor(T, d, "bf16", 98))]
    want = [tim.embed_backward(g, i, V) for i, g in cases]
    torch.cuda.synchronize()
    got = [[tim.embed_backward(g, i, V, stream=streams[n], check=False) for n, (i, g) in enumerate(cases)]
           for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, w) for pair in got for x, w in zip(pair, want))


def test_tied_to_the_head(tim):
    """The other half of a tied matrix's gradient, added to the head's."""
    import torch
    T, d, V = 96, 64, 500
    hidden, gamma = _tensor(T, d, "bf16", 1).contiguous(), torch.ones(d, device="cuda", dtype=torch.bfloat16)
    W, ids = _tensor(V, d, "bf16", 2, size=0.1).contiguous(), _ids(T, V, 3, "any").clamp(min=0)
    _, lse, _ = tim.logprob(hidden, gamma, W, ids, 1.0, 1e-6)
    g = torch.randn(T, device="cuda")
    _, dW = tim.logprob_backward(hidden, gamma, W, ids, lse, g, 1.0, 1e-6)
    _check_grad(tim, _tensor(T, d, "bf16", 4), ids, V, 8.0, before=dW)


@pytest.mark.slow
def test_beyond_2_31_elements(tim):
    """Table, output and gradient of more than 2^31 elements: offsets need 64 bits."""
    import torch
    V, d = 530000, 4104
    table = torch.empty(V, d, dtype=torch.bfloat16, device="cuda")
    for v in range(0, V, 53000):
        table[v:v + 53000] = torch.arange(v, v + 53000, device="cuda")[:, None] % 251
    ids = torch.tensor([0, V - 1, 523300, -1, V - 1], dtype=torch.int32, device="cuda")
    out = tim.embed(table, ids)
    want = (ids.long() % 251).to(torch.bfloat16)[:, None] * (ids >= 0)[:, None]
    assert torch.equal(out, want.expand(5, d))
    table.fill_(7.0)
    tim.embed_backward(out, ids, V, dtype=torch.bfloat16, out_dtable=table)
    assert torch.equal(table[V - 1], 2 * out[1]) and torch.equal(table[523300], out[2])
    table[V - 1] = 0
    table[523300] = 0
    assert not bool(table.any())  # the others, token 0's among them, are 0


@pytest.mark.slow
def test_gradient_of_a_long_batch_beyond_2_31_elements(tim):
    """Rows beyond 2^31 elements of dy, of tokens that lie in several sorts and in one."""
    import torch
    T, V, d = 600000, 5000, 4104
    dy = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    ids = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    at = torch.tensor([0, 3, 140000, 523300, T - 3, T - 1], device="cuda")
    ids[at] = torch.tensor([4999, 7, 7, 7, 4999, 123], dtype=torch.int32, device="cuda")
    dy[at] = torch.tensor([1, 2, 4, 8, 16, 32], dtype=torch.bfloat16, device="cuda")[:, None]
    dy[1] = math.nan  # no token's
    for out in (torch.bfloat16, torch.float32):
        got = tim.embed_backward(dy, ids, V, 3.0, dtype=out)
        for v, want in ((4999, 51.0), (7, 42.0), (123, 96.0)):
            assert bool((got[v] == want).all()), (v, out)
            got[v] = 0
        assert not bool(got.any())
