"""tim.sample on the GPU against the fp64 oracle.

Tokens and kept counts have to be the oracle's wherever no border of a decision lies within
MARGIN of the mass it is compared with.  The bar: every weight is good to 2^-30.5 relative, the
sums are integers of at least 2^50 with a floor of at most one unit a token (V 2^-50 < 2^-31.4),
so two sides of a border are each good to 2^-29.9: 2 x 2^-29.9 < 2e-9.  A row within that margin
is not compared.
logprob and lse are computed as pairs of floats from such sums and rounded once to fp32: half a
step of the value, plus 2^-29.9 for the sum, plus the pairs' roundings (below 2^-40):
tol = 2^-24 |x| + 2^-29.
"""
import math

import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

MARGIN = 2e-9


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


def _logits(T, V, dtype, seed, scale=3.0, pad=0, offset=0):
    """[T, V] on the GPU, as a window of a larger buffer when pad or offset is given."""
    import torch
    g = np.random.default_rng(seed)
    z = (g.normal(size=(T, V)) * scale).astype(np.float32)
    buf = torch.full((T, offset + V + pad), 77.0, dtype=_dtype(dtype), device="cuda")
    buf[:, offset:offset + V] = torch.from_numpy(z).cuda().to(_dtype(dtype))
    return buf[:, offset:offset + V]


def _check(tim, z, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, least=None, **kw):
    import torch
    T = z.shape[0]
    ut = torch.tensor(np.asarray(u, dtype=np.float32), device="cuda")
    got = [t.cpu().numpy() for t in tim.sample(z, ut, temperature, top_k, top_p, min_p, **kw)]

    def at(v, i):
        return v[i].item() if isinstance(v, torch.Tensor) else float(np.float32(v))

    zh, compared = z.double().cpu().numpy(), 0
    for i in range(T):
        r = oracle.sample_row(zh[i], float(np.float32(u[i])), at(temperature, i), int(at(top_k, i)),
                              at(top_p, i), at(min_p, i))
        if r["margin"] < MARGIN:
            continue
        compared += 1
        assert got[0][i] == r["id"], (i, r, [g[i] for g in got])
        assert got[3][i] == r["kept"], (i, r, [g[i] for g in got])
        for g, w in ((got[1][i], r["logprob"]), (got[2][i], r["lse"])):
            assert abs(float(g) - w) <= 2.0 ** -24 * abs(w) + 2.0 ** -29, (i, r, [x[i] for x in got])
    assert compared >= (T if least is None else least)
    return got


SETTINGS = [dict(), dict(temperature=0.7, top_k=5, top_p=0.9), dict(top_p=0.5),
            dict(temperature=1.7, top_p=0.99, min_p=0.01), dict(top_k=1), dict(top_k=40),
            dict(min_p=0.3), dict(temperature=0.0), dict(temperature=0.2, top_k=700)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 31, 255, 1000, 4097, 32003])
def test_sizes_and_settings(tim, dtype, V):
    u = np.random.default_rng(V).random(6).astype(np.float32)
    for n, kw in enumerate(SETTINGS):
        _check(tim, _logits(6, V, dtype, 100 * V + n), u, **kw)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_full_vocabulary_peaked_and_flat(tim, dtype):
    import torch
    V = 151936
    z = _logits(8, V, dtype, 5, scale=1.0)
    g = torch.Generator(device="cuda").manual_seed(3)
    at = torch.randint(0, V, (4, 100), device="cuda", generator=g)
    boost = 18.0 - 2.0 * torch.arange(1, 101, device="cuda").log()
    z[:4].scatter_(1, at, boost.to(z.dtype).expand(4, 100))
    u = np.random.default_rng(9).random(8).astype(np.float32)
    for kw in (dict(), dict(temperature=0.7, top_p=0.95), dict(temperature=0.7, top_k=50, top_p=0.95),
               dict(top_p=0.9, min_p=0.001), dict(min_p=0.05), dict(top_k=20000, top_p=0.8),
               dict(temperature=1.5, top_p=0.999)):
        _check(tim, z, u, **kw)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("offset,pad", [(0, 3), (1, 0), (3, 5), (8, 8)])
def test_rows_at_any_address(tim, dtype, offset, pad):
    u = np.random.default_rng(2).random(5).astype(np.float32)
    z = _logits(5, 1013, dtype, 7, offset=offset, pad=pad)
    for kw in SETTINGS[:4]:
        _check(tim, z, u, **kw)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_ties_go_to_the_lower_id(tim, dtype):
    import torch
    g = np.random.default_rng(4)
    z = torch.from_numpy(g.integers(-3, 4, size=(8, 3001)).astype(np.float32)).cuda().to(_dtype(dtype))
    u = g.random(8).astype(np.float32)
    for kw in (dict(top_k=10), dict(top_k=1000), dict(top_p=0.3), dict(top_k=600, top_p=0.7),
               dict(min_p=1.0), dict(temperature=0.0), dict(top_p=0.9, min_p=0.5)):
        _check(tim, z, u, **kw)
    same = torch.zeros(3, 5000, device="cuda", dtype=_dtype(dtype))  # one value alone
    # top-p on equal tokens: the border falls on a multiple of 1/5000 only by its rounding
    for kw in (dict(), dict(top_k=7), dict(top_k=4999), dict(top_p=0.50013), dict(min_p=1.0)):
        _check(tim, same, [0.1234567, 0.70001, 0.99], **kw)
    zero = torch.zeros(1, 64, device="cuda", dtype=_dtype(dtype))
    zero[0, ::2] = -0.0  # equal to +0
    assert _check(tim, zero, [0.0], top_k=3)[0][0] == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_masked_tokens(tim, dtype):
    import torch
    z = _logits(6, 4100, dtype, 11)
    low = torch.finfo(z.dtype).min
    keep = torch.zeros(4100, dtype=torch.bool, device="cuda")
    keep[torch.tensor([5, 700, 701, 4099], device="cuda")] = True
    z[0:2, ~keep] = -math.inf
    z[2:4, ~keep] = low
    z[4] = low
    z[5] = -math.inf
    z[5, 4000] = low
    u = [0.0, 0.99, 0.4, 0.7, 0.5, 0.5]
    for kw in (dict(), dict(top_k=2), dict(top_k=50), dict(top_p=0.9), dict(min_p=0.1),
               dict(temperature=0.0)):
        # row 4 is 4100 equal tokens: u = 1/2 of them, or of 50 or 2 of them, is a border itself
        got = _check(tim, z, u, least=5, **kw)
        assert all(i in (5, 700, 701, 4099) for i in got[0][:4])
        assert got[0][5] == 4000 and got[3][5] == 1


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_extreme_scales(tim, dtype):
    z = _logits(6, 2003, dtype, 13, scale=3000.0)
    u = np.random.default_rng(6).random(6).astype(np.float32)
    for t in (1e-6, 1e-3, 0.5, 30.0, 1e4, 1e6):
        for kw in (dict(), dict(top_p=0.9), dict(top_k=9), dict(min_p=0.2)):
            _check(tim, z, u, temperature=t, **kw)
    z = _logits(4, 2003, dtype, 14, scale=1e-4)
    _check(tim, z, u[:4], top_p=0.6)
    _check(tim, z, u[:4], temperature=1e-6)


def test_uniform_ends(tim):
    z = _logits(2, 5003, "f32", 15)
    last = float(np.float32(1.0) - np.float32(2.0 ** -24))
    for kw in (dict(), dict(top_k=10), dict(top_p=0.7), dict(min_p=0.1)):
        _check(tim, z, [0.0, last], **kw)


def test_settings_a_row(tim):
    import torch
    T, V = 64, 20011
    z = _logits(T, V, "bf16", 16)
    g = np.random.default_rng(8)
    t = torch.tensor(g.choice([0.0, 0.5, 0.7, 1.0, 1.4], T).astype(np.float32), device="cuda")
    k = torch.tensor(g.choice([-1, 0, 1, 20, 50, 3000, 40000], T).astype(np.int32), device="cuda")
    p = torch.tensor(g.choice([0.1, 0.9, 0.95, 1.0, 2.0], T).astype(np.float32), device="cuda")
    m = torch.tensor(g.choice([0.0, 0.05, 1.0], T).astype(np.float32), device="cuda")
    _check(tim, z, g.random(T).astype(np.float32), t, k, p, m)


def test_bad_rows_are_reported_and_leave_the_others(tim):
    import torch
    z = _logits(7, 999, "f32", 17)
    want = tim.sample(z, torch.full((7,), 0.5, device="cuda"))
    z[1, 500] = math.nan
    z[2, 0] = math.inf
    z[3] = -math.inf
    u = torch.tensor([0.5, 0.5, 0.5, 0.5, 1.0, -0.1, 0.5], device="cuda")
    ws = tim.Workspace(1024)
    got = tim.sample(z, u, workspace=ws, check=False)
    with pytest.raises(tim.TimError):
        ws.check()
    for i in (0, 6):
        assert [g[i].item() for g in got] == [w[i].item() for w in want]
    for i in range(1, 6):
        assert got[0][i] == -1 and got[3][i] == 0
        assert math.isnan(got[1][i]) and math.isnan(got[2][i])
    for bad, code in ((dict(temperature=torch.tensor([-1.0] * 7, device="cuda")), "TIM_ERR_INVALID_ARG"),
                      (dict(top_p=torch.tensor([math.nan] * 7, device="cuda")), "TIM_ERR_INVALID_ARG"),
                      (dict(min_p=torch.tensor([1.5] * 7, device="cuda")), "TIM_ERR_INVALID_ARG")):
        with pytest.raises(tim.TimError, match=code):
            tim.sample(z[:7], u, **bad)
    with pytest.raises(tim.TimError, match="TIM_ERR_NONFINITE"):
        tim.sample(z[3:4], u[:1])
    with pytest.raises(ValueError):
        tim.sample(z.t(), u)
    with pytest.raises(ValueError):
        tim.sample(z, u[:3])


def test_graph_replay_streams_and_outputs(tim):
    """Captured once, replayed on other inputs; on another stream; into the caller's tensors.
    Rows behind the batch are left as they were."""
    import torch
    T, V = 9, 30011
    z = _logits(T, V, "bf16", 18)
    u = torch.rand(T, device="cuda")
    ws = tim.Workspace(1024)
    big = [torch.full((T + 3,), 7, dtype=d, device="cuda")
           for d in (torch.int32, torch.float32, torch.float32, torch.int32)]
    out = tuple(t[:T] for t in big)
    kw = dict(temperature=0.8, top_k=30, top_p=0.9, workspace=ws, check=False)
    tim.sample(z, u, out=out, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tim.sample(z, u, out=out, **kw)
    for seed in (1, 2):
        z.copy_(_logits(T, V, "bf16", 100 + seed))
        u.uniform_()
        graph.replay()
        torch.cuda.synchronize()
        direct = tim.sample(z.clone(), u.clone(), 0.8, 30, 0.9)
        assert all(torch.equal(a, b) for a, b in zip(out, direct))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        other = tim.sample(z, u, 0.8, 30, 0.9, stream=side)
        assert all(torch.equal(a, b) for a, b in zip(out, other))
    assert all(bool((t[T:] == 7).all()) for t in big)


def test_row_results_do_not_depend_on_the_batch(tim):
    import torch
    z = _logits(40, 151936, "bf16", 19)
    u = torch.rand(40, device="cuda")
    for kw in (dict(), dict(top_p=0.9), dict(top_k=50, top_p=0.9)):
        whole = tim.sample(z, u, **kw)
        for i in (0, 17, 39):
            one = tim.sample(z[i:i + 1], u[i:i + 1], **kw)
            assert all(torch.equal(a[i:i + 1], b) for a, b in zip(whole, one))


# A row has 1024, 512, 256 or 128 threads as there are more rows than once, twice or four times the
# SMs (152); the rows of a batch are compared where they are few and by sample where they are many.
MANY = [dict(top_k=50, top_p=0.95, temperature=0.7), dict(top_k=200, top_p=0.9), dict(top_k=900, top_p=0.9),
        dict(top_p=0.9, temperature=0.5), dict(top_p=0.99), dict(min_p=0.1), dict(top_p=0.8, min_p=0.2),
        dict()]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,V", [(152, 9001), (153, 9001), (305, 6007), (609, 6007), (1300, 257)])
def test_many_rows(tim, dtype, T, V):
    import torch
    base = _logits(24, V, dtype, 1000 + T, scale=2.5)
    u = np.random.default_rng(T).random(24).astype(np.float32)
    at = torch.arange(T, device="cuda") % 24
    z, ut = base[at].contiguous(), torch.from_numpy(u).cuda()[at]
    for kw in MANY:
        # 24 rows against the oracle; as a batch the same rows over and over, at every place
        want = _check(tim, base, u, **kw)
        got = tim.sample(z, ut, **kw)
        for g, w in zip(got, want):
            assert torch.equal(g, torch.from_numpy(w).cuda()[at]), kw


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [12, 200, 400, 700])
@pytest.mark.parametrize("rank", [60, 300, 2500])
def test_top_p_on_a_border(tim, dtype, T, rank):
    """top-p is the float32 next to the mass of a row's first `rank` tokens: between border and p
    lie some 2^-26 of the mass, within what a float32 sum leaves open and far outside MARGIN."""
    import torch
    n = 12
    base = _logits(n, 6007, dtype, 77, scale=2.0)
    u = np.random.default_rng(78).random(n).astype(np.float32)
    zh = base.double().cpu().numpy()
    p = np.empty(n, np.float32)
    for i in range(n):
        e = np.sort(np.exp(zh[i] - zh[i].max()))[::-1]
        p[i] = e[:rank].sum() / e.sum()
    at = torch.arange(T, device="cuda") % n
    want = _check(tim, base, u, top_p=torch.from_numpy(p).cuda(), least=n - 3)
    got = tim.sample(base[at].contiguous(), torch.from_numpy(u).cuda()[at],
                     top_p=torch.from_numpy(p).cuda()[at])
    for g, w in zip(got, want):
        assert torch.equal(g, torch.from_numpy(w).cuda()[at])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_largest_vocabulary(tim, dtype):
    import torch
    V = 393216
    z = _logits(3, V, dtype, 21)
    u = np.random.default_rng(22).random(3).astype(np.float32)
    for kw in (dict(), dict(top_p=0.9), dict(top_p=0.99), dict(top_k=50, top_p=0.9),
               dict(top_k=200000, top_p=0.9), dict(min_p=0.02)):
        _check(tim, z, u, **kw)
    with pytest.raises(tim.TimError, match="TIM_ERR_SHAPE"):
        tim.sample(torch.zeros(1, V + 1, device="cuda"), torch.zeros(1, device="cuda"))


def test_one_workspace_for_calls_of_all_sizes_in_turn(tim):
    """Nothing of a call is left in the workspace: calls of other sizes and settings in turn with
    one workspace, scoring's included, give what they give with their own."""
    import torch
    ws = tim.Workspace(1024)
    for T, V, kw in ((700, 5003, dict(top_p=0.97)), (3, 151936, dict(top_p=0.99)), (200, 999, dict()),
                     (40, 50257, dict(top_k=2000, top_p=0.9)), (1, 1, dict(top_k=1)),
                     (700, 5003, dict(top_p=0.97))):
        z = _logits(T, V, "bf16", T + V)
        u = torch.rand(T, device="cuda")
        a = tim.sample(z, u, workspace=ws, **kw)
        b = tim.sample(z, u, **kw)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_calls_at_once(tim):
    """On two streams, each with its own workspace."""
    import torch
    z = _logits(300, 50257, "bf16", 31)
    u = torch.rand(300, device="cuda")
    cases = [dict(top_p=0.97), dict(top_k=3000, top_p=0.9)]
    want = [tim.sample(z, u, **kw) for kw in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    spaces = [tim.Workspace(1024) for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i, kw in enumerate(cases):
            got[i].append(tim.sample(z, u, workspace=spaces[i], stream=streams[i], check=False, **kw))
    torch.cuda.synchronize()
    for i, w in enumerate(want):
        spaces[i].check()
        assert all(torch.equal(x, y) for g in got[i] for x, y in zip(g, w))


def _shapes(V, dtype, seed):
    """Rows of many shapes: flat, steep, rising and falling along the row, one token or one stretch
    far above the rest, logits that lie octaves apart, a few values alone, mostly masked."""
    import torch
    g = np.random.default_rng(seed)
    z = g.normal(size=(12, V)) * 2.0
    z[0] *= 0.05
    z[1] = np.sort(z[1]) * 6
    z[2] = -np.sort(-z[2]) * 6
    z[3, V // 3] += 40
    z[4, V // 2:V // 2 + 50] += 25
    z[5] *= 900
    z[6] = 5000 + z[6] * 2
    z[7] = -9000 + z[7] * 3
    z[8] = g.integers(-2, 3, size=V)
    z[9] = np.where(g.random(V) < 0.6, 1.0, z[9])
    z[10, g.random(V) < 0.9] = -np.inf
    z[11] -= np.linspace(0, 60, V)
    return torch.from_numpy(z.astype(np.float32)).cuda().to(_dtype(dtype))


DEEP = [dict(), dict(temperature=0.05), dict(temperature=40.0), dict(top_p=0.6), dict(top_p=0.999),
        dict(top_p=0.97, temperature=3.0), dict(top_p=0.9, min_p=0.3), dict(top_k=1500),
        dict(top_k=3000, top_p=0.8), dict(top_k=2500, top_p=0.9, min_p=0.05), dict(min_p=0.001)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T", [12, 60, 200, 400, 700])
def test_rows_beyond_the_list(tim, dtype, T):
    import torch
    base = _shapes(5003, dtype, 50)
    u = np.random.default_rng(51).random(12).astype(np.float32)
    at = torch.arange(T, device="cuda") % 12
    z, ut = base[at].contiguous(), torch.from_numpy(u).cuda()[at]
    for kw in DEEP:
        want = _check(tim, base, u, **kw)
        got = tim.sample(z, ut, **kw)
        for i in (0, 3):
            assert torch.equal(got[i], torch.from_numpy(want[i]).cuda()[at]), kw
        for i in (1, 2):  # equal but for the last bit, see the header
            w = torch.from_numpy(want[i]).cuda()[at]
            assert bool(((got[i] - w).abs() <= 2.0 ** -23 * w.abs() + 2.0 ** -29).all()), kw
