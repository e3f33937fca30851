"""tim.verify on the GPU against the fp64 oracle.

Tokens and counts have to be the oracle's wherever no border of a decision lies within MARGIN.  The bar:
p_v and q_v are integers good to 2^-30.3 relative each, so a running sum of max(p - q, 0) is off by
2 x 2^-30.3 of the mass of p at most, and so is the target that it is compared with: 2^-28.3 together.  A
test of acceptance compares two such numbers relative to p(x), a filter's border is the sampler's.
logprob is computed as a pair of floats and rounded once: tol = 2^-24 |x| + 2^-29.
"""
import math

import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

MARGIN = 2.0 ** -28


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


def _problem(B, N, V, dtype, seed, scale=2.0, apart=0.7, pad=(0, 0), offset=(0, 0)):
    """Logits of a target [B, N + 1, V] and of a drafter that agrees up to `apart`, the drafter's stored
    a step at a time, drafts that are likely under the drafter, and uniform numbers."""
    import torch
    g = np.random.default_rng(seed)
    z = (g.normal(size=(B, N + 1, V)) * scale).astype(np.float32)
    q = z[:, :N] + (g.normal(size=(B, N, V)) * apart).astype(np.float32)
    t = torch.full((B, N + 1, offset[0] + V + pad[0]), 77.0, dtype=_dtype(dtype), device="cuda")
    t = t[..., offset[0]:offset[0] + V]
    t.copy_(torch.from_numpy(z))
    d = torch.full((N, B, offset[1] + V + pad[1]), 77.0, dtype=_dtype(dtype), device="cuda")
    d = d[..., offset[1]:offset[1] + V].transpose(0, 1)
    d.copy_(torch.from_numpy(q))
    # each draft among the drafter's best few
    near = np.argsort(-q, axis=2)[..., :min(V, 4)]
    ids = np.take_along_axis(near, g.integers(0, near.shape[2], (B, N, 1)), 2)[..., 0].astype(np.int32)
    return dict(target=t, draft=d, ids=torch.from_numpy(ids).cuda(),
                uniform=torch.from_numpy(g.random((B, N)).astype(np.float32)).cuda(),
                uniform_draw=torch.from_numpy(g.random(B).astype(np.float32)).cuda())


KEYS = ("temperature", "top_k", "top_p", "min_p")
OFF = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)


def _call(tim, p, settings, **kw):
    return tim.verify(p["target"], p["ids"], p["uniform"], p["uniform_draw"], p["draft"], **settings, **kw)


def _check(tim, p, settings=None, draft_settings=None, least=None, **kw):
    import torch
    settings = settings or {}
    if draft_settings is not None:
        kw["draft_settings"] = tuple({**OFF, **draft_settings}[k] for k in KEYS)
    got = _call(tim, p, settings, **kw)
    ids, lp, n = (t.cpu().numpy() for t in got)

    def row(s, b):
        s = {**OFF, **s}
        return [s[k][b].item() if isinstance(s[k], torch.Tensor) else float(np.float32(s[k])) for k in KEYS]

    B, compared = len(ids), 0
    zt = p["target"].double().cpu().numpy()
    zd = None if p["draft"] is None else p["draft"].double().cpu().numpy()
    u, x = p["uniform"].double().cpu().numpy(), p["ids"].cpu().numpy()
    for b in range(B):
        as_int = [[s[0], int(s[1]), s[2], s[3]] for s in (row(settings, b), row(draft_settings or settings, b))]
        r = oracle.ends.verify_sequence(zt[b], None if zd is None else zd[b], x[b], u[b],
                                        p["uniform_draw"][b].item(), *as_int)
        if r["margin"] < MARGIN:
            continue
        compared += 1
        assert ids[b].tolist() == r["ids"] and n[b] == r["accepted"], (b, r, ids[b], n[b])
        for g, w in zip(lp[b], r["logprob"]):
            assert abs(float(g) - w) <= 2.0 ** -24 * abs(w) + 2.0 ** -29, (b, r, lp[b])
    assert compared >= (B if least is None else least)
    return got


SETTINGS = [dict(), dict(temperature=0.7, top_k=5, top_p=0.9), dict(top_p=0.5),
            dict(temperature=1.7, top_p=0.99, min_p=0.01), dict(top_k=1), dict(top_k=40),
            dict(min_p=0.3), dict(temperature=0.0), dict(temperature=0.2, top_k=700)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 31, 255, 1000, 4097, 32003])
def test_sizes_and_settings(tim, dtype, V):
    for n, kw in enumerate(SETTINGS):
        p = _problem(6, 3, V, dtype, 100 * V + n)
        # of two tokens at a low temperature p and q are 1 but for 2^-30, so that what is left of p is
        # no more than the margin and does not decide anything that could be compared
        _check(tim, p, kw, least=4)
        _check(tim, {**p, "draft": None}, kw, least=4)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_full_vocabulary(tim, dtype):
    for V, seed in ((151936, 1), (393216, 2)):
        p = _problem(3, 2, V, dtype, seed, apart=0.4)
        for kw in (dict(), dict(temperature=0.6, top_k=50, top_p=0.95), dict(top_p=0.9), dict(min_p=0.05),
                   dict(top_k=20000, top_p=0.8)):
            # the running sum's steps are 1 / V on average: one in 300 draws lies within the margin
            _check(tim, p, kw, least=2)
            _check(tim, {**p, "draft": None}, kw, least=2)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("offset,pad", [((0, 0), (3, 0)), ((1, 0), (0, 0)), ((3, 3), (5, 5)), ((8, 2), (8, 1))])
def test_rows_at_any_address(tim, dtype, offset, pad):
    p = _problem(7, 3, 1013, dtype, 7, pad=pad, offset=offset)
    for kw in SETTINGS[:4]:
        _check(tim, p, kw)
        _check(tim, {**p, "draft": None}, kw)


@pytest.mark.parametrize("B", [1, 22, 40, 80, 200])
def test_many_sequences(tim, B):
    """Over the sizes at which the first launch takes other numbers of threads a row."""
    import torch
    p = _problem(B, 3, 3001, "bf16", B)
    for kw in (dict(), dict(temperature=0.7, top_k=50, top_p=0.95), dict(top_p=0.97), dict(top_k=2000, top_p=0.9)):
        _check(tim, {**p, "draft": None}, kw, least=B - 1)
        whole = _check(tim, p, kw, least=B - 1)
        b = B // 2
        one = _call(tim, {k: v[b:b + 1] for k, v in p.items()}, kw)
        for w, o in zip(whole, one):
            if o.dtype == torch.float32:
                assert bool(((w[b:b + 1] - o).abs() <= 2.0 ** -23 * o.abs() + 2.0 ** -29).all())
            else:
                assert torch.equal(w[b:b + 1], o)


def test_sequences_on_either_side_of_a_third_of_the_sms(tim):
    """Where the second launch takes other numbers of CTAs a sequence: what they draw is the same."""
    import torch
    B = torch.cuda.get_device_properties(0).multi_processor_count // 3
    p = _problem(B + 1, 3, 3001, "bf16", 5)
    for kw in (dict(), dict(top_k=50, top_p=0.95), dict(temperature=0.7, min_p=0.02)):
        for draft in (p["draft"], None):
            q = {**p, "draft": draft}
            more = _check(tim, q, kw, least=B - 1)
            few = _check(tim, {k: v[:B] if v is not None else v for k, v in q.items()}, kw, least=B - 2)
            assert torch.equal(more[0][:B], few[0]) and torch.equal(more[2][:B], few[2])


@pytest.mark.parametrize("N", [31, 32, 33, 70])
def test_many_drafts(tim, N):
    """A drafter that nearly agrees: accepted runs beyond the 32 positions that are looked at together."""
    p = _problem(6, N, 50, "f32", N, apart=1e-4)
    got = _check(tim, p, least=5)
    assert int(got[2].max()) > 20
    same = {**p, "draft": p["target"][:, :N]}
    assert bool((_check(tim, same)[2] == N).all())  # u q < p where q = p
    assert bool((_check(tim, same, dict(top_k=7, temperature=0.5), least=5)[2] <= N).all())


def test_distributions_that_agree(tim):
    """A draft that neither has, where p and q are the same but for their roundings: from p."""
    import torch
    p = _problem(8, 1, 200, "f32", 31)
    p["target"][:, 0] = p["target"][:, 0].to(torch.bfloat16).float()
    p["draft"] = p["target"][:, :1] + 4.0  # exactly the same
    p["ids"][:, 0] = p["target"][:, 0].argmin(1).int()
    for kw in (dict(top_k=20), dict(min_p=0.3), dict(top_k=20, top_p=0.7, temperature=0.8)):
        ids, _, n = _check(tim, p, kw, least=7)
        assert not bool(n.any())
        assert torch.equal(ids[:, 0], tim.sample(p["target"][:, 0], p["uniform_draw"], **kw)[0])


def test_settings_a_sequence_and_the_drafters_own(tim):
    import torch
    B = 40
    p = _problem(B, 4, 5003, "bf16", 16)
    g = np.random.default_rng(8)
    s = dict(temperature=torch.tensor(g.choice([0.0, 0.5, 0.7, 1.0, 1.4], B).astype(np.float32), device="cuda"),
             top_k=torch.tensor(g.choice([-1, 0, 1, 20, 50, 3000, 40000], B).astype(np.int32), device="cuda"),
             top_p=torch.tensor(g.choice([0.1, 0.9, 0.95, 1.0, 2.0], B).astype(np.float32), device="cuda"),
             min_p=torch.tensor(g.choice([0.0, 0.05, 1.0], B).astype(np.float32), device="cuda"))
    _check(tim, p, s, least=B - 1)
    _check(tim, p, dict(top_k=50), dict(temperature=0.5), least=B - 1)
    _check(tim, p, dict(temperature=0.0), dict(temperature=1.3, top_p=0.9))
    _check(tim, p, dict(temperature=0.7), dict(temperature=0.0), least=B - 1)
    _check(tim, p, s, {k: v.flip(0) for k, v in s.items()}, least=B - 1)


def test_masked_tokens_and_disjoint_supports(tim):
    import torch
    for dtype in ("f32", "bf16", "f16"):
        p = _problem(6, 2, 4100, dtype, 11)
        low = torch.finfo(p["target"].dtype).min
        odd = torch.arange(4100, device="cuda") % 2 == 1
        p["target"][0, :, odd] = -math.inf      # p and q have no token in common
        p["draft"][0, :, ~odd] = -math.inf
        p["ids"][0] |= 1
        p["target"][1, :, 10:] = low
        p["draft"][2, :, 10:] = low
        p["draft"][3] = 0.0                      # flat
        p["target"][4, :, 1:] = -math.inf        # one token alone
        p["ids"][4] = torch.tensor([0, 17], device="cuda")
        p["ids"][5, 0] = 4099
        for kw in (dict(), dict(top_k=50), dict(top_p=0.9), dict(min_p=0.1), dict(temperature=0.0)):
            got = _check(tim, p, kw, least=5)
            assert got[2][0] == 0 and got[0][0, 0] % 2 == 0
            assert got[0][4].tolist() == [0, 0, -1] and got[2][4] == 1


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_extreme_scales(tim, dtype):
    p = _problem(6, 2, 2003, dtype, 13, scale=3000.0, apart=30.0)
    for t in (1e-6, 1e-3, 0.5, 30.0, 1e4, 1e6):
        for kw in (dict(), dict(top_p=0.9), dict(top_k=9), dict(min_p=0.2)):
            _check(tim, p, dict(temperature=t, **kw), least=5)


def test_uniform_ends(tim):
    """At 0 whatever has mass is accepted, and the first token with any is drawn."""
    import torch
    p = _problem(4, 2, 5003, "f32", 15)
    last = float(np.float32(1.0) - np.float32(2.0 ** -24))
    for lo in (0.0, last, 1e-40, 1e-30):
        for draw in (0.0, last):
            p["uniform"].fill_(lo)
            p["uniform_draw"].fill_(draw)
            for kw in (dict(), dict(top_k=10), dict(top_p=0.7)):
                got = _check(tim, p, kw, least=2)
                if lo == 0.0 and not kw:
                    assert bool((got[2] == 2).all())
    # p of the draft 2^-290 and more below the largest: still accepted at 0
    p["target"][0, 0] = 0.0
    p["target"][0, 0, int(p["ids"][0, 0])] = -200.0
    p["uniform"].fill_(0.0)
    assert _call(tim, p, {})[0][0, 0] == p["ids"][0, 0]


def test_one_workspace_for_calls_of_all_sizes_in_turn(tim):
    """Nothing of a call is left in the workspace, nor of the other operators that it serves."""
    import torch
    ws = tim.Workspace(tim.verify_workspace_size(200, 6))
    for n, (B, N, V) in enumerate(((200, 6, 999), (3, 2, 4097), (90, 3, 2003), (200, 1, 64), (1, 40, 501))):
        p = _problem(B, N, V, "bf16", 900 + n)
        for kw in (dict(), dict(top_k=20, top_p=0.9)):
            want = _call(tim, p, kw)
            assert all(torch.equal(a, b) for a, b in zip(want, _call(tim, p, kw, workspace=ws)))
            z = p["target"][:, 0].contiguous()
            tim.sample(z, p["uniform_draw"], workspace=ws, **kw)
            tim.embed_backward(z[:16], torch.arange(min(B, 16), device="cuda", dtype=torch.int32), 16,
                               workspace=ws if ws.nbytes >= tim.embed_backward_workspace_size(16, 16, V) else None)
            assert all(torch.equal(a, b) for a, b in zip(want, _call(tim, p, kw, workspace=ws)))


def test_unequal_drafts(tim):
    """The first -1 ends a sequence's drafts; rows behind are not read."""
    import torch
    p = _problem(6, 4, 999, "bf16", 21, apart=0.1)
    for b, n in enumerate((0, 1, 2, 3, 4, 2)):
        p["ids"][b, n:n + 1] = -1
        p["target"][b, n + 1:] = math.nan
        p["draft"][b, n:] = math.nan
    for kw in (dict(), dict(top_k=20, top_p=0.9)):
        ids, lp, n = _check(tim, p, kw, least=5)
        assert bool((n.cpu() <= torch.tensor([0, 1, 2, 3, 4, 2])).all())
        assert bool((lp[ids < 0] == 0).all())


def test_all_accepted_draws_as_the_sampler(tim):
    import torch
    B, N, V = 30, 2, 30011
    p = _problem(B, N, V, "bf16", 23)
    p["draft"] = p["target"][:, :N]
    kw = dict(temperature=0.8, top_k=30, top_p=0.9)
    for j in range(N):  # drafts within the filters
        p["ids"][:, j] = tim.sample(p["target"][:, j], torch.rand(B, device="cuda"), **kw)[0]
    ids, lp, n = _call(tim, p, kw)
    assert bool((n == N).all())
    want = tim.sample(p["target"][:, N], p["uniform_draw"], **kw)
    assert torch.equal(ids[:, N], want[0])
    assert bool(((lp[:, N] - want[1]).abs() <= 2.0 ** -23 * want[1].abs() + 2.0 ** -29).all())


def test_tokens_are_distributed_as_the_target(tim):
    """65536 sequences with the same logits: the first token's frequencies are p's within six standard
    deviations, whatever the drafter."""
    import torch
    B, V = 65536, 6
    z = torch.tensor([0.5, -1.0, 2.0, 0.0, 1.0, -0.5], device="cuda")
    torch.manual_seed(5)
    for zq in (torch.tensor([2.0, 0.0, 0.0, 0.0, 1.0, -3.0], device="cuda"), torch.zeros(V, device="cuda")):
        for kw in (dict(), dict(temperature=0.7, top_k=4)):
            draft = zq.expand(B, 1, V)
            ids = tim.sample(zq.expand(B, V).contiguous(), torch.rand(B, device="cuda"), **kw)[0].view(B, 1)
            got = tim.verify(z.expand(B, 2, V), ids, torch.rand(B, 1, device="cuda"),
                             torch.rand(B, device="cuda"), draft, **kw)
            p, _, _ = oracle.ends.processed(z.double().cpu().numpy(), kw.get("temperature", 1.0), kw.get("top_k", 0), 1.0, 0.0)
            f = np.bincount(got[0][:, 0].cpu().numpy(), minlength=V) / B
            assert np.all(np.abs(f - p) <= 6 * np.sqrt(p * (1 - p) / B)), (f, p)


def test_bad_sequences_are_reported_and_leave_the_others(tim):
    import torch
    B = 9
    p = _problem(B, 3, 999, "f32", 17, apart=0.01)
    p["uniform"].fill_(0.1)  # all but always accepted
    want = _call(tim, p, {})
    assert bool((want[2] == 3).all())
    p["target"][1, 2, 500] = math.nan
    p["target"][2, 0, 0] = math.inf
    p["draft"][3, 1] = -math.inf
    p["uniform"][4, 1] = 1.0
    p["uniform_draw"][5] = -0.1
    p["ids"][6, 2] = 999
    p["ids"][7, 1] = -2
    ws = tim.Workspace(tim.verify_workspace_size(B, 3))
    ids, lp, n = _call(tim, p, {}, workspace=ws, check=False)
    with pytest.raises(tim.TimError):
        ws.check()
    for b in (0, 8):
        assert torch.equal(ids[b], want[0][b]) and torch.equal(lp[b], want[1][b]) and n[b] == 3
    for b in range(1, 8):
        assert bool((ids[b] == -1).all()) and bool(lp[b].isnan().all()) and n[b] == 0, b
    # a fault behind a refused draft does not count
    q = _problem(1, 3, 999, "f32", 18)
    q["uniform"].fill_(0.999)
    q["ids"][0, 0] = int(q["target"][0, 0].argmin())
    q["draft"][0, 0, q["ids"][0, 0].item()] = 20.0
    want = _call(tim, q, {})
    assert want[2].item() == 0
    q["target"][0, 2, 5] = math.nan
    q["draft"][0, 1, 5] = math.inf
    q["ids"][0, 2] = 5000
    q["uniform"][0, 1] = 2.0
    ids, lp, n = _call(tim, q, {}, workspace=ws)
    assert torch.equal(ids, want[0]) and torch.equal(lp, want[1]) and n.item() == 0
    for bad in (dict(temperature=torch.tensor([-1.0] * B, device="cuda")),
                dict(top_p=torch.tensor([math.nan] * B, device="cuda")),
                dict(min_p=torch.tensor([1.5] * B, device="cuda"))):
        with pytest.raises(tim.TimError, match="TIM_ERR"):
            _call(tim, p, bad)


@pytest.mark.parametrize("B,N", [(200, 6), (700, 3), (40, 12)])
def test_rows_behind_a_refused_draft(tim, B, N):
    """More rows than run at once: which of the rows behind a refused draft are still read does not show.
    Every sequence holds a fault behind a place of its own where it is surely refused."""
    import torch
    V = 3001
    p = _problem(B, N, V, "bf16", B, apart=0.0)
    p["uniform"].fill_(0.5)
    at = torch.arange(B, device="cuda") % (N + 1)
    for b in range(B):
        j = int(at[b])
        if j < N:
            x = int(p["ids"][b, j])
            p["target"][b, j, x] = -math.inf
            p["target"][b, j + 1:] = math.nan
            p["draft"][b, j + 1:] = math.nan
    want = _check(tim, p, least=B - 2)
    assert torch.equal(want[2], at.int())
    for kw in (dict(), dict(top_k=50, top_p=0.9), dict(top_p=0.99)):
        first = _call(tim, p, kw)
        for _ in range(5):
            assert all(torch.equal(x, y) for x, y in zip(first, _call(tim, p, kw)))


def test_refusals(tim):
    import torch
    p = _problem(4, 3, 50, "f32", 19)
    t, d, ids, u, v = (p[k] for k in ("target", "draft", "ids", "uniform", "uniform_draw"))
    for bad in (lambda: tim.verify(t[:, :3], ids, u, v, d), lambda: tim.verify(t, ids.long(), u, v, d),
                lambda: tim.verify(t, ids, u, v, d.half()), lambda: tim.verify(t, ids, u[:, :2], v, d),
                lambda: tim.verify(t, ids, u, v[:3], d), lambda: tim.verify(t, ids, u, v, d[:, :2]),
                lambda: tim.verify(t.transpose(1, 2), ids, u, v, d), lambda: tim.verify(t[0], ids, u, v, d),
                lambda: tim.verify(t, ids, u, v, d, top_k=torch.zeros(3, dtype=torch.int32, device="cuda")),
                lambda: tim.verify(t, ids, u, v, d, out=(torch.empty_like(ids),) * 3)):
        with pytest.raises((ValueError, TypeError)):
            bad()
    for bad in (lambda: tim.verify(t, ids, u, v, d, temperature=-1.0), lambda: tim.verify(t, ids, u, v, d, top_p=0.0),
                lambda: tim.verify(t, ids, u, v, d, draft_settings=(1.0, 0, 1.0, 2.0)),
                lambda: tim.verify(t, ids, u, v, d, workspace=tim.Workspace(1024)),
                lambda: tim.verify(t[:, :1], ids[:, :0], u[:, :0], v)):
        with pytest.raises(tim.TimError):
            bad()


@pytest.mark.parametrize("B,V", [(7, 30011), (90, 7001)])
def test_graph_replay_streams_outputs_and_two_calls_at_once(tim, B, V):
    """With few rows, and with more than run at once."""
    import torch
    N = 3
    p = _problem(B, N, V, "bf16", 18)
    ws = tim.Workspace(tim.verify_workspace_size(B, N))
    big = [torch.full((B + 3, N + 1), 7, dtype=torch.int32, device="cuda"),
           torch.full((B + 3, N + 1), 7.0, device="cuda"),
           torch.full((B + 3,), 7, dtype=torch.int32, device="cuda")]
    out = tuple(t[:B] for t in big)
    kw = dict(temperature=0.8, top_k=30, top_p=0.9)
    _call(tim, p, kw, out=out, workspace=ws, check=False)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _call(tim, p, kw, out=out, workspace=ws, check=False)
    for seed in (101, 102):
        for k, t in _problem(B, N, V, "bf16", seed).items():
            p[k].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        ws.check()
        assert all(torch.equal(a, b) for a, b in zip(out, _check(tim, p, kw, least=B - 2)))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        assert all(torch.equal(a, b) for a, b in zip(out, _call(tim, p, kw, stream=side)))
    assert all(bool((t[B:] == 7).all()) for t in big)
    cases = [dict(top_p=0.97), dict(top_k=3000, top_p=0.9)]
    want = [_call(tim, p, c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    spaces = [tim.Workspace(ws.nbytes) for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i, c in enumerate(cases):
            got[i].append(_call(tim, p, c, workspace=spaces[i], stream=streams[i], check=False))
    torch.cuda.synchronize()
    for i, w in enumerate(want):
        spaces[i].check()
        assert all(torch.equal(x, y) for g in got[i] for x, y in zip(g, w))


def _shapes(V, dtype, seed):
    """Rows of many shapes: flat, steep, rising and falling along the row, one token or one stretch far
    above the rest, logits that lie octaves apart, a few values alone, mostly masked."""
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


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_rows_of_many_shapes(tim, dtype):
    """Every shape as the target's against every shape as the drafter's: all ways in which the sampler's
    kernel finds a row's border."""
    import torch
    V = 5003
    t, d = _shapes(V, dtype, 50), _shapes(V, dtype, 60)
    a, b = torch.meshgrid(torch.arange(12), torch.arange(12), indexing="ij")
    a, b = a.reshape(-1).cuda(), b.reshape(-1).cuda()
    g = np.random.default_rng(51)
    ids = tim.sample(d[b].contiguous(), torch.from_numpy(g.random(144).astype(np.float32)).cuda())[0]
    p = dict(target=t[a].unsqueeze(1).expand(144, 2, V), draft=d[b].unsqueeze(1).contiguous(), ids=ids.view(144, 1),
             uniform=torch.from_numpy(g.random((144, 1)).astype(np.float32)).cuda(),
             uniform_draw=torch.from_numpy(g.random(144).astype(np.float32)).cuda())
    for kw in (dict(), dict(temperature=0.05), dict(temperature=40.0), dict(top_p=0.6), dict(top_p=0.999),
               dict(top_p=0.9, min_p=0.3), dict(top_k=1500), dict(top_k=2500, top_p=0.9, min_p=0.05), dict(min_p=0.001)):
        _check(tim, p, kw, least=130)


@pytest.mark.slow
def test_beyond_2_31_elements(tim):
    """Logits of more than 2^31 elements: offsets need 64 bits."""
    import torch
    B, N, V = 2400, 5, 151936
    t = torch.zeros(B, N + 1, V, dtype=torch.bfloat16, device="cuda")
    ids = torch.randint(0, V, (B, N), device="cuda", dtype=torch.int32)
    last = torch.randint(0, V, (B,), device="cuda")
    t[:, :N].scatter_(2, ids.long().unsqueeze(2), 100.0)
    t[:, N].scatter_(1, last.unsqueeze(1), 100.0)
    got = tim.verify(t, ids, torch.rand(B, N, device="cuda"), torch.rand(B, device="cuda"), t[:, :N])
    assert torch.equal(got[0][:, :N], ids) and torch.equal(got[0][:, N], last.int())
    ids[-1, 2] = (ids[-1, 2] + 1) % V
    got = tim.verify(t, ids, torch.rand(B, N, device="cuda"), torch.rand(B, device="cuda"))
    assert got[2][-1] == 2 and got[0][-1, 2] == (ids[-1, 2] - 1) % V
