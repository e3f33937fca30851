"""What is measured of the operators at the two ends of a model: the verification of drafted tokens, the
embedding lookup and its gradient, and the residual update with the norms around a block.

``run`` computes them in plain torch operations, or, where ``own`` is true, with the library's calls.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {"f32": 4, "bf16": 2, "f16": 2}
V_FULL = 151936  # the vocabulary of this repository's benchmark


def listed():
    def verify(name, B, N, V, dtype, **kw):
        c = dict(name=name, op="verify", B=B, N=N, V=V, dtype=dtype, pad=0, temperature=1.0, top_k=0,
                 top_p=1.0, min_p=0.0, mixed=False, certain=False, short=0.0)
        c.update(kw)
        return c

    def embed(name, op, T, V, d, dtype, **kw):
        c = dict(name=name, op=op, T=T, V=V, d=d, dtype=dtype, pad=0, masked=0.0)
        c.update(kw)
        return c

    def norm(name, op, T, d, dtype, **kw):
        c = dict(name=name, op=op, T=T, d=d, dtype=dtype, pad=0, gate="none", post=False, pre=True,
                 scale=1.0)
        c.update(kw)
        return c

    return [
        # one request with three drafted tokens: latency
        verify("verify_one", 1, 3, V_FULL, "bf16", temperature=0.7, top_k=50, top_p=0.95),
        # a decoding batch whose requests bring settings of their own and have unequal drafts
        verify("verify_batch_mixed", 48, 3, V_FULL, "bf16", mixed=True, short=0.3),
        # rollouts for training: the whole distribution, no filter
        verify("verify_rollout_plain", 128, 4, V_FULL, "bf16"),
        # tokens proposed by lookup in the prompt (no draft distribution), small odd vocabulary
        verify("verify_lookup_odd", 13, 5, 32003, "f16", pad=5, certain=True, temperature=1.3, min_p=0.05),
        # a decoding step's tokens: latency
        embed("embed_decode", "embed", 64, V_FULL, 4096, "bf16"),
        # the benchmark's batch of tokens
        embed("embed_batch", "embed", 32768, V_FULL, 4096, "bf16"),
        # the gradient of the benchmark's batch, an eighth of the rows padding
        embed("embed_grad", "embed_grad", 32768, V_FULL, 4096, "bf16", masked=0.125),
        # a small odd training piece through autograd
        embed("embed_train_odd", "embed_train", 777, 32003, 1000, "f16", masked=0.1),
        # a decoding step's residual update between two blocks: latency
        norm("norm_decode", "norm", 64, 4096, "bf16"),
        # the forward of the benchmark's batch, norms before and after the block
        norm("norm_batch", "norm", 32768, 4096, "bf16", post=True, gate="channel"),
        # the gradient of a batch with a gate a token
        norm("norm_grad", "norm_grad", 16384, 4096, "bf16", post=True, gate="token", scale=0.22),
        # a small odd training piece in fp32 through autograd, a gate an element
        norm("norm_train_odd", "norm_train", 333, 1001, "f32", post=True, gate="full", pad=3, scale=0.5),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["verify", "verify", "embed", "embed_grad", "embed_train", "norm", "norm_grad",
                     "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "f32", "f16"])
    e = SIZES[dtype]
    pad = rng.choice([0, 0, 0, rng.randint(1, 100)])
    if op == "verify":
        V = rng.choice([V_FULL, _log_uniform(rng, 1000, V_FULL)])
        N = rng.randint(1, 8)
        rows = 128 * 9 * V_FULL * 2 // (V * e)
        return dict(op=op, B=_log_uniform(rng, 1, max(1, min(256, rows // (2 * N + 1)))), N=N, V=V,
                    dtype=dtype, pad=pad,
                    temperature=rng.choice([1.0, round(rng.uniform(0.3, 1.5), 2)]),
                    top_k=rng.choice([0, 0, 1, _log_uniform(rng, 2, 1000)]),
                    top_p=rng.choice([1.0, round(rng.uniform(0.3, 0.99), 3)]),
                    min_p=rng.choice([0.0, 0.0, round(rng.uniform(0.01, 0.2), 3)]),
                    mixed=rng.random() < 0.3, certain=rng.random() < 0.25,
                    short=rng.choice([0.0, round(rng.uniform(0.1, 0.6), 2)]))
    if op.startswith("embed"):
        V = rng.choice([V_FULL, _log_uniform(rng, 1000, V_FULL)])
        d = rng.choice([2048, 4096, _log_uniform(rng, 8, 8192)])
        if V * d * e > V_FULL * 4096 * 2:
            d = max(8, V_FULL * 4096 * 2 // (V * e))
        most = max(1, min(32768, 32768 * 4096 * 2 // (d * e * (2 if op == "embed_train" else 1))))
        return dict(op=op, T=_log_uniform(rng, 1, most), V=V, d=d, dtype=dtype, pad=pad,
                    masked=rng.choice([0.0, round(rng.uniform(0.05, 0.5), 2)]))
    d = rng.choice([2048, 4096, _log_uniform(rng, 8, 8192)])
    cost = {"norm": 5, "norm_grad": 8, "norm_train": 13}[op]  # arrays moved, at most
    most = max(1, min(32768, 32768 * 4096 * 2 * 4 // (d * e * cost)))
    return dict(op=op, T=_log_uniform(rng, 1, most), d=d, dtype=dtype, pad=pad,
                gate=rng.choice(["none", "none", "channel", "token", "full"]),
                post=rng.random() < 0.5, pre=rng.random() < 0.8,
                scale=rng.choice([1.0, round(rng.uniform(0.1, 1.5), 3)]))


# ------------------------------------------------------------------------------- inputs

def _rand(g, *size):
    return torch.rand(*size, generator=g, device="cuda")


def _randn(g, *size):
    return torch.randn(*size, generator=g, device="cuda")


def _padded(x, pad, dtype):
    """The rows of x in a buffer of wider rows."""
    buf = torch.zeros(*x.shape[:-1], x.shape[-1] + pad, dtype=dtype, device="cuda")
    out = buf[..., :x.shape[-1]]
    out.copy_(x)
    return out


KEYS = ("temperature", "top_k", "top_p", "min_p")


def _prepare_verify(case, g):
    """Target logits as a language model's head gives them, a normal bulk far below a few favoured
    tokens, and a draft model that agrees up to noise.  Drafted tokens are drawn from the draft's
    processed distribution."""
    B, N, V, dtype = case["B"], case["N"], case["V"], DTYPES[case["dtype"]]
    s = dict(case=case)
    if case["mixed"]:
        menu = torch.tensor([[0.0, 0, 1.0, 0.0], [0.7, 50, 0.95, 0.0], [1.0, 0, 1.0, 0.0],
                             [0.6, 20, 0.95, 0.05], [1.0, 0, 0.9, 0.0], [0.8, 0, 1.0, 0.05]],
                            device="cuda")
        pick = menu[torch.randint(0, len(menu), (B,), generator=g, device="cuda")]
        for i, k in enumerate(KEYS):
            s[k] = pick[:, i].to(torch.int32 if k == "top_k" else torch.float32).contiguous()
    else:
        for k in KEYS:
            s[k] = case[k]
    target = torch.empty(B, N + 1, V + case["pad"], dtype=dtype, device="cuda")[..., :V]
    # the drafter writes a step at a time: [N, B, V]
    draft = torch.empty(N, B, V + case["pad"], dtype=dtype, device="cuda")[..., :V].transpose(0, 1)
    ids = torch.empty(B, N, dtype=torch.int64, device="cuda")
    n = min(200, V // 2)
    for j in range(N + 1):
        start = torch.randint(0, V, (B, 1), generator=g, device="cuda")
        stride = max(1, V // n)
        jitter = torch.randint(0, stride, (B, n), generator=g, device="cuda")
        favoured = (start + torch.arange(n, device="cuda") * stride + jitter) % V
        peak = 6.0 + 14.0 * _rand(g, B, 1)
        fall = 0.3 + 2.0 * _rand(g, B, 1)
        rank = torch.arange(1, n + 1, device="cuda", dtype=torch.float32)
        top = peak - fall * rank.log() + 0.5 * _randn(g, B, n)
        bulk = 2.0 * _randn(g, B, V)
        target[:, j].copy_(bulk.scatter(1, favoured, top))
        if j == N:
            break
        near = bulk.add_(0.7 * _randn(g, B, V)).scatter_(1, favoured, top + 0.7 * _randn(g, B, n))
        draft[:, j].copy_(near)
        cum = _processed(draft[:, j], s).cumsum(1)
        at = _rand(g, B, 1).double() * cum[:, -1:]
        ids[:, j] = (cum <= at).sum(1).clamp(max=V - 1)
    if case["short"] > 0:  # requests with fewer drafts
        ends = torch.where(_rand(g, B) < case["short"], torch.randint(0, N, (B,), generator=g, device="cuda"),
                           torch.full((B,), N, device="cuda"))
        ids = torch.where(torch.arange(N, device="cuda") < ends.view(B, 1), ids, torch.full_like(ids, -1))
    s.update(target=target, draft=None if case["certain"] else draft, ids=ids.to(torch.int32),
             uniform=_rand(g, B, N), uniform_draw=_rand(g, B))
    return s


def _frequencies(V):
    """How often the tokens of a vocabulary occur, the most frequent first: Zipf's law."""
    p = 1.0 / (torch.arange(V, dtype=torch.float64) + 10.0)
    return p / p.sum()


def _prepare_embed(case, g):
    T, V, d, dtype = case["T"], case["V"], case["d"], DTYPES[case["dtype"]]
    cdf = _frequencies(V).cumsum(0).cuda()
    rank = torch.searchsorted(cdf, _rand(g, T).double()).clamp(max=V - 1)
    ids = (rank * 7919 + torch.randint(0, V, (1,), generator=g, device="cuda")) % V  # spread over the ids
    if case["masked"] > 0:
        ids = torch.where(_rand(g, T) < case["masked"], torch.full_like(ids, -1), ids)
    s = dict(case=case, ids=ids.to(torch.int32), scale=math.sqrt(d))
    if case["op"] != "embed_grad":
        s["table"] = _padded(0.02 * _randn(g, V, d), case["pad"], dtype)
    if case["op"] == "embed_train":
        s["table"] = s["table"].detach().contiguous().requires_grad_(True)
    if case["op"] != "embed":
        s["dy"] = _padded(1e-2 * _randn(g, T, d), case["pad"], dtype)
    return s


def _prepare_norm(case, g):
    T, d, dtype = case["T"], case["d"], DTYPES[case["dtype"]]
    size = 0.5 + 2.0 * _rand(g, T, 1)
    h = size * _randn(g, T, d)
    h[:, :: max(1, d // 5)] *= 20.0  # the few large channels of a residual stream
    s = dict(case=case, x=_padded(0.7 * _randn(g, T, d), case["pad"], dtype), eps=1e-6)
    s["gamma"] = (1.0 + 0.2 * _randn(g, d)).to(dtype) if case["pre"] else None
    s["gamma_post"] = (0.5 + 0.2 * _randn(g, d)).to(dtype) if case["post"] else None
    gate = {"none": None, "channel": (d,), "token": (T, 1), "full": (T, d)}[case["gate"]]
    s["gate"] = None if gate is None else torch.sigmoid(_randn(g, *gate)).to(dtype)
    s["h"] = _padded(h, case["pad"], dtype)
    if case["op"] == "norm_grad":  # what the forward kept: the new residual stream, the block's output
        s["h"] = _padded(_plain_norm(s)[0], case["pad"], dtype)
    if case["op"] != "norm":
        s["dy"] = _padded(1e-2 * _randn(g, T, d), case["pad"], dtype) if case["pre"] else None
        s["dh"] = _padded(1e-2 * _randn(g, T, d), case["pad"], dtype)
    if case["op"] == "norm_train":
        for k in ("h", "x", "gamma", "gamma_post", "gate"):
            if s[k] is not None:
                s[k] = s[k].detach().requires_grad_(True)
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "verify":
        return _prepare_verify(case, g)
    if case["op"].startswith("embed"):
        return _prepare_embed(case, g)
    return _prepare_norm(case, g)


# ------------------------------------------------------------------------------- plain forms

def _per_row(v, n, device):
    if isinstance(v, torch.Tensor):
        return v.double().view(n, 1)
    # a setting given as a number is a 32-bit one
    return torch.full((n, 1), v, dtype=torch.float32, device=device).double()


def _processed(z, settings):
    """The distribution left of each row of logits [n, V] after temperature, top-k, top-p and min-p, in
    64 bits: a token next to a border is kept or not."""
    z32 = z.float()
    n, V = z32.shape
    dev = z32.device
    tau, k, top_p, min_p = (_per_row(settings[i], n, dev) for i in KEYS)
    greedy = tau == 0
    tau = torch.where(greedy, torch.ones_like(tau), tau)
    k = torch.where(greedy, torch.ones_like(k), torch.where(k <= 0, torch.full_like(k, V), k))
    zs, order = torch.sort(z32, dim=1, descending=True, stable=True)
    w = torch.exp((zs.double() - zs[:, :1].double()) / tau)
    keep = (torch.arange(V, device=dev) < k) & (zs > -math.inf)
    wk = w * keep
    cum = wk.cumsum(1)
    keep &= (cum - wk < top_p * cum[:, -1:]) | (top_p >= 1)
    keep &= w >= min_p
    w *= keep
    w /= w.sum(1, keepdim=True)
    return torch.zeros_like(w).scatter_(1, order, w)


def _plain_verify(s):
    B, N1, V = s["target"].shape
    N = N1 - 1
    dev = s["target"].device
    settings = {k: s[k].repeat_interleave(N1) if isinstance(s[k], torch.Tensor) else s[k] for k in KEYS}
    p = _processed(s["target"].reshape(B * N1, V), settings).view(B, N1, V)
    x = s["ids"].long()
    drafted = (x >= 0).int().cumprod(1)
    at = x.clamp(min=0).unsqueeze(2)
    px = p[:, :N].gather(2, at).squeeze(2)
    if s["draft"] is None:
        qx = torch.ones_like(px)
    else:
        settings = {k: s[k].repeat_interleave(N) if isinstance(s[k], torch.Tensor) else s[k] for k in KEYS}
        q = _processed(s["draft"].reshape(B * N, V), settings).view(B, N, V)
        qx = q.gather(2, at).squeeze(2)
    accepted = ((s["uniform"].double() * qx < px).int() * drafted).cumprod(1).sum(1)
    rejected = accepted < drafted.sum(1)
    b = torch.arange(B, device=dev)
    last = p[b, accepted]
    where = accepted.clamp(max=N - 1)
    if s["draft"] is None:
        r = last.scatter(1, x[b, where].clamp(min=0).unsqueeze(1), 0.0)
    else:
        r = (last - q[b, where]).clamp(min=0)
    r = torch.where(rejected.unsqueeze(1) & (r.sum(1, keepdim=True) > 0), r, last)
    cum = r.cumsum(1)
    y = (cum <= s["uniform_draw"].double().view(B, 1) * cum[:, -1:]).sum(1).clamp(max=V - 1)
    pos = torch.arange(N1, device=dev)
    ids = torch.where(pos < accepted.unsqueeze(1), torch.cat([x, x[:, :1]], 1), torch.full((B, N1), -1, device=dev))
    ids[b, accepted] = y
    lp = p.gather(2, ids.clamp(min=0).unsqueeze(2)).squeeze(2).log()
    lp = torch.where(ids >= 0, lp, torch.zeros_like(lp)).float()
    return ids.to(torch.int32), lp, accepted.to(torch.int32)


def _plain_embed(s):
    live = (s["ids"] >= 0).unsqueeze(1)
    out = s["table"].detach()[s["ids"].clamp(min=0).long()].float() * s["scale"]
    return torch.where(live, out, torch.zeros_like(out)).to(s["table"].dtype)


def _plain_embed_grad(s):
    V, dy = s["case"]["V"], s["dy"]
    live = s["ids"] >= 0
    out = torch.zeros(V, dy.shape[1], dtype=torch.float32, device=dy.device)
    rows = torch.where(live.unsqueeze(1), dy.float() * s["scale"], torch.zeros((), device=dy.device))
    return out.index_add_(0, s["ids"].clamp(min=0).long(), rows).to(dy.dtype)


def _plain_norm(s):
    x, eps = s["x"].detach().float(), s["eps"]
    if s["gamma_post"] is not None:
        x = x * torch.rsqrt((x * x).mean(1, keepdim=True) + eps) * s["gamma_post"].detach().float()
    if s["gate"] is not None:
        x = x * s["gate"].detach().float()
    h = (s["h"].detach().float() + s["case"]["scale"] * x).to(s["x"].dtype)
    if s["gamma"] is None:
        return h, None
    z = h.float()
    y = z * torch.rsqrt((z * z).mean(1, keepdim=True) + eps) * s["gamma"].detach().float()
    return h, y.to(h.dtype)


def _plain_norm_grad(s, h):
    """From the new residual stream h and the block's output."""
    x, dH, eps, dtype = s["x"].detach().float(), s["dh"].float(), s["eps"], s["x"].dtype
    d_gamma = d_post = d_gate = None
    if s["gamma"] is not None:
        z, dy, w = h.float(), s["dy"].float(), s["gamma"].detach().float()
        r = torch.rsqrt((z * z).mean(1, keepdim=True) + eps)
        d_gamma = (dy * z * r).sum(0, dtype=torch.float64).float()
        dH = dH + r * w * dy - z * (r * r * r * (w * dy * z).mean(1, keepdim=True))
    n = x
    if s["gamma_post"] is not None:
        w1 = s["gamma_post"].detach().float()
        r1 = torch.rsqrt((x * x).mean(1, keepdim=True) + eps)
        n = x * r1 * w1
    dn = s["case"]["scale"] * dH
    if s["gate"] is not None:
        kind = s["case"]["gate"]
        full = dn * n
        d_gate = (full.sum(0, dtype=torch.float64).float() if kind == "channel" else
                  full.sum(1, keepdim=True, dtype=torch.float64).float() if kind == "token" else full)
        dn = dn * s["gate"].detach().float()
    dx = dn
    if s["gamma_post"] is not None:
        d_post = (dn * x * r1).sum(0, dtype=torch.float64).float()
        dx = r1 * w1 * dn - x * (r1 * r1 * r1 * (w1 * dn * x).mean(1, keepdim=True))
    if d_gate is not None and s["case"]["gate"] == "full":
        d_gate = d_gate.to(dtype)
    return [dH.to(dtype), dx.to(dtype)] + [t for t in (d_gamma, d_post, d_gate) if t is not None]


# ------------------------------------------------------------------------------- one pass

def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        if op == "verify":
            return _plain_verify(s)
        if op == "embed":
            return _plain_embed(s)
        if op == "embed_grad":
            return _plain_embed_grad(s)
        if op == "embed_train":
            return _plain_embed(s), _plain_embed_grad(s)
        if op == "norm":
            return [t for t in _plain_norm(s) if t is not None]
        if op == "norm_grad":
            return _plain_norm_grad(s, s["h"])
        h, y = _plain_norm(s)
        grads = _plain_norm_grad(s, h)
        like = [t for t in (s["gamma"], s["gamma_post"], s["gate"]) if t is not None]
        grads[2:] = [a.to(t.dtype) for a, t in zip(grads[2:], like)]
        return [t for t in (h, y) if t is not None] + grads
    import rollout_logprob_consistency_gb300 as tim
    if op == "verify":
        if "workspace" not in s:  # a user's program keeps one
            s["workspace"] = tim.Workspace(tim.verify_workspace_size(c["B"], c["N"]))
        return tim.verify(s["target"], s["ids"], s["uniform"], s["uniform_draw"], s["draft"],
                          s["temperature"], s["top_k"], s["top_p"], s["min_p"],
                          workspace=s["workspace"], check=False)
    if op.startswith("embed"):
        if "workspace" not in s:
            s["workspace"] = tim.Workspace(tim.embed_backward_workspace_size(c["T"], c["V"], c["d"]))
        ws = s["workspace"]
        if op == "embed":
            return tim.embed(s["table"], s["ids"], s["scale"], workspace=ws, check=False)
        if op == "embed_grad":
            return tim.embed_backward(s["dy"], s["ids"], c["V"], s["scale"], dtype=s["dy"].dtype,
                                      workspace=ws, check=False)
        out = tim.embedding(s["table"], s["ids"], s["scale"], workspace=ws, check=False)
        grad, = torch.autograd.grad(out, s["table"], s["dy"])
        return out.detach(), grad
    how = dict(gamma_post=s["gamma_post"], gate=s["gate"], scale=c["scale"])
    if op == "norm":
        h, y = tim.residual_norm(s["h"], s["x"], s["gamma"], s["eps"], **how)
        return [t for t in (h, y) if t is not None]
    if "workspace" not in s:
        s["workspace"] = tim.Workspace(tim.residual_norm_backward_workspace_size(c["T"], c["d"]))
    if op == "norm_grad":
        grads = tim.residual_norm_backward(s["h"], s["x"], s["dh"], s["dy"], s["gamma"], s["eps"],
                                           workspace=s["workspace"], **how)
        return [t for t in grads if t is not None]
    h, y = tim.block_residual(s["h"], s["x"], s["gamma"], s["eps"], workspace=s["workspace"], **how)
    leaves = [s[k] for k in ("h", "x", "gamma", "gamma_post", "gate") if s[k] is not None]
    outs, into = ((h, y), (s["dh"], s["dy"])) if y is not None else ((h,), (s["dh"],))
    grads = torch.autograd.grad(outs, leaves, into)
    return [t.detach() for t in outs] + list(grads)


def work(case):
    e = SIZES[case["dtype"]]
    if case["op"] == "verify":
        B, N, V = case["B"], case["N"], case["V"]
        full = 1.0 - case["short"] / 2 * (N + 1) / N  # of the drafted rows
        rows = B * (1 + N * full) + (0 if case["certain"] else B * N * full)
        return {"bytes": rows * V * e + B * (16 * N + 16), "flops": 4 * rows * V}
    T, d = case["T"], case["d"]
    if case["op"].startswith("embed"):
        V, live = case["V"], 1.0 - case["masked"]
        rows = float(-torch.expm1(-T * live * _frequencies(V)).sum())  # distinct tokens, as expected
        fwd = {"bytes": rows * d * e + T * d * e + 4 * T, "flops": T * live * d}
        bwd = {"bytes": live * T * d * e + V * d * e + 4 * T, "flops": 2 * T * live * d}
        if case["op"] == "embed":
            return fwd
        if case["op"] == "embed_grad":
            return bwd
        return {k: fwd[k] + bwd[k] for k in fwd}
    n = T * d
    gate = {"none": 0, "channel": d, "token": T, "full": n}[case["gate"]]
    fwd = {"bytes": (3 + case["pre"]) * n * e + gate * e, "flops": 10 * n}
    bwd = {"bytes": (5 + case["pre"]) * n * e + gate * e * (2 if case["gate"] == "full" else 1),
           "flops": 25 * n}
    if case["op"] == "norm":
        return fwd
    if case["op"] == "norm_grad":
        return bwd
    return {k: fwd[k] + bwd[k] for k in fwd}


# ------------------------------------------------------------------------------- 64 bits

def _number(x, i):  # a setting given as a number is a 32-bit one
    return x[i].item() if isinstance(x, torch.Tensor) else float(torch.tensor(float(x)))


def _log_processed(z, tau, k, p, mp):
    """ln of the processed distribution of one row in 64 bits, -inf for what is filtered out."""
    z = z.double()
    out = torch.full_like(z, -math.inf)
    order = torch.argsort(z, descending=True, stable=True)
    if tau == 0:
        out[order[0]] = 0.0
        return out
    if 0 < k < len(z):
        order = order[: int(k)]
    x = z[order] / tau
    lq = x - torch.logsumexp(x, 0)
    if p < 1:
        n = 1 + int((lq.exp().cumsum(0)[:-1] < p).sum())
        order, x = order[:n], x[:n]
    if mp > 0:
        ok = x - x[0] >= math.log(mp)
        order, x = order[ok], x[ok]
    out[order] = x - torch.logsumexp(x, 0)
    return out


@torch.no_grad()
def _exact_verify(s):
    B, N = s["ids"].shape
    lp = torch.zeros(B, N + 1, dtype=torch.float64, device="cuda")
    for b in range(B):
        settings = [_number(s[k], b) for k in KEYS]
        for j in range(N + 1):
            log_p = _log_processed(s["target"][b, j], *settings)
            x = int(s["ids"][b, j]) if j < N else -1
            r = log_p.exp()
            if x >= 0:
                if s["draft"] is None:
                    q = torch.zeros_like(r)
                    q[x] = 1.0
                else:
                    q = _log_processed(s["draft"][b, j], *settings).exp()
                if s["uniform"][b, j].double() * q[x] < r[x]:
                    lp[b, j] = log_p[x]
                    continue
                rest = torch.relu(r - q)
                r = rest if rest.sum() > 0 else r
            ids = r.nonzero().view(-1)
            cdf = r[ids].cumsum(0)
            at = torch.searchsorted(cdf, s["uniform_draw"][b].double() * cdf[-1], right=True)
            lp[b, j] = log_p[ids[at.clamp(max=len(ids) - 1)]]
            break
    return None, lp, None


@torch.no_grad()
def exact(case, seed):
    """From the definitions in 64 bits: the scores of the tokens that a verification yields, row by row;
    the lookup and the sums of its gradient; the residual update, its gradients by autograd."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "verify":
        return _exact_verify(s)
    if op.startswith("embed"):
        live = (s["ids"] >= 0).nonzero().view(-1)
        ids, scale = s["ids"][live].long(), _number(s["scale"], 0)
        res = []
        if op != "embed_grad":
            out = torch.zeros(case["T"], case["d"], dtype=torch.float64, device="cuda")
            out[live] = s["table"].detach().double()[ids] * scale
            res.append(out)
        if op != "embed":
            grad = torch.zeros(case["V"], case["d"], dtype=torch.float64, device="cuda")
            res.append(grad.index_add_(0, ids, s["dy"][live].double()).mul_(scale))
        return res[0] if len(res) == 1 else tuple(res)

    names = [k for k in ("h", "x", "gamma", "gamma_post", "gate") if s[k] is not None]
    t = {k: s[k].detach().double().requires_grad_(op != "norm") for k in names}
    scale = _number(case["scale"], 0)

    def unit(v):
        return v / (v.pow(2).mean(1, keepdim=True) + s["eps"]).sqrt()

    with torch.enable_grad():
        n = t["x"] if s["gamma_post"] is None else unit(t["x"]) * t["gamma_post"]
        step = scale * n * (t["gate"] if s["gate"] is not None else 1.0)
        # the stream is kept in its own type: a rounding that gradients pass straight through
        before = t["h"] if op != "norm_grad" else t["h"].detach() - step.detach()
        if op == "norm_grad":
            before.requires_grad_(True)
        sum_ = before + step
        h = sum_ if op == "norm_grad" else sum_ + (sum_.to(s["x"].dtype).double() - sum_).detach()
        y = unit(h) * t["gamma"] if s["gamma"] is not None else None
        outs = [v for v in (sum_, y) if v is not None]
        if op == "norm":
            return [v.detach() for v in outs]
        leaves = [before if k == "h" else t[k] for k in names]
        into = [s["dh"].double()] + ([s["dy"].double()] if y is not None else [])
        grads = torch.autograd.grad([h] + outs[1:], leaves, into)
    return list(grads) if op == "norm_grad" else [v.detach() for v in outs] + list(grads)
