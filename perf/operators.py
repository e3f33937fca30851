"""What is measured of the operators on a [T, V] logits matrix: the sampler (temperature, top-k, top-p
and min-p, from given uniform numbers) and the distillation loss from a teacher's top logits, alone,
through autograd, and with its gradient in one call.

``run`` computes them in plain torch operations, or, where ``own`` is true, with the library's calls.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {"f32": 4, "bf16": 2, "f16": 2}
V_FULL = 151936  # the vocabulary of this repository's benchmark


def listed():
    def sample(name, T, V, dtype, **kw):
        c = dict(name=name, op="sample", T=T, V=V, dtype=dtype, pad=0, temperature=1.0, top_k=0,
                 top_p=1.0, min_p=0.0, mixed=False)
        c.update(kw)
        return c

    def distill(name, op, T, V, dtype, K, **kw):
        c = dict(name=name, op=op, T=T, V=V, dtype=dtype, pad=0, K=K, temperature=1.0,
                 kind="forward", tail=False, masked=0.0)
        c.update(kw)
        return c

    return [
        # one request decoding alone: latency
        sample("sample_one", 1, V_FULL, "bf16", temperature=0.7, top_k=50, top_p=0.95),
        # a decoding batch whose requests bring settings of their own, some greedy, some unfiltered
        sample("sample_batch_mixed", 96, V_FULL, "bf16", mixed=True),
        # the same batch after the engine widened its logits to fp32, nucleus sampling only
        sample("sample_batch_topp", 128, V_FULL, "f32", temperature=0.7, top_p=0.95),
        # on-policy rollouts for training: the whole distribution, no filter
        sample("sample_rollout_plain", 512, V_FULL, "bf16"),
        # small odd vocabulary with a padded row stride, min-p
        sample("sample_odd_minp", 37, 32003, "f16", pad=5, temperature=1.3, min_p=0.05),
        # many rows at once, the usual top-k and top-p
        sample("sample_rows_topk", 1024, V_FULL, "bf16", temperature=0.7, top_k=50, top_p=0.95),
        # evaluation of the loss alone: one long response
        distill("distill_eval", "forward", 2048, V_FULL, "bf16", 64),
        # a short ragged piece, rows that start at odd addresses
        distill("distill_eval_odd", "forward", 33, 32003, "f32", 20, kind="reverse", tail=True),
        # a training step through autograd
        distill("distill_autograd", "autograd", 1024, V_FULL, "bf16", 64, temperature=2.0, tail=True),
        # a training step with token weights known beforehand: loss and gradient in one call
        distill("distill_step", "step", 2048, V_FULL, "bf16", 64, masked=0.25),
        # the same in fp32 with a long teacher head, reverse KL
        distill("distill_step_f32", "step", 512, V_FULL, "f32", 256, kind="reverse", tail=True),
        # a short odd training piece
        distill("distill_step_odd", "step", 19, 50257, "f16", 8, temperature=1.5, masked=0.3),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["sample", "sample", "forward", "autograd", "step", "step"])
    V = rng.choice([V_FULL, _log_uniform(rng, 1000, V_FULL)])
    dtype = rng.choice(["bf16", "bf16", "f32", "f16"])
    most = 1024 if op == "sample" else 2048
    most = max(1, min(most, most * V_FULL * 2 // (V * SIZES[dtype] * (2 if op == "autograd" else 1))))
    c = dict(op=op, T=_log_uniform(rng, 1, min(most, 4096)), V=V, dtype=dtype,
             pad=rng.choice([0, 0, 0, rng.randint(1, 100)]))
    if op == "sample":
        c.update(temperature=rng.choice([1.0, round(rng.uniform(0.3, 1.5), 2)]),
                 top_k=rng.choice([0, 0, 1, _log_uniform(rng, 2, 1000)]),
                 top_p=rng.choice([1.0, round(rng.uniform(0.3, 0.99), 3)]),
                 min_p=rng.choice([0.0, 0.0, round(rng.uniform(0.01, 0.2), 3)]),
                 mixed=rng.random() < 0.3)
    else:
        c.update(K=_log_uniform(rng, 1, 512), temperature=rng.choice([1.0, round(rng.uniform(0.5, 3.0), 2)]),
                 kind=rng.choice(["forward", "reverse"]), tail=rng.random() < 0.5,
                 masked=rng.choice([0.0, round(rng.uniform(0.1, 0.6), 2)]))
    return c


def _logits(case, g, favoured):
    """Logits as a language model's head gives them: a normal bulk far below a few favoured tokens,
    some rows nearly decided and some undecided.  [T, V] in a [T, V + pad] buffer."""
    T, V = case["T"], case["V"]
    buf = torch.empty(T, V + case["pad"], dtype=DTYPES[case["dtype"]], device="cuda")
    n = favoured.shape[1]
    peak = 6.0 + 14.0 * torch.rand(T, 1, generator=g, device="cuda")
    fall = 0.3 + 2.0 * torch.rand(T, 1, generator=g, device="cuda")
    rank = torch.arange(1, n + 1, device="cuda", dtype=torch.float32)
    top = peak - fall * rank.log() + 0.5 * torch.randn(T, n, generator=g, device="cuda")
    z = buf[:, :V]
    z.copy_(torch.randn(T, V, generator=g, device="cuda").mul_(2.0).scatter_(1, favoured, top))
    return z, top


def _distinct(T, n, V, g):
    """[T, n] token ids, distinct within a row."""
    start = torch.randint(0, V, (T, 1), generator=g, device="cuda")
    stride = max(1, V // n)
    jitter = torch.randint(0, stride, (T, n), generator=g, device="cuda")
    return (start + torch.arange(n, device="cuda") * stride + jitter) % V


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T, V = case["T"], case["V"]
    if case["op"] == "sample":
        z, _ = _logits(case, g, _distinct(T, min(200, V // 2), V, g))
        s = dict(case=case, logits=z, uniform=torch.rand(T, generator=g, device="cuda"))
        keys = ("temperature", "top_k", "top_p", "min_p")
        if case["mixed"]:
            menu = torch.tensor([[0.0, 0, 1.0, 0.0], [0.7, 50, 0.95, 0.0], [1.0, 0, 1.0, 0.0],
                                 [0.6, 20, 0.95, 0.05], [1.0, 0, 0.9, 0.0], [0.8, 0, 1.0, 0.05]],
                                device="cuda")
            pick = menu[torch.randint(0, len(menu), (T,), generator=g, device="cuda")]
            for i, k in enumerate(keys):
                s[k] = pick[:, i].to(torch.int32 if k == "top_k" else torch.float32).contiguous()
        else:
            for k in keys:
                s[k] = case[k]
        return s
    K = min(case["K"], V // 2)
    ids = _distinct(T, K, V, g)
    z, top = _logits(case, g, ids)
    # the teacher agrees with the student up to noise; its head holds most of its mass
    t = top + 0.7 * torch.randn(T, K, generator=g, device="cuda")
    t, order = t.sort(dim=1, descending=True)
    ids = ids.gather(1, order)
    held = 0.6 + 0.39 * torch.rand(T, 1, generator=g, device="cuda")
    lp = torch.log_softmax(t, dim=1) + held.log()
    if case["masked"] > 0:  # rows of the prompt: no entries
        off = torch.rand(T, 1, generator=g, device="cuda") < case["masked"]
        off[0] = False
        ids = torch.where(off, torch.full_like(ids, -1), ids)
    live = (ids[:, 0] >= 0).float()
    s = dict(case=case, logits=z, ids=ids.to(torch.int32), lp=lp.contiguous(),
             weight=(live / live.sum().clamp(min=1.0)).contiguous())
    if case["op"] == "autograd":
        s["logits"] = z.detach().requires_grad_(True)
    return s


# ------------------------------------------------------------------------------- plain forms

def _per_row(v, T, device):
    if isinstance(v, torch.Tensor):
        return v.double().view(T, 1)
    # a setting given as a number is a 32-bit one
    return torch.full((T, 1), v, dtype=torch.float32, device=device).double()


def _plain_sample(s):
    z32 = s["logits"].float()
    T, V = z32.shape
    dev = z32.device
    tau, k, top_p, min_p = (_per_row(s[n], T, dev) for n in ("temperature", "top_k", "top_p", "min_p"))
    greedy = tau == 0
    tau = torch.where(greedy, torch.ones_like(tau), tau)
    k = torch.where(greedy, torch.ones_like(k), torch.where(k <= 0, torch.full_like(k, V), k))
    zs, order = torch.sort(z32, dim=1, descending=True, stable=True)
    top = zs[:, :1].double()
    w = torch.exp((zs.double() - top) / tau)  # 64 bits: a token next to a border is kept or not
    keep = (torch.arange(V, device=dev) < k) & (zs > -math.inf)
    wk = w * keep
    cum = wk.cumsum(1)
    keep &= (cum - wk < top_p * cum[:, -1:]) | (top_p >= 1)
    keep &= w >= min_p
    wid = torch.zeros_like(w).scatter_(1, order, w * keep)
    cum = wid.cumsum(1)
    S = cum[:, -1:]
    tok = (cum <= s["uniform"].double().view(T, 1) * S).sum(1, keepdim=True).clamp(max=V - 1)
    lse = top / tau + torch.log(S)
    lp = z32.gather(1, tok).double() / tau - lse
    return (tok.view(T).to(torch.int32), lp.view(T).float(), lse.view(T).float(),
            keep.sum(1).to(torch.int32))


def _plain_distill(s, grad_loss=None):
    c = s["case"]
    tau = float(torch.tensor(c["temperature"], dtype=torch.float32))
    z = s["logits"].detach()
    T, V = z.shape
    e = torch.zeros(T, V + 1, dtype=torch.float32, device=z.device)  # a last column for no entry
    x = z.float() / tau
    m = x.amax(1, keepdim=True)
    torch.exp(x - m, out=e[:, :V])
    valid = (s["ids"] >= 0) & (s["lp"] > -math.inf)
    ids = torch.where(valid, s["ids"], torch.zeros_like(s["ids"])).long()
    # 64 bits for the K terms of a row: the loss is a difference of near numbers
    xk = z.gather(1, ids).double() / tau
    ek = torch.where(valid, torch.exp(xk - m), torch.zeros_like(xk))
    at = torch.where(valid, ids, torch.full_like(ids, V))
    rest = e.scatter(1, at, 0.0).sum(1, keepdim=True, dtype=torch.float64)
    P0 = ek.sum(1, keepdim=True)
    S = rest + P0
    lse = m + torch.log(S)
    lq = s["lp"].double()
    q = torch.where(valid, torch.exp(lq), torch.zeros_like(lq))
    Q = q.sum(1, keepdim=True)
    qr = 1.0 - Q
    tail = torch.full_like(Q, bool(c["tail"]), dtype=torch.bool) & (qr > 2.0 ** -20) & (rest > 0)
    qr = torch.where(tail, qr, torch.zeros_like(qr))
    pk, pr, P = ek / S, rest / S, P0 / S
    a = torch.where(valid, xk - lse - lq, torch.zeros_like(lq))  # ln p - ln q
    ar = torch.where(tail, torch.log(pr) - torch.log(torch.where(tail, qr, torch.ones_like(qr))),
                     torch.zeros_like(pr))
    if c["kind"] == "forward":
        loss = -(q * a).sum(1, keepdim=True) - qr * ar
        c_rest = Q - torch.where(tail, qr * P / pr, torch.zeros_like(pr))
        g_head = pk * (Q + qr) - q
    else:
        tr = torch.where(tail, pr, torch.zeros_like(pr))
        loss = (pk * a).sum(1, keepdim=True) + tr * ar
        B = (pk * (a + 1)).sum(1, keepdim=True) + tr * (ar + 1)
        c_rest = torch.where(tail, ar + 1, torch.zeros_like(ar)) - B
        g_head = pk * (a + 1 - B)
    empty = ~valid.any(1, keepdim=True)
    zero = torch.zeros_like(loss)
    loss = torch.where(empty, zero, loss).view(-1).float()
    if grad_loss is None:
        return loss, torch.where(empty, zero, lse).view(-1).float()
    scale = torch.where(empty, zero, grad_loss.double().view(-1, 1) / tau)
    d = e.mul_((c_rest * scale / S).float()).scatter_(1, at, (g_head * scale).float())
    return loss, d[:, :V].to(z.dtype)


# ------------------------------------------------------------------------------- one pass

def run(state):
    c = state["case"]
    if not own:
        if c["op"] == "sample":
            return _plain_sample(state)
        return _plain_distill(state, None if c["op"] == "forward" else state["weight"])
    import rollout_logprob_consistency_gb300 as tim
    if "workspace" not in state:  # a user's program keeps one
        state["workspace"] = tim.Workspace(1024)
    ws = state["workspace"]
    if c["op"] == "sample":
        return tim.sample(state["logits"], state["uniform"], state["temperature"], state["top_k"],
                          state["top_p"], state["min_p"], workspace=ws, check=False)
    args = (state["logits"], state["ids"], state["lp"])
    how = dict(temperature=c["temperature"], kind=c["kind"], tail=c["tail"], workspace=ws, check=False)
    if c["op"] == "forward":
        loss, lse, _ = tim.distill(*args, **how)
        return loss, lse
    if c["op"] == "step":
        return tim.distill_grad(*args, state["weight"], **how)
    loss = tim.distill_loss(*args, **how)
    grad, = torch.autograd.grad(loss, state["logits"], state["weight"])
    return loss.detach(), grad


def work(case):
    n, e = case["T"] * case["V"], SIZES[case["dtype"]]
    if case["op"] == "sample":
        return {"bytes": n * e + case["T"] * 20, "flops": 4 * n}
    live = 1.0 - case["masked"]
    small = case["T"] * (8 * case["K"] + 8)
    if case["op"] == "forward":
        return {"bytes": live * n * e + small, "flops": live * 4 * n}
    return {"bytes": (1 + live) * n * e + small + 4 * case["T"], "flops": live * 8 * n}


# ------------------------------------------------------------------------------- 64 bits

@torch.no_grad()
def exact(case, seed):
    """Row by row in 64 bits: the scores of the token that the sampler's definition gives, or the
    loss and its gradient from the buckets (a head token each, the others together)."""
    s = prepare(case, seed)
    T, V = s["logits"].shape

    def number(x, i):  # a setting given as a number is a 32-bit one
        return x[i].item() if isinstance(x, torch.Tensor) else float(torch.tensor(float(x)))

    if case["op"] == "sample":
        lps, lses = [], []
        for i in range(T):
            z = s["logits"][i].double()
            tau, k, p, mp = (number(s[n], i) for n in ("temperature", "top_k", "top_p", "min_p"))
            if tau == 0:
                lps.append(torch.zeros((), dtype=torch.float64, device=z.device))
                lses.append(z.max())
                continue
            x = z / tau
            logp = x - torch.logsumexp(x, 0)
            order = torch.argsort(z, descending=True, stable=True)
            if 0 < k < V:
                order = order[: int(k)]
            lq = logp[order] - torch.logsumexp(logp[order], 0)
            if p < 1:
                order = order[: 1 + int((lq.exp().cumsum(0)[:-1] < p).sum())]
            order = order[logp[order] - logp[order[0]] >= (math.log(mp) if mp > 0 else -math.inf)]
            kept = torch.sort(order).values
            lse = torch.logsumexp(x[kept], 0)
            cdf = (x[kept] - lse).exp().cumsum(0)
            at = torch.searchsorted(cdf, s["uniform"][i].double(), right=True)
            lps.append(x[kept[at.clamp(max=len(kept) - 1)]] - lse)
            lses.append(lse)
        return None, torch.stack(lps), torch.stack(lses), None

    tau = number(case["temperature"], 0)
    with_grad = case["op"] != "forward"
    loss = torch.zeros(T, dtype=torch.float64, device="cuda")
    lse = torch.zeros(T, dtype=torch.float64, device="cuda")
    grad = torch.zeros(T, V if with_grad else 0, dtype=torch.float64, device="cuda")
    for i in range(T):
        on = (s["ids"][i] >= 0) & (s["lp"][i] > -math.inf)
        ids, lq = s["ids"][i][on].long(), s["lp"][i][on].double()
        if not len(ids):
            continue
        x = s["logits"][i].double() / tau
        lse[i] = torch.logsumexp(x, 0)
        logp = x - lse[i]
        outside = torch.ones(V, dtype=torch.bool, device="cuda")
        outside[ids] = False
        lk = logp[ids]
        lr = torch.logsumexp(logp.masked_fill(~outside, -math.inf), 0)
        qr = 1.0 - lq.exp().sum()
        tail = bool(case["tail"]) and bool(qr > 2.0 ** -20) and bool(lr > -math.inf)
        if tail:
            lk, lq = torch.cat([lk, lr.view(1)]), torch.cat([lq, qr.log().view(1)])
        if case["kind"] == "forward":
            loss[i] = (lq.exp() * (lq - lk)).sum()
            by = -lq.exp()  # dL / d ln p of each bucket
        else:
            loss[i] = (lk.exp() * (lk - lq)).sum()
            by = lk.exp() * (lk - lq + 1)
        if with_grad:
            p = logp.exp()
            g = -p * by.sum()  # every ln p has -p_v from the normaliser
            g[ids] += by[: len(ids)]
            if tail:
                g += torch.where(outside, p * (by[-1] / lr.exp()), torch.zeros_like(p))
            grad[i] = g * (s["weight"][i].double() / tau)
    return (loss, grad) if with_grad else (loss, lse)
