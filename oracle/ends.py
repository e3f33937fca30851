"""fp64 oracle for the operators at a model's two ends: the verification of drafted tokens, the
embedding lookup and its gradient, the residual update with the norms around a block.
TEST INFRASTRUCTURE ONLY.

Straight from the definitions in include/tim.h, in 64 bits.
"""
from __future__ import annotations

import math

import numpy as np


# ----------------------------------------------------------------------------- embedding

def embed(table, ids, scale: float):
    table = np.asarray(table, dtype=np.float64)
    out = np.zeros((len(ids), table.shape[1]))
    for t, v in enumerate(ids):
        if v >= 0:
            out[t] = scale * table[v]
    return out


def embed_backward(dy, ids, V: int, scale: float):
    """(the gradient, scale sum |dy|, how many rows a token has)."""
    dy = np.asarray(dy, dtype=np.float64)
    ids = np.asarray(ids)
    grad, size = np.zeros((V, dy.shape[1])), np.zeros((V, dy.shape[1]))
    on = ids >= 0
    np.add.at(grad, ids[on], dy[on])
    np.add.at(size, ids[on], np.abs(dy[on]))
    return scale * grad, abs(scale) * size, np.bincount(ids[on], minlength=V)


# ----------------------------------------------------------------------------- residual norm

def residual_norm(h, x, gamma, gamma_post, gate, scale: float, eps: float):
    """(h' unrounded, scale g n); gate broadcastable to [T, d] or None."""
    h, x = np.asarray(h, np.float64), np.asarray(x, np.float64)
    n = x
    if gamma_post is not None:
        n = x / np.sqrt(np.mean(x * x, 1, keepdims=True) + eps) * gamma_post
    step = scale * n * (1.0 if gate is None else gate)
    return h + step, step


def norm_rows(h, gamma, eps: float):
    h = np.asarray(h, np.float64)
    return h / np.sqrt(np.mean(h * h, 1, keepdims=True) + eps) * gamma


def residual_norm_backward(h, x, dh, dy, gamma, gamma_post, gate, scale: float, eps: float):
    """dict of the gradients, each a pair (value, E): E 2^-24 bounds what fp32 arithmetic may be off.

    A sum over a row is 32 additions in a thread at most and 10 among threads; with the products of its
    terms below 45 roundings of the terms' sizes.  r = 1 / sqrt(mean + eps): half the 43 of its sum and
    4 of its own, below 26; r^3 below 80."""
    x = np.asarray(x, np.float64)
    T, d = x.shape
    H, EH = np.zeros((T, d)), np.zeros((T, d))
    out = {}
    if dh is not None:
        H, EH = H + dh, EH + 3 * np.abs(dh)
    if gamma is not None:
        if dy is not None:
            r = 1.0 / np.sqrt(np.mean(h * h, 1, keepdims=True) + eps)
            a = r * gamma * dy
            size = np.abs(h) * r ** 3 / d * np.sum(np.abs(gamma * dy * h), 1, keepdims=True)
            H = H + a - h * (r ** 3 / d * np.sum(gamma * dy * h, 1, keepdims=True))
            EH = EH + 33 * np.abs(a) + 130 * size
            out["dgamma"] = (np.sum(dy * h * r, 0), (T + 70) * np.sum(np.abs(dy * h * r), 0))
        else:
            out["dgamma"] = (np.zeros(d), np.zeros(d))
    out["dresidual"] = (H, EH)
    n, r1 = x, 1.0
    if gamma_post is not None:
        r1 = 1.0 / np.sqrt(np.mean(x * x, 1, keepdims=True) + eps)
        n = x * r1 * gamma_post
    g = 1.0 if gate is None else gate
    dn = scale * g * H
    E = np.abs(scale * g) * EH + 3 * np.abs(dn)
    if gate is not None:
        full, Ef = scale * n * H, np.abs(scale * n) * EH + 32 * np.abs(scale * n * H)
        axes = {(T, d): None, (d,): 0, (T, 1): 1}[np.shape(gate) if d > 1 or np.ndim(gate) == 1 else (T, 1)]
        if axes is None:
            out["dgate"] = (full, Ef)
        else:
            k = (T + 70) if axes == 0 else 45
            out["dgate"] = (np.sum(full, axes, keepdims=axes == 1),
                            np.sum(Ef + k * np.abs(full), axes, keepdims=axes == 1))
    if gamma_post is None:
        out["dblock"] = (dn, E)
    else:
        b = gamma_post * dn
        out["dgamma_post"] = (np.sum(dn * x * r1, 0),
                              np.sum(np.abs(x * r1) * E + (T + 70) * np.abs(dn * x * r1), 0))
        c = r1 ** 3 / d
        out["dblock"] = (r1 * b - x * c * np.sum(b * x, 1, keepdims=True),
                         np.abs(r1 * gamma_post) * E + 30 * np.abs(r1 * b) + np.abs(x) * c *
                         np.sum(np.abs(gamma_post * x) * E + 130 * np.abs(b * x), 1, keepdims=True))
    return out


# ----------------------------------------------------------------------------- verification

NO_REST = 2.0 ** -28  # of max(p - q, 0), below which p is drawn from


def processed(z, temperature: float, top_k: int, top_p: float, min_p: float):
    """(p [V], ln p [V], how near the nearest border of a filter lies)."""
    z = np.asarray(z, dtype=np.float64)
    V = z.shape[0]
    lp = np.full(V, -np.inf)
    order = np.lexsort((np.arange(V), -z))
    if temperature == 0.0:
        lp[order[0]] = 0.0
        return np.exp(lp), lp, math.inf
    order = order[z[order] > -np.inf]
    if 0 < top_k < V:
        order = order[:top_k]
    s = (z[order] - z[order[0]]) / temperature
    w = np.exp(s)
    keep, margin = w >= min_p, math.inf
    if top_p < 1.0:
        before = np.concatenate(([0.0], np.cumsum(w)[:-1])) / np.sum(w)
        keep &= before < top_p
        margin = float(np.min(np.abs(before - top_p)))
    lp[order[keep]] = s[keep] - math.log(np.sum(w[keep]))
    return np.exp(lp), lp, margin


def verify_sequence(target, draft, ids, uniform, uniform_draw: float, settings, draft_settings=None):
    """ids, logprob [N + 1], accepted, and ``margin``: how near the nearest border of a decision lies,
    in units of the mass of p (of an acceptance: relative to p of the token)."""
    N = len(ids)
    out, lps, margin = [], [], math.inf
    for j in range(N + 1):
        p, lp, m = processed(target[j], *settings)
        margin = min(margin, m)
        x = int(ids[j]) if j < N else -1
        r = p
        if x >= 0:
            if draft is None:
                q, lq = np.zeros_like(p), 0.0
                q[x] = 1.0
            else:
                q, lq, m = processed(draft[j], *(draft_settings or settings))
                lq = lq[x]
                margin = min(margin, m)
            # u q(x) < p(x), which both may lie below the range of a number
            ln_uq = lq + (math.log(uniform[j]) if uniform[j] > 0 else -math.inf)
            if lp[x] > -math.inf and ln_uq > -math.inf:
                margin = min(margin, abs(ln_uq - lp[x]))
            if ln_uq < lp[x]:
                out.append(x)
                lps.append(float(lp[x]))
                continue
            rest = np.maximum(p - q, 0.0)
            margin = min(margin, abs(rest.sum() - NO_REST))
            if rest.sum() >= NO_REST:
                r = rest
        c = np.cumsum(r)
        at = int(np.searchsorted(c, uniform_draw * c[-1], side="right"))
        y = min(at, int(np.nonzero(r)[0][-1]))
        if uniform_draw > 0:
            margin = min(margin, float(np.min(np.abs(c - uniform_draw * c[-1]))))
        out.append(y)
        lps.append(float(lp[y]))
        break
    n = len(out) - 1
    pad = N + 1 - len(out)
    return dict(ids=out + [-1] * pad, logprob=lps + [0.0] * pad, accepted=n, margin=margin)
