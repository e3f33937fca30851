"""fp64 oracle for the operators on a logits matrix: the sampler and the distillation loss.
TEST INFRASTRUCTURE ONLY.

One row at a time, straight from the definitions in include/tim.h; nothing is fused and no
border is found by anything but a sort and running sums in 64 bits.
"""
from __future__ import annotations

import math

import numpy as np

TAIL_FLOOR = 2.0 ** -20


def sample_row(z, u: float, temperature: float, top_k: int, top_p: float, min_p: float) -> dict:
    """Token, logprob, lse and number kept of one row, and ``margin``: how near, in units of the
    kept mass (top-p: of the top-k mass), the nearest border of a decision lies."""
    z = np.asarray(z, dtype=np.float64)
    V = z.shape[0]
    order = np.lexsort((np.arange(V), -z))
    if temperature == 0.0:
        x = int(order[0])
        return dict(id=x, logprob=0.0, lse=float(z[x]), kept=1, margin=math.inf)
    order = order[z[order] > -np.inf]
    if 0 < top_k < V:
        order = order[:top_k]
    s = z[order] / temperature
    w = np.exp(s - s[0])
    margin = math.inf
    keep = np.ones(len(order), dtype=bool)
    if top_p < 1.0:
        before = np.concatenate(([0.0], np.cumsum(w)[:-1])) / np.sum(w)
        keep = before < top_p
        margin = float(np.min(np.abs(before - top_p)))
    keep &= w >= min_p
    ids = np.sort(order[keep])
    s = z[ids] / temperature
    m = float(np.max(s))
    e = np.exp(s - m)
    c = np.cumsum(e)
    S = float(c[-1])
    at = int(np.searchsorted(c, u * S, side="right"))
    at = min(at, len(ids) - 1)
    margin = min(margin, float(np.min(np.abs(c - u * S))) / S if u > 0 else math.inf)
    lse = m + math.log(S)
    return dict(id=int(ids[at]), logprob=float(s[at] - lse), lse=lse, kept=int(len(ids)),
                margin=margin)


def distill_row(z, ids, lp, temperature: float, kind: str, tail: bool):
    """(loss, lse, dL/dz) of one row."""
    z = np.asarray(z, dtype=np.float64)
    lp = np.asarray(lp, dtype=np.float64)
    ids = np.asarray(ids, dtype=np.int64)
    on = (ids >= 0) & (lp > -np.inf)
    ids, lq = ids[on], lp[on]
    if ids.size == 0:
        return 0.0, 0.0, np.zeros_like(z)
    s = z / temperature
    m = np.max(s)
    lse = float(m + np.log(np.sum(np.exp(s - m))))
    logp = s - lse
    p = np.exp(logp)
    q = np.exp(lq)
    head = np.zeros(z.shape[0], dtype=bool)
    head[ids] = True
    pr = float(np.sum(p[~head]))
    qr = 1.0 - float(np.sum(q))
    tail = tail and qr > TAIL_FLOOR and pr > 0.0
    with np.errstate(invalid="ignore", divide="ignore"):
        if kind == "forward":
            loss = float(np.sum(np.where(q > 0, q * (lq - logp[ids]), 0.0)))
            by_head, by_rest = -q, 0.0      # dL / d ln p of a bucket
            if tail:
                loss += qr * (math.log(qr) - math.log(pr))
                by_rest = -qr
        else:
            pk = p[ids]
            a = logp[ids] - lq
            loss = float(np.sum(np.where(pk > 0, pk * a, 0.0)))
            by_head, by_rest = np.where(pk > 0, pk * (a + 1.0), 0.0), 0.0
            if tail:
                ar = math.log(pr) - math.log(qr)
                loss += pr * ar
                by_rest = pr * (ar + 1.0)
    g = -p * (np.sum(by_head) + by_rest)
    g[ids] += by_head
    if tail:
        g[~head] += by_rest * p[~head] / pr
    return loss, lse, g / temperature
