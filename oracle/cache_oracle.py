"""Shared-prefix decode attention and cache eviction, from their definitions in
float64 (plain numpy loops; test infrastructure only)."""
from __future__ import annotations

import math

import numpy as np


def _f64(x):
    return x.detach().cpu().double().numpy() if hasattr(x, "detach") else np.asarray(x, np.float64)


def prefix_attention(q, kp, vp, k, v, lens, weights=None):
    """One decode step: q [B, T, H, d]; prefix kp, vp [G, Np, d]; own caches
    k, v [B, G, C, d] with lens[b] valid rows, the last T of them the new
    tokens.  Query t of sequence b sees the prefix and own rows
    x <= lens[b] - T + t.  Returns (o [B, T, H, d], lse [B, T, H], weights
    [B, G, C]: the given ones plus the softmax weight every own key received,
    absum [B, T, H, d]: sum of the softmax weights times |v|, reach [B, T, H]:
    largest sum over the head dim of |q k| / sqrt(d) of a seen key)."""
    q, kp, vp, k, v = (_f64(x) for x in (q, kp, vp, k, v))
    B, T, H, d = q.shape
    G, C = k.shape[1], k.shape[2]
    r = H // G
    o, absum = np.zeros((B, T, H, d)), np.zeros((B, T, H, d))
    lse, reach = np.full((B, T, H), -np.inf), np.zeros((B, T, H))
    w = np.zeros((B, G, C)) if weights is None else _f64(weights).copy()
    for b in range(B):
        for t in range(T):
            n = min(max(int(lens[b]) - T + t + 1, 0), C)
            for h in range(H):
                g = h // r
                keys = np.concatenate([kp[g], k[b, g, :n]])
                vals = np.concatenate([vp[g], v[b, g, :n]])
                if len(keys) == 0:
                    continue
                s = keys @ q[b, t, h] / math.sqrt(d)
                e = np.exp(s - s.max())
                p = e / e.sum()
                o[b, t, h] = p @ vals
                absum[b, t, h] = p @ np.abs(vals)
                lse[b, t, h] = s.max() + math.log(e.sum())
                reach[b, t, h] = (np.abs(keys) @ np.abs(q[b, t, h])).max() / math.sqrt(d)
                w[b, g, :n] += p[len(kp[g]):]
    return o, lse, w, absum, reach


def evict_plan(weights, positions, length, budget, first, recent):
    """The rows of one (sequence, group) that move: (from, to), both ascending.
    Kept are the first min(length, budget) rows under (always-staying rows,
    weight descending, row ascending); kept rows past that count go to the
    dropped rows before it."""
    n = min(length, budget)
    w = np.asarray(weights[:length], dtype=np.float64)
    pos = np.asarray(positions[:length], dtype=np.int64)
    if n == length:
        return np.zeros(0, np.int64), np.zeros(0, np.int64)
    stays = (pos < first) | (pos > pos.max() - recent)
    score = [(not stays[x], math.inf if math.isnan(w[x]) else -w[x], x) for x in range(length)]
    kept = {x for _, _, x in sorted(score)[:n]}
    to = np.array([x for x in range(n) if x not in kept], dtype=np.int64)
    frm = np.array([x for x in range(n, length) if x in kept], dtype=np.int64)
    return frm, to


def evict(k, v, weights, positions, lens, budget, first, recent):
    """Eviction on copies of k, v [B, G, C, d], weights, positions [B, G, C]:
    (k, v, weights, positions, new_lens) as numpy arrays of the given types
    (bf16 tensors stay torch tensors)."""
    k, v = k.clone(), v.clone()
    w, pos = np.array(weights, copy=True), np.array(positions, copy=True)
    new = []
    for b, ln in enumerate(int(x) for x in lens):
        n = min(ln, budget)
        new.append(n)
        for g in range(w.shape[1]):
            frm, to = evict_plan(w[b, g], pos[b, g], ln, budget, first, recent)
            for f, t in zip(frm, to):
                k[b, g, t], v[b, g, t] = k[b, g, f], v[b, g, f]
                w[b, g, t], pos[b, g, t] = w[b, g, f], pos[b, g, f]
            w[b, g, n:ln], pos[b, g, n:ln] = 0.0, -1
    return k, v, w, pos, np.array(new, dtype=np.int32)
