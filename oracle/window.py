"""Plain numpy oracle of the calls around the verify and the cache, in 64 bits:
logit adjustment, rotary positions, accumulated attention and eviction.

Written from the definitions in include/spec_verify.h, loops over requests,
rows and tokens, no kernel's order of operations.
"""
from __future__ import annotations

import math

import numpy as np

from . import kv


def _bit(words, t):
    return (int(words[t // 32]) >> (t % 32)) & 1


# ------------------------------------------------------------------ logits
def adjust(logits, out, tokens=None, token_lens=None, prompt_lens=None, repetition=None, frequency=None, presence=None,
           bias_ids=None, bias_values=None, allowed=None, allowed_rows=None, draft_tokens=None, draft_lens=None,
           masks=None):
    """logits [B, R, V] float64; returns `out` (what lies behind a request's last row) with the adjusted rows."""
    B, R, V = logits.shape
    out = np.array(out, dtype=np.float64)
    counted = any(x is not None for x in (repetition, frequency, presence))
    for b in range(B):
        rows = R
        if draft_lens is not None:
            rows = int(draft_lens[b]) + 1 if 0 <= draft_lens[b] < R else 0
        prompt, said = set(), {}
        if counted and tokens is not None:
            n = len(tokens[b]) if token_lens is None else min(max(int(token_lens[b]), 0), len(tokens[b]))
            p = 0 if prompt_lens is None else min(max(int(prompt_lens[b]), 0), n)
            prompt = {int(t) for t in tokens[b][:p]}
            for t in tokens[b][p:n]:
                said[int(t)] = said.get(int(t), 0) + 1
        for r in range(rows):
            x = logits[b, r].astype(np.float64).copy()
            c = dict(said)
            if counted and draft_tokens is not None:
                for m, t in enumerate(draft_tokens[b]):
                    before = m < r if masks is None else m > 0 and _bit(masks[b, r], m)
                    if before:
                        c[int(t)] = c.get(int(t), 0) + 1
            if counted:
                for t in prompt | set(c):
                    if not 0 <= t < V:
                        continue
                    if repetition is not None:
                        x[t] = x[t] / repetition[b] if x[t] > 0 else x[t] * repetition[b]
                    if t in c:
                        x[t] -= (0.0 if frequency is None else frequency[b]) * c[t]
                        x[t] -= 0.0 if presence is None else presence[b]
            if bias_ids is not None:
                for t, v in zip(bias_ids[b], bias_values[b]):
                    if 0 <= t < V:
                        x[t] += v
            if allowed is not None:
                a = b * R + r if allowed_rows is None else int(allowed_rows[b, r])
                if a >= len(allowed):
                    x[:] = -np.inf
                elif a >= 0:
                    for t in range(V):
                        if not _bit(allowed[a], t):
                            x[t] = -np.inf
            out[b, r] = x
    return out


# ------------------------------------------------------------------ rotary positions
def positions(B, W, starts, masks=None):
    p = np.zeros((B, W), dtype=object)
    for b in range(B):
        for i in range(W):
            depth = i if masks is None else max(0, sum(_bit(masks[b, i], m) for m in range(W)) - 1)
            p[b, i] = int(starts[b]) + depth
    return p


def _turn(position, f):
    """Sine and cosine of position * f, the product exact (integers over a power of two) and reduced by a
    period of 200 bits."""
    n, d = float(f).as_integer_ratio()
    tau = 2 * 0x3243F6A8885A308D313198A2E03707344A4093822299F31D0082EFA98EC4E6C89  # 2 pi 2^256
    x = (abs(position * n) << 256) // d % tau
    a = math.copysign(1.0, position * n) * (x / 2 ** 256)
    return math.sin(a), math.cos(a)


def rotate(x, out, starts, inv_freq, interleaved=False, gain=1.0, window_lens=None, masks=None):
    """x [B, W, heads, D] float64; returns `out` with the rotated rows."""
    B, W, _, D = x.shape
    out, pairs = np.array(out, dtype=np.float64), len(inv_freq)
    pos = positions(B, W, starts, masks)
    for b in range(B):
        w = W if window_lens is None else int(window_lens[b])
        if not 0 <= w <= W:
            continue
        for i in range(w):
            out[b, i] = x[b, i]
            for p in range(pairs):
                s, c = _turn(pos[b, i], inv_freq[p])
                u, v = (2 * p, 2 * p + 1) if interleaved else (p, p + pairs)
                a, z = x[b, i, :, u], x[b, i, :, v]
                out[b, i, :, u] = gain * (a * c - z * s)
                out[b, i, :, v] = gain * (z * c + a * s)
    return out


# ------------------------------------------------------------------ accumulated attention
def weigh(q, lse, pool, scales, tables, seq_lens, out, window_lens=None, scale=None, weights=None, decay=1.0):
    """Returns (out, spread): `out` [B, H, T] with the weights of each request's positions, and the largest
    scale * sum |q_d k_d| of the rows of each KV head [B, H]."""
    B, W, Hq, D = q.shape
    N, _, H, tpb, _ = pool.shape
    scale = D ** -0.5 if scale is None else scale
    out = np.array(out, dtype=np.float64)
    spread = np.zeros((B, H))
    T = out.shape[2]
    for b in range(B):
        w, s = W if window_lens is None else int(window_lens[b]), int(seq_lens[b])
        if s < 0 or not 0 <= w <= W or s + w > tables.shape[1] * tpb:
            continue
        for h in range(H):
            for t in range(min(s + w, T)):
                x = float(decay) * float(weights[b, h, t]) if weights is not None and t < s else 0.0
                blk = kv._mapped(tables, N, b, t, tpb)
                if blk is None:
                    out[b, h, t] = np.nan
                    continue
                k = kv.decode(pool[blk, 0, h, t % tpb]) * float(scales[blk, 0, h])
                heads = slice(h * (Hq // H), (h + 1) * (Hq // H))
                i0 = max(0, t - s)
                e = lse[b, i0:w, heads]
                a = scale * (q[b, i0:w, heads] @ k)
                with np.errstate(invalid="ignore"):
                    p = np.where(e == -np.inf, 0.0, np.exp(a - np.where(e == -np.inf, 0.0, e)))
                if p.size:
                    spread[b, h] = max(spread[b, h], abs(scale) * (np.abs(q[b, i0:w, heads]) @ np.abs(k)).max())
                out[b, h, t] = x + p.sum()
    return out, spread


# ------------------------------------------------------------------ eviction
def evict(weights, pool, scales, tables, seq_lens, keep, first=0, recent=0, held=None, out_weights=None):
    """Returns (new_lens, kept, out_weights, free, pool, scales)."""
    pool, scales = pool.copy(), scales.astype(np.float64)
    N, _, H, tpb, _ = pool.shape
    B, _, T = weights.shape
    kept = np.full((B, H, keep), -1, np.int32)
    out = np.zeros((B, H, keep), np.float32) if out_weights is None else out_weights.copy()
    new, free = np.array(seq_lens, np.int32).copy(), np.zeros(B, np.int32)
    for b in range(B):
        n = int(seq_lens[b])
        if n < 0 or n > T or n > tables.shape[1] * tpb or any(
                kv._mapped(tables, N, b, t, tpb) is None for t in range(0, n, tpb)):
            continue
        new[b] = min(n, keep)
        if held is not None:
            free[b] = max(0, int(held[b]) - -(-int(new[b]) // tpb))
        for h in range(H):
            if n <= keep:
                kept[b, h, :n] = np.arange(n)
                out[b, h, :n] = weights[b, h, :n]
                continue
            # by weight from the largest, by position among equals; NaN last
            middle = sorted(range(first, n - recent), key=lambda t: (
                (1, 0.0, t) if np.isnan(weights[b, h, t]) else (0, -float(weights[b, h, t]), t)))
            stay = sorted([*range(first), *middle[:keep - first - recent], *range(n - recent, n)])
            kept[b, h] = stay
            out[b, h, :keep] = weights[b, h, stay]
            at = [(int(tables[b, t // tpb]), t % tpb) for t in stay]
            for kind in range(2):
                rows = [(pool[blk, kind, h, off].copy(), float(scales[blk, kind, h])) for blk, off in at]
                for j0 in range(0, keep, tpb):
                    part = rows[j0:j0 + tpb]
                    blk, top = int(tables[b, j0 // tpb]), max(s for _, s in part)
                    for off, (codes, s) in enumerate(part):
                        pool[blk, kind, h, off] = codes if s == top else kv.encode(kv.decode(codes) * kv._over(s, top))
                    scales[blk, kind, h] = top
    return new, kept, out, free, pool, scales
