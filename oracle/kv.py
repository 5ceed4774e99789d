"""Plain numpy oracle of the paged 8-bit KV cache calls, in 64 bits.

Written from the definitions in include/spec_verify.h: loops over requests,
rows and blocks, no kernel's order of operations.  e4m3: 1 sign, 4 exponent
bits (bias 7), 3 mantissa bits, subnormals of 2^-9, no infinities, NaN at
0x7f; the largest value is 448.
"""
from __future__ import annotations

import math

import numpy as np


def _values():
    v = np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)])
    v[127] = np.nan
    return np.concatenate([v, -v])


E4M3 = _values()


def decode(codes):
    return E4M3[np.asarray(codes, dtype=np.uint8)]


def encode(x):
    """Nearest e4m3 code, ties to the even code; not finite: NaN (0x7f)."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    grid = E4M3[:127]
    hi = np.clip(np.searchsorted(grid, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    down, up = a - grid[lo], grid[hi] - a
    code = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.signbit(x), code + 128, code)
    return np.where(np.isfinite(x), code, 127).astype(np.uint8)


def scale_for(amax):
    """The least power of two s >= 2^-126 with amax <= 448 s; 0 for 0."""
    if amax == 0:
        return 0.0
    e = -126
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def _over(a, b):
    return a / b if b > 0 else 0.0


def _finite_amax(x):
    x = np.abs(np.asarray(x, dtype=np.float64))
    x = x[np.isfinite(x)]
    return float(x.max()) if x.size else 0.0


def _wins(window_lens, B, W):
    return [W] * B if window_lens is None else [int(x) for x in window_lens]


def _mapped(tables, num_blocks, b, t, tpb):
    if t < 0 or t >= tables.shape[1] * tpb:
        return None
    blk = int(tables[b, t // tpb])
    return blk if 0 <= blk < num_blocks else None


# ------------------------------------------------------------------ blocks
def reserve(seq_lens, window_lens, tables, held, free, count, tpb, W):
    """Returns (slots, granted, tables, held, count)."""
    tables, held, count = tables.copy(), held.copy(), int(count)
    B, cols = tables.shape
    win = _wins(window_lens, B, W)
    slots = np.full((B, W), -1, np.int32)
    granted = np.full(B, -1, np.int32)
    dry = False
    for b in range(B):
        s, w, h = int(seq_lens[b]), win[b], int(held[b])
        if s < 0 or not 0 <= w <= W or not 0 <= h <= cols or -(-(s + w) // tpb) > cols:
            continue
        need = max(0, -(-(s + w) // tpb) - h)
        if need and (dry or need > (count if 0 <= count <= len(free) else 0)):
            dry = True
            continue
        for i in range(need):
            count -= 1
            tables[b, h + i] = free[count]
        held[b] = h + need
        granted[b] = w
        for i in range(w):
            blk = int(tables[b, (s + i) // tpb])
            if 0 <= blk < len(free):
                slots[b, i] = blk * tpb + (s + i) % tpb
    return slots, granted, tables, held, count


def release(tables, held, counts, free, count):
    """Returns (tables, held, free, count)."""
    tables, held, free, count = tables.copy(), held.copy(), free.copy(), int(count)
    n = [int(c) if 0 <= h <= tables.shape[1] and 0 <= c <= h else 0 for c, h in zip(counts, held)]
    if count < 0 or count + sum(n) > len(free):
        return tables, held, free, count
    for b in reversed(range(len(n))):
        for _ in range(n[b]):
            held[b] -= 1
            free[count] = tables[b, held[b]]
            tables[b, held[b]] = -1
            count += 1
    return tables, held, free, count


def tree_masks(paths, N):
    B, P, L = paths.shape
    bits = np.zeros((B, N, -(-N // 32) * 32), dtype=np.uint8)
    for b in range(B):
        for path in paths[b]:
            if path[0] != 0:
                continue
            path = path[:np.flatnonzero(path < 0)[0]] if (path < 0).any() else path
            if (path >= N).any():
                bits[b] = 0
                break
            for d in range(len(path)):
                bits[b, path[d], path[:d + 1]] = 1
    return np.packbits(bits, axis=-1, bitorder="little").view(np.int32)


def mask_bits(masks, W):
    m = np.ascontiguousarray(masks).view(np.uint8)
    return np.unpackbits(m, axis=-1, bitorder="little")[:, :, :W].astype(bool)


# ------------------------------------------------------------------ the cache's contents
def _write(pool, scales, blk, first, rows, least):
    """rows [n, 2, H, D] (true values, NaN for what is not finite) into block
    blk from offset first; least [2, H]: the scale the rows ask for."""
    for kind in range(2):
        for h in range(pool.shape[2]):
            new, old = float(least[kind, h]), float(scales[blk, kind, h])
            if first and old >= new:
                new = old
            elif first:
                pool[blk, kind, h, :first] = encode(decode(pool[blk, kind, h, :first]) * _over(old, new))
            scales[blk, kind, h] = new
            pool[blk, kind, h, first:first + len(rows)] = encode(rows[:, kind, h] * _over(1.0, new))


def store(k, v, pool, scales, tables, seq_lens, window_lens=None):
    """k, v [B, W, H, D] float64; pool uint8; returns (pool, scales)."""
    pool, scales = pool.copy(), scales.astype(np.float64)
    n, _, H, tpb, D = pool.shape
    B, W = k.shape[:2]
    for b, w in enumerate(_wins(window_lens, B, W)):
        s = int(seq_lens[b])
        if s < 0 or not 0 < w <= W or s + w > tables.shape[1] * tpb:
            continue
        if any(_mapped(tables, n, b, t, tpb) is None for t in range(s, s + w)):
            continue
        t = s
        while t < s + w:
            end = min(s + w, (t // tpb + 1) * tpb)
            x = np.stack([k[b, t - s:end - s], v[b, t - s:end - s]], 1).astype(np.float64)
            least = np.array([[scale_for(_finite_amax(x[:, i, h])) for h in range(H)] for i in range(2)])
            _write(pool, scales, _mapped(tables, n, b, t, tpb), t % tpb, x, least)
            t = end
    return pool, scales


def relocate(pool, scales, tables, base_lens, nodes, accepted):
    pool, scales = pool.copy(), scales.astype(np.float64)
    N, _, H, tpb, D = pool.shape
    for b in range(len(base_lens)):
        n, base, path = int(accepted[b]), int(base_lens[b]), [int(x) for x in nodes[b]]
        if n <= 0 or n >= len(path) or path[0] != 0 or any(path[j] <= path[j - 1] for j in range(1, n + 1)):
            continue
        src = [base + path[j] for j in range(1, n + 1)]
        dst = [base + j for j in range(1, n + 1)]
        if any(_mapped(tables, N, b, t, tpb) is None for t in src + dst):
            continue
        codes = np.stack([pool[_mapped(tables, N, b, t, tpb), :, :, t % tpb] for t in src])
        had = np.stack([scales[_mapped(tables, N, b, t, tpb)] for t in src])
        j = 0
        while j < n:
            end = min(n, (dst[j] // tpb + 1) * tpb - base - 1)
            blk = _mapped(tables, N, b, dst[j], tpb)
            _write(pool, scales, blk, dst[j] % tpb, decode(codes[j:end]) * had[j:end, :, :, None],
                   had[j:end].max(0))
            j = end
    return pool, scales


# ------------------------------------------------------------------ attention
def attend(q, pool, scales, tables, seq_lens, window_lens=None, masks=None, scale=None):
    """q [B, W, Hq, D] float64.  Returns a dict: out, lse, and for error
    bounds amp [B, W, Hq, D] = sum p |v|, spread [B, W, Hq] = the largest
    scale * sum |q_d k_d| and keys [B, W, Hq] = the number of seen positions.
    Rows behind a window's end are zero."""
    B, W, Hq, D = q.shape
    N, _, H, tpb, _ = pool.shape
    scale = D ** -0.5 if scale is None else scale
    r = dict(out=np.zeros(q.shape), lse=np.zeros((B, W, Hq)), amp=np.zeros(q.shape), spread=np.zeros((B, W, Hq)),
             keys=np.zeros((B, W, Hq)))
    bits = None if masks is None else mask_bits(masks, W)
    for b, w in enumerate(_wins(window_lens, B, W)):
        s = int(seq_lens[b])
        if s < 0 or not 0 <= w <= W or s + w > tables.shape[1] * tpb:
            r["out"][b], r["lse"][b] = np.nan, np.nan
            continue
        T = s + w
        blocks = [_mapped(tables, N, b, t, tpb) for t in range(0, T, tpb)]
        if any(x is None for x in blocks):
            r["out"][b, :w], r["lse"][b, :w] = np.nan, np.nan
            continue
        if T == 0:
            continue
        x = decode(pool[blocks]) * scales[blocks].astype(np.float64)[..., None, None]
        see = np.ones((w, T), dtype=bool)
        see[:, s:] = np.tril(np.ones((w, w), dtype=bool)) if bits is None else bits[b, :w, :w]
        for hq in range(Hq):
            k, v = (x[:, kind, hq // (Hq // H)].reshape(-1, D)[:T] for kind in (0, 1))
            qh = q[b, :w, hq]
            for i in range(w):
                t = np.flatnonzero(see[i])
                r["keys"][b, i, hq] = len(t)
                if not len(t):
                    r["lse"][b, i, hq] = -math.inf
                    continue
                a = scale * (k[t] @ qh[i])
                m = a.max()
                p = np.exp(a - m)
                z = p.sum()
                r["lse"][b, i, hq] = m + math.log(z) if np.isfinite(z) else np.nan
                r["out"][b, i, hq] = p @ v[t] / z
                r["amp"][b, i, hq] = p @ np.abs(v[t]) / z
                r["spread"][b, i, hq] = abs(scale) * (np.abs(k[t]) @ np.abs(qh[i])).max()
    return r
