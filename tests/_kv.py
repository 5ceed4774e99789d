"""Cases of the paged 8-bit KV cache shared by its tests."""
import numpy as np

from oracle import kv


def cache(rng, lens, H, D, tpb, spare=3, extra_cols=1, spread=1.0, stale="random"):
    """Pages in shuffled order for requests that reach `lens`; codes of rows
    past a request's end are arbitrary bytes, NaN codes among them."""
    per = -(-np.asarray(lens) // tpb)
    cols = max(1, int(per.max(initial=0)) + extra_cols)
    n = int(per.sum()) + spare
    perm = rng.permutation(n)
    tables = np.full((len(lens), cols), -1, np.int32)
    at = 0
    for b, p in enumerate(per):
        tables[b, :p] = perm[at:at + p]
        at += p
    pool = rng.integers(0, 256, (n, 2, H, tpb, D)).astype(np.uint8)
    scales = np.zeros((n, 2, H), np.float32)
    for b, T in enumerate(lens):
        for t0 in range(0, int(T), tpb):
            m = min(tpb, int(T) - t0)
            x = rng.normal(0, 1, (2, H, m, D)) * np.exp(spread * rng.normal(0, 1, (2, H, 1, 1)))
            blk = tables[b, t0 // tpb]
            for kind in range(2):
                for h in range(H):
                    s = kv.scale_for(np.abs(x[kind, h]).max())
                    pool[blk, kind, h, :m] = kv.encode(x[kind, h] / s)
                    scales[blk, kind, h] = s
    unused = np.setdiff1d(np.arange(n), tables)
    scales[unused] = 1.0
    return pool, scales, tables


def random_paths(rng, N, P, L):
    """Root-to-leaf paths of a random tree whose nodes' ids exceed their parents'."""
    parent, depth = [-1], [0]
    for n in range(1, N):
        ok = [m for m in range(n) if depth[m] < L - 1]
        m = int(rng.choice(ok))
        parent.append(m)
        depth.append(depth[m] + 1)
    leaves = [n for n in range(N) if n not in parent[1:]] or [0]
    paths = np.full((P, L), -1, np.int32)
    for p in range(min(P, len(leaves))):
        chain, n = [], leaves[p]
        while n >= 0:
            chain.append(n)
            n = parent[n]
        paths[p, :len(chain)] = chain[::-1]
    return paths


def to_bf16(x):
    """float64 -> nearest bfloat16 (as float64), ties to even."""
    import torch
    return torch.from_numpy(np.asarray(x, np.float64)).to(torch.float32).to(torch.bfloat16).double().numpy()


def to_f16(x):
    return np.asarray(x).astype(np.float16).astype(np.float64)
