"""The 8-bit paged KV cache beside the verify calls: what a decode step runs.

One step of speculative decoding writes a window of draft tokens behind each
request's committed prefix, lets every window token attend to the prefix and
to its own ancestors in the window, verifies, and keeps the accepted rows.
Five operators, each in its plain form (elementary torch operations in 32
bits) and through the library's calls:

  paging    blocks for the windows taken from a free list, block tables and
            slot maps built on the device, and the blocks given back
  masks     each tree node's ancestors as bits, from the paths
  store     the window's K and V rows rounded to e4m3 into the pages, one
            power-of-two scale for each block of tokens and head
  attend    attention of the window's rows over the paged 8-bit cache
  relocate  the accepted nodes' rows gathered behind the prefix, rescaled
            where a row changes to a block of another scale

The cache: kv_pool [num_blocks, 2, Hkv, tokens_per_block, D] e4m3 (0 = K,
1 = V), kv_scales [num_blocks, 2, Hkv] float32; logical position t of request
b is row t % tokens_per_block of block block_tables[b, t // tokens_per_block].
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # a serving step of 64 requests with 7 drafts each
        dict(name="paging_b64_w8", op="paging", B=64, W=8, tpb=32, lo=128, hi=2048),
        # the largest batch a call takes
        dict(name="paging_b8192_w4", op="paging", B=8192, W=4, tpb=16, lo=1, hi=4096),
        # the tree workload's shape: 60 nodes, three levels under the root
        dict(name="masks_b16_n60_l4", op="masks", B=16, N=60, P=60, L=4),
        # deep, wide trees of many requests
        dict(name="masks_b64_n509_l17", op="masks", B=64, N=509, P=301, L=17),
        # the rows of 7 drafts and the bonus position, ragged, one layer
        dict(name="store_b64_w8_d128_bf16", op="store", B=64, W=8, Hq=32, Hkv=8, D=128, tpb=32, lo=128, hi=2048,
             ragged=True, dtype="bf16"),
        # prompts of odd length written in one call
        dict(name="store_b4_w4001_d64_f16", op="store", B=4, W=4001, Hq=16, Hkv=4, D=64, tpb=64, lo=0, hi=300,
             ragged=True, dtype="f16"),
        # one request, one token: the latency of a plain decode step
        dict(name="attend_b1_w1_c1000_d128_bf16", op="attend", B=1, W=1, Hq=32, Hkv=8, D=128, tpb=16, lo=1000, hi=1000,
             ragged=False, tree=False, dtype="bf16"),
        # 3 drafts and the bonus position of 256 requests: bound by the cache's bytes
        dict(name="attend_b256_w4_c8192_d128_bf16", op="attend", B=256, W=4, Hq=32, Hkv=8, D=128, tpb=32, lo=512,
             hi=8192, ragged=True, tree=False, dtype="bf16"),
        # the tree workload's windows over long prefixes: 240 rows per KV head
        dict(name="attend_tree_b16_n60_c8192_d128_bf16", op="attend", B=16, W=60, Hq=32, Hkv=8, D=128, tpb=64, lo=512,
             hi=8192, ragged=False, tree=True, dtype="bf16"),
        # prompt chunks of odd length behind cached prefixes: bound by the products
        dict(name="attend_b3_w2049_c4500_d64_f16", op="attend", B=3, W=2049, Hq=16, Hkv=4, D=64, tpb=48, lo=0, hi=4500,
             ragged=True, tree=False, dtype="f16"),
        # the tree workload's accepted rows, one layer
        dict(name="relocate_b16_n60_l4_d128", op="relocate", B=16, N=60, L=4, Hkv=8, D=128, tpb=16, lo=128, hi=2048),
        # long accepted paths of many requests
        dict(name="relocate_b256_n120_l17_d64", op="relocate", B=256, N=120, L=17, Hkv=8, D=64, tpb=32, lo=1, hi=1000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["paging", "masks", "store", "attend", "attend", "attend", "relocate"])
    tpb = rng.choice([16, 32, 48, 64, 128])
    lo = rng.choice([0, 1, rng.randint(2, 600)])
    D = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "f16"])
    Hkv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8])
    if op == "paging":
        return dict(op=op, B=_log(rng, 1, 8192), W=_log(rng, 1, 65), tpb=tpb, lo=lo, hi=lo + _log(rng, 1, 4000))
    if op == "masks":
        N = _log(rng, 2, 1000)
        return dict(op=op, B=_log(rng, 1, 64), N=N, P=rng.randint(1, min(N, 300)), L=rng.randint(2, 20))
    if op == "store":
        if rng.random() < 0.5:
            B, W = _log(rng, 1, 256), rng.randint(1, 65)
        else:
            B, W = rng.randint(1, 4), _log(rng, 64, 4000)
        return dict(op=op, B=B, W=W, Hq=Hkv * group, Hkv=Hkv, D=D, tpb=tpb, lo=lo, hi=lo + _log(rng, 1, 2000),
                    ragged=rng.random() < 0.5, dtype=dtype)
    if op == "relocate":
        L = rng.randint(2, 20)
        return dict(op=op, B=_log(rng, 1, 256), N=rng.randint(2 * L, 128), L=L, Hkv=Hkv, D=D, tpb=tpb, lo=lo,
                    hi=lo + _log(rng, 1, 2000))
    form = rng.choice(["token", "chain", "chain", "tree", "prompt"])
    W = {"token": 1, "chain": rng.randint(2, 16), "tree": rng.randint(8, 128), "prompt": _log(rng, 64, 2000)}[form]
    rows = W * Hkv * group
    hi = lo + _log(rng, 16, 60000 if form == "token" else 12000)
    hi = min(hi, lo + max(16, 280_000_000 // rows - W - lo))
    most = min(256, 9_000_000 // (Hkv * (lo + hi)), 150_000_000 // (rows * (hi + W)), 800_000 // rows)
    return dict(op=op, B=_log(rng, 1, max(1, most)), W=W, Hq=Hkv * group, Hkv=Hkv, D=D, tpb=tpb, lo=lo, hi=hi,
                ragged=form != "token" and rng.random() < 0.5, tree=form == "tree", dtype=dtype)


# ------------------------------------------------------------------ inputs
def _lens(c):
    """The case's prefix lengths, spread evenly over [lo, hi] (a seed permutes them)."""
    return np.round(np.linspace(c["lo"], c["hi"], c["B"])).astype(np.int64)


def _wins(c):
    """The case's window lengths: W, or spread over [1, W] with every prefix length getting any of them."""
    if not c.get("ragged"):
        return np.full(c["B"], c["W"], dtype=np.int64)
    return 1 + (np.arange(c["B"], dtype=np.int64) * 5 + c["W"] - 1) % c["W"]


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _tree_paths(rng, N, P, L):
    """Root-to-leaf node lists of a random tree whose nodes are numbered level by level; -1 padded."""
    # nodes per level: the root, then levels that grow to a common width
    width = max(1, -(-(N - 1) // (L - 1)))
    level = np.concatenate([[0], 1 + np.minimum(np.arange(N - 1) // width, L - 2)])
    parent = np.full(N, -1)
    for n in range(1, N):
        parent[n] = 0 if level[n] == 1 else rng.choice(np.flatnonzero(level == level[n] - 1))
    leaves = np.setdiff1d(np.arange(N), parent)
    rng.shuffle(leaves)
    paths = np.full((P, L), -1)
    for p, n in enumerate(np.sort(leaves[:P])):
        chain = []
        while n >= 0:
            chain.append(n)
            n = parent[n]
        paths[p, :len(chain)] = chain[::-1]
    return paths


def _cache(c, rng, g, ends):
    """Pages in shuffled order and quantised contents for requests that reach at most `ends`."""
    tpb, H, D = c["tpb"], c["Hkv"], c["D"]
    per = -(-ends // tpb)
    cols = max(1, int(per.max()))
    blocks = int(per.sum()) + 3
    perm = rng.permutation(blocks)
    tables = np.full((c["B"], cols), -1, dtype=np.int64)
    tables[np.arange(cols)[None, :] < per[:, None]] = perm[:int(per.sum())]
    pool = torch.empty((blocks, 2, H, tpb, D), dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.empty((blocks, 2, H), dtype=torch.float32, device=DEV)
    # each head its own level, a few large channels, each block some spread
    level = torch.exp(0.7 * torch.randn((1, 2, H, 1, 1), generator=g, device=DEV))
    level = level * (1 + 5 * (torch.rand((1, 2, H, 1, D), generator=g, device=DEV) < 0.04))
    at = max(1, (1 << 27) // (2 * H * tpb * D))
    for b0 in range(0, blocks, at):
        n = min(at, blocks - b0)
        x = torch.randn((n, 2, H, tpb, D), generator=g, device=DEV) * level
        x *= torch.exp(0.3 * torch.randn((n, 2, H, 1, 1), generator=g, device=DEV))
        s = _scale_for(x.abs().amax((-1, -2)))
        pool[b0:b0 + n] = (x / s[..., None, None]).to(torch.float8_e4m3fn)
        scales[b0:b0 + n] = s
    return _i32(tables), pool, scales


def prepare(case, seed):
    c = case
    rng = np.random.default_rng(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(c)
    if c["op"] == "masks":
        s["paths"] = _i32(np.stack([_tree_paths(rng, c["N"], c["P"], c["L"]) for _ in range(c["B"])]))
        return s
    lens = rng.permutation(_lens(c))
    B, tpb = c["B"], c["tpb"]
    s["seq_lens"] = _i32(lens)
    if c["op"] == "paging":
        W = c["W"]
        wins = rng.integers(0, W + 1, B) if W > 1 else np.ones(B, dtype=np.int64)
        held = -(-lens // tpb)
        need = -(-(lens + wins) // tpb) - held
        cols = int((held - (-W // tpb) + 1).max())
        blocks = int((held - (-W // tpb) + 1).sum()) + 5
        perm = rng.permutation(blocks)
        tables = np.full((B, cols), -1, dtype=np.int64)
        tables[np.arange(cols)[None, :] < held[:, None]] = perm[:int(held.sum())]
        free = np.full(blocks, -1, dtype=np.int64)
        spare = blocks - int(held.sum())
        free[:spare] = perm[int(held.sum()):]
        s.update(window_lens=_i32(wins), tables=_i32(tables), held=_i32(held), free=_i32(free), count=_i32([spare]),
                 give=_i32(need))
        return s
    H, D = c["Hkv"], c["D"]
    if c["op"] == "relocate":
        N, L = c["N"], c["L"]
        n = rng.integers(0, L, B)
        n[0] = L - 1
        nodes = np.full((B, L), -1, dtype=np.int64)
        nodes[:, 0] = 0
        for b in range(B):
            # accepted nodes beyond the places that the rows move to
            nodes[b, 1:1 + n[b]] = np.sort(rng.choice(np.arange(L, N), n[b], replace=False))
        s["tables"], s["pool"], s["scales"] = _cache(c, rng, g, lens + N)
        s["nodes"], s["accepted"] = _i32(nodes), _i32(n)
        return s
    t = TYPES[c["dtype"]]
    W, Hq = c["W"], c["Hq"]
    wins = _wins(c)
    s["window_lens"] = _i32(wins) if c["ragged"] else None
    s["tables"], s["pool"], s["scales"] = _cache(c, rng, g, lens + W)
    # q, k and v as a projection leaves them: slices of one row per token
    qkv = torch.randn((B, W, Hq + 2 * H, D), generator=g, device=DEV)
    qkv *= torch.exp(0.3 * torch.randn((B, W, Hq + 2 * H, 1), generator=g, device=DEV))
    qkv = qkv.to(t)
    s["q"], s["k"], s["v"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + H], qkv[:, :, Hq + H:]
    if c["op"] == "attend":
        s["masks"] = None
        if c["tree"]:
            L = min(W, 5)
            paths = np.stack([_tree_paths(rng, W, W, L) for _ in range(B)])
            bits = np.zeros((B, W, W), dtype=bool)
            for b in range(B):
                for path in paths[b]:
                    path = path[path >= 0]
                    for d in range(len(path)):
                        bits[b, path[d], path[:d + 1]] = True
            words = -(-W // 32)
            packed = np.zeros((B, W, words * 32), dtype=np.uint8)
            packed[:, :, :W] = bits
            s["masks"] = torch.from_numpy(np.packbits(packed, axis=-1, bitorder="little").view(np.int32).copy()).to(DEV)
        # rows behind a window's end are left as they are
        s["out"] = torch.zeros((B, W, Hq, D), dtype=t, device=DEV)
        s["lse"] = torch.zeros((B, W, Hq), dtype=torch.float32, device=DEV)
    return s


# ------------------------------------------------------------------ plain forms
def _scale_for(amax):
    """The smallest power of two with amax <= 448 * scale (0 for 0)."""
    m, e = torch.frexp(amax)
    s = torch.ldexp(torch.ones_like(amax), torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126))
    return torch.where(amax > 0, s, torch.zeros_like(amax))


def _ratio(a, b):
    return torch.where(b > 0, a / b, torch.zeros_like(a))


def _paging(s):
    tpb, W = s["tpb"], s["W"]
    seq, win, held, tables, free = s["seq_lens"], s["window_lens"], s["held"], s["tables"], s["free"]
    cols = tables.shape[1]
    need = ((seq + win + tpb - 1) // tpb - held).clamp(min=0)
    upto = need.cumsum(0)
    ok = (upto <= s["count"]) | (need == 0)
    need = torch.where(ok, need, 0)
    first = upto - need
    col = torch.arange(cols, device=DEV)[None, :]
    i = col - held[:, None]
    take = (i >= 0) & (i < need[:, None])
    at = (s["count"] - 1 - first[:, None] - i).clamp(0, free.numel() - 1)
    tables.copy_(torch.where(take, free[at.long()], tables))
    held += need
    s["count"] -= need.sum()
    granted = torch.where(ok, win, -1).to(torch.int32)
    j = torch.arange(W, device=DEV)[None, :]
    t = seq[:, None] + j
    blk = torch.gather(tables, 1, (t // tpb).clamp(max=cols - 1).long())
    slots = torch.where(j < granted[:, None], blk * tpb + t % tpb, -1).to(torch.int32)
    # the blocks go back: the last `give` of each table
    give = torch.where((s["give"] >= 0) & (s["give"] <= held), s["give"], 0)
    first = give.cumsum(0) - give
    total = give.sum()
    i = col - (held - give)[:, None]
    back = (i >= 0) & (i < give[:, None])
    at = s["count"] + total - 1 - first[:, None] - i
    at = torch.where(back, at, free.numel()).long()
    grown = torch.cat([free, free.new_zeros(1)])
    grown.scatter_(0, at.reshape(-1), torch.where(back, tables, 0).reshape(-1))
    free.copy_(torch.where(torch.arange(free.numel(), device=DEV) < s["count"] + total, grown[:-1], free))
    tables.masked_fill_(back, -1)
    held -= give
    s["count"] += total
    return slots, granted, tables, held, free, s["count"]


def _masks(s):
    paths, N = s["paths"].long(), s["N"]
    B, P, L = paths.shape
    used = (paths[:, :, 0] == 0)[:, :, None] & (paths >= 0).cumprod(2).bool()
    node = torch.where(used, paths, N)
    words = -(-N // 32)
    bits = torch.zeros((B, N + 1, words * 32 + 1), dtype=torch.bool, device=DEV)
    d = torch.arange(L, device=DEV)
    row = node[:, :, :, None].expand(B, P, L, L)
    anc = node[:, :, None, :].expand(B, P, L, L)
    on = (d[None, :] <= d[:, None]) & (row < N) & (anc < N)
    b = torch.arange(B, device=DEV)[:, None, None, None].expand(B, P, L, L)
    bits[b, torch.where(on, row, N), torch.where(on, anc, words * 32)] = True
    word = bits[:, :N, :words * 32].reshape(B, N, words, 32)
    value = (word.long() << torch.arange(32, device=DEV)).sum(-1)
    return torch.where(value >= 1 << 31, value - (1 << 32), value).to(torch.int32)


def _store(s):
    seq, tables, pool, scales, tpb = s["seq_lens"].long(), s["tables"].long(), s["pool"], s["scales"], s["tpb"]
    B, W, H, D = s["k"].shape
    win = torch.full((B,), W, device=DEV) if s["window_lens"] is None else s["window_lens"].long()
    x = torch.stack([s["k"], s["v"]], 2).float()  # [B, W, 2, H, D]
    i = torch.arange(W, device=DEV)[None, :]
    real = i < win[:, None]
    t = seq[:, None] + i
    page = t // tpb - (seq // tpb)[:, None]  # pages of the window, from its first
    pages = (W - 1) // tpb + 2
    amax = torch.where(real[:, :, None, None], x.abs().amax(-1), 0)
    new = torch.zeros((B, pages, 2, H), device=DEV)
    new.scatter_reduce_(1, page[:, :, None, None].expand(B, W, 2, H), amax, "amax")
    new = _scale_for(new)
    # the first page's live rows keep their values under the larger scale
    first = tables.gather(1, (seq // tpb).clamp(max=tables.shape[1] - 1)[:, None])[:, 0]
    live = (torch.arange(tpb, device=DEV)[None, :] < (seq % tpb)[:, None]) & (win > 0)[:, None]
    some = live.any(1)
    rows = first[some]
    old = scales[rows]
    new[some, 0] = torch.maximum(new[some, 0], old)
    kept = pool[rows].float()
    moved = (kept * _ratio(old, new[some, 0])[..., None, None]).to(torch.float8_e4m3fn)
    keep = live[some][:, None, None, :, None]
    pool[rows] = torch.where(keep, moved.float(), kept).to(torch.float8_e4m3fn)
    # the new rows
    touched = torch.zeros((B, pages), device=DEV).scatter_reduce_(1, page, real.float(), "amax") > 0
    at = ((seq // tpb)[:, None] + torch.arange(pages, device=DEV)).clamp(max=tables.shape[1] - 1)
    scales[tables.gather(1, at)[touched]] = new[touched]
    q = x * _ratio(torch.ones_like(new), new).gather(1, page[:, :, None, None].expand(B, W, 2, H))[..., None]
    blk = tables.gather(1, (t // tpb).clamp(max=tables.shape[1] - 1))
    pool.view(torch.uint8).permute(0, 3, 1, 2, 4)[blk[real], (t % tpb)[real]] = \
        q[real].to(torch.float8_e4m3fn).view(torch.uint8)
    return pool, scales


def _attend(s):
    seq, tables, tpb = s["seq_lens"].long(), s["tables"].long().clamp(min=0), s["tpb"]
    B, W, Hq, D = s["q"].shape
    H = s["Hkv"]
    win = torch.full((B,), W, device=DEV) if s["window_lens"] is None else s["window_lens"].long()
    T = tables.shape[1] * tpb
    x = s["pool"][tables].float() * s["scales"][tables][..., None, None]  # [B, cols, 2, H, tpb, D]
    x = x.permute(2, 0, 3, 1, 4, 5).reshape(2, B, H, T, D)
    i = torch.arange(W, device=DEV)
    pos = torch.arange(T, device=DEV)
    j = pos[None, :] - seq[:, None]  # the window's place of each position
    if s["masks"] is None:
        see = j[:, None, :] <= i[None, :, None]
    else:
        word = s["masks"].long().gather(2, (j.clamp(0, W - 1) // 32)[:, None, :].expand(B, W, T))
        see = (j < 0)[:, None, :] | (((word >> (j.clamp(min=0) % 32)[:, None, :]) & 1) == 1) & (j < W)[:, None, :]
    see = see & (j < win[:, None])[:, None, :]
    q = s["q"].float().reshape(B, W, H, Hq // H, D).permute(0, 2, 1, 3, 4).reshape(B, H, -1, D)
    a = (q @ x[0].transpose(-1, -2)).reshape(B, H, W, Hq // H, T) / math.sqrt(D)
    a = a.masked_fill(~see[:, None, :, None, :], -math.inf)
    top = a.amax(-1, keepdim=True)
    p = torch.exp(a - top.clamp(min=-1e30))
    del a
    z = p.sum(-1, keepdim=True)
    v = torch.where((j < win[:, None])[:, None, :, None], x[1], 0)
    o = (p.reshape(B, H, -1, T) @ v).reshape(B, H, W, Hq // H, D) / z.clamp(min=1e-37)
    lse = (top + torch.log(z))[..., 0]
    row = (i[None, :] < win[:, None])[:, :, None]
    o = torch.where(row[..., None], o.permute(0, 2, 1, 3, 4).reshape(B, W, Hq, D), 0)
    lse = torch.where(row, lse.permute(0, 2, 1, 3).reshape(B, W, Hq), 0)
    return o.to(s["q"].dtype), lse


def _relocate(s):
    seq, tables, pool, scales, tpb = s["seq_lens"].long(), s["tables"].long(), s["pool"], s["scales"], s["tpb"]
    nodes, n = s["nodes"].long(), s["accepted"].long()
    B, L = nodes.shape
    H, D = s["Hkv"], s["D"]
    j = torch.arange(1, L, device=DEV)[None, :]
    real = j <= n[:, None]

    def place(t):
        blk = tables.gather(1, (t // tpb).clamp(0, tables.shape[1] - 1))
        return blk, t % tpb

    codes = pool.view(torch.uint8).permute(0, 3, 1, 2, 4)
    blk, off = place(seq[:, None] + nodes[:, 1:].clamp(min=0))
    x = codes[blk, off].view(torch.float8_e4m3fn).float()  # [B, L - 1, 2, H, D]
    had = torch.where(real[:, :, None, None], scales[blk], 0)
    t = seq[:, None] + j
    start = (seq + 1) // tpb
    page = t // tpb - start[:, None]
    pages = (L - 2) // tpb + 2
    new = torch.zeros((B, pages, 2, H), device=DEV)
    new.scatter_reduce_(1, page[:, :, None, None].expand(B, L - 1, 2, H), had, "amax")
    live = (torch.arange(tpb, device=DEV)[None, :] < ((seq + 1) % tpb)[:, None]) & (n > 0)[:, None]
    some = live.any(1)
    rows = tables.gather(1, start.clamp(max=tables.shape[1] - 1)[:, None])[:, 0][some]
    old = scales[rows]
    new[some, 0] = torch.maximum(new[some, 0], old)
    kept = pool[rows].float()
    moved = (kept * _ratio(old, new[some, 0])[..., None, None]).to(torch.float8_e4m3fn)
    pool[rows] = torch.where(live[some][:, None, None, :, None], moved.float(), kept).to(torch.float8_e4m3fn)
    touched = torch.zeros((B, pages), device=DEV).scatter_reduce_(1, page, real.float(), "amax") > 0
    at = (start[:, None] + torch.arange(pages, device=DEV)).clamp(max=tables.shape[1] - 1)
    scales[tables.gather(1, at)[touched]] = new[touched]
    y = x * _ratio(had, new.gather(1, page[:, :, None, None].expand(B, L - 1, 2, H)))[..., None]
    blk, off = place(t)
    codes[blk[real], off[real]] = y[real].to(torch.float8_e4m3fn).view(torch.uint8)
    return pool, scales


def run(state):
    s = state
    if not own:
        return {"paging": _paging, "masks": _masks, "store": _store, "attend": _attend, "relocate": _relocate}[s["op"]](s)
    import speculative_decoding_verification_row_gb300 as sv
    if s["op"] == "paging":
        slots, granted = sv.reserve_blocks(s["seq_lens"], s["tables"], s["held"], s["free"], s["count"], s["tpb"],
                                           s["W"], window_lens=s["window_lens"])
        sv.release_blocks(s["tables"], s["held"], s["give"], s["free"], s["count"])
        return slots, granted, s["tables"], s["held"], s["free"], s["count"]
    if s["op"] == "masks":
        return sv.tree_masks(s["paths"], s["N"])
    if s["op"] == "store":
        sv.store_kv(s["k"], s["v"], s["pool"], s["scales"], s["tables"], s["seq_lens"], window_lens=s["window_lens"])
        return s["pool"], s["scales"]
    if s["op"] == "attend":
        return sv.attend_kv(s["q"], s["pool"], s["scales"], s["tables"], s["seq_lens"], window_lens=s["window_lens"],
                            masks=s["masks"], out=s["out"], out_lse=s["lse"])
    sv.relocate_quantised_kv(s["pool"], s["scales"], s["tables"], s["seq_lens"], s["nodes"], s["accepted"])
    return s["pool"], s["scales"]


# ------------------------------------------------------------------ work
def work(case):
    c = case
    if c["op"] == "masks":
        return {"bytes": 4.0 * c["B"] * (c["P"] * c["L"] + c["N"] * -(-c["N"] // 32)), "flops": 0.0}
    lens, B = _lens(c), c["B"]
    if c["op"] == "paging":
        # lengths, windows, held, give; the slots; a window's new blocks written, read and given back
        return {"bytes": 4.0 * B * (6 + c["W"] + 4 * max(1, c["W"] / 2 / c["tpb"])), "flops": 0.0}
    H, D = c["Hkv"], c["D"]
    if c["op"] == "relocate":
        rows = B * c["L"] / 2 * 2 * H
        return {"bytes": rows * (2 * D + 8), "flops": rows * D}
    wins = _wins(c)
    size = 2
    if c["op"] == "store":
        rows = float(wins.sum()) * 2 * H
        return {"bytes": rows * D * (size + 1) + rows / c["tpb"] * 4, "flops": 3.0 * rows * D}
    seen = lens + wins
    pages = -(-seen // c["tpb"])
    rows = wins * c["Hq"]
    kv = float((seen * 2 * H * D + pages * 2 * H * 4).sum())
    near = wins * wins if c["tree"] else wins * (wins + 1) // 2
    pairs = float(((lens * wins + near) * c["Hq"]).sum())
    return {"bytes": kv + float(rows.sum()) * (2 * size * D + 4), "flops": 4.0 * pairs * D}


# ------------------------------------------------------------------ 64 bits
def _e4m3_values():
    """The 128 values of the codes without a sign: 3 bits of mantissa, exponent bias 7, NaN at 127."""
    v = [m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)]
    v[127] = math.nan
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _values(codes):
    u = codes.contiguous().view(torch.uint8).int()
    return _e4m3_values()[u & 127] * torch.where(u > 127, -1.0, 1.0).double()


def _nearest(x):
    """x rounded to the e4m3 values, ties to the even code (|x| <= 448)."""
    grid = _e4m3_values()[:127]
    a = x.abs().contiguous()
    hi = torch.searchsorted(grid, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    down, up = a - grid[lo], grid[hi] - a
    code = torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    return torch.sign(x) * grid[code]


def _need(amax):
    return 0.0 if amax == 0 else 2.0 ** math.ceil(math.log2(amax / 448.0))


def _exact_pages(values, scales, blk, first, rows, src):
    """Writes `rows` [n, 2, H, D] (true values) with the least scales `src` [2, H] from offset `first` of block blk."""
    new = src if first == 0 else torch.maximum(src, scales[blk])
    ratio = torch.where(new > 0, 1 / new.clamp(min=1e-300), 0.0)[:, :, None, None]
    if first:
        values[blk, :, :, :first] = _nearest(values[blk, :, :, :first] * scales[blk][:, :, None, None] * ratio)
    values[blk, :, :, first:first + rows.shape[0]] = _nearest(rows.permute(1, 2, 0, 3) * ratio)
    scales[blk] = new


def exact(case, seed):
    c = case
    if c["op"] in ("paging", "masks"):
        return None
    s = prepare(c, seed)
    seq, tables, tpb = s["seq_lens"].tolist(), s["tables"].tolist(), c["tpb"]
    if c["op"] == "attend":
        return _exact_attend(s, seq, tables)
    if c["op"] == "store" and sum(_wins(c)) / tpb + c["B"] > 4000:
        return None
    values, scales = _values(s["pool"]), s["scales"].double()
    if c["op"] == "store":
        win = [c["W"]] * c["B"] if s["window_lens"] is None else s["window_lens"].tolist()
        for b in range(c["B"]):
            at, end = seq[b], seq[b] + win[b]
            while at < end:
                to = min(end, (at // tpb + 1) * tpb)
                x = torch.stack([s["k"][b, at - seq[b]:to - seq[b]], s["v"][b, at - seq[b]:to - seq[b]]], 1).double()
                least = x.abs().amax((0, 3)).tolist()
                least = torch.tensor([[_need(a) for a in r] for r in least], dtype=torch.float64, device=DEV)
                _exact_pages(values, scales, tables[b][at // tpb], at % tpb, x, least)
                at = to
        return values, scales
    nodes, n = s["nodes"].tolist(), s["accepted"].tolist()
    for b in range(c["B"]):
        if n[b] < 1:
            continue
        src = [seq[b] + nodes[b][j] for j in range(1, n[b] + 1)]
        had = torch.stack([scales[tables[b][t // tpb]] for t in src])
        x = torch.stack([values[tables[b][t // tpb], :, :, t % tpb] for t in src]) * had[..., None]
        at, end = seq[b] + 1, seq[b] + n[b] + 1
        while at < end:
            to = min(end, (at // tpb + 1) * tpb)
            i, k = at - seq[b] - 1, to - seq[b] - 1
            _exact_pages(values, scales, tables[b][at // tpb], at % tpb, x[i:k], had[i:k].amax(0))
            at = to
    return values, scales


def _exact_attend(s, seq, tables):
    B, W, Hq, D = s["q"].shape
    H, tpb = s["Hkv"], s["tpb"]
    out = torch.zeros((B, W, Hq, D), dtype=torch.float64, device=DEV)
    lse = torch.zeros((B, W, Hq), dtype=torch.float64, device=DEV)
    win = [W] * B if s["window_lens"] is None else s["window_lens"].tolist()
    bits = None
    if s["masks"] is not None:
        m = s["masks"].cpu().numpy().view(np.uint8)
        bits = torch.from_numpy(np.unpackbits(m, axis=-1, bitorder="little")[:, :, :W].astype(bool)).to(DEV)
    for b in range(B):
        w, T = win[b], seq[b] + win[b]
        if w == 0:
            continue
        blocks = torch.tensor(tables[b][:-(-T // tpb)], device=DEV)
        x = _values(s["pool"][blocks]) * s["scales"][blocks].double()[..., None, None]
        see = torch.ones((w, T), dtype=torch.bool, device=DEV)
        see[:, seq[b]:] = torch.ones((w, w), dtype=torch.bool, device=DEV).tril() if bits is None else bits[b, :w, :w]
        for h in range(Hq):
            k, v = (x[:, kind, h // (Hq // H)].reshape(-1, D)[:T] for kind in (0, 1))
            a = torch.einsum("wd,td->wt", s["q"][b, :w, h].double(), k) * D ** -0.5
            a[~see] = -math.inf
            lse[b, :w, h] = torch.logsumexp(a, 1)
            out[b, :w, h] = torch.softmax(a, 1) @ v
    return out, lse
