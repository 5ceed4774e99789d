"""What a decode step needs around the verify calls and the 8-bit paged cache.

Before a verify the target's logits are penalised, biased and masked; before
the store and the attention the window's queries and keys are rotated to their
positions; and a cache that has grown to its budget drops the positions that
drew the least attention.  Five operators, each in its plain form (elementary
torch operations in 32 bits, angles in 64) and through the library's calls:

  adjust        penalties for repeated tokens, biases and grammar masks on the
                logits of a window's rows, each row with the draft tokens
                before it
  rotate        rotary positions of a window's queries and keys
  rotate_store  the same, the keys and values going straight into the cache
  weigh         the attention that each cached position drew from a window's
                rows, added to a running weight
  evict         the positions of least weight dropped from the cache, the
                others moved together

The cache: kv_pool [num_blocks, 2, Hkv, tokens_per_block, D] e4m3 (0 = K,
1 = V), kv_scales [num_blocks, 2, Hkv] float32; logical position t of request
b is row t % tokens_per_block of block block_tables[b, t // tokens_per_block].
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one request, one token, a short conversation: the latency of a plain decode step
        dict(name="adjust_b1_r1_v32000_f32", op="adjust", form="chain", B=1, R=1, V=32000, T=700, bias=8, penalties=True,
             grammars=0, inplace=False, ragged=False, dtype="f32"),
        # 7 drafts and the bonus row of 64 requests with a few thousand tokens each
        dict(name="adjust_b64_r8_v128256_bf16", op="adjust", form="chain", B=64, R=8, V=128256, T=4096, bias=16,
             penalties=True, grammars=0, inplace=False, ragged=False, dtype="bf16"),
        # tree windows under penalties and a grammar
        dict(name="adjust_tree_b16_n60_v151936_bf16", op="adjust", form="tree", B=16, R=60, V=151936, T=2000, bias=0,
             penalties=True, grammars=40, inplace=False, ragged=False, dtype="bf16"),
        # a grammar alone, written into the logits themselves
        dict(name="adjust_grammar_b256_r4_v129280_bf16", op="adjust", form="chain", B=256, R=4, V=129280, T=0, bias=0,
             penalties=False, grammars=64, inplace=True, ragged=False, dtype="bf16"),
        # 7 drafts and the bonus position of 64 requests, one layer
        dict(name="rotate_b64_w8_d128_bf16", op="rotate", B=64, W=8, Hq=32, Hkv=8, D=128, rot=128, interleaved=False,
             ramp=1.0, tree=False, lo=128, hi=2048, ragged=True, dtype="bf16"),
        # prompts of odd length, a quarter of the head rotated, far positions
        dict(name="rotate_b4_w4001_d128_f16", op="rotate", B=4, W=4001, Hq=32, Hkv=4, D=128, rot=32, interleaved=True,
             ramp=8.0, tree=False, lo=0, hi=120000, ragged=False, dtype="f16"),
        # the tree workload's windows, rotated by their depth and stored
        dict(name="rotate_store_tree_b16_n60_d128_bf16", op="rotate_store", B=16, W=60, Hq=32, Hkv=8, D=128, rot=128,
             interleaved=False, ramp=1.0, tree=True, tpb=32, lo=128, hi=2048, ragged=False, dtype="bf16"),
        # prompts of odd length stored in one call
        dict(name="rotate_store_b8_w2001_d64_f16", op="rotate_store", B=8, W=2001, Hq=16, Hkv=4, D=64, rot=64,
             interleaved=True, ramp=4.0, tree=False, tpb=64, lo=0, hi=300, ragged=False, dtype="f16"),
        # 3 drafts and the bonus position of 64 requests over long prefixes: bound by the cache's bytes
        dict(name="weigh_b64_w4_c8192_d128_bf16", op="weigh", B=64, W=4, Hq=32, Hkv=8, D=128, tpb=32, lo=512, hi=8192,
             ragged=True, decay=0.99, dtype="bf16"),
        # prompt chunks of odd length behind cached prefixes: bound by the products and exponentials
        dict(name="weigh_b2_w2049_c4500_d64_f16", op="weigh", B=2, W=2049, Hq=16, Hkv=4, D=64, tpb=48, lo=0, hi=4500,
             ragged=False, decay=1.0, dtype="f16"),
        # one long request over its budget
        dict(name="evict_b1_c16000_k4096_d128", op="evict", B=1, Hkv=8, D=128, tpb=16, lo=16000, hi=16000, keep=4096,
             first=4, recent=256),
        # a batch of requests, most of them over the budget
        dict(name="evict_b64_c8192_k2048_d128", op="evict", B=64, Hkv=8, D=128, tpb=32, lo=1500, hi=8192, keep=2048,
             first=4, recent=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adjust", "adjust", "rotate", "rotate_store", "weigh", "weigh", "evict"])
    tpb = rng.choice([16, 32, 48, 64, 128])
    lo = rng.choice([0, 1, rng.randint(2, 600)])
    D = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "f16"])
    Hkv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8])
    if op == "adjust":
        form = rng.choice(["chain", "chain", "tree"])
        V = _log(rng, 500, 160000)
        R = rng.randint(1, 17) if form == "chain" else rng.randint(4, 120)
        B = _log(rng, 1, max(1, min(256, 140_000_000 // (R * V))))
        inplace = rng.random() < 0.3  # then what can be done twice: the grammar
        return dict(op=op, form=form, B=B, R=R, V=V, T=0 if inplace else _log(rng, 1, 12000),
                    bias=0 if inplace else rng.choice([0, 1, rng.randint(2, 300)]), penalties=not inplace,
                    grammars=_log(rng, 1, 64) if inplace else rng.choice([0, rng.randint(1, 64)]), inplace=inplace,
                    ragged=form == "chain" and R > 1 and rng.random() < 0.5, dtype=rng.choice(["bf16", "f32"]))
    if op in ("rotate", "rotate_store"):
        tree = rng.random() < 0.3
        if tree or rng.random() < 0.5:
            B, W = _log(rng, 1, 256), rng.randint(1, 65)
        else:
            B, W = rng.randint(1, 4), _log(rng, 64, 4000)
        c = dict(op=op, B=B, W=W, Hq=Hkv * group, Hkv=Hkv, D=D, rot=rng.choice([D, D, D // 2, 16, D - 16]),
                 interleaved=rng.random() < 0.5, ramp=rng.choice([1.0, 2.0, 8.0, 32.0]), tree=tree, lo=lo,
                 hi=lo + _log(rng, 1, 2000 if op == "rotate_store" else 500000), ragged=rng.random() < 0.5, dtype=dtype)
        return c if op == "rotate" else dict(c, tpb=tpb)
    if op == "evict":
        hi = lo + _log(rng, 16, 20000)
        keep = max(1, int(hi * rng.uniform(0.05, 0.9)))
        first = rng.choice([0, min(4, keep // 4)])
        return dict(op=op, B=_log(rng, 1, max(1, min(128, 4_000_000 // (Hkv * hi)))), Hkv=Hkv, D=D, tpb=tpb, lo=lo, hi=hi,
                    keep=keep, first=first, recent=int((keep - first) * rng.choice([0, 0.1, 0.5])))
    form = rng.choice(["token", "chain", "chain", "prompt"])
    W = {"token": 1, "chain": rng.randint(2, 16), "prompt": _log(rng, 64, 2000)}[form]
    rows = W * Hkv * group
    hi = lo + _log(rng, 16, 60000 if form == "token" else 12000)
    hi = min(hi, lo + max(16, 280_000_000 // rows - W - lo))
    most = min(128, 4_500_000 // (Hkv * (lo + hi)), 200_000_000 // (rows * (hi + W)))
    return dict(op=op, B=_log(rng, 1, max(1, most)), W=W, Hq=Hkv * group, Hkv=Hkv, D=D, tpb=tpb, lo=lo, hi=hi,
                ragged=form != "token" and rng.random() < 0.5, decay=rng.choice([1.0, 0.99, 0.5]), dtype=dtype)


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


def _tree_masks(rng, B, N, depth):
    """Ancestor bits [B, N, ceil(N / 32)] int32 of random trees, a node's own bit among them; parents stand before their children."""
    bits = np.zeros((B, N, -(-N // 32) * 32), dtype=np.uint8)
    for b in range(B):
        level = np.zeros(N, dtype=np.int64)
        bits[b, 0, 0] = 1
        for n in range(1, N):
            ok = np.flatnonzero(level[:n] < depth)
            p = int(ok[rng.integers(0, len(ok))])
            level[n] = level[p] + 1
            bits[b, n] = bits[b, p]
            bits[b, n, n] = 1
    return torch.from_numpy(np.packbits(bits, axis=-1, bitorder="little").view(np.int32).copy()).to(DEV)


def _bits(words, n):
    """The first n bits of the last axis's 32-bit words, as truth values."""
    b = (words.long()[..., None] >> torch.arange(32, device=DEV)) & 1
    return b.reshape(*words.shape[:-1], -1)[..., :n] == 1


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


def _frequencies(rot, ramp):
    """Radians per position of each pair, in 64 bits, and the gain of cos and sin: base 10000; for a context
    extended `ramp` times the slow pairs are divided by it, the fast ones kept, those between blended."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = 10000.0 ** (-2 * i / rot)
    if ramp == 1.0:
        return f.to(DEV), 1.0
    turns = 4096 * f / (2 * math.pi)  # over the trained context
    kept = ((turns - 1) / (32 - 1)).clamp(0, 1)
    return (f / ramp * (1 - kept) + f * kept).to(DEV), 0.1 * math.log(ramp) + 1


def _tokens(rng, shape, V):
    """Token ids of which a few are frequent: log-uniform ranks, scattered over the vocabulary."""
    rank = np.floor(np.exp(rng.random(shape) * math.log(V))).astype(np.int64) - 1
    return (rank * 7919 + 13) % V


def _prepare_adjust(c, s, rng, g):
    B, R, V, T = c["B"], c["R"], c["V"], c["T"]
    t = TYPES[c["dtype"]]
    s["logits"] = torch.empty((B, R, V), dtype=t, device=DEV)
    for b in range(B):
        s["logits"][b] = 2.5 * torch.randn((R, V), generator=g, device=DEV)
    s["out"] = s["logits"] if c["inplace"] else torch.zeros_like(s["logits"])
    for k in ("tokens", "token_lens", "prompt_lens", "repetition", "frequency", "presence", "bias_ids", "bias_values",
              "allowed", "allowed_rows", "draft_tokens", "masks", "draft_lens"):
        s[k] = None
    s["masks"] = _tree_masks(rng, B, R, 8) if c["form"] == "tree" else None
    if c["form"] == "tree" or R > 1:
        s["draft_tokens"] = _i32(_tokens(rng, (B, R if c["form"] == "tree" else R - 1), V))
    if c["ragged"]:
        s["draft_lens"] = _i32((np.arange(B) * 5 + R - 1) % R)
    if c["penalties"]:
        s["tokens"] = _i32(_tokens(rng, (B, T), V))
        lens = rng.integers(-(-T // 2), T + 1, B)
        lens[rng.integers(0, B)] = T
        s["token_lens"] = _i32(lens)
        s["prompt_lens"] = _i32((lens * rng.random(B)).astype(np.int64))
        on = rng.random(B) < 0.8
        s["repetition"], s["frequency"], s["presence"] = (
            torch.from_numpy(np.where(on, x, n).astype(np.float32)).to(DEV)
            for x, n in ((rng.uniform(1.0, 1.3, B), 1.0), (rng.uniform(0, 1, B), 0.0), (rng.uniform(-0.5, 1, B), 0.0)))
    if c["bias"]:
        ids = np.stack([rng.permutation(V)[:c["bias"]] for _ in range(B)])
        ids = np.where(np.arange(ids.shape[1])[None, :] < rng.integers(1, ids.shape[1] + 1, B)[:, None], ids, -1)
        s["bias_ids"] = _i32(ids)
        values = np.where(rng.random(ids.shape) < 0.1, -np.inf, rng.uniform(-10, 10, ids.shape))
        s["bias_values"] = torch.from_numpy(values.astype(np.float32)).to(DEV)
    if c["grammars"]:
        n, words = c["grammars"], -(-V // 32)
        # inside a string nearly everything may follow, between a structure's parts a few tokens
        some = torch.rand((n, words * 32), generator=g, device=DEV)
        share = torch.where(torch.arange(n, device=DEV) % 2 == 0, 0.9, 0.001)
        bit = some < share[:, None]
        bit[:, 5] = True
        word = (bit.reshape(n, words, 32).long() << torch.arange(32, device=DEV)).sum(-1)
        s["allowed"] = torch.where(word >= 1 << 31, word - (1 << 32), word).to(torch.int32)
        s["allowed_rows"] = _i32(np.where(rng.random((B, R)) < 0.25, -1, rng.integers(0, n, (B, R))))


def _k_rows(s, T):
    """The cached keys of positions 0..T-1, [B, Hkv, T, D] float32 (any values behind a request's end)."""
    tables, tpb = s["tables"].long().clamp(min=0), s["tpb"]
    cols = -(-T // tpb)
    k = s["pool"][:, 0][tables[:, :cols]].float() * s["scales"][:, 0][tables[:, :cols]][..., None, None]
    return k.permute(0, 2, 1, 3, 4).reshape(s["B"], s["Hkv"], -1, s["D"])[:, :, :T]


def _scores(s, lo, hi):
    """scale * q . k of requests lo..hi-1 in 32 bits, [n, Hkv, W, group, T], -inf where a row sees nothing."""
    part = dict(s, B=hi - lo, tables=s["tables"][lo:hi])
    B, W, Hq, D = s["q"][lo:hi].shape
    H = s["Hkv"]
    T = s["tables"].shape[1] * s["tpb"]
    k = _k_rows(part, T)
    q = s["q"][lo:hi].float().reshape(B, W, H, Hq // H, D).permute(0, 2, 1, 3, 4).reshape(B, H, -1, D)
    a = (q @ k.transpose(-1, -2)).reshape(B, H, W, Hq // H, T) / math.sqrt(D)
    seq = s["seq_lens"][lo:hi].long()
    win = torch.full_like(seq, W) if s["window_lens"] is None else s["window_lens"][lo:hi].long()
    i = torch.arange(W, device=DEV)
    j = torch.arange(T, device=DEV)[None, :] - seq[:, None]  # the window's place of each position
    see = (j[:, None, :] <= i[None, :, None]) & (i[None, :] < win[:, None])[:, :, None]
    return a.masked_fill(~see[:, None, :, None, :], -math.inf)


def prepare(case, seed):
    c = case
    rng = np.random.default_rng(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(c)
    if c["op"] == "adjust":
        _prepare_adjust(c, s, rng, g)
        return s
    lens = rng.permutation(_lens(c))
    B, H, D = c["B"], c["Hkv"], c["D"]
    s["seq_lens"] = _i32(lens)
    if c["op"] == "evict":
        s["tables"], s["pool"], s["scales"] = _cache(c, rng, g, lens)
        T = s["tables"].shape[1] * c["tpb"]
        # few positions draw most of the attention; the weights of many have fallen to nothing
        w = torch.exp(2.5 * torch.randn((B, H, T), generator=g, device=DEV))
        s["weights"] = torch.where(torch.rand((B, H, T), generator=g, device=DEV) < 0.1, 0.0, w)
        s["out_weights"] = torch.zeros((B, H, c["keep"]), device=DEV)
        return s
    t = TYPES[c["dtype"]]
    W, Hq = c["W"], c["Hq"]
    wins = _wins(c)
    s["window_lens"] = _i32(wins) if c["ragged"] else None
    # q, k and v as a projection leaves them: slices of one row per token
    qkv = torch.randn((B, W, Hq + 2 * H, D), generator=g, device=DEV)
    qkv *= torch.exp(0.3 * torch.randn((B, W, Hq + 2 * H, 1), generator=g, device=DEV))
    qkv = qkv.to(t)
    s["q"], s["k"], s["v"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + H], qkv[:, :, Hq + H:]
    if c["op"] in ("rotate", "rotate_store"):
        s["inv_freq"], s["gain"] = _frequencies(c["rot"], c["ramp"])
        s["masks"] = _tree_masks(rng, B, W, 8) if c["tree"] else None
        # rows behind a window's end are left as they are
        s["out_q"] = torch.zeros((B, W, Hq, D), dtype=t, device=DEV)
        s["out_k"] = torch.zeros((B, W, H, D), dtype=t, device=DEV)
        if c["op"] == "rotate_store":
            s["tables"], s["pool"], s["scales"] = _cache(c, rng, g, lens + W)
            # positions were dropped from the cache before: it is shorter than the text
            s["starts"] = _i32(lens + rng.integers(0, 5000, B))
        return s
    s["tables"], s["pool"], s["scales"] = _cache(c, rng, g, lens + W)
    T = s["tables"].shape[1] * c["tpb"]
    # as the attention of these rows leaves it
    at = max(1, 400_000_000 // (W * Hq * T))
    lse = [torch.logsumexp(_scores(s, b, min(B, b + at)).double(), -1).float() for b in range(0, B, at)]
    lse = torch.cat(lse).permute(0, 2, 1, 3).reshape(B, W, Hq)
    s["lse"] = torch.where(lse == -math.inf, 0, lse).contiguous()  # 0 behind a window's end
    # what some steps before have left, of the size of what this one adds
    s["weights"] = torch.exp(1.5 * torch.randn((B, H, T), generator=g, device=DEV)) * (W * Hq / H / T)
    s["out"] = torch.zeros((B, H, T), device=DEV)
    return s


# ------------------------------------------------------------------ plain forms
def _scale_for(amax):
    """The smallest power of two with amax <= 448 * scale (0 for 0)."""
    m, e = torch.frexp(amax)
    s = torch.ldexp(torch.ones_like(amax), torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126))
    return torch.where(amax > 0, s, torch.zeros_like(amax))


def _ratio(a, b):
    return torch.where(b > 0, a / b, torch.zeros_like(a))


def _adjust(s):
    B, R, V = s["logits"].shape
    x = s["logits"].float()
    if s["penalties"]:
        T = s["tokens"].shape[1]
        i = torch.arange(T, device=DEV)[None, :]
        real, prompt = i < s["token_lens"][:, None], i < s["prompt_lens"][:, None]
        tokens = s["tokens"].long()
        count = torch.zeros((B, V), device=DEV).scatter_add_(1, tokens, (real & ~prompt).float())
        asked = torch.zeros((B, V), device=DEV).scatter_add_(1, tokens, (real & prompt).float()) > 0
        count = count[:, None, :].expand(B, R, V)
        if s["draft_tokens"] is not None:
            draft = s["draft_tokens"].long()
            M = draft.shape[1]
            m = torch.arange(M, device=DEV)
            if s["masks"] is None:  # row i comes behind drafts 0..i-1
                before = (m[None, :] < torch.arange(R, device=DEV)[:, None])[None].expand(B, R, M)
            else:  # row n comes behind node n and its ancestors; node 0 is among the tokens
                before = _bits(s["masks"], M) & (m > 0)
            count = count.scatter_add(2, draft[:, None, :].expand(B, R, M), before.float())
        r, f, p = (s[k][:, None, None] for k in ("repetition", "frequency", "presence"))
        again = torch.where(x > 0, x / r, x * r)
        x = torch.where((count > 0) | asked[:, None, :], again, x)
        x = torch.where(count > 0, x - f * count - p, x)
    if s["bias_ids"] is not None:
        add = torch.zeros((B, V + 1), device=DEV)
        ids = s["bias_ids"].long()
        add.scatter_add_(1, torch.where(ids < 0, V, ids), s["bias_values"])
        x = x + add[:, None, :V]
    if s["allowed"] is not None:
        rows = s["allowed_rows"].long()
        fine = _bits(s["allowed"], V)[rows.clamp(min=0)] | (rows < 0)[..., None]
        x = torch.where(fine, x, -math.inf)
    x = x.to(s["logits"].dtype)
    if s["draft_lens"] is not None:  # rows behind a request's last one are left as they are
        x = torch.where((torch.arange(R, device=DEV)[None, :] <= s["draft_lens"][:, None])[..., None], x, s["out"])
    s["out"].copy_(x)
    return s["out"]


def _turned(s, x):
    """x [B, W, heads, D] rotated to its rows' positions, in x's type."""
    B, W, _, D = x.shape
    rot = 2 * s["inv_freq"].numel()
    start = s["starts"] if s["op"] == "rotate_store" else s["seq_lens"]
    i = torch.arange(W, device=DEV)[None, :]
    if s["masks"] is not None:  # a node's depth
        i = _bits(s["masks"], W).sum(-1) - 1
    angle = (start[:, None] + i).double()[..., None] * s["inv_freq"]
    cos, sin = ((f(angle) * s["gain"]).float()[:, :, None, :] for f in (torch.cos, torch.sin))
    y = x[..., :rot].float()
    if s["interleaved"]:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y.to(x.dtype), x[..., rot:]], -1)


def _behind(s, y, out):
    """y where a row is of its request's window, else what `out` holds."""
    if s["window_lens"] is None:
        return y
    return torch.where((torch.arange(y.shape[1], device=DEV)[None, :] < s["window_lens"][:, None])[..., None, None], y, out)


def _rotate(s):
    return _behind(s, _turned(s, s["q"]), s["out_q"]), _behind(s, _turned(s, s["k"]), s["out_k"])


def _rotate_store(s):
    q, k = _turned(s, s["q"]), _turned(s, s["k"])
    seq, tables, pool, scales, tpb = s["seq_lens"].long(), s["tables"].long(), s["pool"], s["scales"], s["tpb"]
    B, W, H, D = k.shape
    win = torch.full((B,), W, device=DEV) if s["window_lens"] is None else s["window_lens"].long()
    x = torch.stack([k, s["v"]], 2).float()  # [B, W, 2, H, D]
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
    pool[rows] = torch.where(live[some][:, None, None, :, None], moved.float(), kept).to(torch.float8_e4m3fn)
    # the new rows
    touched = torch.zeros((B, pages), device=DEV).scatter_reduce_(1, page, real.float(), "amax") > 0
    at = ((seq // tpb)[:, None] + torch.arange(pages, device=DEV)).clamp(max=tables.shape[1] - 1)
    scales[tables.gather(1, at)[touched]] = new[touched]
    y = x * _ratio(torch.ones_like(new), new).gather(1, page[:, :, None, None].expand(B, W, 2, H))[..., None]
    blk = tables.gather(1, (t // tpb).clamp(max=tables.shape[1] - 1))
    pool.view(torch.uint8).permute(0, 3, 1, 2, 4)[blk[real], (t % tpb)[real]] = \
        y[real].to(torch.float8_e4m3fn).view(torch.uint8)
    return _behind(s, q, s["out_q"]), pool, scales


def _weigh(s):
    B, T = s["B"], s["weights"].shape[2]
    seq = s["seq_lens"].long()
    win = torch.full_like(seq, s["W"]) if s["window_lens"] is None else s["window_lens"].long()
    lse = s["lse"].reshape(B, s["W"], s["Hkv"], -1).permute(0, 2, 1, 3)[..., None]
    new = torch.exp(_scores(s, 0, B) - lse).sum((2, 3))
    t = torch.arange(T, device=DEV)[None, None, :]
    new = new + torch.where(t < seq[:, None, None], s["decay"] * s["weights"], 0)
    return torch.where(t < (seq + win)[:, None, None], new, s["out"])


def _evict(s):
    w, tables, pool, scales, tpb = s["weights"], s["tables"].long(), s["pool"], s["scales"], s["tpb"]
    B, H, T = w.shape
    seq, keep, D = s["seq_lens"].long(), s["keep"], s["D"]
    t = torch.arange(T, device=DEV)[None, None, :]
    n = seq[:, None, None]
    # those that always stay before those that may, by weight, the lowest position first; nothing behind the end
    must = (t < s["first"]) | (t >= n - s["recent"])
    rank = torch.where(t < n, torch.where(must, math.inf, w), -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :keep]
    if T < keep:
        order = torch.cat([order, order.new_zeros((B, H, keep - T))], -1)
    j = torch.arange(keep, device=DEV)[None, None, :]
    real = j < n
    kept = torch.sort(torch.where(real, order, T), -1).values
    at = torch.where(real, kept, 0)
    weights = torch.where(real, w.gather(2, at), s["out_weights"])
    # the rows, each with its block's scale; a block that receives rows gets the largest among theirs
    blk = tables[:, None, :].expand(B, H, -1).gather(2, at // tpb).clamp(min=0)
    h = torch.arange(H, device=DEV)[None, :, None].expand(B, H, keep)
    codes = pool.view(torch.uint8)
    x = codes[blk, :, h, at % tpb].view(torch.float8_e4m3fn).float()  # [B, H, keep, 2, D]
    had = torch.where(real[..., None], scales[blk, :, h], 0)  # [B, H, keep, 2]
    page = (j // tpb).expand(B, H, keep)
    pages = -(-keep // tpb)
    new = torch.zeros((B, H, pages, 2), device=DEV)
    new.scatter_reduce_(2, page[..., None].expand(B, H, keep, 2), had, "amax")
    y = x * _ratio(had, new.gather(2, page[..., None].expand(B, H, keep, 2)))[..., None]
    over = (real & (n > keep)).expand(B, H, keep)
    to = tables[:, None, :].expand(B, H, -1).gather(2, page.clamp(max=tables.shape[1] - 1))
    codes[to[over], :, h[over], (j % tpb).expand(B, H, keep)[over]] = y[over].to(torch.float8_e4m3fn).view(torch.uint8)
    cols = min(pages, tables.shape[1])
    whole = (seq > keep)[:, None, None].expand(B, H, cols)
    hh = torch.arange(H, device=DEV)[None, :, None].expand(B, H, cols)
    scales[tables[:, None, :cols].expand(B, H, cols)[whole], :, hh[whole]] = new[:, :, :cols][whole]
    return seq.clamp(max=keep).to(torch.int32), torch.where(real, kept, -1).to(torch.int32), weights, pool, scales


def run(state):
    s = state
    if not own:
        return {"adjust": _adjust, "rotate": _rotate, "rotate_store": _rotate_store, "weigh": _weigh,
                "evict": _evict}[s["op"]](s)
    import speculative_decoding_verification_row_gb300 as sv
    if s["op"] == "adjust":
        return sv.adjust_logits(s["logits"], tokens=s["tokens"], token_lens=s["token_lens"], prompt_lens=s["prompt_lens"],
                                repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"],
                                bias_ids=s["bias_ids"], bias_values=s["bias_values"], allowed=s["allowed"],
                                allowed_rows=s["allowed_rows"], draft_tokens=s["draft_tokens"],
                                draft_lens=s["draft_lens"], masks=s["masks"], out=s["out"])
    if s["op"] == "rotate":
        return sv.rotate_qk(s["q"], s["k"], s["seq_lens"], s["inv_freq"], interleaved=s["interleaved"], gain=s["gain"],
                            window_lens=s["window_lens"], masks=s["masks"], out_q=s["out_q"], out_k=s["out_k"])
    if s["op"] == "rotate_store":
        q = sv.rotate_store_kv(s["q"], s["k"], s["v"], s["inv_freq"], s["pool"], s["scales"], s["tables"], s["seq_lens"],
                               starts=s["starts"], interleaved=s["interleaved"], gain=s["gain"],
                               window_lens=s["window_lens"], masks=s["masks"], out_q=s["out_q"])
        return q, s["pool"], s["scales"]
    if s["op"] == "weigh":
        return sv.weigh_kv(s["q"], s["lse"], s["pool"], s["scales"], s["tables"], s["seq_lens"],
                           window_lens=s["window_lens"], weights=s["weights"], decay=s["decay"], out=s["out"])
    lens, kept, weights, _ = sv.evict_kv(s["weights"], s["pool"], s["scales"], s["tables"], s["seq_lens"], s["keep"],
                                         first=s["first"], recent=s["recent"], out_weights=s["out_weights"])
    return lens, kept, weights, s["pool"], s["scales"]


# ------------------------------------------------------------------ work
def work(case):
    c = case
    B = c["B"]
    if c["op"] == "adjust":
        size = 4 if c["dtype"] == "f32" else 2
        rows = B * c["R"] if not c["ragged"] else float((1 + (np.arange(B) * 5 + c["R"] - 1) % c["R"]).sum())
        around = 4.0 * B * (0.75 * c["T"] + 2 * c["bias"] + 3 + 2 * c["R"]) + c["grammars"] * c["V"] / 8
        # in place, the tokens that a grammar bans are written (of three quarters of the rows, 0.55 of a row) and none is read
        return {"bytes": around + rows * c["V"] * size * (0.41 if c["inplace"] else 2.0), "flops": 0.0}
    lens, H, D = _lens(c), c["Hkv"], c["D"]
    if c["op"] == "evict":
        over = lens > c["keep"]
        rows = float(over.sum()) * c["keep"] * 2 * H
        kept = float(np.minimum(lens, c["keep"]).sum()) * H
        return {"bytes": 4.0 * H * float(lens.sum()) + 8 * kept + rows * (2 * D + 8 / c["tpb"]), "flops": 0.0}
    wins = _wins(c)
    if c["op"] in ("rotate", "rotate_store"):
        heads = float(wins.sum()) * (c["Hq"] + H)
        moved = 4.0 * D * heads
        if c["op"] == "rotate_store":
            moved = float(wins.sum()) * D * (4 * c["Hq"] + 2 * H * 3 + 2 * H * 4 / c["tpb"] / D)
        return {"bytes": moved, "flops": 3.0 * heads * c["rot"]}
    seen = lens + wins
    pages = -(-seen // c["tpb"])
    rows = wins * c["Hq"]
    pairs = float(((lens * wins + wins * (wins + 1) // 2) * c["Hq"]).sum())
    read = float((seen * H * D + pages * H * 4 + lens * H * 4).sum()) + float(rows.sum()) * (2 * D + 4)
    return {"bytes": read + 4.0 * H * float(seen.sum()), "flops": 2.0 * pairs * D}


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


def _exact_adjust(s):
    out = s["out"].double().clone()
    B, R, V = out.shape
    none = torch.zeros(0, dtype=torch.int64, device=DEV)
    bits = None if s["masks"] is None else _bits(s["masks"], R).tolist()
    for b in range(B):
        said = asked = none
        if s["penalties"]:
            n, p = int(s["token_lens"][b]), int(s["prompt_lens"][b])
            said, asked = s["tokens"][b, p:n].long(), s["tokens"][b, :p].long()
        last = R - 1 if s["draft_lens"] is None else int(s["draft_lens"][b])
        for i in range(last + 1):
            x = s["logits"][b, i].double()
            if s["penalties"]:
                mine = []
                if s["draft_tokens"] is not None:
                    mine = range(i) if bits is None else [m for m in range(1, R) if bits[b][i][m]]
                here = s["draft_tokens"][b].long()[list(mine)] if len(mine) else none
                token, times = torch.unique(torch.cat([said, here]), return_counts=True)
                r, f, p = (float(s[k][b]) for k in ("repetition", "frequency", "presence"))
                any_ = torch.unique(torch.cat([token, asked]))
                x[any_] = torch.where(x[any_] > 0, x[any_] / r, x[any_] * r)
                x[token] -= f * times + p
            if s["bias_ids"] is not None:
                m = s["bias_ids"][b] >= 0
                x[s["bias_ids"][b][m].long()] += s["bias_values"][b][m].double()
            if s["allowed"] is not None and int(s["allowed_rows"][b, i]) >= 0:
                x[~_bits(s["allowed"][int(s["allowed_rows"][b, i])], V)] = -math.inf
            out[b, i] = x
    return out


def _exact_turned(s, x, out):
    """The rows of each window as complex numbers times exp(i position frequency)."""
    y = out.double().clone()
    B, W, heads, D = x.shape
    rot = 2 * s["inv_freq"].numel()
    start = (s["starts"] if s["op"] == "rotate_store" else s["seq_lens"]).tolist()
    for b in range(B):
        w = W if s["window_lens"] is None else int(s["window_lens"][b])
        place = torch.arange(W, device=DEV).double()
        if s["masks"] is not None:
            place = _bits(s["masks"][b], W).double().sum(-1) - 1
        turn = torch.polar(torch.full((W, rot // 2), s["gain"], dtype=torch.float64, device=DEV),
                           torch.outer(place + start[b], s["inv_freq"]))[:, None, :]
        z = x[b].double()
        if s["interleaved"]:
            p = torch.view_as_real(torch.view_as_complex(z[..., :rot].reshape(W, heads, -1, 2).contiguous()) * turn).flatten(-2)
        else:
            p = torch.complex(z[..., :rot // 2].contiguous(), z[..., rot // 2:rot].contiguous()) * turn
            p = torch.cat([p.real, p.imag], -1)
        y[b, :w] = torch.cat([p, z[..., rot:]], -1)[:w]
    return y


def _exact_store(s):
    values, scales = _values(s["pool"]), s["scales"].double()
    tpb, tables = s["tpb"], s["tables"].tolist()
    k = _exact_turned(s, s["k"], s["out_k"]).to(s["k"].dtype)  # the cache takes the rotated keys in their type
    for b in range(s["B"]):
        at = first = int(s["seq_lens"][b])
        end = at + (s["W"] if s["window_lens"] is None else int(s["window_lens"][b]))
        while at < end:
            to, blk, off = min(end, (at // tpb + 1) * tpb), tables[b][at // tpb], at % tpb
            x = torch.stack([k[b, at - first:to - first], s["v"][b, at - first:to - first]], 1).double()
            need = torch.tensor([[_need(a) for a in r] for r in x.abs().amax((0, 3)).tolist()], dtype=torch.float64, device=DEV)
            new = need if off == 0 else torch.maximum(need, scales[blk])
            ratio = torch.where(new > 0, 1 / new.clamp(min=1e-300), 0.0)[:, :, None, None]
            if off:
                values[blk, :, :, :off] = _nearest(values[blk, :, :, :off] * scales[blk][:, :, None, None] * ratio)
            values[blk, :, :, off:off + to - at] = _nearest(x.permute(1, 2, 0, 3) * ratio)
            scales[blk] = new
            at = to
    return values, scales


def _exact_weigh(s):
    out = s["out"].double().clone()
    B, W, Hq, D = s["q"].shape
    H, tpb = s["Hkv"], s["tpb"]
    for b in range(B):
        n = int(s["seq_lens"][b])
        w = W if s["window_lens"] is None else int(s["window_lens"][b])
        blocks = s["tables"][b, :-(-(n + w) // tpb)].long()
        k = _values(s["pool"][blocks, 0]) * s["scales"][blocks, 0].double()[..., None, None]
        k = k.permute(1, 0, 2, 3).reshape(H, -1, D)[:, :n + w]
        see = torch.ones((w, n + w), dtype=torch.bool, device=DEV)
        see[:, n:] = torch.ones((w, w), dtype=torch.bool, device=DEV).tril()
        out[b, :, :n] = s["decay"] * s["weights"][b, :, :n].double()
        out[b, :, n:n + w] = 0
        for h in range(Hq):
            a = s["q"][b, :w, h].double() @ k[h // (Hq // H)].T * D ** -0.5
            p = torch.exp(a - s["lse"][b, :w, h].double()[:, None]) * see
            out[b, h // (Hq // H), :n + w] += p.sum(0)
    return out


def _exact_evict(s):
    values, scales = _values(s["pool"]), s["scales"].double()
    out = s["out_weights"].double().clone()
    tpb, keep, tables = s["tpb"], s["keep"], s["tables"].long()
    for b in range(s["B"]):
        n = int(s["seq_lens"][b])
        for h in range(s["Hkv"]):
            w = s["weights"][b, h, :n].double()
            if n <= keep:
                out[b, h, :n] = w
                continue
            free = keep - s["first"] - s["recent"]
            pos = torch.arange(s["first"], n - s["recent"], device=DEV)
            # by weight, then by position
            by = pos[torch.sort(-w[pos], stable=True).indices[:free]]
            kept = torch.cat([torch.arange(s["first"], device=DEV), by.sort().values, torch.arange(n - s["recent"], n, device=DEV)])
            out[b, h, :keep] = w[kept]
            src, dst = tables[b, kept // tpb], tables[b, torch.arange(keep, device=DEV) // tpb]
            for kind in range(2):
                x = values[src, kind, h, kept % tpb] * scales[src, kind, h][:, None]
                new = torch.zeros(scales.shape[0], dtype=torch.float64, device=DEV)
                new.scatter_reduce_(0, dst, scales[src, kind, h], "amax")
                ratio = torch.where(new > 0, 1 / new.clamp(min=1e-300), 0.0)
                values[dst, kind, h, torch.arange(keep, device=DEV) % tpb] = _nearest(x * ratio[dst][:, None])
                scales[dst, kind, h] = new[dst]
    return None, None, out, values, scales


def exact(case, seed):
    c = case
    if c["op"] == "rotate_store" and sum(_wins(c)) / c["tpb"] + c["B"] > 4000:
        return None
    s = prepare(c, seed)
    if c["op"] == "adjust":
        return _exact_adjust(s)
    if c["op"] == "rotate":
        return _exact_turned(s, s["q"], s["out_q"]), _exact_turned(s, s["k"], s["out_k"])
    if c["op"] == "rotate_store":
        return (_exact_turned(s, s["q"], s["out_q"]), *_exact_store(s))
    return _exact_weigh(s) if c["op"] == "weigh" else _exact_evict(s)
