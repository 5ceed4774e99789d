"""The calls around the verify and the cache as a decode step uses them
together: rotated and stored, attended, weighed, penalised, verified, moved,
rolled back and evicted.  Each call's result is held against the oracle on the
inputs that it got; the same steps captured in one graph give the same bits."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_row_gb300 as sv
from oracle import kv, window
from _kv import random_paths

pytestmark = pytest.mark.gpu

B, N, L, H, G, D, TPB, V, KEEP = 3, 12, 5, 2, 4, 64, 16, 600, 96


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _state(seed):
    rng = np.random.default_rng(seed)
    cols, blocks = 16, 64
    s = dict(pool=torch.zeros((blocks, 2, H, TPB, D), dtype=torch.uint8, device="cuda"),
             scales=torch.zeros((blocks, 2, H), device="cuda"), tables=_i32(np.full((B, cols), -1)), held=_i32([0] * B),
             free=_i32(rng.permutation(blocks)), count=_i32([blocks]), seq=_i32([0] * B), text=_i32([0] * B),
             w=torch.zeros((B, H, cols * TPB), device="cuda"), said=_i32(np.zeros((B, 400))), said_n=_i32([0] * B),
             prompt_n=_i32([0] * B))
    s["paths"] = _i32(np.stack([random_paths(rng, N, N, L) for _ in range(B)]))
    s["masks"] = sv.tree_masks(s["paths"], N)
    s["freq"], s["gain"] = sv.rotary_frequencies(D, scaling="ramp", factor=4.0, original_len=64, device="cuda")
    for k, lo, hi in (("rep", 1.0, 1.3), ("fre", 0, 0.5), ("pre", 0, 0.5)):
        s[k] = torch.from_numpy(rng.uniform(lo, hi, B).astype(np.float32)).cuda()
    allowed = rng.integers(-2**31, 2**31, (2, -(-V // 32))) | 0x55555555
    s["allowed"], s["rows"] = _i32(allowed), _i32(rng.integers(-1, 2, (B, N)))
    return s, rng


def _inputs(rng, W):
    d = dict(qkv=torch.from_numpy(rng.normal(0, 1, (B, W, (G + 2) * H, D))).cuda().bfloat16())
    d["logits"] = torch.from_numpy(rng.normal(0, 2, (B, N, V))).cuda().bfloat16()
    d["tree"] = torch.zeros((B, N), dtype=torch.int32, device="cuda")
    return d


def _split(qkv):
    return qkv[:, :, :G * H], qkv[:, :, G * H:G * H + H], qkv[:, :, G * H + H:]


def _np(t):
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def _prefill(s, rng):
    lens = np.array([90, 50, 7])
    x = _inputs(rng, 90)
    q, k, v = _split(x["qkv"])
    win = _i32(lens)
    sv.reserve_blocks(s["seq"], s["tables"], s["held"], s["free"], s["count"], TPB, 90, window_lens=win)
    qr = sv.rotate_store_kv(q, k, v, s["freq"], s["pool"], s["scales"], s["tables"], s["seq"], starts=s["text"],
                            gain=s["gain"], window_lens=win)
    _, lse = sv.attend_kv(qr, s["pool"], s["scales"], s["tables"], s["seq"], window_lens=win, want_lse=True)
    sv.weigh_kv(qr, lse, s["pool"], s["scales"], s["tables"], s["seq"], window_lens=win, out=s["w"])
    s["said"][:, :90] = _i32(rng.integers(0, V, (B, 90)))
    for k in ("seq", "text", "said_n", "prompt_n"):
        s[k].copy_(win)


def _propose(s, x):
    """Draft tokens that the penalised target partly accepts: each node its parent's greedy token."""
    bits = kv.mask_bits(_np(s["masks"]), N)
    want = torch.zeros((B, N), dtype=torch.int32)
    for _ in range(L):  # a level at a time: a node's penalties know the drafts before it
        adj = sv.adjust_logits(x["logits"], tokens=s["said"], token_lens=s["said_n"], prompt_lens=s["prompt_n"],
                               repetition=s["rep"], frequency=s["fre"], presence=s["pre"], allowed=s["allowed"],
                               allowed_rows=s["rows"], draft_tokens=_i32(want.numpy()), masks=s["masks"])
        best = adj.float().argmax(-1).cpu()
        for b in range(B):
            for n in range(1, N):
                anc = np.flatnonzero(bits[b, n])
                if len(anc) > 1:
                    want[b, n] = best[b, anc[-2]] if n % 3 else 5
    x["tree"].copy_(want)


def _step(s, x, seen=None):
    def note(name, **kw):
        if seen is not None:
            seen[name] = {k: _np(v) for k, v in kw.items()}
    q, k, v = _split(x["qkv"])
    sv.reserve_blocks(s["seq"], s["tables"], s["held"], s["free"], s["count"], TPB, N)
    qr = sv.rotate_store_kv(q, k, v, s["freq"], s["pool"], s["scales"], s["tables"], s["seq"], starts=s["text"],
                            gain=s["gain"], masks=s["masks"])
    out, lse = sv.attend_kv(qr, s["pool"], s["scales"], s["tables"], s["seq"], masks=s["masks"], want_lse=True)
    note("attend", q=q, qr=qr, pool=s["pool"], scales=s["scales"], tables=s["tables"], seq=s["seq"], out=out, lse=lse,
         text=s["text"])
    adj = sv.adjust_logits(x["logits"], tokens=s["said"], token_lens=s["said_n"], prompt_lens=s["prompt_n"],
                           repetition=s["rep"], frequency=s["fre"], presence=s["pre"], allowed=s["allowed"],
                           allowed_rows=s["rows"], draft_tokens=x["tree"], masks=s["masks"])
    note("adjust", said=s["said"], said_n=s["said_n"], adj=adj)
    tok, n, _, nodes = sv.verify_tree(adj, x["tree"], s["paths"])
    sv.relocate_quantised_kv(s["pool"], s["scales"], s["tables"], s["seq"], nodes, n)
    # the accepted path is a chain now: its rows of q and lse
    at = nodes.clamp(min=0).long()
    qa = qr.gather(1, at[:, :, None, None].expand(B, L, G * H, D))
    la = lse.gather(1, at[:, :, None].expand(B, L, G * H))
    before = s["w"].clone()
    sv.weigh_kv(qa, la, s["pool"], s["scales"], s["tables"], s["seq"], window_lens=n + 1, weights=s["w"], decay=0.9,
                out=s["w"])
    note("weigh", qa=qa, la=la, pool=s["pool"], scales=s["scales"], tables=s["tables"], seq=s["seq"], n=n, before=before,
         w=s["w"])
    new, _, give = sv.rollback_paged(s["seq"], n, N - 1, TPB, blocks_held=s["held"])
    sv.release_blocks(s["tables"], s["held"], give, s["free"], s["count"])
    pool, scales, w = s["pool"].clone(), s["scales"].clone(), s["w"].clone()
    old = new.clone()
    _, kept, _, give = sv.evict_kv(s["w"], s["pool"], s["scales"], s["tables"], new, KEEP, first=4, recent=16,
                                   blocks_held=s["held"], out_lens=new, out_weights=s["w"])
    note("evict", pool=pool, scales=scales, tables=s["tables"], w=w, old=old, held=s["held"], new=new, kept=kept, give=give,
         out=s["w"], moved=s["pool"], rescaled=s["scales"])
    sv.release_blocks(s["tables"], s["held"], give, s["free"], s["count"])
    s["seq"].copy_(new)
    s["text"] += n + 1
    slot = s["said_n"][:, None] + torch.arange(L, device="cuda")
    mine = torch.arange(L, device="cuda")[None] <= n[:, None]
    s["said"].scatter_(1, slot.long(), torch.where(mine, tok, s["said"].gather(1, slot.long())))
    s["said_n"] += n + 1
    return out, adj, tok, n, kept


def _check(s, x, seen):
    a = seen["attend"]
    masks = _np(s["masks"])
    want = window.rotate(a["q"], np.zeros_like(a["q"]), a["text"], _np(s["freq"]), False, s["gain"], None, masks)
    tol = 2.0 ** -21 * s["gain"] * 2 * np.abs(a["q"]).max() + 2.0 ** -8 * np.abs(want)
    assert (np.abs(a["qr"] - want) <= tol).all()
    r = kv.attend(a["qr"], a["pool"], a["scales"], a["tables"], a["seq"], masks=masks)
    # weights to 11 bits, out to 8; scores to fp32
    assert (np.abs(a["out"] - r["out"]) <= 2.0 ** -8 * np.abs(r["out"]) + 2.0 ** -9 * r["amp"]).all()
    assert (np.abs(a["lse"] - r["lse"]) <= 1e-4).all()
    d = seen["adjust"]
    adj = window.adjust(_np(x["logits"]), np.zeros((B, N, V)), d["said"], d["said_n"], _np(s["prompt_n"]), _np(s["rep"]),
                        _np(s["fre"]), _np(s["pre"]), allowed=_np(s["allowed"]), allowed_rows=_np(s["rows"]),
                        draft_tokens=_np(x["tree"]), masks=masks)
    fine = np.isfinite(adj)
    assert np.array_equal(fine, np.isfinite(d["adj"]))
    assert (np.abs(adj[fine] - d["adj"][fine]) <= 2.0 ** -8 * np.abs(adj[fine]) + 1e-5).all()
    w = seen["weigh"]
    want, spread = window.weigh(w["qa"], w["la"], w["pool"], w["scales"], w["tables"], w["seq"], w["before"], w["n"] + 1, None,
                                w["before"], np.float32(0.9))
    # as test_evict.py derives it
    rel = np.expm1(spread.max() * (D + 3) * 2.0 ** -23) + 2.0 ** -20
    assert (np.abs(w["w"] - want) <= rel * np.abs(want)).all()
    e = seen["evict"]
    mark = e["w"].astype(np.float32)
    new, kept, out, give, pool, scales = window.evict(mark, e["pool"], e["scales"], e["tables"], e["old"], KEEP, 4, 16,
                                                      e["held"], mark)
    assert np.array_equal(e["new"], new) and np.array_equal(e["kept"], kept) and np.array_equal(e["give"], give)
    assert np.array_equal(e["out"], out) and np.array_equal(e["rescaled"], scales)
    nan = (pool & 127) == 127
    assert np.array_equal(e["moved"][~nan], pool[~nan])
    return e["old"].max() > KEEP


def test_steps_of_a_request_that_outgrows_its_budget():
    s, rng = _state(0)
    _prefill(s, rng)
    evicted = accepted = 0
    for _ in range(4):
        x = _inputs(rng, N)
        _propose(s, x)
        seen = {}
        n = _step(s, x, seen)[3]
        evicted += _check(s, x, seen)
        accepted += int(n.sum())
        assert (n >= 0).all() and (s["seq"] <= KEEP).all()
        # every block is held once or free
        held = sorted(s["free"][:s["count"].item()].tolist() + [t for t in s["tables"].flatten().tolist() if t >= 0])
        assert held == list(range(s["free"].numel()))
    assert evicted and accepted and (s["text"] > s["seq"]).any()


def test_a_captured_step_gives_the_same_bits():
    s, rng = _state(1)
    _prefill(s, rng)
    xs = []
    t = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    want = []
    for _ in range(3):
        x = _inputs(rng, N)
        _propose(t, x)
        xs.append(x)
        want.append([y.clone() for y in _step(t, x)])
    buf = {k: v.clone() for k, v in xs[0].items()}
    keep = {k: v.clone() for k, v in s.items() if isinstance(v, torch.Tensor)}
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        _step(s, buf)  # the allocations before the capture
    torch.cuda.synchronize()
    for k, v in keep.items():
        s[k].copy_(v)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = _step(s, buf)
    for x, w in zip(xs, want):
        for k in buf:
            buf[k].copy_(x[k])
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, w))
    for k in keep:
        assert torch.equal(s[k], t[k]), k
