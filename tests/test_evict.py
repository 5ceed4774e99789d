"""Accumulated attention weights and eviction from the paged 8-bit cache:
oracle pins and refusals on the CPU, the CUDA calls against the oracle on the
GPU.

weigh_kv's tolerance.  A score is a sum of D products that are exact in fp32,
added by tensor cores that may cut bits below 2^-23 of the partial sum: D *
2^-23 of the sum of magnitudes ("spread", times the scale); the scale's product
and the subtraction of lse round by 2^-24 of their results (|score| <= spread,
|score - lse| <= 2 spread + the sum of what is left of exp), the product with
log2(e) as much again.  exp2 is off by 2^-22.  That is a relative error of each
weight; the sum of n weights adds at most (n / 64 + 64) roundings of 2^-24, the
decayed weight two.

evict_kv has no tolerance: its choice, its moves and its roundings are defined
to the bit."""
import ctypes
import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_row_gb300 as sv
from oracle import kv, window
from _kv import cache, to_bf16, to_f16
from test_kv_store import BAD_CACHES, _fake_cache

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ CPU
def test_weights_of_the_oracle_are_the_attentions():
    """The weights of a window's rows sum to their number, and weighing V by them is the sum of the outputs."""
    rng = np.random.default_rng(0)
    H, G, D, W, s = 2, 3, 64, 4, 21
    pool, scales, tables = cache(rng, [s + W], H, D, 16)
    q = rng.normal(0, 1, (1, W, H * G, D))
    r = kv.attend(q, pool, scales, tables, [s])
    w, _ = window.weigh(q, r["lse"], pool, scales, tables, [s], np.zeros((1, H, s + W)))
    assert np.allclose(w.sum(-1), W * G)
    v = np.stack([kv.decode(pool[tables[0, t // 16], 1, :, t % 16]) * scales[tables[0, t // 16], 1][:, None]
                  for t in range(s + W)], 1)
    assert np.allclose((w[0, :, :, None] * v).sum(1), r["out"][0].reshape(W, H, G, D).sum((0, 2)))


def test_oracle_evict_hand_example():
    D, tpb = 64, 16
    pool = np.zeros((3, 2, 1, tpb, D), np.uint8)
    scales = np.array([1.0, 4.0, 0.5], np.float32).reshape(3, 1, 1).repeat(2, 1)
    tables = np.array([[2, 0, 1]], np.int32)
    for t in range(48):
        pool[tables[0, t // tpb], :, 0, t % tpb] = kv.encode(np.full(D, 1.0 + t % 8))
    w = np.zeros((1, 1, 48), np.float32)
    w[0, 0, [5, 20, 40]], w[0, 0, 30] = 3.0, np.nan
    new, kept, out, free, p, s = window.evict(w, pool, scales, tables, [48], 18, first=1, recent=2, held=[3])
    # 0 stays; 46 and 47 stay; 5, 20 and 40 by weight; then the lowest positions of weight 0
    assert kept[0, 0].tolist() == [0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 20, 40, 46, 47]
    assert new.tolist() == [18] and free.tolist() == [1] and out[0, 0, 5] == 3.0
    # block 2 receives rows of scales 0.5 and 4 (from 46 on the second block's): the largest
    assert s[2, 0, 0] == 4.0 and s[0, 0, 0] == 4.0 and s[1, 0, 0] == 4.0
    get = lambda j: kv.decode(p[tables[0, j // tpb], 0, 0, j % tpb, 0]) * s[tables[0, j // tpb], 0, 0]  # noqa: E731
    for j, t in enumerate(kept[0, 0]):
        assert get(j) == (1.0 + t % 8) * scales[tables[0, t // tpb], 0, 0]


def _fake_weigh(**o):
    f = 16 * 1024
    s = (ctypes.c_int64 * 3)(256, 128, 64)
    a = dict(size=ctypes.sizeof(sv.WeighParams), q=f, q_strides=s, dtype=sv.SPEC_BF16, B=2, W=3, q_heads=4, seq_lens=f,
             window_lens=None, lse=f, scale=0.1, weights=f, decay=1.0, out=f, T=100)
    a.update(o)
    return sv.WeighParams(*[a[n] for n, _ in sv.WeighParams._fields_])


def _fake_evict(**o):
    f = 16 * 1024
    a = dict(size=ctypes.sizeof(sv.EvictParams), weights=f, T=100, B=2, seq_lens=f, keep=20, first=4, recent=6, new_lens=f,
             kept=f, out_weights=2 * f, T_out=20, blocks_held=f, free_blocks=f)
    a.update(o)
    return sv.EvictParams(*[a[n] for n, _ in sv.EvictParams._fields_])


def test_refusals_before_any_launch():
    lib = sv.lib()
    odd = (ctypes.c_int64 * 3)(256, 132, 64)

    def weigh(cache, p, scratch=16 * 1024, size=1 << 24):
        return lib.spec_weigh_kv(cache, p, scratch, size, None)

    def evict(cache, p, scratch=16 * 1024, size=1 << 24):
        return lib.spec_evict_kv(cache, p, scratch, size, None)
    for B, H, keep, tpb in ((0, 1, 1, 16), (8193, 1, 1, 16), (1, 0, 1, 16), (1, 1025, 1, 16), (1, 1, 0, 16),
                            (1, 1, 2**30 + 1, 16), (1, 1, 1, 8), (1, 1, 1, 24), (1, 1, 1, 1040)):
        assert lib.spec_evict_scratch_size(B, H, keep, tpb) == 0
    need = lib.spec_evict_scratch_size(2, 2, 20, 16)
    for bad in (dict(scratch=None), dict(scratch=16 * 1024 + 128), dict(size=need - 1)):
        assert evict(_fake_cache(), _fake_evict(), **bad) == sv.SPEC_EWORKSPACE
    for B, W, q, k, D in ((0, 1, 4, 2, 64), (8193, 1, 4, 2, 64), (1, 0, 4, 2, 64), (1, 65537, 4, 2, 64), (1, 1, 4, 3, 64),
                          (1, 1, 0, 1, 64), (1, 1, 4, 0, 64), (1, 1, 16386, 2, 64), (1, 1, 4, 2, 96)):
        assert lib.spec_weigh_scratch_size(B, W, q, k, D) == 0
    for W in (3, 300):
        need = lib.spec_weigh_scratch_size(2, W, 4, 2, 64)
        for bad in (dict(scratch=None), dict(scratch=16 * 1024 + 128), dict(size=need - 1)):
            assert weigh(_fake_cache(), _fake_weigh(W=W), **bad) == sv.SPEC_EWORKSPACE
    for bad in BAD_CACHES:
        assert weigh(_fake_cache(**bad), _fake_weigh()) == sv.SPEC_EINVAL, bad
        assert evict(_fake_cache(**bad), _fake_evict()) == sv.SPEC_EINVAL, bad
    for bad in (dict(size=8), dict(q=None), dict(q=16 * 1024 + 4), dict(q_strides=odd), dict(dtype=sv.SPEC_F32), dict(B=0),
                dict(B=8193), dict(W=0), dict(W=65537), dict(q_heads=0), dict(q_heads=3), dict(q_heads=16386),
                dict(seq_lens=None), dict(lse=None), dict(out=None), dict(T=0), dict(scale=math.nan), dict(scale=3e38),
                dict(decay=math.inf), dict(B=8192, W=65536, q_heads=16)):
        assert weigh(_fake_cache(), _fake_weigh(**bad)) == sv.SPEC_EINVAL, bad
    for bad in (dict(size=8), dict(weights=None), dict(T=0), dict(B=0), dict(B=8193), dict(seq_lens=None), dict(keep=0),
                dict(keep=2**30 + 1, T_out=2**31 - 1), dict(first=-1), dict(recent=-1), dict(first=15),
                dict(first=2**31 - 1), dict(new_lens=None), dict(kept=None), dict(out_weights=None), dict(T_out=19),
                dict(out_weights=16 * 1024), dict(blocks_held=None), dict(free_blocks=None)):
        assert evict(_fake_cache(), _fake_evict(**bad)) == sv.SPEC_EINVAL, bad
    long = dict(max_blocks=2**26, tokens_per_block=32)
    assert weigh(_fake_cache(**long), _fake_weigh()) == sv.SPEC_EINVAL
    assert evict(_fake_cache(**long), _fake_evict()) == sv.SPEC_EINVAL
    assert weigh(_fake_cache(), None) == evict(_fake_cache(), None) == sv.SPEC_EINVAL
    assert weigh(None, _fake_weigh()) == evict(None, _fake_evict()) == sv.SPEC_EINVAL


_NO_GPU = pytest.mark.skipif(torch.cuda.is_available(),
                             reason="a call that is not refused would read the addresses made up here")
_F = 1 << 20
_CACHE = dict(pool=9 * _F, scales=10 * _F, block_tables=11 * _F)


@_NO_GPU
@pytest.mark.parametrize("W", [3, 300])
def test_weigh_refuses_arrays_that_overlap(W):
    lib, f, B, H, T = sv.lib(), _F, 2, 2, 100
    row = (ctypes.c_int64 * 3)(W * 512, 512, 64)

    def call(scratch=12 * f, cache=(), **o):
        a = dict(q=f, q_strides=row, W=W, seq_lens=4 * f, window_lens=5 * f, lse=6 * f, weights=7 * f, out=8 * f, B=B, T=T)
        return lib.spec_weigh_kv(_fake_cache(**{**_CACHE, **dict(cache)}), _fake_weigh(**{**a, **o}), scratch, 1 << 24, None)
    n = B * H * T * 4
    for o in (dict(), dict(out=7 * f), dict(weights=None), dict(out=7 * f + n), dict(weights=8 * f + n), dict(window_lens=None),
              dict(out=f + 4 * 128, T=2, q_strides=(ctypes.c_int64 * 3)(W * 512, 512, 64), B=1), dict(lse=7 * f),
              dict(q_strides=(ctypes.c_int64 * 3)(0, 512, 64))):  # not refused: there is no GPU
        assert call(**o) == sv.SPEC_ECUDA, o
    for o in (dict(out=7 * f + 4), dict(out=7 * f - n + 4), dict(out=6 * f + 8), dict(out=f), dict(out=4 * f), dict(out=5 * f + 4),
              dict(out=9 * f), dict(out=10 * f), dict(out=11 * f), dict(scratch=f), dict(scratch=7 * f), dict(scratch=8 * f),
              dict(scratch=6 * f), dict(scratch=11 * f)):
        assert call(**o) == sv.SPEC_EINVAL, o


@_NO_GPU
def test_evict_refuses_arrays_that_overlap():
    lib, f = sv.lib(), _F
    row = 2 * 2 * 4  # bytes a position: 2 requests, 2 heads

    def call(scratch=12 * f, cache=(), **o):
        a = dict(weights=f, seq_lens=2 * f, new_lens=3 * f, kept=4 * f, out_weights=5 * f, blocks_held=6 * f, free_blocks=7 * f)
        return lib.spec_evict_kv(_fake_cache(**{**_CACHE, **dict(cache)}), _fake_evict(**{**a, **o}), scratch, 1 << 20, None)
    for o in (dict(), dict(new_lens=2 * f), dict(out_weights=f, T_out=100), dict(new_lens=2 * f, out_weights=f, T_out=100),
              dict(blocks_held=None, free_blocks=None), dict(out_weights=f + 100 * row), dict(kept=5 * f + 20 * row),
              dict(free_blocks=3 * f + 8)):  # not refused: there is no GPU
        assert call(**o) == sv.SPEC_ECUDA, o
    for o in (dict(new_lens=2 * f + 4), dict(out_weights=f + 4), dict(out_weights=f + 4, T_out=100), dict(out_weights=f + 100 * row - 4),
              dict(kept=f), dict(kept=5 * f + 20 * row - 4), dict(free_blocks=3 * f + 4), dict(free_blocks=6 * f), dict(new_lens=6 * f + 4),
              dict(kept=9 * f), dict(out_weights=10 * f), dict(out_weights=11 * f), dict(scratch=f), dict(scratch=4 * f), dict(scratch=11 * f),
              dict(cache=dict(scales=9 * f + 64)), dict(cache=dict(pool=f)), dict(cache=dict(block_tables=9 * f + 4))):
        assert call(**o) == sv.SPEC_EINVAL, o


# ------------------------------------------------------------------ GPU: weights
def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _gpu(*arrays):
    return [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in arrays]


def _weigh_case(rng, lens, W, Hq, H, D, tpb, dtype, wins=None, amp=1.0):
    B = len(lens)
    wins = np.full(B, W) if wins is None else np.asarray(wins)
    pool, scales, tables = cache(rng, np.maximum(lens, 0) + np.clip(wins, 0, W), H, D, tpb)
    q = amp * rng.normal(0, 1, (B, W, Hq, D))
    q = to_bf16(q) if dtype == "bf16" else to_f16(q)
    lse = kv.attend(q, pool, scales, tables, lens, np.clip(wins, 0, W))["lse"].astype(np.float32)
    return q, lse, pool, scales, tables, wins


def _check_weigh(q, lse, pool, scales, tables, lens, wins, dtype, T, weights=None, decay=1.0, scale=None, strided=False):
    B, W, Hq, D = q.shape
    H = pool.shape[2]
    qd = torch.from_numpy(q).to(TYPES[dtype]).cuda()
    if strided:
        qd = torch.cat([qd, qd[:, :, :1]], 2)[:, :, :Hq]
    p, s, tb = _gpu(pool, scales, tables)
    out = torch.full((B, H, T), -3.0, device="cuda")
    wd = None if weights is None else torch.from_numpy(weights).cuda()
    got = sv.weigh_kv(qd, torch.from_numpy(lse).cuda(), p, s, tb, _i32(lens), window_lens=_i32(wins), scale=scale,
                      weights=wd, decay=decay, out=out)
    assert got is out
    got = got.double().cpu().numpy()
    want, spread = window.weigh(q, lse.astype(np.float64), pool, scales, tables, lens, np.full((B, H, T), -3.0), wins, scale,
                                weights, np.float32(decay))
    assert np.array_equal(np.isnan(got), np.isnan(want))
    n = W * Hq // H
    top = spread.max() if spread.size else 0
    rel = math.expm1(top * (D * 2.0 ** -23 + 6 * 2.0 ** -24) + 16 * 2.0 ** -24) + 2.0 ** -21 + (n / 64 + 64) * 2.0 ** -24
    fine = np.isfinite(want)
    err = np.abs(got - want)[fine]
    assert (err <= rel * np.abs(want[fine]) + 1e-37).all(), (err / np.maximum(np.abs(want[fine]), 1e-30)).max()
    return got, want


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("lens,W,Hq,H,D,tpb", [([0], 1, 1, 1, 64, 16), ([1, 16, 63], 1, 4, 2, 128, 16),
                                               ([100, 0, 257], 5, 8, 2, 64, 32), ([15, 400], 16, 10, 2, 128, 48),
                                               ([70], 60, 16, 2, 128, 64), ([0, 33], 130, 4, 1, 64, 16),
                                               ([300], 33, 40, 8, 128, 128), ([5], 300, 5, 5, 128, 1024),
                                               ([1000, 3], 64, 1, 1, 64, 80), ([130], 257, 12, 2, 128, 32),
                                               ([40, 700], 8, 8, 2, 64, 16), ([40, 700], 11, 6, 2, 128, 32),
                                               ([3000], 20, 8, 2, 64, 64), ([1000], 400, 8, 2, 64, 32)])
def test_weigh_matches_oracle(dtype, lens, W, Hq, H, D, tpb):
    rng = np.random.default_rng(W + D)
    lens = np.asarray(lens)
    wins = rng.integers(0, W + 1, len(lens))
    wins[0] = W
    q, lse, pool, scales, tables, wins = _weigh_case(rng, lens, W, Hq, H, D, tpb, dtype, wins)
    T = int((lens + wins).max()) + 7
    w = np.exp(rng.normal(0, 2, (len(lens), H, T))).astype(np.float32)
    _check_weigh(q, lse, pool, scales, tables, lens, wins, dtype, T, w, 0.75)
    _check_weigh(q, lse, pool, scales, tables, lens, wins, dtype, max(1, T // 2), strided=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 64)])
def test_shares_of_many_steps(dtype, D):
    """88 steps of 64 rows over 15 units a head: each CTA stages some 14 steps, four or five by each of its staging warps.
    Neighbouring steps' rows differ in size and direction, so a row of another step shows; and equal calls give
    equal bits.  The lse are no attention's: in fp16 some weights pass fp32's largest value (e^89; scores reach 150),
    and read inf."""
    rng = np.random.default_rng(15)
    H, G, W, tpb, s = 2, 4, 1400, 32, 2300
    pool, scales, tables = cache(rng, [s + W], H, D, tpb)
    q = rng.normal(0, 1, (1, W, H * G, D)) * np.where(np.arange(W) // 16 % 2, 1.0, 0.25)[None, :, None, None]
    q = to_bf16(q) if dtype == "bf16" else to_f16(q)
    lse = (5.0 + rng.normal(0, 1, (1, W, H * G))).astype(np.float32)
    p, sc, tb, ld = _gpu(pool, scales, tables, lse)
    qd = torch.from_numpy(q).to(TYPES[dtype]).cuda()
    one = sv.weigh_kv(qd, ld, p, sc, tb, _i32([s]))
    for _ in range(30):
        assert torch.equal(sv.weigh_kv(qd, ld, p, sc, tb, _i32([s])), one)
    want, spread = window.weigh(q, lse.astype(np.float64), pool, scales, tables, [s], np.zeros((1, H, s + W)))
    got = one.double().cpu().numpy()[:, :, :s + W]
    # the bound of the file's head
    rel = math.expm1(spread.max() * (D * 2.0 ** -23 + 6 * 2.0 ** -24) + 16 * 2.0 ** -24) + 2.0 ** -21 + (W * G / 64 + 64) * 2.0 ** -24
    top = float(np.finfo(np.float32).max)
    beyond = want > top
    assert not ((want > top * (1 - rel)) & (want < top * (1 + rel))).any()  # none that may be either
    assert np.isinf(got[beyond]).all()
    assert (np.abs(got - want)[~beyond] <= rel * want[~beyond]).all()


@pytest.mark.gpu
def test_an_empty_window_decays():
    rng = np.random.default_rng(1)
    q, lse, pool, scales, tables, wins = _weigh_case(rng, np.array([50, 70]), 3, 4, 2, 64, 16, "bf16", [0, 2])
    w = rng.random((2, 2, 80)).astype(np.float32)
    got, _ = _check_weigh(q, lse, pool, scales, tables, np.array([50, 70]), wins, "bf16", 80, w, 0.5)
    assert np.array_equal(got[0, :, :50], (0.5 * w[0, :, :50]).astype(np.float64)) and (got[0, :, 50:] == -3).all()


@pytest.mark.gpu
def test_large_scores_nan_and_rows_without_weight():
    rng = np.random.default_rng(2)
    lens = np.array([40, 40])
    q, lse, pool, scales, tables, wins = _weigh_case(rng, lens, 9, 4, 2, 64, 16, "bf16", amp=12.0)
    _check_weigh(q, lse, pool, scales, tables, lens, wins, "bf16", 60)
    lse[0, 3], lse[1, 2, 1] = -np.inf, np.nan
    pool[tables[0, 1], 0, 1, 4] = 127  # a key of NaN
    q[1, 8, 3, 5] = np.nan
    got, want = _check_weigh(q, lse, pool, scales, tables, lens, wins, "bf16", 60)
    assert np.isnan(got[0, 1, 20]) and np.isfinite(got[0, 1, :20]).all() and np.isnan(got[1, 0, :43]).all()


@pytest.mark.gpu
def test_bad_requests_and_blocks():
    rng = np.random.default_rng(3)
    lens = np.array([40, -1, 30, 500, 33])
    wins = np.array([3, 3, 5, 3, -1])
    B = len(lens)
    pool, scales, tables = cache(rng, [44] * B, 1, 64, 16)
    tables[0, 1], tables[2, 2] = len(pool), -2
    q = to_bf16(rng.normal(0, 1, (B, 4, 2, 64)))
    got, _ = _check_weigh(q, np.full((B, 4, 2), 4.0, np.float32), pool, scales, tables, lens, wins, "bf16", 64)
    assert np.isnan(got[0, 0, 16:32]).all() and np.isfinite(got[0, 0, :16]).all()
    assert (got[[1, 2, 3, 4]] == -3).all()  # window 5 of 4, lengths out of range


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,W,D", [("bf16", 4, 128), ("f16", 4, 64), ("bf16", 64, 64), ("f16", 64, 128), ("bf16", 400, 128),
                                       ("f16", 400, 64)])
def test_weights_of_exact_scores(dtype, W, D):
    """Rows and keys of whole numbers, as many bits as their types hold, whose scores are exact in fp32 in any order
    (below 2^24), less an lse that is a multiple of the same unit.  What is left to round: the product of y = score - lse
    with log2(e), 2^-24 |y|, and that constant, 2^-25 |y|; exp2, 2^-22; and the sums, one 2^-24 an addition on a
    weight's way (rows in a lane or a step of 64, then steps, shuffles and parts).  A bf16 row's first element is 2^28,
    where the keys are 0: the others are 2^-28 of it."""
    rng = np.random.default_rng(W + D)
    H, G, tpb, s = 2, 4, 16, 700
    bits = 8 if dtype == "bf16" else 11
    unit = 2.0 ** (-13 if dtype == "bf16" else -16)
    q = rng.integers(-2 ** bits + 1, 2 ** bits, (W, H, G, D)).astype(np.float64)
    n = s + W
    k = rng.integers(-15, 16, (n, H, D)).astype(np.float64)
    if dtype == "bf16":
        q[..., 0], k[..., 0] = 2.0 ** 28, 0
    S = np.einsum("ihgd,thd->ihgt", q, k) * unit
    S[np.broadcast_to((np.arange(n)[None] > s + np.arange(W)[:, None])[:, None, None], S.shape)] = -np.inf
    top = S.max(-1, keepdims=True)
    lse = np.round((top + np.log(np.exp(S - top).sum(-1, keepdims=True))) / unit) * unit
    y = S - lse
    p = np.exp(y)
    want = p.sum((0, 2))
    adds = 33 + W * G // 64 + 16
    bound = (p * (1.5 * 2.0 ** -24 * np.abs(np.where(p > 0, y, 0)) + 2.0 ** -22)).sum((0, 2)) + adds * 2.0 ** -24 * want
    cols = -(-n // tpb)
    tables = rng.permutation(cols).astype(np.int32)[None]
    pool = np.zeros((cols, 2, H, tpb, D), np.uint8)
    for t in range(n):
        pool[tables[0, t // tpb], 0, :, t % tpb] = kv.encode(k[t])
    pd, tb = _gpu(pool, tables)
    qd = torch.from_numpy(q.reshape(1, W, H * G, D)).to(TYPES[dtype]).cuda()
    assert np.array_equal(qd.double().cpu().numpy().reshape(q.shape), q)
    ld = torch.from_numpy(lse.astype(np.float32).reshape(1, W, H * G)).cuda()
    got = sv.weigh_kv(qd, ld, pd, torch.ones((cols, 2, H), device="cuda"), tb, _i32([s]), scale=unit)
    err = np.abs(got[0, :, :n].double().cpu().numpy() - want)
    assert (err <= bound + 1e-37).all(), (err / bound).max()


@pytest.mark.gpu
def test_weights_of_an_attention_sum_to_its_rows():
    rng = np.random.default_rng(4)
    for W, lens in ((3, [5000, 1, 700]), (700, [1300, 0, 5])):
        B, Hq, H, D, tpb = 3, 16, 4, 128, 32
        per = max(lens) + W
        cols = -(-per // tpb)
        pool = torch.zeros((B * cols, 2, H, tpb, D), dtype=torch.uint8, device="cuda")
        scales = torch.zeros((B * cols, 2, H), device="cuda")
        tables = _i32(rng.permutation(B * cols).reshape(B, cols))
        at = _i32([0] * B)
        x = torch.from_numpy(rng.normal(0, 1, (B, max(lens), H, D))).cuda().bfloat16()
        sv.store_kv(x, x, pool, scales, tables, at, window_lens=_i32(lens))
        q, k = (torch.from_numpy(rng.normal(0, 1, (B, W, h, D))).cuda().bfloat16() for h in (Hq, H))
        sv.store_kv(k, k, pool, scales, tables, _i32(lens))
        _, lse = sv.attend_kv(q, pool, scales, tables, _i32(lens), want_lse=True)
        out = sv.weigh_kv(q, lse, pool, scales, tables, _i32(lens))
        total = out.double().sum(-1)
        # each weight is exp of a rounded score less a rounded lse
        assert (total / (W * Hq / H) - 1).abs().max() < 1e-4
        again = sv.weigh_kv(q, lse, pool, scales, tables, _i32(lens), weights=out, decay=1.0, out=out.clone())
        w2 = out.clone()
        sv.weigh_kv(q, lse, pool, scales, tables, _i32(lens), weights=w2, out=w2)  # in place
        assert torch.equal(again, w2)


@pytest.mark.gpu
@pytest.mark.parametrize("W", [3, 90])
def test_weigh_beside_an_attention_on_another_stream_and_captured(W):
    rng = np.random.default_rng(12)
    lens = np.array([900, 30])
    q, lse, pool, scales, tables, wins = _weigh_case(rng, lens, W, 8, 2, 64, 16, "bf16")
    qd = torch.from_numpy(q).cuda().bfloat16()
    p, s, tb, ld = _gpu(pool, scales, tables, lse)
    seq = _i32(lens)
    one = sv.weigh_kv(qd, ld, p, s, tb, seq)
    att = sv.attend_kv(qd, p, s, tb, seq)[0]
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):  # both kinds take tensor memory
        w = sv.weigh_kv(qd, ld, p, s, tb, seq, stream=a)
        x = sv.attend_kv(qd, p, s, tb, seq, stream=b)[0]
    torch.cuda.synchronize()
    assert torch.equal(w, one) and torch.equal(x, att)
    # accumulated three times, eagerly and in two graphs of one call each
    def call(w):
        return sv.weigh_kv(qd, ld, p, s, tb, seq, weights=w, decay=0.5, out=w)
    want = torch.zeros_like(one)
    for _ in range(3):
        call(want)
    got = torch.zeros_like(one)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            call(got)
    got.zero_()
    for g in (graphs[0], graphs[1], graphs[0]):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.gpu
def test_weigh_in_a_pool_over_4_gb():
    H, D, tpb, N = 8, 128, 64, 36000  # 4.7 GB
    pool = torch.zeros((N, 2, H, tpb, D), dtype=torch.uint8, device="cuda")
    scales = torch.ones((N, 2, H), device="cuda")
    tables = _i32([[0, N - 1, N - 2]])
    pool[N - 2:, 0, :, :, 0] = 0x38  # 1.0
    q = torch.zeros((1, 1, H, D), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 2.0
    out = sv.weigh_kv(q, torch.zeros((1, 1, H), device="cuda"), pool, scales, tables, _i32([150]), scale=1.0)
    want = torch.exp(torch.where(torch.arange(151, device="cuda") < 64, 0.0, 2.0))
    assert (out[0, :, :151] / want - 1).abs().max() < 1e-6 and not out[0, :, 151:].any()


@pytest.mark.gpu
@pytest.mark.parametrize("W", [2, 50])
def test_weights_shifted_against_the_output_are_refused(W):
    rng = np.random.default_rng(16)
    pool, scales, tables = _gpu(*cache(rng, [30, 61], 2, 64, 16))
    q = torch.zeros((2, W, 4, 64), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((2, W, 4), device="cuda")
    buf = torch.zeros(2 * 2 * 64 + 4, device="cuda")
    with pytest.raises(sv.SpecError):
        sv.weigh_kv(q, lse, pool, scales, tables, _i32([20, 9]), weights=buf[:256].view(2, 2, 64), out=buf[4:].view(2, 2, 64))
    assert not buf.any()


# ------------------------------------------------------------------ GPU: eviction
def _check_evict(w, pool, scales, tables, lens, keep, first=0, recent=0, held=None, extra=0, inplace=False):
    B, H, T = w.shape
    p, s, tb, wd = _gpu(pool, scales, tables, w)
    seq = _i32(lens)
    hd = None if held is None else _i32(held)
    if inplace:
        ow, ol = wd, seq
        mark = w[:, :, :]
    else:
        mark = np.full((B, H, keep + extra), -3.0, np.float32)
        ow, ol = torch.from_numpy(mark).cuda(), None
    new, kept, out, free = sv.evict_kv(wd, p, s, tb, seq, keep, first=first, recent=recent, blocks_held=hd, out_lens=ol,
                                       out_weights=ow)
    r = window.evict(w, pool, scales, tables, lens, keep, first, recent, held, mark)
    assert new.cpu().numpy().tolist() == r[0].tolist()
    assert np.array_equal(kept.cpu().numpy(), r[1])
    assert np.array_equal(out.cpu().numpy(), r[2], equal_nan=True)
    if held is not None:
        assert free.cpu().numpy().tolist() == r[3].tolist()
    assert np.array_equal(s.cpu().numpy().astype(np.float64), r[5])
    got, want = p.cpu().numpy(), r[4]
    nan = (got & 127) == 127  # NaN codes may differ in sign
    assert np.array_equal(nan, (want & 127) == 127) and np.array_equal(got[~nan], want[~nan])
    return new, kept, out


@pytest.mark.gpu
@pytest.mark.parametrize("lens,H,D,tpb,keep,first,recent", [
    ([1], 1, 64, 16, 1, 0, 0), ([17, 5, 16], 2, 64, 16, 16, 0, 0), ([40, 100, 33], 2, 128, 16, 33, 4, 7),
    ([300, 299, 0], 1, 64, 32, 100, 100, 0), ([300], 3, 64, 48, 77, 0, 77), ([600, 70], 2, 64, 64, 64, 3, 61),
    ([1500, 1100], 2, 64, 1024, 1050, 4, 20), ([1300], 1, 128, 560, 1200, 0, 5), ([2100, 1024], 1, 64, 16, 1024, 1, 1),
    ([5000], 1, 64, 16, 2500, 4, 100), ([513] * 9, 1, 64, 128, 512, 0, 0), ([1000], 2, 128, 16, 1, 0, 0)])
def test_evict_matches_oracle(lens, H, D, tpb, keep, first, recent):
    rng = np.random.default_rng(keep)
    pool, scales, tables = cache(rng, lens, H, D, tpb)
    T = max(lens) + 3
    for kind in range(3):
        w = np.exp(rng.normal(0, 3, (len(lens), H, T))).astype(np.float32)
        if kind == 1:  # many equal, zeros of both signs, negative and not finite ones
            w = np.round(rng.normal(0, 1, w.shape)).astype(np.float32)
            w[rng.random(w.shape) < 0.05] = np.nan
            w[rng.random(w.shape) < 0.05] = np.inf
            w[rng.random(w.shape) < 0.05] = -np.inf
            w[rng.random(w.shape) < 0.1] = -0.0
        if kind == 2:
            w[:] = 0
        held = [-(-n // tpb) + 1 for n in lens]
        _check_evict(w, pool, scales, tables, lens, keep, first, recent, held, extra=kind)
    _check_evict(np.exp(rng.normal(0, 3, (len(lens), H, T))).astype(np.float32)[:, :, :max(T, keep)], pool, scales, tables,
                 lens, min(keep, T), min(first, T), min(recent, T - min(first, T)), inplace=True)


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,D,keep", [(20, 8, 64, 40), (39, 8, 128, 33), (77, 8, 64, 20), (77, 8, 128, 24)])
def test_evict_of_many_heads(B, H, D, keep):
    """More heads than SMs: other sizes of CTAs and of the moved slices."""
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 90, B)
    pool, scales, tables = cache(rng, lens, H, D, 16)
    w = np.exp(rng.normal(0, 2, (B, H, 90))).astype(np.float32)
    _check_evict(w, pool, scales, tables, lens, keep, 2, 5, -(-lens // 16))


@pytest.mark.gpu
@pytest.mark.parametrize("lens,H,keep", [([40001], 1, 15000), ([13001, 8300, 2500] + [60] * 17, 8, 3000)])
def test_weights_in_place_beyond_the_registers(lens, H, keep):
    """A CTA's registers hold 16384 weights of few heads and 8192 with more heads than SMs; what is behind is read as the
    kept weights are written below it.  Many weights are equal."""
    rng = np.random.default_rng(18)
    pool, scales, tables = cache(rng, lens, H, 64, 64)
    w = np.round(np.exp(rng.normal(0, 1, (len(lens), H, max(lens)))), 1).astype(np.float32)
    _check_evict(w, pool, scales, tables, lens, keep, 4, 500, [-(-n // 64) for n in lens], inplace=True)
    _check_evict(w, pool, scales, tables, lens, keep, 4, 500, extra=3)


@pytest.mark.gpu
def test_untouched_requests():
    rng = np.random.default_rng(7)
    lens = np.array([90, 90, -3, 90, 200, 90, 0, 95])
    pool, scales, tables = cache(rng, np.clip(lens, 0, 100), 2, 64, 16)
    tables[1, 3], tables[3, 0] = -1, len(pool)
    w = rng.random((8, 2, 92)).astype(np.float32)  # too few for the last
    new, kept, _ = _check_evict(w, pool, scales, tables, lens, 40, 2, 3, [9] * 8)
    assert new.tolist() == [40, 90, -3, 90, 200, 40, 0, 95]
    assert (kept[[1, 2, 3, 4, 6, 7]] == -1).all()


@pytest.mark.gpu
def test_scales_that_differ_widely():
    rng = np.random.default_rng(8)
    pool, scales, tables = cache(rng, [700, 650], 2, 64, 16, spread=4.0)
    scales[tables[0, 3]] = 0.0
    pool[tables[0, 3]] = 0
    w = rng.random((2, 2, 700)).astype(np.float32)
    _check_evict(w, pool, scales, tables, [700, 650], 250, 4, 30)


@pytest.mark.gpu
def test_long_requests_and_repeated_eviction():
    """200 000 positions of one head; and the same call twice on what it leaves."""
    rng = np.random.default_rng(9)
    n, keep, tpb = 200000, 70000, 16
    cols = -(-n // tpb)
    pool = torch.randint(0, 127, (cols, 2, 1, tpb, 64), dtype=torch.uint8, device="cuda")
    scales = torch.exp2(torch.randint(-3, 4, (cols, 2, 1), device="cuda").float())
    tables = _i32(rng.permutation(cols)[None])
    w = torch.from_numpy(rng.random((1, 1, n)).astype(np.float32)).cuda()
    val = pool[tables[0].long()].view(torch.float8_e4m3fn).float() * scales[tables[0].long()][..., None, None]
    val = val.transpose(0, 1).reshape(2, cols * tpb, 64)
    seq = _i32([n])
    new, kept, out, _ = sv.evict_kv(w, pool, scales, tables, seq, keep, first=100, recent=1000, out_lens=seq)
    at = kept[0, 0].long()
    assert new is seq and seq.item() == keep and (at[1:] > at[:-1]).all()
    assert torch.equal(out[0, 0], w[0, 0, at])
    middle = w[0, 0, 100:n - 1000]
    assert torch.equal(torch.sort(middle, descending=True).values[:keep - 1100].sort().values,
                       w[0, 0, at[100:keep - 1000]].sort().values)
    got = pool[tables[0].long()].view(torch.float8_e4m3fn).float() * scales[tables[0].long()][..., None, None]
    got = got.transpose(0, 1).reshape(2, cols * tpb, 64)[:, :keep]
    want = val[:, at]
    # codes whose scale grew (at most 2^6 times) are rounded again below the normal range: half of 2^-9 of the new scale
    top = scales[tables[0].long()][:-(-keep // tpb), :, 0].repeat_interleave(tpb, 0)[:keep].t()[..., None]
    assert ((got - want).abs() <= 2.0 ** -10 * top).all()
    before = pool.clone()
    lens2, kept2, _, _ = sv.evict_kv(out, pool, scales, tables, seq, keep, first=100, recent=1000)
    assert lens2.item() == keep and torch.equal(kept2[0, 0].long(), torch.arange(keep, device="cuda"))
    assert torch.equal(pool, before)


@pytest.mark.gpu
def test_kept_weights_shifted_against_the_weights_are_refused():
    rng = np.random.default_rng(17)
    pool, scales, tables = _gpu(*cache(rng, [30, 61], 2, 64, 16))
    old = pool.clone()
    buf = torch.zeros(2 * 2 * 64 + 4, device="cuda")
    with pytest.raises(sv.SpecError):
        sv.evict_kv(buf[4:].view(2, 2, 64), pool, scales, tables, _i32([30, 60]), 20, out_weights=buf[:256].view(2, 2, 64))
    assert torch.equal(pool, old) and not buf.any()


@pytest.mark.gpu
def test_captured_and_on_another_stream():
    rng = np.random.default_rng(10)
    lens, keep = [500, 300, 20], 100
    pool, scales, tables = cache(rng, lens, 2, 64, 16)
    w = [rng.random((3, 2, 500)).astype(np.float32) for _ in range(2)]
    p, s, tb, wd = _gpu(pool, scales, tables, w[0])
    seq = _i32(lens)
    outs = dict(out_lens=torch.empty_like(seq), out_kept=torch.empty((3, 2, keep), dtype=torch.int32, device="cuda"),
                out_weights=torch.zeros((3, 2, keep), device="cuda"))
    stream = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.evict_kv(wd, p, s, tb, seq, keep, recent=9, **outs)
    for x in w:
        r = window.evict(x, pool, scales, tables, lens, keep, 0, 9)
        for t, a in ((p, pool), (s, scales), (wd, x)):
            t.copy_(torch.from_numpy(a))
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(outs["out_kept"].cpu().numpy(), r[1]) and np.array_equal(s.cpu().numpy(), r[5])
        for t, a in ((p, pool), (s, scales)):
            t.copy_(torch.from_numpy(a))
        torch.cuda.synchronize()
        kept = sv.evict_kv(wd, p, s, tb, seq, keep, recent=9, stream=stream)[1]
        stream.synchronize()
        assert np.array_equal(kept.cpu().numpy(), r[1]) and np.array_equal(s.cpu().numpy(), r[5])


@pytest.mark.gpu
def test_binding_refusals():
    rng = np.random.default_rng(11)
    pool, scales, tables = _gpu(*cache(rng, [30, 61], 2, 64, 16))
    seq = _i32([30, 58])
    w = torch.zeros((2, 2, 64), device="cuda")
    q = torch.zeros((2, 3, 4, 64), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((2, 3, 4), device="cuda")

    def weigh(q=q, lse=lse, **kw):
        return sv.weigh_kv(q, lse, pool, scales, tables, seq, **kw)
    for bad in (dict(q=q.float()), dict(q=q[:, :, :3]), dict(q=q[:1]), dict(lse=lse[:, :2]), dict(lse=lse.double()),
                dict(weights=w[:, :1]), dict(weights=w.double()), dict(weights=w, out=w[:, :, :9]), dict(out=lse),
                dict(out=w.cpu()), dict(window_lens=seq.long())):
        with pytest.raises(ValueError):
            weigh(**bad)
    for bad in (dict(decay=math.nan), dict(scale=math.inf)):
        with pytest.raises(sv.SpecError):
            weigh(**bad)

    def evict(w=w, keep=20, **kw):
        return sv.evict_kv(w, pool, scales, tables, seq, keep, **kw)
    held = _i32([2, 4])
    for bad in (dict(keep=0), dict(first=15, recent=6), dict(first=-1), dict(recent=-1), dict(w=w[:, :1]), dict(w=w.half()),
                dict(out_weights=w[:, :, :19].contiguous()), dict(out_kept=torch.zeros((2, 2, 19), dtype=torch.int32, device="cuda")),
                dict(out_lens=seq.long()), dict(out_free=held), dict(blocks_held=held, out_free=held),
                dict(blocks_held=seq, out_lens=seq), dict(out_weights=scales),
                dict(out_lens=held, blocks_held=held)):
        with pytest.raises(ValueError):
            evict(**bad)
