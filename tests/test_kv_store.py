"""The quantising store and the relocation of accepted rows in the paged
8-bit cache: oracle pins on the CPU, the CUDA calls against the oracle on the
GPU.  Both define their roundings completely, so codes and scales are compared
for equality."""
import ctypes

import numpy as np
import pytest
import torch

import speculative_decoding_verification_row_gb300 as sv
from oracle import kv
from _kv import cache, random_paths, to_bf16, to_f16


# ------------------------------------------------------------------ oracle pins (CPU)
def test_e4m3_table_and_rounding_match_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(kv.decode(codes.numpy()), want, equal_nan=True)
    x = np.concatenate([np.random.default_rng(0).normal(0, 1, 20000) * 10.0 ** np.linspace(-4, 2, 20000),
                        want[np.isfinite(want)], (want[:126] + want[1:127]) / 2])  # values and every tie
    x = x[np.abs(x) <= 448].astype(np.float32)
    got = kv.encode(x.astype(np.float64))
    assert np.array_equal(got, torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert kv.encode([np.inf, -np.inf, np.nan]).tolist() == [127] * 3


@pytest.mark.parametrize("amax,want", [(0.0, 0.0), (448.0, 1.0), (np.nextafter(448.0, 449), 2.0), (224.0, 0.5),
                                       (1.0, 2.0 ** -8), (1e-45, 2.0 ** -126), (3e38, 2.0 ** 120)])
def test_scale_rule(amax, want):
    assert kv.scale_for(amax) == want


def test_store_grows_a_live_block_and_restarts_a_dead_one():
    H, D, tpb = 1, 64, 16
    pool = np.zeros((2, 2, H, tpb, D), np.uint8)
    scales = np.zeros((2, 2, H), np.float32)
    tables = np.array([[0, 1]], np.int32)
    one = np.ones((1, 3, H, D))
    pool, scales = kv.store(one, one, pool, scales, tables, [0])
    assert (scales[0] == 2.0 ** -8).all()
    pool, scales = kv.store(4 * one, 4 * one, pool, scales, tables, [3])  # rows 3..5, four times larger
    assert (scales[0] == 2.0 ** -6).all()
    x = kv.decode(pool[0, 0, 0, :6, 0]) * scales[0, 0, 0]
    assert x.tolist() == [1, 1, 1, 4, 4, 4]
    pool, scales = kv.store(one, one, pool, scales, tables, [0])  # from the first row: the old scale is gone
    assert (scales[0] == 2.0 ** -8).all()


def test_relocate_hand_example():
    # rows 0..5 hold 1, 2, 4, ... in blocks of 2 rows; base 1, nodes 0, 2, 4
    H, D, tpb = 1, 64, 2
    pool = np.zeros((4, 2, H, tpb, D), np.uint8)
    scales = np.ones((4, 2, H), np.float32)
    scales[2] = 4.0
    tables = np.array([[3, 0, 2, 1]], np.int32)
    for t in range(6):
        blk = tables[0, t // 2]
        pool[blk, :, :, t % 2] = kv.encode(2.0 ** t / scales[blk, 0, 0])
    p, s = kv.relocate(pool, scales, tables, [1], [[0, 2, 4]], [2])
    get = lambda t: kv.decode(p[tables[0, t // 2], 0, 0, t % 2, 0]) * s[tables[0, t // 2], 0, 0]  # noqa: E731
    assert [get(t) for t in range(4)] == [1, 2, 8, 32]  # logical 2 <- 3, 3 <- 5
    assert s[0, 0, 0] == 4.0 and s[3, 0, 0] == 1.0
    same, _ = kv.relocate(pool, scales, tables, [1], [[0, 2, 1]], [2])
    assert np.array_equal(same, pool)


def _fake_cache(**o):
    f = 16 * 1024
    a = dict(size=ctypes.sizeof(sv.KvCache), pool=f, scales=f, block_tables=f, num_blocks=4, max_blocks=2,
             tokens_per_block=16, kv_heads=2, head_dim=64)
    a.update(o)
    return sv.KvCache(*[a[n] for n, _ in sv.KvCache._fields_])


BAD_CACHES = [dict(size=8), dict(pool=None), dict(pool=16 * 1024 + 8), dict(scales=None), dict(block_tables=None),
              dict(num_blocks=0), dict(max_blocks=0), dict(tokens_per_block=8), dict(tokens_per_block=24),
              dict(tokens_per_block=1040), dict(kv_heads=0), dict(kv_heads=1025), dict(head_dim=96)]


def test_refusals_before_any_launch():
    lib, f = sv.lib(), ctypes.c_void_p(16 * 1024)
    s3 = (ctypes.c_int64 * 3)(128, 128, 64)

    def store(cache, k=f, v=f, ks=s3, vs=s3, dt=1, seq=f, B=2, W=3):
        return lib.spec_store_kv(ctypes.byref(cache), k, ks, v, vs, dt, seq, None, B, W, None)

    def move(cache, base=f, nodes=f, n=f, B=2, L=4):
        return lib.spec_relocate_quantised_kv(ctypes.byref(cache), base, nodes, n, B, L, None)
    for bad in BAD_CACHES:
        assert store(_fake_cache(**bad)) == sv.SPEC_EINVAL, bad
        assert move(_fake_cache(**bad)) == sv.SPEC_EINVAL, bad
    odd = (ctypes.c_int64 * 3)(128, 132, 64)
    for bad in (dict(k=None), dict(v=ctypes.c_void_p(16 * 1024 + 4)), dict(ks=odd), dict(vs=odd), dict(dt=0), dict(dt=3),
                dict(seq=None), dict(B=0), dict(B=8193), dict(W=0), dict(W=65537)):
        assert store(_fake_cache(), **bad) == sv.SPEC_EINVAL, bad
    for bad in (dict(base=None), dict(nodes=None), dict(n=None), dict(B=0), dict(L=0), dict(L=65)):
        assert move(_fake_cache(), **bad) == sv.SPEC_EINVAL, bad


def test_param_structs_match_the_header(tmp_path):
    import os
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "spec_verify.h"', "int main(void) {"]
    want = []
    for cname, py in (("spec_kv_cache", sv.KvCache), ("spec_attend_params", sv.AttendParams)):
        lines.append(f'  printf("%zu\\n", sizeof({cname}));')
        want.append(ctypes.sizeof(py))
        for name, _ in py._fields_:
            lines.append(f'  printf("%zu\\n", offsetof({cname}, {name}));')
            want.append(getattr(py, name).offset)
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["  return 0;", "}"]))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", inc, str(src), "-o", str(exe)], check=True)
    assert [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()] == want


# ------------------------------------------------------------------ GPU parity
def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def same_cache(pool, scales, want_pool, want_scales, touched=None):
    got = pool.view(torch.uint8).cpu().numpy()
    # the sign of a NaN is not part of its value
    nan = (got & 127) == 127
    assert np.array_equal(nan, (want_pool & 127) == 127)
    assert np.array_equal(np.where(nan, 0, got), np.where(nan, 0, want_pool))
    assert np.array_equal(scales.cpu().numpy().astype(np.float64), want_scales)


@pytest.mark.gpu
@pytest.mark.parametrize("B,W,H,D,tpb,hi,dt", [(1, 1, 1, 64, 16, 0, "bf16"), (5, 1, 2, 128, 16, 50, "f16"),
                                               (7, 8, 3, 128, 32, 100, "bf16"), (4, 61, 2, 64, 16, 33, "f16"),
                                               (3, 200, 1, 128, 128, 90, "bf16"), (2, 700, 2, 128, 256, 3, "f16"),
                                               (3, 50, 2, 64, 48, 95, "bf16")])
def test_store_matches_the_oracle(B, W, H, D, tpb, hi, dt):
    rng = np.random.default_rng(B * 1000 + W)
    seq = rng.integers(0, hi + 1, B)
    if B > 1:
        seq[1] = seq[1] // tpb * tpb  # a window that starts a block
    win = rng.integers(0, W + 1, B)
    win[0] = W
    pool, scales, tables = cache(rng, seq + W, H, D, tpb)
    # rows like a projection's: strided slices, per-token spread of 2^-20 .. 2^12, zeros, not finite
    x = rng.normal(0, 1, (B, W, 3 * H + 1, D)) * 2.0 ** rng.integers(-20, 13, (B, W, 1, 1))
    x = (to_bf16 if dt == "bf16" else to_f16)(x)
    x[rng.random(x.shape[:3]) < 0.1] = 0
    x[0, 0, H, :3] = [np.inf, -np.inf, np.nan]
    if B > 4:
        tables[2, seq[2] // tpb] = -1   # an unmapped window: nothing is stored
        win[3] = W + 1
        seq[4] = -1
    t = dev(x).to(torch.bfloat16 if dt == "bf16" else torch.float16)
    k, v = t[:, :, H:2 * H], t[:, :, 2 * H:3 * H]
    want = kv.store(x[:, :, H:2 * H], x[:, :, 2 * H:3 * H], pool, scales, tables, seq, win)
    dp, ds = dev(pool), dev(scales)
    for _ in range(1 if B > 2 else 2):  # storing the same window again changes nothing more
        sv.store_kv(k, v, dp, ds, dev(tables), dev(seq.astype(np.int32)), window_lens=dev(win.astype(np.int32)))
        same_cache(dp, ds, *want)


@pytest.mark.gpu
@pytest.mark.parametrize("B,W,H,D,tpb", [(3300, 2, 5, 64, 16), (2500, 17, 3, 128, 16)])
def test_store_of_many_requests(B, W, H, D, tpb):
    # so many blocks that one CTA takes all heads of a block, the last round of them not full
    rng = np.random.default_rng(B)
    seq = rng.integers(0, 20, B)
    win = rng.integers(0, W + 1, B)
    pool, scales, tables = cache(rng, seq + W, H, D, tpb, extra_cols=0)
    x = to_bf16(rng.normal(0, 1, (B, W, 2 * H, D)) * 2.0 ** rng.integers(-9, 10, (B, W, 1, 1)))
    tables[7, seq[7] // tpb] = -1
    win[7], win[8], seq[9] = W, W + 1, -1
    t = dev(x).to(torch.bfloat16)
    dp, ds = dev(pool), dev(scales)
    sv.store_kv(t[:, :, :H], t[:, :, H:], dp, ds, dev(tables), dev(seq.astype(np.int32)),
                window_lens=dev(win.astype(np.int32)))
    same_cache(dp, ds, *kv.store(x[:, :, :H], x[:, :, H:], pool, scales, tables, seq, win))


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -140, 2.0 ** 125])
def test_store_of_extreme_rows(scale):
    # all zero, below the least scale, at the top of the type's range
    rng = np.random.default_rng(1)
    pool, scales, tables = cache(rng, np.array([20]), 1, 64, 16)
    x = to_bf16(rng.uniform(-1, 1, (1, 4, 1, 64)) * scale)
    t = dev(x).to(torch.bfloat16)
    x = t.double().cpu().numpy()
    for s in (16, 10):  # a fresh block, and one with live rows
        dp, ds = dev(pool), dev(scales)
        sv.store_kv(t, t, dp, ds, dev(tables), dev(np.array([s], np.int32)))
        same_cache(dp, ds, *kv.store(x, x, pool, scales, tables, [s]))


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,L,H,D,tpb", [(16, 60, 4, 8, 128, 16), (9, 128, 64, 2, 64, 16), (6, 40, 17, 3, 128, 32),
                                           (3, 70, 40, 1, 64, 48)])
def test_relocate_matches_the_oracle(B, N, L, H, D, tpb):
    rng = np.random.default_rng(N * 10 + L)
    base = rng.integers(0, 70, B)
    base[0] = tpb - 1  # the first row moved to starts a block
    pool, scales, tables = cache(rng, base + N, H, D, tpb, spread=4.0)
    nodes = np.full((B, L), -1, np.int32)
    nodes[:, 0] = 0
    n = rng.integers(1, L, B)
    for b in range(B):
        nodes[b, 1:1 + n[b]] = np.sort(rng.choice(np.arange(1, N), n[b], replace=False))
    n[1] = 0
    if B > 5:
        n[2] = -1
        nodes[3, 1] = 0                                  # not increasing
        tables[4, (base[4] + 1) // tpb] = -1             # unmapped
        nodes[5, 1:1 + n[5]] = np.arange(1, 1 + n[5])    # already in place
    want = kv.relocate(pool, scales, tables, base, nodes, n)
    dp, ds = dev(pool), dev(scales)
    sv.relocate_quantised_kv(dp.view(torch.float8_e4m3fn), ds, dev(tables), dev(base.astype(np.int32)), dev(nodes),
                             dev(n.astype(np.int32)))
    same_cache(dp, ds, *want)
    assert not np.array_equal(want[0], pool)


@pytest.mark.gpu
def test_relocate_moves_the_values_of_the_unscaled_call():
    # with one scale everywhere the codes move as relocate_accepted_kv moves rows
    rng = np.random.default_rng(3)
    B, N, L, H, D, tpb = 4, 30, 6, 2, 64, 16
    base = rng.integers(0, 40, B).astype(np.int32)
    pool, scales, tables = cache(rng, base + N, H, D, tpb)
    scales[:] = 0.5
    paths = np.stack([random_paths(rng, N, 1, L)[0] for _ in range(B)])
    n = ((paths >= 0).sum(1) - 1).astype(np.int32)
    rows = dev(pool.transpose(0, 3, 1, 2, 4).reshape(-1, 2 * H * D))  # token-major rows
    sv.relocate_accepted_kv(rows, dev(tables), dev(base), dev(paths), dev(n), tpb)
    dp, ds = dev(pool), dev(scales)
    sv.relocate_quantised_kv(dp, ds, dev(tables), dev(base), dev(paths), dev(n))
    got = dp.cpu().numpy().transpose(0, 3, 1, 2, 4).reshape(-1, 2 * H * D)
    assert np.array_equal(got, rows.cpu().numpy())
    assert (ds == 0.5).all()
