"""Rotary positions of a window's queries and keys, alone and on the way into
the cache: oracle pins and refusals on the CPU, the CUDA calls against the
oracle on the GPU.

Tolerance of a rotated element gain (a cos - b sin): the angle is off by at
most 2^-30 turns from its reduction, 2^-32 from cutting it to 32 bits and
2^-25 half turns from its rounding to fp32, 2^-23 radians in all; sine and
cosine are rounded by CUDA's sincospif to 2 ulp, 2^-23; the gain and three
operations round by 2^-24 each.  In all at most 2^-21 gain (|a| + |b|), and
then the type's rounding, eps / 2 of the value."""
import ctypes
import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_row_gb300 as sv
from oracle import kv, window
from _kv import cache, random_paths, to_bf16, to_f16

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ CPU
def test_oracle_turns_exactly_far_out():
    for p, f in ((1, 1.0), (7, 0.3), (-5, 0.11), (12345, 1e-3)):
        assert window._turn(p, f) == pytest.approx((math.sin(p * f), math.cos(p * f)), abs=1e-14)
    # 2^30 radians: 170891318 turns and 5.92...; and additivity, which a lost product would break
    s, c = window._turn(2**30, 1.0)
    s1, c1 = window._turn(2**30 - 3, 1.0)
    assert math.isclose(s, s1 * math.cos(3) + c1 * math.sin(3), abs_tol=1e-15)
    assert math.isclose(c, c1 * math.cos(3) - s1 * math.sin(3), abs_tol=1e-15)


@pytest.mark.parametrize("inter", [False, True])
def test_oracle_keeps_lengths_and_differences(inter):
    rng = np.random.default_rng(0)
    q, k = rng.normal(0, 1, (2, 1, 4, 1, 32))
    f, _ = sv.rotary_frequencies(16)
    f = f.numpy()

    def dot(a, b):
        x = window.rotate(np.repeat(q[:1, :1], 1, 1)[:, :1], np.zeros((1, 1, 1, 32)), [a], f, inter)
        y = window.rotate(k[:1, :1], np.zeros((1, 1, 1, 32)), [b], f, inter)
        return float((x * y).sum())
    assert dot(5, 2) == pytest.approx(dot(1005, 1002), abs=1e-12)  # only the distance counts
    x = window.rotate(q, np.zeros_like(q), [9], f, inter, gain=1.5)
    assert np.allclose((x[..., :16] ** 2).sum(-1), 2.25 * (q[..., :16] ** 2).sum(-1))
    assert np.array_equal(x[..., 16:], q[..., 16:])


def test_frequencies():
    f, gain = sv.rotary_frequencies(8, 10000.0)
    assert f.dtype == torch.float64 and gain == 1.0
    assert f.tolist() == pytest.approx([1, 0.1, 0.01, 0.001])
    assert sv.rotary_frequencies(8, scaling="linear", factor=4)[0].tolist() == pytest.approx([x / 4 for x in f.tolist()])
    b = sv.rotary_frequencies(8, scaling="base", factor=4)[0]
    assert b[0] == 1 and b[-1].item() == pytest.approx(0.001 / 4)
    for name, g in (("ramp", 0.1 * math.log(8) + 1), ("smooth", 1.0)):
        r, gain = sv.rotary_frequencies(64, scaling=name, factor=8, original_len=4096)
        f = sv.rotary_frequencies(64)[0]
        turns = 4096 * f / (2 * math.pi)
        assert gain == pytest.approx(g)
        assert torch.equal(r[turns >= 32], f[turns >= 32])
        assert torch.allclose(r[turns <= 1], f[turns <= 1] / 8, rtol=1e-15)
        assert ((r <= f) & (r >= f / 8 * (1 - 1e-15))).all()
    assert sv.rotary_frequencies(8, scaling="linear", factor=1)[0].tolist() == sv.rotary_frequencies(8)[0].tolist()
    for bad in (dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=8, base=0.0), dict(rot_dim=8, factor=0.5),
                dict(rot_dim=8, scaling="dynamic"), dict(rot_dim=8, scaling="ramp"),
                dict(rot_dim=8, scaling="smooth", original_len=100, fast=1.0, slow=1.0),
                dict(rot_dim=2, scaling="base", factor=2.0)):
        with pytest.raises(ValueError):
            sv.rotary_frequencies(**bad)


def _fake(**o):
    f = 16 * 1024
    s = (ctypes.c_int64 * 3)(256, 128, 64)
    a = dict(size=ctypes.sizeof(sv.RotateParams), q=f, k=f, out_q=f, out_k=f, q_strides=s, k_strides=s, out_q_strides=s,
             out_k_strides=s, dtype=sv.SPEC_BF16, B=2, W=3, q_heads=4, k_heads=2, head_dim=64, starts=f, window_lens=None,
             masks=None, inv_freq=f, pairs=32, interleaved=0, gain=1.0)
    a.update(o)
    return sv.RotateParams(*[a[n] for n, _ in sv.RotateParams._fields_])


_ODD = (ctypes.c_int64 * 3)(256, 132, 64)
_OTHER = (ctypes.c_int64 * 3)(512, 128, 64)
BAD = [dict(size=8), dict(dtype=sv.SPEC_F32), dict(dtype=9), dict(B=0), dict(B=8193), dict(W=0), dict(W=65537),
       dict(head_dim=24), dict(head_dim=528), dict(head_dim=0), dict(pairs=0), dict(pairs=12), dict(pairs=40),
       dict(starts=None), dict(inv_freq=None), dict(gain=math.inf), dict(gain=math.nan), dict(masks=16 * 1024, W=1025),
       dict(q=None), dict(q_heads=0), dict(k_heads=-1), dict(q_heads=16385), dict(q=16 * 1024 + 8), dict(q_strides=_ODD),
       dict(out_q=16 * 1024 + 2), dict(out_q_strides=_ODD), dict(out_q_strides=_OTHER)]


@pytest.mark.parametrize("bad", BAD, ids=lambda b: ",".join(b))
def test_refusals_before_any_launch(bad):
    lib = sv.lib()
    assert lib.spec_rotate_qk(_fake(**bad), None) == sv.SPEC_EINVAL
    from test_kv_store import _fake_cache
    s3 = (ctypes.c_int64 * 3)(128, 128, 64)
    f = 16 * 1024
    if "out_q_strides" not in bad:
        assert lib.spec_rotate_store_kv(_fake_cache(), _fake(out_k=None, **bad), f, s3, f, f, 1 << 30, None) == sv.SPEC_EINVAL


def test_refusals_of_each_call():
    from test_kv_store import BAD_CACHES, _fake_cache
    lib, f = sv.lib(), 16 * 1024
    s3, odd = (ctypes.c_int64 * 3)(128, 128, 64), (ctypes.c_int64 * 3)(128, 132, 64)
    assert lib.spec_rotate_qk(None, None) == sv.SPEC_EINVAL
    for bad in (dict(out_q=None), dict(out_k=None), dict(q=None, q_heads=0, k=None, k_heads=0, out_q=None, out_k=None),
                dict(q=None, q_heads=0)):
        assert lib.spec_rotate_qk(_fake(**bad), None) == sv.SPEC_EINVAL, bad

    def store(c=None, p=None, v=f, vs=s3, seq=f, scratch=f, size=1 << 30):
        return lib.spec_rotate_store_kv(c or _fake_cache(), p or _fake(out_k=None), v, vs, seq, scratch, size, None)
    for W in (3, 40):
        need = lib.spec_rotate_store_scratch_size(2, W, 2, 64, 16)
        for bad in (dict(scratch=None), dict(scratch=f + 64), dict(size=need - 1)):
            assert store(p=_fake(out_k=None, W=W), **bad) == sv.SPEC_EWORKSPACE
    for bad in ((0, 1, 1, 64, 16), (8193, 1, 1, 64, 16), (1, 0, 1, 64, 16), (1, 65537, 1, 64, 16), (1, 1, 0, 64, 16),
                (1, 1, 1025, 64, 16), (1, 1, 1, 96, 16), (1, 1, 1, 64, 8), (1, 1, 1, 64, 1040), (1, 1, 1, 64, 24)):
        assert lib.spec_rotate_store_scratch_size(*bad) == 0
    for bad in BAD_CACHES:
        assert store(c=_fake_cache(**bad)) == sv.SPEC_EINVAL, bad
    for bad in (dict(), dict(out_k=None, k_heads=3), dict(out_k=None, head_dim=128), dict(out_k=None, out_q=None),
                dict(out_k=None, k=None, k_heads=0)):
        assert store(p=_fake(**bad)) == sv.SPEC_EINVAL, bad
    assert store(v=None) == store(vs=odd) == store(v=f + 4) == store(seq=None) == sv.SPEC_EINVAL
    assert lib.spec_rotate_store_kv(None, _fake(out_k=None), f, s3, f, f, 1 << 30, None) == sv.SPEC_EINVAL


@pytest.mark.skipif(torch.cuda.is_available(), reason="a call that is not refused would read the addresses made up here")
def test_the_stride_of_an_axis_of_one_element_does_not_count():
    f = 1 << 20
    other = (ctypes.c_int64 * 3)(512, 128, 64)
    one = dict(q=f, out_q=f, k=None, k_heads=0, out_k=None, starts=2 * f, inv_freq=3 * f, out_q_strides=other, W=2, q_heads=2)
    assert sv.lib().spec_rotate_qk(_fake(**one, B=1), None) == sv.SPEC_ECUDA  # not refused: there is no GPU
    assert sv.lib().spec_rotate_qk(_fake(**one, B=2), None) == sv.SPEC_EINVAL


_NO_GPU = pytest.mark.skipif(torch.cuda.is_available(),
                             reason="a call that is not refused would read the addresses made up here")


def _s3(*s):
    return (ctypes.c_int64 * 3)(*s)


def _placed(**o):
    """Arguments that lie apart: B 2, W 3, q of 4 heads and k of 2, slices of one row of 8 heads per token."""
    f, row = 1 << 20, 8 * 64
    s = _s3(3 * row, row, 64)
    a = dict(q=f, k=f + 4 * 128, out_q=2 * f, out_k=2 * f + 4 * 128, q_strides=s, k_strides=s, out_q_strides=s, out_k_strides=s,
             starts=3 * f, inv_freq=4 * f)
    a.update(o)
    return _fake(**a)


_F, _ROW = 1 << 20, 8 * 64 * 2  # bytes of a token's row
OVERLAPS = [dict(out_q=_F + 128), dict(out_q=_F + 16), dict(out_q=_F - _ROW), dict(out_k=_F), dict(out_k=2 * _F + 3 * 128),
            dict(out_k=2 * _F + 3 * 128 + _ROW, out_k_strides=_s3(_ROW // 2, 3 * _ROW // 2, 64)),
            dict(out_q_strides=_s3(3 * 512, 248, 64)), dict(out_q_strides=_s3(3 * 512, 512, 56)), dict(out_q_strides=_s3(0, 512, 64)),
            dict(out_q_strides=_s3(1024, 512, 64)), dict(q=2 * _F, out_q=2 * _F, q_strides=_s3(0, 512, 64), out_q_strides=_s3(0, 512, 64)),
            dict(starts=2 * _F + 4 * 128 + 60), dict(inv_freq=2 * _F + 5 * _ROW), dict(out_q_strides=_s3(-3 * 512, 512, 64), k=2 * _F - 3 * _ROW)]
APART = [dict(), dict(out_q=_F, out_k=_F + 4 * 128), dict(out_q=_F + 6 * 3 * _ROW), dict(q=2 * _F + 6 * 128, k=_F, q_heads=2),
         dict(starts=2 * _F + 6 * 128), dict(out_k=2 * _F + 5 * 128 + _ROW, out_k_strides=_s3(_ROW // 2, 3 * _ROW // 2, 64)),
         dict(out_q_strides=_s3(-3 * 512, 512, 64)), dict(k=_F), dict(q_strides=_s3(0, 0, 0)),
         dict(inv_freq=2 * _F + 6 * _ROW), dict(out_q_strides=_s3(64, 512, 128), out_q=2 * _F, k=None, k_heads=0, out_k=None)]


@_NO_GPU
def test_arrays_that_overlap_are_refused():
    from test_kv_store import _fake_cache
    lib, f = sv.lib(), _F
    for o in APART:  # not refused: there is no GPU
        assert lib.spec_rotate_qk(_placed(**o), None) == sv.SPEC_ECUDA, o
    for o in OVERLAPS:
        assert lib.spec_rotate_qk(_placed(**o), None) == sv.SPEC_EINVAL, o

    def store(v=6 * f, seq=7 * f, scratch=8 * f, cache=(), **o):
        c = _fake_cache(**{**dict(pool=9 * f, scales=10 * f, block_tables=11 * f), **dict(cache)})
        return lib.spec_rotate_store_kv(c, _placed(out_k=None, **o), v, _s3(3 * 512, 512, 64), seq, scratch, 1 << 20, None)
    assert store() == store(out_q=_F) == store(v=_F + 4 * 128) == store(starts=7 * f) == sv.SPEC_ECUDA
    for o in (dict(out_q=6 * f - _ROW), dict(out_q=_F + 128), dict(seq=2 * f), dict(scratch=2 * f), dict(scratch=_F + 4 * 128, W=40),
              dict(v=9 * f + 4096), dict(cache=dict(scales=9 * f + 4)), dict(cache=dict(block_tables=9 * f)),
              dict(out_q=9 * f), dict(scratch=10 * f), dict(seq=10 * f + 28), dict(out_q_strides=_s3(3 * 512, 8, 64))):
        assert store(**o) == sv.SPEC_EINVAL, o


def test_meeting_of_strided_arrays_by_enumeration(tmp_path):
    """csrc/apart.cuh against the sets of bytes, for small arrays of any strides."""
    import os
    import shutil
    import subprocess
    if shutil.which("g++") is None:
        pytest.skip("no C++ compiler")
    csrc = os.path.join(os.path.dirname(os.path.abspath(sv.__file__)), "csrc")
    src = tmp_path / "meet.cpp"
    src.write_text(f"""#include <cstdio>
#include "{csrc}/apart.cuh"
int main() {{
  long p[2], st[2][3], n[2][3], run[2];
  while (true) {{
    sv::Span s[2];
    for (int k = 0; k < 2; ++k) {{
      if (scanf("%ld %ld %ld %ld %ld %ld %ld %ld", &p[k], &st[k][0], &st[k][1], &st[k][2], &n[k][0], &n[k][1], &n[k][2], &run[k]) != 8) return 0;
      const int64_t x[3] = {{st[k][0], st[k][1], st[k][2]}};
      s[k] = sv::strided((const void*)p[k], x, n[k][0], n[k][1], n[k][2], run[k], 2);
    }}
    printf("%d %d\\n", sv::meet(s[0], s[1]), sv::folds(s[0]));
  }}
}}
""")
    exe = tmp_path / "meet"
    subprocess.run(["g++", "-std=c++17", "-x", "c++", str(src), "-o", str(exe)], check=True)
    rng = np.random.default_rng(0)
    lines, want = [], []
    for _ in range(3000):
        sets = []
        for _ in range(2):
            n, run = rng.integers(1, 5, 3), int(rng.integers(1, 6))
            st = rng.integers(-3, 4, 3) * rng.choice([1, 3, 7, 20], 3)
            p = int(rng.integers(1000, 1150))
            lines.append(" ".join(str(x) for x in (p, *st, *n, run)))
            at = [p + 2 * int(i * st[0] + j * st[1] + k * st[2]) + e for i in range(n[0]) for j in range(n[1]) for k in range(n[2])
                  for e in range(2 * run)]
            sets.append(at)
        want.append((int(bool(set(sets[0]) & set(sets[1]))), int(len(set(sets[0])) != len(sets[0]))))
    out = subprocess.run([str(exe)], input="\n".join(lines), capture_output=True, text=True, check=True).stdout.split()
    got = list(zip(map(int, out[0::2]), map(int, out[1::2])))
    assert got == want and 300 < sum(w[0] for w in want) < 2700 and 300 < sum(w[1] for w in want) < 2700


# ------------------------------------------------------------------ GPU
def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _qkv(rng, B, W, Hq, H, D, dtype, pad=0):
    """Slices of one row per token, as a fused projection leaves them."""
    x = torch.from_numpy(rng.normal(0, 1, (B, W, Hq + 2 * H, D + pad))).to(TYPES[dtype]).cuda()[..., :D]
    return x[:, :, :Hq], x[:, :, Hq:Hq + H], x[:, :, Hq + H:]


def _close(got, x, want, rot, gain, inter, dtype):
    x = np.abs(x)
    half = rot // 2
    bound = np.zeros_like(x)
    if inter:
        s = x[..., 0:rot:2] + x[..., 1:rot:2]
        bound[..., 0:rot:2] = bound[..., 1:rot:2] = s
    else:
        s = x[..., :half] + x[..., half:rot]
        bound[..., :half] = bound[..., half:rot] = s
    eps = torch.finfo(TYPES[dtype])
    tol = 2.0 ** -21 * abs(gain) * bound + np.maximum(eps.eps / 2 * np.abs(want), eps.smallest_normal * eps.eps)
    err = np.abs(got - want)
    assert (err <= tol).all(), (err - tol).max()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("B,W,Hq,H,D,rot,inter", [(1, 1, 1, 1, 16, 16, False), (2, 3, 8, 2, 64, 64, False),
                                                  (2, 3, 8, 2, 64, 64, True), (3, 5, 5, 1, 128, 32, False),
                                                  (3, 5, 5, 1, 128, 112, True), (1, 9, 40, 8, 128, 128, False),
                                                  (1, 2, 3, 3, 512, 512, False), (1, 2, 3, 3, 512, 496, True),
                                                  (2, 2, 4, 2, 80, 16, False), (1, 40, 2, 1, 192, 64, True)])
def test_rotate_matches_oracle(dtype, B, W, Hq, H, D, rot, inter):
    rng = np.random.default_rng(D + rot)
    q, k, _ = _qkv(rng, B, W, Hq, H, D, dtype)
    starts = rng.integers(0, 131072, B)
    starts[0] = 2**30 if rot > 32 else -77
    f, gain = sv.rotary_frequencies(rot, scaling="ramp", factor=8, original_len=4096, device="cuda")
    oq, ok = sv.rotate_qk(q, k, _i32(starts), f, interleaved=inter, gain=gain)
    for x, y in ((q, oq), (k, ok)):
        x = x.double().cpu().numpy()
        want = window.rotate(x, np.zeros_like(x), starts, f.cpu().numpy(), inter, gain)
        _close(y.double().cpu().numpy(), x, want, rot, gain, inter, dtype)


@pytest.mark.gpu
def test_frequencies_of_any_size():
    rng = np.random.default_rng(1)
    q, _, _ = _qkv(rng, 4, 3, 2, 1, 64, "f16")
    f = np.array([0.0, 1.0, -1.0, 2.0**32, 1e-12, -3e-5, 6.283185307179586, 2.0**-64, 1e-300, 3.5, 1e4, -2.0**31, 0.5,
                  2.0**-33, 7.7e-9, 1e-7] * 2)
    starts = np.array([2**31 - 3, -2**31, 123456789, 0])
    got, none = sv.rotate_qk(q, None, _i32(starts), torch.from_numpy(f).cuda())
    x = q.double().cpu().numpy()
    # 2^32 radians a position at 2^31: 2^63 radians, whose reduction by 1 / (2 pi) in 64 bits is off by 2^-3 turns and more:
    # the bound of the header holds while position * inv_freq stays below 2^34
    want = window.rotate(x, np.zeros_like(x), starts, f)
    sure = np.abs(f) <= 8
    keep = np.concatenate([sure, sure])
    a, b, w = (z[..., keep] for z in (got.double().cpu().numpy(), x, want))
    _close(a, b, w, int(keep.sum()), 1.0, False, "f16")
    assert none is None and torch.isfinite(got).all()


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
def test_windows_trees_strides_and_in_place(inter):
    rng = np.random.default_rng(2)
    B, W, Hq, H, D, rot = 3, 37, 4, 2, 64, 48
    q, k, _ = _qkv(rng, B, W, Hq, H, D, "bf16", pad=8)
    paths = np.stack([random_paths(rng, W - 4, W, 7) for _ in range(B)])  # the last nodes are on no path
    masks = kv.tree_masks(paths, W)
    lens, starts = np.array([W, 0, 20]), np.array([5, 6, 70000])
    f, _ = sv.rotary_frequencies(rot, device="cuda")
    for m in (None, masks):
        md = None if m is None else _i32(m)
        oq, ok = sv.rotate_qk(q, k, _i32(starts), f, interleaved=inter, window_lens=_i32(lens), masks=md)
        for x, y in ((q, oq), (k, ok)):
            x = x.double().cpu().numpy()
            want = window.rotate(x, np.zeros_like(x), starts, f.cpu().numpy(), inter, 1.0, lens, m)
            _close(y.double().cpu().numpy(), x, want, rot, 1.0, inter, "bf16")
            assert not y[1].any() and not y[2, 20:].any()
        # in place, on strided slices: the same bits, and nothing else written
        whole = torch.cat([q, k], 2).clone()
        a, b = whole[:, :, :Hq], whole[:, :, Hq:]
        old = whole.clone()
        ra, rb = sv.rotate_qk(a, b, _i32(starts), f, interleaved=inter, window_lens=_i32(lens), masks=md, out_q=a, out_k=b)
        assert ra is a and rb is b
        for x, y, z in ((a, oq, old[:, :, :Hq]), (b, ok, old[:, :, Hq:])):
            assert torch.equal(x[0], y[0]) and torch.equal(x[2, :20], y[2, :20])
            assert torch.equal(x[1], z[1]) and torch.equal(x[2, 20:], z[2, 20:])
        k2 = sv.rotate_qk(None, k, _i32(starts), f, interleaved=inter, window_lens=_i32(lens), masks=md)
        assert k2[0] is None and torch.equal(k2[1], ok)
    bad = sv.rotate_qk(q, k, _i32(starts), f, window_lens=_i32([-1, W + 1, 1]))[0]
    assert not bad[:2].any() and bad[2, 0].any()


STORE = [(1, 1, 1, 1, 64, 16), (2, 5, 8, 2, 128, 16), (3, 40, 4, 2, 64, 32), (2, 33, 2, 1, 128, 32), (2, 200, 4, 4, 64, 64),
         (1, 150, 4, 2, 128, 64), (2, 130, 2, 1, 128, 48), (1, 1100, 2, 1, 64, 1024), (5, 8, 32, 8, 128, 1024),
         (2, 70, 3, 3, 64, 80), (300, 4, 2, 8, 64, 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("B,W,Hq,H,D,tpb", STORE)
@pytest.mark.parametrize("inter,rot", [(False, 1.0), (True, 1.0), (False, 0.25), (True, 0.75)])
def test_rotating_store_is_the_two_calls(dtype, B, W, Hq, H, D, tpb, inter, rot):
    rng = np.random.default_rng(W + D)
    lens = rng.integers(0, 3 * tpb, B)
    wins = rng.integers(0, W + 1, B)
    wins[0] = W
    pool, scales, tables = cache(rng, lens + W, H, D, tpb)
    if B > 2:
        tables[1, 0] = -1  # what a bad table leaves out is left out by both
        lens[2] = -1
    pool, scales, tables = torch.from_numpy(pool).cuda(), torch.from_numpy(scales).cuda(), _i32(tables)
    q, k, v = _qkv(rng, B, W, Hq, H, D, dtype)
    f, gain = sv.rotary_frequencies(int(rot * D), scaling="ramp", factor=4, original_len=2048, device="cuda")
    starts = _i32(rng.integers(0, 200000, B))
    masks = None
    if W <= 40 and B < 100:
        masks = _i32(kv.tree_masks(np.stack([random_paths(rng, W, W, 9) for _ in range(B)]), W))
    for win, m in ((_i32(wins), None), (None, masks)):
        args = dict(interleaved=inter, gain=gain, window_lens=win, masks=m)
        p2, s2 = pool.clone(), scales.clone()
        q2, k2 = sv.rotate_qk(q, k, starts, f, **args)
        sv.store_kv(k2, v, p2, s2, tables, _i32(lens), window_lens=win)
        p1, s1 = pool.clone(), scales.clone()
        q1 = sv.rotate_store_kv(q, k, v, f, p1, s1, tables, _i32(lens), starts=starts, **args)
        assert torch.equal(q1, q2) and torch.equal(p1, p2) and torch.equal(s1, s2)


# (B, W, Hq, H, D, tpb) of one launch: min(W, tpb) * D / 8 at most 64
ONE_LAUNCH = [(3, 1, 32, 8, 128, 16), (4, 3, 8, 2, 128, 16), (4, 4, 4, 4, 128, 32), (2, 2, 2, 1, 128, 1024), (5, 4, 10, 5, 128, 48),
              (4, 8, 4, 2, 64, 16), (3, 7, 6, 3, 64, 16), (2, 5, 2, 1, 64, 48), (3, 6, 7, 7, 64, 32)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("B,W,Hq,H,D,tpb", ONE_LAUNCH)
@pytest.mark.parametrize("inter,rot", [(False, 1.0), (True, 1.0), (False, 0.25), (True, 0.75)])
def test_one_launch_is_the_two_calls(dtype, B, W, Hq, H, D, tpb, inter, rot):
    """Windows of a decode step, across a block's end and inside it, as chains and as trees."""
    assert sv.lib().spec_rotate_store_scratch_size(B, W, H, D, tpb) == 256  # no scratch for rotated keys
    rng = np.random.default_rng(W * D + tpb)
    lens = 2 * tpb - 1 - np.arange(B) * (W // 2)  # the first window crosses the end of its block, the last ones end there
    lens[-1] = 0
    pool, scales, tables = cache(rng, lens + W, H, D, tpb)
    pool, scales, tables = torch.from_numpy(pool).cuda(), torch.from_numpy(scales).cuda(), _i32(tables)
    q, k, v = _qkv(rng, B, W, Hq, H, D, dtype)
    k *= torch.from_numpy(np.exp(rng.normal(0, 1, (B, W, 1, 1)))).to(k.dtype).cuda()  # some grow their block's scale
    f, gain = sv.rotary_frequencies(int(rot * D), scaling="ramp", factor=4, original_len=2048, device="cuda")
    starts = _i32(rng.integers(0, 200000, B))
    masks = _i32(kv.tree_masks(np.stack([random_paths(rng, W, W, 4) for _ in range(B)]), W))
    wins = rng.integers(0, W + 1, B)
    wins[0] = W
    for win, m in ((None, None), (_i32(wins), None), (None, masks), (_i32(wins), masks)):
        args = dict(interleaved=inter, gain=gain, window_lens=win, masks=m)
        p2, s2 = pool.clone(), scales.clone()
        q2, k2 = sv.rotate_qk(q, k, starts, f, **args)
        sv.store_kv(k2, v, p2, s2, tables, _i32(lens), window_lens=win)
        p1, s1 = pool.clone(), scales.clone()
        q1 = sv.rotate_store_kv(q, k, v, f, p1, s1, tables, _i32(lens), starts=starts, **args)
        assert torch.equal(q1, q2) and torch.equal(p1, p2) and torch.equal(s1, s2)
        assert not torch.equal(p1, pool)


@pytest.mark.gpu
@pytest.mark.parametrize("B,W,Hq,H,D,inter", [(1300, 4, 8, 8, 128, False), (2600, 4, 6, 3, 128, True), (1300, 8, 8, 8, 64, False)])
def test_one_launch_of_a_large_batch(B, W, Hq, H, D, inter):
    """So many blocks that a CTA takes all (kind, head) pairs of one, which share its angles."""
    tpb = 16
    assert sv.lib().spec_rotate_store_scratch_size(B, W, H, D, tpb) == 256
    assert B * 2 * -(-2 * H // 4) > 8 * 152 * 8  # where the CTAs change
    rng = np.random.default_rng(B)
    tables = _i32(rng.permutation(2 * B).reshape(B, 2))
    pool = torch.from_numpy(rng.integers(0, 256, (2 * B, 2, H, tpb, D)).astype(np.uint8)).cuda()
    scales = torch.from_numpy(np.exp2(rng.integers(-9, -4, (2 * B, 2, H))).astype(np.float32)).cuda()
    lens = rng.integers(0, 2 * tpb - W + 1, B)
    q, k, v = _qkv(rng, B, W, Hq, H, D, "bf16")
    f, _ = sv.rotary_frequencies(D, device="cuda")
    starts = _i32(rng.integers(0, 5000, B))
    win = _i32(rng.integers(0, W + 1, B))
    masks = _i32(np.broadcast_to(kv.tree_masks(random_paths(rng, W, W, 4)[None], W), (B, W, 1)))
    for args in (dict(window_lens=win), dict(masks=masks)):
        p2, s2 = pool.clone(), scales.clone()
        q2, k2 = sv.rotate_qk(q, k, starts, f, interleaved=inter, **args)
        sv.store_kv(k2, v, p2, s2, tables, _i32(lens), window_lens=args.get("window_lens"))
        p1, s1 = pool.clone(), scales.clone()
        q1 = sv.rotate_store_kv(q, k, v, f, p1, s1, tables, _i32(lens), starts=starts, interleaved=inter, **args)
        assert torch.equal(q1, q2) and torch.equal(p1, p2) and torch.equal(s1, s2)


@pytest.mark.gpu
def test_rotating_store_starts_at_the_cursor():
    rng = np.random.default_rng(4)
    pool, scales, tables = (torch.from_numpy(x).cuda() for x in cache(rng, [30, 61], 2, 64, 16))
    q, k, v = _qkv(rng, 2, 4, 4, 2, 64, "bf16")
    f, _ = sv.rotary_frequencies(64, device="cuda")
    seq = _i32([20, 50])
    a = sv.rotate_store_kv(q, k, v, f, pool, scales, tables, seq)
    assert torch.equal(a, sv.rotate_qk(q, None, seq, f)[0])
    inplace = q.clone()
    assert sv.rotate_store_kv(inplace, k, v, f, pool, scales, tables, seq, out_q=inplace) is inplace
    assert torch.equal(inplace, a)


@pytest.mark.gpu
@pytest.mark.parametrize("W", [3, 40])
def test_keys_and_values_of_one_array(W):
    """k and v are only read, so they may be one array, as for store_kv; in one launch and in two."""
    rng = np.random.default_rng(9)
    lens = np.array([20, 5])
    pool, scales, tables = (torch.from_numpy(x).cuda() for x in cache(rng, lens + W, 2, 64, 16))
    q, k, _ = _qkv(rng, 2, W, 4, 2, 64, "bf16")
    f, _ = sv.rotary_frequencies(64, device="cuda")
    p2, s2 = pool.clone(), scales.clone()
    q2, k2 = sv.rotate_qk(q, k, _i32(lens), f)
    sv.store_kv(k2, k, p2, s2, tables, _i32(lens))
    q1 = sv.rotate_store_kv(q, k, k, f, pool, scales, tables, _i32(lens))
    assert torch.equal(q1, q2) and torch.equal(pool, p2) and torch.equal(scales, s2)


@pytest.mark.gpu
def test_in_place_through_a_view_with_another_stride_on_an_axis_of_one_element():
    rng = np.random.default_rng(10)
    f, _ = sv.rotary_frequencies(64, device="cuda")
    for shape, stride in (((1, 3, 4, 64), (8, 256, 64, 1)), ((2, 1, 4, 64), (256, 24, 64, 1)), ((2, 3, 1, 64), (192, 64, 640, 1))):
        x = torch.from_numpy(rng.normal(0, 1, shape)).cuda().bfloat16()
        s = _i32(rng.integers(0, 100, shape[0]))
        want = sv.rotate_qk(x, None, s, f)[0]
        view = x.as_strided(shape, stride)
        assert torch.equal(view, x) and view.stride() != x.stride()
        assert sv.rotate_qk(x, None, s, f, out_q=view)[0] is view and torch.equal(x, want)


@pytest.mark.gpu
def test_outputs_that_overlap_are_refused():
    rng = np.random.default_rng(11)
    q, k, v = _qkv(rng, 2, 5, 4, 2, 64, "bf16")
    f, _ = sv.rotary_frequencies(64, device="cuda")
    s = _i32([3, 4])
    buf = torch.zeros(2 * 5 * 8 * 64 + 1024, dtype=torch.bfloat16, device="cuda")
    x, y = buf[:5120].view(2, 5, 8, 64)[:, :, :4], buf[64:5184].view(2, 5, 8, 64)[:, :, :4]
    rows = buf.as_strided((2, 5, 4, 64), (1280, 248, 64, 1))  # a row's end is the next one's beginning
    for kw in (dict(q=x, out_q=y), dict(q=q, out_q=rows), dict(q=q, k=k, out_q=x, out_k=buf[192:5312].view(2, 5, 8, 64)[:, :, :2])):
        with pytest.raises(sv.SpecError):
            sv.rotate_qk(kw["q"], kw.get("k"), s, f, out_q=kw["out_q"], out_k=kw.get("out_k"))
    one = torch.zeros((1, 1, 4, 64), dtype=torch.bfloat16, device="cuda").expand(2, 5, 4, 64)
    with pytest.raises(ValueError):
        sv.rotate_qk(one, None, s, f, out_q=one)
    pool, scales, tables = (torch.from_numpy(z).cuda() for z in cache(rng, [30, 61], 2, 64, 16))
    for out in (rows, buf):
        with pytest.raises((ValueError, sv.SpecError)):
            sv.rotate_store_kv(x, k, v, f, pool, scales, tables, s, out_q=y if out is buf else out)
    assert not buf.any()
    # rows between each other's rows are apart: q, k and both outputs in one array
    all4 = torch.zeros((2, 5, 12, 64), dtype=torch.bfloat16, device="cuda")
    all4[:, :, :4], all4[:, :, 8:10] = q, k
    got = sv.rotate_qk(all4[:, :, :4], all4[:, :, 8:10], s, f, out_q=all4[:, :, 4:8], out_k=all4[:, :, 10:])
    want = sv.rotate_qk(q, k, s, f)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
def test_largest_windows():
    rng = np.random.default_rng(5)
    W = sv.SPEC_MAX_WINDOW
    q, k, _ = _qkv(rng, 1, W, 1, 1, 64, "bf16")
    f, _ = sv.rotary_frequencies(64, device="cuda")
    oq, _ = sv.rotate_qk(q, k, _i32([1000]), f)
    for i in (0, 1, 40000, W - 1):
        one = sv.rotate_qk(q[:, i:i + 1], None, _i32([1000 + i]), f)[0]
        assert torch.equal(one, oq[:, i:i + 1])


@pytest.mark.gpu
def test_binding_refusals():
    rng = np.random.default_rng(6)
    q, k, v = _qkv(rng, 2, 3, 4, 2, 64, "bf16")
    f, _ = sv.rotary_frequencies(64, device="cuda")
    s = _i32([0, 1])

    def call(q=q, k=k, s=s, f=f, **kw):
        return sv.rotate_qk(q, k, s, f, **kw)
    for bad in (dict(f=f.float()), dict(f=f[:12]), dict(f=torch.cat([f, f])), dict(f=f.cpu()), dict(s=s.long()),
                dict(s=s[:1]), dict(q=q.float()), dict(k=k.half()), dict(k=k[:, :2]), dict(q=q[..., 1:49]),
                dict(q=None, k=None), dict(q=None, out_q=q), dict(out_q=k), dict(out_q=q.half()),
                dict(out_q=torch.zeros_like(q[:, :1]).expand(2, 3, 4, 64)),
                dict(out_k=q[:, :, :2], out_q=q), dict(window_lens=s.float()),
                dict(masks=torch.zeros((2, 3, 2), dtype=torch.int32, device="cuda")), dict(q=q.cpu())):
        with pytest.raises(ValueError):
            call(**bad)
    pool, scales, tables = (torch.from_numpy(x).cuda() for x in cache(rng, [30, 61], 2, 64, 16))

    def store(q=q, k=k, v=v, f=f, **kw):
        return sv.rotate_store_kv(q, k, v, f, pool, scales, tables, s, **kw)
    for bad in (dict(v=v.half()), dict(v=v[:, :2]), dict(k=q), dict(f=f[:4]), dict(out_q=q[:, :2]), dict(q=q[:1]),
                dict(starts=s[:1])):
        with pytest.raises(ValueError):
            store(**bad)
    with pytest.raises((ValueError, sv.SpecError)):
        call(gain=math.nan)


@pytest.mark.gpu
def test_store_rounds_like_the_oracle():
    """The whole path against the oracle: rotation, the keys' type, the cache's codes."""
    rng = np.random.default_rng(8)
    for dtype, rnd in (("bf16", to_bf16), ("f16", to_f16)):
        pool, scales, tables = cache(rng, [60, 45], 2, 64, 16)
        q, k, v = _qkv(rng, 2, 20, 2, 2, 64, dtype)
        f, _ = sv.rotary_frequencies(64, device="cuda")
        seq, starts = np.array([40, 25]), np.array([4000, 25])
        p, s = torch.from_numpy(pool).cuda(), torch.from_numpy(scales).cuda()
        sv.rotate_store_kv(q, k, v, f, p, s, _i32(tables), _i32(seq), starts=_i32(starts))
        kr = rnd(window.rotate(k.double().cpu().numpy(), np.zeros(k.shape), starts, f.cpu().numpy()))
        wp, ws = kv.store(kr, v.double().cpu().numpy(), pool, scales, tables, seq)
        got, want = (kv.decode(a) * b[..., None, None] for a, b in
                     ((p.cpu().numpy(), s.cpu().numpy().astype(np.float64)), (wp, ws)))
        live = np.isfinite(want)
        assert np.array_equal(live, np.isfinite(got))
        # a key rounded the other way in its type is at most one e4m3 step off: 2^-3 of it, or 2^-9 of the scale
        step = np.maximum(2.0 ** -3 * np.abs(want), 2.0 ** -9 * np.broadcast_to(ws[..., None, None], want.shape))
        assert (np.abs(got - want)[live] <= step[live]).all()
        assert (got == want)[live].mean() > 0.99
