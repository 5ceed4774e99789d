"""Attention over the paged 8-bit cache: oracle pins on the CPU, the CUDA
call against the 64-bit oracle on the GPU.

Error bound of one output element, from the steps of the computation (u =
2^-24 is fp32's half step, eps(T) / 2 the output type's):
  scores   a dot product of D exact products summed in fp32 in any order is
           off by at most D u sum|q_d k_d|; the products with the two scales
           and log2(e) and the subtraction of the maximum add a few u of the
           score: delta = (D + 8) u spread in all, spread = scale sum|q_d k_d|
  weights  exp2 within 2^-21, rounded to fp16: 2^-11; weights below fp16's
           normal range (relative to the row's largest, scaled up by at least
           2^8) are off by at most 2^-32
  sums     over n keys in fp32: n u each for numerator and denominator
so |out - exact| <= (2 delta + 2^-11 + 2^-20 + 2 n u) A + n 2^-32 vmax
                    + eps(T) / 2 |out| + the type's least step,
A = sum p |v| / sum p.  lse: delta + 2^-20 + n u + 4 u |lse|.
"""
import ctypes

import numpy as np
import pytest
import torch

import speculative_decoding_verification_row_gb300 as sv
from oracle import kv
from _kv import cache, random_paths, to_bf16, to_f16
from test_kv_store import BAD_CACHES, _fake_cache

U = 2.0 ** -24


# ------------------------------------------------------------------ oracle pins (CPU)
def test_oracle_matches_a_dense_softmax():
    rng = np.random.default_rng(0)
    H, G, D, tpb, seq, w = 2, 3, 64, 16, 21, 5
    pool, scales, tables = cache(rng, np.array([seq + w]), H, D, tpb)
    q = rng.normal(0, 1, (1, w, H * G, D))
    r = kv.attend(q, pool, scales, tables, [seq])
    x = torch.from_numpy((kv.decode(pool[tables[0, :2]]) * scales[tables[0, :2]][..., None, None]))
    k, v = (x[:, i].permute(1, 0, 2, 3).reshape(H, -1, D)[:, :seq + w].repeat_interleave(G, 0) for i in (0, 1))
    qt = torch.from_numpy(q[0]).transpose(0, 1)
    see = torch.ones(w, seq + w, dtype=torch.bool).tril(seq)
    want = torch.nn.functional.scaled_dot_product_attention(qt, k, v, attn_mask=see)
    assert np.allclose(r["out"][0], want.transpose(0, 1).numpy(), rtol=1e-12, atol=1e-12)


def test_oracle_empty_rows_and_chain_masks():
    rng = np.random.default_rng(1)
    pool, scales, tables = cache(rng, np.array([4]), 1, 64, 16)
    q = rng.normal(0, 1, (1, 4, 1, 64))
    chain = kv.tree_masks(np.arange(4, dtype=np.int32)[None, None], 4)
    a, b = kv.attend(q, pool, scales, tables, [0]), kv.attend(q, pool, scales, tables, [0], masks=chain)
    assert np.array_equal(a["out"], b["out"])
    chain[0, 2] = 0
    c = kv.attend(q, pool, scales, tables, [0], masks=chain)
    assert (c["out"][0, 2] == 0).all() and c["lse"][0, 2, 0] == -np.inf and np.array_equal(c["out"][0, 3], a["out"][0, 3])


def test_refusals_before_any_launch():
    lib, f = sv.lib(), 16 * 1024
    ok = dict(size=ctypes.sizeof(sv.AttendParams), q=f, q_strides=(ctypes.c_int64 * 3)(256, 128, 64), dtype=1, B=2, W=3,
              q_heads=4, seq_lens=f, window_lens=None, masks=None, scale=0.125, out=f, out_lse=None)

    def call(cache=None, scratch=f, nbytes=1 << 40, **o):
        a = dict(ok, **o)
        prm = sv.AttendParams(*[a[n] for n, _ in sv.AttendParams._fields_])
        return lib.spec_attend_kv(ctypes.byref(cache or _fake_cache()), ctypes.byref(prm), scratch, nbytes, None)
    for bad in BAD_CACHES:
        assert call(cache=_fake_cache(**bad)) == sv.SPEC_EINVAL, bad
    odd = (ctypes.c_int64 * 3)(256, 130, 64)
    for bad in (dict(size=8), dict(q=None), dict(q=f + 8), dict(q_strides=odd), dict(dtype=0), dict(dtype=3), dict(B=0),
                dict(B=8193), dict(W=0), dict(W=65537), dict(q_heads=3), dict(q_heads=0), dict(seq_lens=None),
                dict(out=None), dict(out=f + 4), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(W=1025, masks=f)):
        assert call(**bad) == sv.SPEC_EINVAL, bad
    assert call(scratch=None) == call(scratch=f + 16) == call(nbytes=16) == sv.SPEC_EWORKSPACE
    s = lib.spec_attend_scratch_size
    assert s(2, 3, 4, 2, 64) > 0
    assert s(0, 3, 4, 2, 64) == s(2, 0, 4, 2, 64) == s(2, 3, 3, 2, 64) == s(2, 3, 4, 2, 80) == 0
    cpu = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sv.attend_kv(cpu, torch.zeros((1, 2, 2, 16, 64), dtype=torch.uint8), torch.zeros((1, 2, 2)),
                     torch.zeros((1, 1), dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


@pytest.mark.parametrize("scale", [3e38, -3e38, 2.4e38])
def test_a_scale_whose_log2_form_is_infinite_is_refused(scale):
    # it would turn scores of 0 into NaN
    f = 16 * 1024
    prm = sv.AttendParams(ctypes.sizeof(sv.AttendParams), f, (ctypes.c_int64 * 3)(256, 128, 64), 1, 2, 3, 4, f, None, None,
                          scale, f, None)
    rc = sv.lib().spec_attend_kv(ctypes.byref(_fake_cache()), ctypes.byref(prm), f, 1 << 40, None)
    assert rc == sv.SPEC_EINVAL


def test_tensor_memory_is_taken_behind_the_wait_for_the_kernel_before():
    # A launch that may start before the kernel in front has ended must not hold
    # what that kernel may still ask for.  Checked in the source: on a GPU the
    # other order would hang, and only beside another program's kernel.
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "speculative_decoding_verification_row_gb300", "csrc", "attend_tiles.cu")) as f:
        kernel = f.read().split("attend_tiles_kernel(", 1)[1]
    assert kernel.count("tcgen05.alloc") == kernel.count("griddepcontrol.wait") == 1
    assert kernel.index("griddepcontrol.wait") < kernel.index("tcgen05.alloc")


# ------------------------------------------------------------------ GPU parity
def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def i32(a):
    return dev(np.asarray(a, np.int32))


def make_q(rng, shape, dt, amp=1.0):
    q = (to_bf16 if dt == "bf16" else to_f16)(rng.normal(0, amp, shape))
    return q, dev(q).to(torch.bfloat16 if dt == "bf16" else torch.float16)


def check(out, lse, r, dt, D, rows, vmax):
    """rows [B, W]: the rows a call writes."""
    eps = 2.0 ** -8 if dt == "bf16" else 2.0 ** -11
    got, want = out.double().cpu().numpy()[rows], r["out"][rows]
    n, spread, amp = r["keys"][rows][..., None], r["spread"][rows][..., None], r["amp"][rows]
    delta = (D + 8) * U * spread
    tol = (2 * delta + 2.0 ** -11 + 2.0 ** -20 + 2 * n * U) * amp + n * 2.0 ** -32 * vmax + eps * np.abs(want) + 2.0 ** -25
    assert np.array_equal(np.isnan(got), np.isnan(want))
    fine = ~np.isnan(want)
    bad = np.abs(got - want)[fine] > tol[fine]
    assert not bad.any(), f"{bad.mean():.2%} of {bad.size} outside, worst {(np.abs(got - want)[fine] / tol[fine]).max():.3f}"
    if lse is not None:
        got, want = lse.double().cpu().numpy()[rows], r["lse"][rows]
        assert np.array_equal(np.isneginf(got), np.isneginf(want)) and np.array_equal(np.isnan(got), np.isnan(want))
        fine = np.isfinite(want)
        tol = delta[..., 0] + 2.0 ** -20 + n[..., 0] * U + 4 * U * np.abs(np.where(fine, want, 0))
        assert (np.abs(got - np.where(fine, want, 0))[fine] <= tol[fine]).all()


def run_case(rng, seq, win, W, H, G, D, tpb, dt, masks=None, spread=1.0, amp=1.0, scale=None, edit=None):
    seq, win = np.asarray(seq), np.asarray(win)
    B = len(seq)
    pool, scales, tables = cache(rng, seq + win, H, D, tpb, spread=spread)
    if edit:
        edit(pool, scales, tables)
    q, dq = make_q(rng, (B, W, H * G, D), dt, amp)
    r = kv.attend(q, pool, scales, tables, seq, win, masks, scale)
    out = torch.full(dq.shape, 7.0, dtype=dq.dtype, device="cuda")
    lse = torch.full(dq.shape[:3], 7.0, device="cuda")
    sv.attend_kv(dq, dev(pool), dev(scales), i32(tables), i32(seq), window_lens=i32(win),
                 masks=None if masks is None else i32(masks), scale=scale, out=out, out_lse=lse)
    rows = np.arange(W)[None] < win[:, None]
    live = [b for b in range(B) if win[b]]
    x = kv.decode(pool)[:, 1] * scales[:, 1][..., None, None]
    check(out, lse, r, dt, D, rows, np.nanmax(np.abs(np.where(np.isnan(x), 0, x))) if live else 0)
    assert (out[dev(~rows)] == 7).all() and (lse[dev(~rows)] == 7).all()  # padded rows stay
    return out, lse


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("G,tpb,seq", [(1, 16, [0]), (4, 16, [1]), (8, 16, [15, 16, 17]), (4, 32, [999]),
                                       (16, 48, [63, 0, 130]), (5, 64, [127, 128, 129, 500]), (24, 16, [300, 31])])
def test_single_token(D, dt, G, tpb, seq):
    rng = np.random.default_rng(G * 100 + len(seq))
    run_case(rng, seq, [1] * len(seq), 1, 2, G, D, tpb, dt)


@pytest.mark.gpu
@pytest.mark.parametrize("W,H,G,D,tpb,dt,hi", [(2, 1, 1, 64, 16, "bf16", 40), (4, 2, 4, 128, 32, "bf16", 700),
                                               (8, 2, 4, 128, 32, "f16", 300), (8, 1, 8, 64, 16, "bf16", 600),
                                               (17, 2, 4, 128, 64, "bf16", 260), (33, 1, 8, 64, 128, "f16", 400),
                                               (65, 2, 5, 128, 48, "bf16", 200), (130, 1, 3, 64, 16, "f16", 333)])
def test_chain_windows(W, H, G, D, tpb, dt, hi):
    rng = np.random.default_rng(W)
    B = 5
    seq = rng.integers(0, hi + 1, B)
    win = rng.integers(0, W + 1, B)
    seq[0], win[0], win[1] = 0, W, W
    win[2] = 0
    run_case(rng, seq, win, W, H, G, D, tpb, dt)


@pytest.mark.gpu
@pytest.mark.parametrize("W,L,H,G,D,tpb,dt", [(8, 4, 1, 1, 64, 16, "bf16"), (12, 5, 2, 1, 128, 16, "f16"),
                                              (60, 4, 2, 4, 128, 64, "bf16"), (64, 9, 1, 2, 64, 32, "f16"),
                                              (100, 12, 2, 3, 128, 16, "bf16"), (300, 20, 1, 1, 64, 48, "f16")])
def test_tree_windows(W, L, H, G, D, tpb, dt):
    rng = np.random.default_rng(W + L)
    seq = np.array([0, 37, 200])
    paths = np.stack([random_paths(rng, W, W, L) for _ in seq])
    paths[1, -W // 3:] = -1  # some nodes on no path: at an empty prefix their rows see nothing
    paths[0, -W // 2:] = -1
    masks = kv.tree_masks(paths, W)
    run_case(rng, seq, [W, W, W - 1], W, H, G, D, tpb, dt, masks=masks)


@pytest.mark.gpu
@pytest.mark.parametrize("G,W", [(2, 3), (8, 12)])
def test_empty_rows(G, W):
    rng = np.random.default_rng(9)
    masks = np.zeros((2, W, 1), np.int32)
    masks[:, 1] = 0b10
    out, lse = run_case(rng, [0, 20], [W, W], W, 2, G, 64, 16, "bf16", masks=masks)
    assert (out[0, 0] == 0).all() and torch.isneginf(lse[0, 0]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("G,W", [(1, 2), (4, 4), (4, 40), (8, 40)])
@pytest.mark.parametrize("kind", [0, 1])
def test_nan_in_unseen_places(G, W, kind):
    # NaN codes in a window row reach the tokens that see it and no others;
    # rows past the end hold arbitrary bytes already
    rng = np.random.default_rng(W + kind)
    seq, H, D, tpb = [19, 0, 300], 2, 128, 16

    def edit(pool, scales, tables):
        for b, s in enumerate(seq):
            t = s + W - 1
            pool[tables[b, t // tpb], kind, 0, t % tpb, 5] = 0x7f
            pool[tables[b, t // tpb], kind, 1, t % tpb, :] = 0xff
    run_case(rng, seq, [W] * 3, W, H, G, D, tpb, "bf16", edit=edit)
    masks = np.zeros((3, W, -(-W // 32)), np.int32)
    masks[:, :, 0] = 1  # everybody sees token 0; token 1 of the window sees the NaN row
    masks[:, 1, (W - 1) // 32] |= np.int32(np.uint32(1 << ((W - 1) % 32)).view(np.int32))
    run_case(rng, seq, [W] * 3, W, H, G, D, tpb, "bf16", masks=masks, edit=edit)


@pytest.mark.gpu
@pytest.mark.parametrize("G,W", [(1, 1), (4, 4), (4, 40)])
def test_nan_in_the_prefix_reaches_every_row(G, W):
    rng = np.random.default_rng(3)

    def edit(pool, scales, tables):
        pool[tables[0, 2], 1, 0, 7, 9] = 0x7f
        pool[tables[1, 1], 0, 1, 3, 9] = 0xff
    out, _ = run_case(rng, [70, 70], [W, W], W, 2, G, 64, 16, "f16", edit=edit)
    assert torch.isnan(out[0, 0, 0, 9]) and torch.isnan(out[1, 0, G]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("G,W", [(1, 1), (4, 4), (4, 40)])
def test_bad_requests_read_nan_and_leave_the_others(G, W):
    rng = np.random.default_rng(4)
    seq, win = [100, 50, -1, 40, 3, 90], [W, W, W, W + 1, -1, W]
    B, H, D, tpb = 6, 2, 64, 16
    pool, scales, tables = cache(rng, np.full(B, 100 + W), H, D, tpb)
    tables[1, 2] = len(pool)     # a block that does not exist
    tables[5, (90 + W - 1) // tpb] = -1  # an unmapped block in the window
    q, dq = make_q(rng, (B, W, H * G, D), "bf16")
    out, lse = sv.attend_kv(dq, dev(pool), dev(scales), i32(tables), i32(seq), window_lens=i32(win), want_lse=True)
    r = kv.attend(q, pool, scales, tables, seq, win)
    assert all(torch.isnan(out[b]).all() and torch.isnan(lse[b]).all() for b in (1, 2, 3, 4, 5))
    rows = np.zeros((B, W), bool)
    rows[0] = True
    check(out, lse, r, "bf16", D, rows, np.nanmax(np.abs(kv.decode(pool[:, 1]))) * scales[:, 1].max())
    # a window past the table's end
    o2, _ = sv.attend_kv(dq, dev(pool), dev(scales), i32(tables[:, :3]), i32([48 - W] + [60] * 5))
    assert torch.isfinite(o2[0].float()).all() and torch.isnan(o2[1]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("G,W", [(2, 1), (4, 4), (4, 40)])
def test_scales_and_levels(G, W):
    rng = np.random.default_rng(6)
    # blocks of very different scales, steep and flat scores, a negative scale, zero blocks
    run_case(rng, [200, 333], [W, W], W, 2, G, 128, 16, "bf16", spread=6.0, amp=0.05)
    run_case(rng, [200, 333], [W, W], W, 2, G, 64, 16, "f16", amp=30.0)
    run_case(rng, [200, 333], [W, W], W, 2, G, 64, 32, "bf16", scale=-0.3)
    run_case(rng, [200, 333], [W, W], W, 2, G, 64, 32, "bf16", scale=0.0)

    def zero(pool, scales, tables):
        pool[tables[0, 1]], scales[tables[0, 1]] = 0, 0
        scales[tables[1]] *= np.float32(0.7)  # not a power of two
    run_case(rng, [200, 333], [W, W], W, 2, G, 64, 16, "bf16", edit=zero)


@pytest.mark.gpu
@pytest.mark.parametrize("G,W", [(2, 1), (4, 16)])
def test_many_light_keys_beside_a_heavy_one(G, W):
    # one position holds about half of the mass, 20000 alike ones the rest:
    # weights far below the largest still count
    rng = np.random.default_rng(7)
    H, D, tpb, T = 1, 64, 64, 20000 // 64 * 64

    def edit(pool, scales, tables):
        pool[tables[0]] = 0
        pool[tables[0], 1] = kv.encode(rng.uniform(0.5, 1.5, pool[tables[0], 1].shape))
        pool[tables[0, 0], 0, 0, 0] = kv.encode(1.0)
        pool[tables[0, 0], 1, 0, 0] = kv.encode(-1.0)
        scales[:] = 1
    seq = T - W
    pool, scales, tables = cache(rng, np.array([T]), H, D, tpb, extra_cols=0)
    edit(pool, scales, tables)
    q = to_bf16(np.full((1, W, G, D), np.log(2e4) / D))
    r = kv.attend(q, pool, scales, tables, [seq], scale=1.0)
    out, lse = sv.attend_kv(dev(q).to(torch.bfloat16), dev(pool), dev(scales), i32(tables), i32([seq]), scale=1.0,
                            want_lse=True)
    check(out, lse, r, "bf16", D, np.ones((1, W), bool), 1.5)


@pytest.mark.gpu
def test_strided_queries_and_defaults():
    rng = np.random.default_rng(8)
    B, W, H, G, D, tpb = 3, 4, 2, 2, 64, 16
    seq = [40, 7, 90]
    pool, scales, tables = cache(rng, np.array(seq) + W, H, D, tpb)
    q, dq = make_q(rng, (B, W, H * G + 2 * H, D), "bf16")
    r = kv.attend(q[:, :, :H * G], pool, scales, tables, seq)
    a = [dev(pool).view(torch.float8_e4m3fn), dev(scales), i32(tables), i32(seq)]
    for x in (dq[:, :, :H * G], dq[:, :, :H * G].transpose(1, 2).contiguous().transpose(1, 2)):
        out, lse = sv.attend_kv(x, *a)
        assert lse is None
        check(out, None, r, "bf16", D, np.ones((B, W), bool), 100)
    with pytest.raises(ValueError):
        sv.attend_kv(dq[:, :, :H * G, ::2], *a)
    with pytest.raises(ValueError):
        sv.attend_kv(dq[:, :, :3], *a)
    with pytest.raises(ValueError):
        sv.attend_kv(dq[:2, :, :H * G], *a)
    with pytest.raises(ValueError):
        sv.attend_kv(dq[:, :, :H * G].contiguous(), *a, out=torch.empty((B, W, H * G, D), device="cuda"))
    with pytest.raises(ValueError):
        sv.attend_kv(dq[:, :, :H * G], *a, masks=torch.zeros((B, W), dtype=torch.int32, device="cuda"))
    with pytest.raises(sv.SpecError):
        sv.attend_kv(dq[:, :, :H * G], *a, scratch=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.gpu
def test_streams_graphs_and_repeats():
    # two captured graphs replayed on two streams at once, eager calls between
    # them, and the same bits every time
    rng = np.random.default_rng(10)
    B, H, D, tpb = 6, 2, 128, 16
    runs = []
    for W, G in ((1, 4), (20, 8)):
        seq = rng.integers(500, 1500, B)
        pool, scales, tables = cache(rng, seq + W, H, D, tpb)
        _, dq = make_q(rng, (B, W, H * G, D), "bf16")
        args = [dq, dev(pool), dev(scales), i32(tables), i32(seq)]
        want, want_lse = sv.attend_kv(*args, want_lse=True)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            sv.attend_kv(*args)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got, got_lse = sv.attend_kv(*args, want_lse=True)
        runs.append((args, want, want_lse, g, got, got_lse, side))
    for _ in range(5):
        for args, want, want_lse, g, got, got_lse, side in runs:
            with torch.cuda.stream(side):
                g.replay()
            eager, _ = sv.attend_kv(*args, stream=runs[0][6])
            other, _ = sv.attend_kv(*args, stream=side.cuda_stream)
            torch.cuda.synchronize()
            assert torch.equal(eager, want) and torch.equal(other, want)
    for args, want, want_lse, g, got, got_lse, side in runs:
        assert torch.equal(got, want) and torch.equal(got_lse, want_lse)


@pytest.mark.gpu
def test_offsets_beyond_32_bits():
    # a pool of over 4 GB; the request's blocks lie at its two ends
    H, D, tpb, W = 8, 128, 128, 4
    n = (1 << 32) // (2 * H * tpb * D) + 200
    rng = np.random.default_rng(11)
    small, scales, tables = cache(rng, np.array([500 + W]), H, D, tpb, spare=0, extra_cols=0)
    pool = torch.zeros((n, 2, H, tpb, D), dtype=torch.uint8, device="cuda")
    at = np.array([0, n - 1, n - 2, n - 150])[:len(small)]
    pool[torch.from_numpy(at).cuda()] = dev(small)
    big_scales = torch.ones((n, 2, H), device="cuda")
    big_scales[torch.from_numpy(at).cuda()] = dev(scales)
    q, dq = make_q(rng, (1, W, H * 4, D), "bf16")
    r = kv.attend(q, small, scales, tables, [500])
    out, lse = sv.attend_kv(dq, pool, big_scales, i32(at[tables]), i32([500]), want_lse=True)
    check(out, lse, r, "bf16", D, np.ones((1, W), bool), 500)
    k, dk = make_q(rng, (1, W, H, D), "bf16")
    sv.store_kv(dk, dk, pool, big_scales, i32(at[tables]), i32([500]))
    want, want_s = kv.store(k, k, small, scales, tables, [500])
    assert np.array_equal(pool[torch.from_numpy(at).cuda()].cpu().numpy(), want)


@pytest.mark.gpu
def test_a_step_of_tree_decoding():
    """The calls as a step makes them: blocks, rows, attention, verify,
    relocation, rollback, blocks back; the next step's attention then reads
    exactly the accepted tokens."""
    import oracle
    import workloads
    rng = np.random.default_rng(12)
    w = workloads.make("tree_b16_n60_l4_v151936_bf16", seed=3, B=4, V=4096)
    B, N, L = w["B"], w["N"], w["L"]
    H, G, D, tpb = 2, 4, 64, 16
    seq = np.array([30, 0, 47, 100], np.int32)
    pool0, scales0, _ = cache(rng, seq, H, D, tpb, spare=40)
    n = len(pool0)
    held = -(-seq // tpb)
    order = rng.permutation(n)
    tables = np.full((B, 12), -1, np.int32)
    at = 0
    for b in range(B):
        tables[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    scales0[:] = np.exp2(rng.integers(-6, -3, scales0.shape))
    pool0 &= 0x77  # no NaN codes
    free = np.full(n, -1, np.int32)
    free[:n - at] = order[at:]
    d = dict(seq=i32(seq), tables=i32(tables), held=i32(held), free=i32(free), count=i32([n - at]))
    pool, scales = dev(pool0), dev(scales0.astype(np.float32))
    k, dk = make_q(rng, (B, N, H, D), "bf16")
    v, dv = make_q(rng, (B, N, H, D), "bf16")
    q, dq = make_q(rng, (B, N, H * G, D), "bf16")
    # the step
    slots, granted = sv.reserve_blocks(d["seq"], d["tables"], d["held"], d["free"], d["count"], tpb, N)
    masks = sv.tree_masks(i32(w["paths"]), N)
    sv.store_kv(dk, dv, pool, scales, d["tables"], d["seq"])
    out, lse = sv.attend_kv(dq, pool, scales, d["tables"], d["seq"], masks=masks, want_lse=True)
    logits = dev(w["target"].view(np.int16)).view(torch.bfloat16)
    tok, acc, best, nodes = sv.verify_tree(logits, i32(w["tree_tokens"]), i32(w["paths"]))
    sv.relocate_quantised_kv(pool, scales, d["tables"], d["seq"], nodes, acc)
    new, _, spare = sv.rollback_paged(d["seq"], acc, N - 1, tpb, blocks_held=d["held"])
    sv.release_blocks(d["tables"], d["held"], spare, d["free"], d["count"])
    # the oracle's step
    slots_o, granted_o, t_o, h_o, c_o = kv.reserve(seq, None, tables, held, free, n - at, tpb, N)
    assert np.array_equal(slots.cpu().numpy(), slots_o) and (granted == N).all()
    p_o, s_o = kv.store(k, v, pool0, scales0, t_o, seq)
    m_o = kv.tree_masks(w["paths"].astype(np.int32), N)
    r = kv.attend(q, p_o, s_o, t_o, seq, masks=m_o)
    check(out, lse, r, "bf16", D, np.ones((B, N), bool), 100)
    o = oracle.verify(w)
    assert np.array_equal(nodes.cpu().numpy(), o["accepted_nodes"]) and (o["num_accepted"] > 0).any()
    p_o, s_o = kv.relocate(p_o, s_o, t_o, seq, o["accepted_nodes"], o["num_accepted"])
    assert np.array_equal(pool.cpu().numpy(), p_o) and np.array_equal(scales.cpu().numpy(), s_o)
    len_o = seq + o["num_accepted"] + 1
    give = np.maximum(0, h_o - -(-len_o // tpb))
    t_o, h_o, f_o, c_o = kv.release(t_o, h_o, give, free, c_o)
    assert np.array_equal(new.cpu().numpy(), len_o)
    for got, want in ((d["tables"], t_o), (d["held"], h_o), (d["free"], f_o), (d["count"], [c_o])):
        assert np.array_equal(got.cpu().numpy(), want)
    # the next step: one more token behind the accepted rows
    _, dq = make_q(rng, (B, 1, H * G, D), "bf16")
    sv.reserve_blocks(new, d["tables"], d["held"], d["free"], d["count"], tpb, 1)
    sv.store_kv(dk[:, :1], dv[:, :1], pool, scales, d["tables"], new)
    out, lse = sv.attend_kv(dq, pool, scales, d["tables"], new, want_lse=True)
    r = kv.attend(dq.double().cpu().numpy(), pool.cpu().numpy(), scales.cpu().numpy(), d["tables"].cpu().numpy(), len_o)
    check(out, lse, r, "bf16", D, np.ones((B, 1), bool), 100)


@pytest.mark.gpu
@pytest.mark.parametrize("G,W,D,B,seq", [(4, 40, 64, 2, 9000), (8, 30, 128, 3, 20000), (1, 4, 64, 1, 60000), (4, 4, 128, 40, 3000)])
def test_long_prefixes(G, W, D, B, seq):
    # many tiles per CTA: every ring of the kernels wraps several times.  The
    # oracle's rows are those of one request; the others are its copies.
    rng = np.random.default_rng(D)
    H, tpb = 1, 64
    pool, scales, tables = cache(rng, np.array([seq + W]), H, D, tpb)
    tables = np.repeat(tables, B, 0)
    q, dq = make_q(rng, (1, W, H * G, D), "bf16", 0.3)
    r = kv.attend(q, pool, scales, tables[:1], [seq])
    for _ in range(3):
        out, lse = sv.attend_kv(dq.repeat(B, 1, 1, 1), dev(pool), dev(scales), i32(tables), i32([seq] * B), want_lse=True)
    for b in range(B):
        check(out[b:b + 1], lse[b:b + 1], r, "bf16", D, np.ones((1, W), bool), np.abs(np.nan_to_num(kv.decode(pool))).max() * scales.max())


@pytest.mark.gpu
@pytest.mark.parametrize("G,W", [(1, 1), (2, 1), (3, 2), (8, 1), (5, 3)])
@pytest.mark.parametrize("D", [64, 128])
def test_one_request_over_every_sm(G, W, D):
    # one KV head's keys spread over hundreds of CTAs: the join of many parts, by
    # as many warps per row as the row count leaves
    run_case(np.random.default_rng(G), [30011], [W], W, 1, G, D, 32, "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("G,W", [(1, 1), (4, 4), (4, 40)])
@pytest.mark.parametrize("col", [0, 3, 5])
def test_block_ids_out_of_range_in_the_prefix(G, W, col):
    # every id outside [0, num_blocks) reads NaN, whatever its value
    rng = np.random.default_rng(col)
    H, D, tpb, seq = 2, 64, 16, 100
    pool, scales, tables = cache(rng, np.full(7, seq + W), H, D, tpb)
    ids = np.array([-1, -2, -3, -2 ** 31, len(pool), 2 ** 31 - 1], np.int64)
    tables[1:, col] = ids
    q, dq = make_q(rng, (7, W, H * G, D), "bf16")
    out, lse = sv.attend_kv(dq, dev(pool), dev(scales), i32(tables), i32([seq] * 7), want_lse=True)
    for b in range(1, 7):
        assert torch.isnan(out[b]).all() and torch.isnan(lse[b]).all(), ids[b - 1]
    r = kv.attend(q, pool, scales, tables, [seq] * 7)
    rows = np.zeros((7, W), bool)
    rows[0] = True
    check(out, lse, r, "bf16", D, rows, np.nanmax(np.abs(kv.decode(pool[:, 1]))) * scales[:, 1].max())


def near(out, r, D, rows, vmax, least):
    """check's bound for bf16 outputs far from 1: vmax [..] is the largest
    p_t |v_t| over the largest p_t of the positions that a row sees, `least`
    half the least step of the values."""
    got, want = out.double().cpu().numpy()[rows], r["out"][rows]
    n, spread, amp = r["keys"][rows][..., None], r["spread"][rows][..., None], r["amp"][rows]
    tol = ((2 * (D + 8) * U * spread + 2.0 ** -11 + 2.0 ** -20 + 2 * n * U) * amp + n * 2.0 ** -32 * vmax
           + 2.0 ** -8 * np.abs(want) + least)
    assert np.isfinite(got).all()
    worst = (np.abs(got - want) / tol).max()
    assert worst <= 1, f"worst {worst:.3g} of the bound"


@pytest.mark.gpu
@pytest.mark.parametrize("B,G,W,D", [(1, 1, 1, 128), (900, 1, 2, 64), (1, 4, 40, 128), (200, 4, 40, 64)])
def test_values_at_the_top_of_the_types_range(B, G, W, D):
    # Thousands of alike keys: a sum of V that is not yet divided by the weights'
    # would pass the largest float.  One request is cut into many parts; of many
    # requests most lie in one CTA whole.
    rng = np.random.default_rng(B + W)
    H, tpb, seq = 1, 64, 3000
    pool, scales, tables = cache(rng, np.array([seq + W]), H, D, tpb, extra_cols=0)
    pool[:, 0] = kv.encode(rng.normal(0, 0.01, pool[:, 0].shape))
    pool[:, 1] = kv.encode(rng.uniform(200, 448, pool[:, 1].shape))
    scales[:, 0], scales[:, 1] = 1, 2.0 ** 119
    q, dq = make_q(rng, (1, W, H * G, D), "bf16")
    r = kv.attend(q, pool, scales, tables, [seq])
    out, lse = sv.attend_kv(dq.repeat(B, 1, 1, 1), dev(pool), dev(scales), i32(np.repeat(tables, B, 0)), i32([seq] * B),
                            want_lse=True)
    for b in range(0, B, 1 if B < 10 else 53):
        near(out[b:b + 1], r, D, np.ones((1, W), bool), 448 * 2.0 ** 119, 0)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()


@pytest.mark.gpu
@pytest.mark.parametrize("G,W", [(1, 4), (4, 4), (4, 40), (3, 130)])
@pytest.mark.parametrize("ratio", [16, 20, 30, 60, 110])
@pytest.mark.parametrize("prefix", [1, 25])
def test_unseen_values_take_no_bits(G, W, ratio, prefix):
    # the window's last token begins a block whose V scale is 2^ratio times the
    # others'; the tokens before it do not see it and are exact to their own values
    rng = np.random.default_rng(W + ratio)
    H, D, tpb = 2, 64, 16
    seq = 16 * (prefix + (W + 14) // 16) - (W - 1)
    pool, scales, tables = cache(rng, np.array([seq + W]), H, D, tpb)
    last = tables[0, (seq + W - 1) // tpb]
    seen = np.setdiff1d(tables[0, :(seq + W - 1) // tpb], last)
    vmax = np.nanmax(np.abs(kv.decode(pool[seen, 1]) * scales[seen, 1][..., None, None]))
    scales[last, 1] = 2.0 ** ratio * scales[seen, 1].max()
    q, dq = make_q(rng, (1, W, H * G, D), "bf16")
    r = kv.attend(q, pool, scales, tables, [seq])
    out, lse = sv.attend_kv(dq, dev(pool), dev(scales), i32(tables), i32([seq]), want_lse=True)
    rows = np.ones((1, W), bool)
    rows[0, -1] = False
    check(out, lse, r, "bf16", D, rows, vmax)
    near(out, r, D, ~rows, 448 * scales[last, 1].max(), 2.0 ** -25)


@pytest.mark.gpu
@pytest.mark.parametrize("G,W", [(1, 1), (4, 4), (4, 40)])
@pytest.mark.parametrize("where", [0, 5, 11])
def test_a_light_key_of_large_values(G, W, where):
    # one key weighs 2^-60 of the others and its V is 2^40 times theirs: what it
    # adds (2^-20) leaves the others' bits alone, wherever it stands
    rng = np.random.default_rng(where)
    H, D, tpb, seq = 1, 64, 16, 192
    pool, scales, tables = cache(rng, np.array([seq + W]), H, D, tpb)
    pool[:, 0] = kv.encode(0.0)
    pool[:, 1] = kv.encode(rng.uniform(0.5, 1.5, pool[:, 1].shape))
    blk = tables[0, where]
    pool[blk, 0] = kv.encode(-1.0)
    scales[:] = 1
    scales[blk, 1] = 2.0 ** 40
    q, dq = make_q(rng, (1, W, H * G, D), "bf16", 0)
    q[:], _ = 1.0, dq.fill_(1.0)
    scale = 60 * np.log(2) / D  # the block's scores are 60 below the others' in log2 units
    r = kv.attend(q, pool, scales, tables, [seq], scale=float(np.float32(scale)))
    out, lse = sv.attend_kv(dq, dev(pool), dev(scales), i32(tables), i32([seq]), scale=scale, want_lse=True)
    check(out, lse, r, "bf16", D, np.ones((1, W), bool), 1.5)


@pytest.mark.gpu
@pytest.mark.parametrize("G,W", [(1, 1), (4, 4), (4, 40)])
@pytest.mark.parametrize("exps", [(127,), (-130,), (-138,), (-126, -100), (100, -100, 0), (127, -149)])
def test_value_scales_over_all_of_fp32(G, W, exps):
    rng = np.random.default_rng(len(exps))
    H, D, tpb, seq = 2, 64, 16, 300
    pool, scales, tables = cache(rng, np.array([seq + W]), H, D, tpb)
    if max(exps) > 119:  # V of at most 1 times the largest scale
        pool[:, 1] = kv.encode(rng.uniform(-1, 1, pool[:, 1].shape))
    else:
        pool[:, 1] = kv.encode(rng.uniform(-448, 448, pool[:, 1].shape))
    scales[:, 1] = np.ldexp(np.float32(1), rng.choice(exps, scales[:, 1].shape)).astype(np.float32)
    if len(exps) == 1:
        scales[:, 1] *= np.float32(1.375)  # not a power of two
    q, dq = make_q(rng, (1, W, H * G, D), "bf16")
    r = kv.attend(q, pool, scales, tables, [seq])
    out, lse = sv.attend_kv(dq, dev(pool), dev(scales), i32(tables), i32([seq]), want_lse=True)
    x = np.abs(kv.decode(pool[:, 1]) * scales[:, 1].astype(np.float64)[..., None, None])
    near(out, r, D, np.ones((1, W), bool), np.nanmax(x), 2.0 ** -133)
    assert np.allclose(lse.cpu().numpy(), r["lse"], rtol=0, atol=1e-3)


@pytest.mark.gpu
@pytest.mark.parametrize("G,W", [(1, 1), (4, 4), (4, 40)])
def test_a_value_scale_of_zero(G, W):
    # codes times 0 are 0, in a block whose weights count all the same
    rng = np.random.default_rng(5)

    def edit(pool, scales, tables):
        scales[tables[0, 1:4], 1] = 0
        scales[tables[1], 1] = 0  # nothing but zeros
        pool[:, 1][(pool[:, 1] & 127) == 127] = 0
    out, lse = run_case(rng, [200, 70], [W, W], W, 2, G, 64, 16, "bf16", edit=edit)
    assert (out[1] == 0).all() and torch.isfinite(lse).all()


@pytest.mark.gpu
@pytest.mark.parametrize("G,W", [(1, 1), (4, 4), (4, 40)])
def test_scales_of_minus_zero(G, W):
    rng = np.random.default_rng(6)

    def edit(pool, scales, tables):
        scales[tables[0, 1:4]] = -0.0
        scales[tables[1]] = -0.0
        pool[(pool & 127) == 127] = 0
    out, lse = run_case(rng, [200, 70], [W, W], W, 2, G, 64, 16, "bf16", edit=edit)
    assert (out[1] == 0).all() and torch.isfinite(lse).all()


@pytest.mark.gpu
@pytest.mark.parametrize("G,W", [(1, 1), (4, 4), (4, 40)])
@pytest.mark.parametrize("exp", [4, 8, 12])
def test_scores_of_millions(G, W, exp):
    # scores up to 2^26, where fp32 hardly tells one from the next: a weighted mean of V all the same
    rng = np.random.default_rng(exp)
    H, D, tpb, seq = 2, 64, 16, 400
    pool, scales, tables = cache(rng, np.array([seq + W]), H, D, tpb)
    pool[:, 1] = kv.encode(rng.uniform(-1, 1, pool[:, 1].shape))
    scales[:, 1], scales[:, 0] = 1, 2.0 ** exp
    q, dq = make_q(rng, (1, W, H * G, D), "f16", 20.0)
    out, lse = sv.attend_kv(dq, dev(pool), dev(scales), i32(tables), i32([seq]), want_lse=True)
    r = kv.attend(q, pool, scales, tables, [seq])
    assert out.abs().max() <= 1
    assert (np.abs(lse.double().cpu().numpy() - r["lse"]) <= (D + 8) * U * r["spread"] + 100).all()


@pytest.mark.gpu
@pytest.mark.parametrize("tpb", [80, 256, 1024])
@pytest.mark.parametrize("G,W,D", [(4, 1, 128), (2, 7, 64), (8, 33, 128), (4, 70, 64)])
def test_large_and_odd_blocks(tpb, G, W, D):
    rng = np.random.default_rng(tpb + W)
    run_case(rng, [0, tpb - 1, 1500], [W, W, W // 2], W, 2, G, D, tpb, "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("B,G,W", [(1, 4, 1), (3, 4, 4), (1, 4, 40), (5, 2, 90)])
@pytest.mark.parametrize("fill", [0, 0x7f, 0xff])
def test_scratch_may_hold_anything(B, G, W, fill):
    rng = np.random.default_rng(B)
    H, D, tpb, seq = 2, 128, 16, [2000, 0, 77, 500, 1][:B]
    pool, scales, tables = cache(rng, np.array(seq) + W, H, D, tpb)
    _, dq = make_q(rng, (B, W, H * G, D), "bf16")
    a = [dq, dev(pool), dev(scales), i32(tables), i32(seq)]
    want, want_lse = sv.attend_kv(*a, want_lse=True)
    need = sv.lib().spec_attend_scratch_size(B, W, H * G, H, D)
    scratch = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
    for _ in range(2):  # also: what the call itself left there
        out, lse = sv.attend_kv(*a, want_lse=True, scratch=scratch)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.gpu
def test_stored_scales_of_a_pool_beyond_32_bits():
    H, D, tpb, W = 8, 128, 128, 4
    n = (1 << 32) // (2 * H * tpb * D) + 200
    rng = np.random.default_rng(12)
    small, scales, tables = cache(rng, np.array([510 + W]), H, D, tpb, spare=0, extra_cols=0)
    at = np.array([0, n - 1, n - 2, n - 150, n - 3])[:len(small)]
    where = torch.from_numpy(at).cuda()
    pool = torch.zeros((n, 2, H, tpb, D), dtype=torch.uint8, device="cuda")
    pool[where] = dev(small)
    big = torch.ones((n, 2, H), device="cuda")
    big[where] = dev(scales)
    k, dk = make_q(rng, (1, W, H, D), "bf16", 30.0)
    sv.store_kv(dk, dk, pool, big, i32(at[tables]), i32([510]))
    want, want_s = kv.store(k, k, small, scales, tables, [510])
    assert np.array_equal(pool[where].cpu().numpy(), want)
    assert np.array_equal(big[where].double().cpu().numpy(), want_s) and not np.array_equal(want_s, scales)
    others = torch.ones(n, dtype=torch.bool, device="cuda")
    others[where] = False
    assert (big[others] == 1).all()


@pytest.mark.gpu
def test_a_captured_step_of_tree_decoding():
    # every call of a step in one graph, replayed twice on the state of its start
    import oracle
    import workloads
    rng = np.random.default_rng(13)
    w = workloads.make("tree_b16_n60_l4_v151936_bf16", seed=4, B=4, V=4096)
    B, N = w["B"], w["N"]
    H, G, D, tpb = 2, 4, 64, 16
    seq = np.array([30, 0, 47, 100], np.int32)
    pool0, scales0, tables = cache(rng, seq, H, D, tpb, spare=40, extra_cols=5)
    n, held = len(pool0), (-(-seq // tpb)).astype(np.int32)
    pool0 &= 0x77  # no NaN codes
    free = np.full(n, -1, np.int32)
    spare = rng.permutation(np.setdiff1d(np.arange(n), tables))
    free[:len(spare)] = spare
    start = [pool0, scales0, tables, held, free, np.array([len(spare)], np.int32)]
    k, dk = make_q(rng, (B, N, H, D), "bf16")
    v, dv = make_q(rng, (B, N, H, D), "bf16")
    q, dq = make_q(rng, (B, N, H * G, D), "bf16")
    state = [dev(x) for x in start]
    pool, scales, dtab, dheld, dfree, count = state
    dseq, paths, tree = i32(seq), i32(w["paths"]), i32(w["tree_tokens"])
    logits = dev(w["target"].view(np.int16)).view(torch.bfloat16)
    ws = sv.Workspace()

    def step():
        slots, granted = sv.reserve_blocks(dseq, dtab, dheld, dfree, count, tpb, N)
        masks = sv.tree_masks(paths, N)
        sv.store_kv(dk, dv, pool, scales, dtab, dseq)
        out, lse = sv.attend_kv(dq, pool, scales, dtab, dseq, masks=masks, want_lse=True)
        _, acc, _, nodes = sv.verify_tree(logits, tree, paths, workspace=ws)
        sv.relocate_quantised_kv(pool, scales, dtab, dseq, nodes, acc)
        new, _, give = sv.rollback_paged(dseq, acc, N - 1, tpb, blocks_held=dheld)
        sv.release_blocks(dtab, dheld, give, dfree, count)
        return slots, granted, masks, out, lse, acc, nodes, new

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        slots, granted, masks, out, lse, acc, nodes, new = step()
    # the oracle's step
    slots_o, granted_o, t_o, h_o, c_o = kv.reserve(seq, None, tables, held, free, len(spare), tpb, N)
    m_o = kv.tree_masks(w["paths"].astype(np.int32), N)
    p_o, s_o = kv.store(k, v, pool0, scales0, t_o, seq)
    r = kv.attend(q, p_o, s_o, t_o, seq, masks=m_o)
    o = oracle.verify(w)
    p_o, s_o = kv.relocate(p_o, s_o, t_o, seq, o["accepted_nodes"], o["num_accepted"])
    len_o = seq + o["num_accepted"] + 1
    t_o, h_o, f_o, c_o = kv.release(t_o, h_o, np.maximum(0, h_o - -(-len_o // tpb)), free, c_o)
    for _ in range(2):
        for x, x0 in zip(state, start):
            x.copy_(dev(x0))
        for x in (slots, granted, masks, acc, nodes, new, out, lse):
            x.zero_()
        g.replay()
        torch.cuda.synchronize()
        for got, want in ((slots, slots_o), (granted, granted_o), (masks, m_o), (acc, o["num_accepted"]),
                          (nodes, o["accepted_nodes"]), (new, len_o), (pool, p_o), (scales, s_o), (dtab, t_o),
                          (dheld, h_o), (dfree, f_o), (count, [c_o])):
            assert np.array_equal(got.cpu().numpy(), want)
        check(out, lse, r, "bf16", D, np.ones((B, N), bool), 100)


@pytest.mark.gpu
@pytest.mark.parametrize("G,D", [(1, 64), (2, 128)])
def test_the_longest_window(G, D):
    # a prompt of 65536 tokens; a row of it is the row of a window of one behind its prefix
    rng = np.random.default_rng(D)
    H, tpb, W = 1, 64, 65536
    pool, scales, tables = cache(rng, np.array([W]), H, D, tpb)
    q, dq = make_q(rng, (1, W, H * G, D), "bf16")
    out, lse = sv.attend_kv(dq, dev(pool), dev(scales), i32(tables), i32([0]), want_lse=True)
    for i in (0, 1, 127, 128, 4095, 32768, 65534, 65535):
        r = kv.attend(q[:, i:i + 1], pool, scales, tables, [i])
        check(out[:, i:i + 1], lse[:, i:i + 1], r, "bf16", D, np.ones((1, 1), bool), 448 * scales.max())
    assert torch.isfinite(out).all()


@pytest.mark.gpu
@pytest.mark.parametrize("W,H,G,D", [(1, 1, 1, 64), (1, 1, 4, 128), (3, 1, 16, 64)])
def test_the_largest_batch(W, H, G, D):
    # 8192 requests of 0 to 60 positions over shared pages
    rng = np.random.default_rng(W)
    B, tpb = 8192, 16
    pool, scales, tables = cache(rng, np.array([60 + W]), H, D, tpb)
    seq = rng.integers(0, 61, B)
    _, dq = make_q(rng, (B, W, H * G, D), "f16")
    out, lse = sv.attend_kv(dq, dev(pool), dev(scales), i32(np.repeat(tables, B, 0)), i32(seq), want_lse=True)
    for b in [0, 1, B - 1] + list(rng.integers(0, B, 40)):
        r = kv.attend(dq[b:b + 1].double().cpu().numpy(), pool, scales, tables, seq[b:b + 1])
        check(out[b:b + 1], lse[b:b + 1], r, "f16", D, np.ones((1, W), bool), 448 * scales.max())


@pytest.mark.gpu
@pytest.mark.parametrize("W,H,G", [(1, 1024, 1), (1, 1024, 16), (2, 1024, 16)])
def test_the_most_heads(W, H, G):
    rng = np.random.default_rng(G)
    D, tpb, seq = 64, 16, [17, 3]
    pool, scales, tables = cache(rng, np.array(seq) + W, H, D, tpb)
    k, dk = make_q(rng, (2, W, H, D), "bf16")
    p, s = dev(pool), dev(scales)
    sv.store_kv(dk, dk, p, s, i32(tables), i32(seq))
    q, dq = make_q(rng, (2, W, H * G, D), "bf16")
    out, lse = sv.attend_kv(dq, p, s, i32(tables), i32(seq), want_lse=True)
    pool, scales = kv.store(k, k, pool, scales, tables, seq)
    assert np.array_equal(s.double().cpu().numpy(), scales)
    r = kv.attend(q, pool, scales, tables, seq)
    check(out, lse, r, "bf16", D, np.ones((2, W), bool), 448 * scales.max())


@pytest.mark.gpu
def test_the_widest_tree():
    rng = np.random.default_rng(1024)
    W, H, G, D, tpb = 1024, 1, 2, 64, 32
    paths = random_paths(rng, W, W, 33)[None]
    masks = kv.tree_masks(paths, W)
    run_case(rng, [70], [W], W, H, G, D, tpb, "bf16", masks=masks)
