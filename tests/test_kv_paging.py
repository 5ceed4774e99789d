"""Block reservation and release, and the tree's ancestor masks: oracle pins
on the CPU, the CUDA calls against the oracle on the GPU (whole numbers, so
every comparison is for equality)."""
import ctypes

import numpy as np
import pytest
import torch

import speculative_decoding_verification_row_gb300 as sv
from oracle import kv
from _kv import random_paths


# ------------------------------------------------------------------ oracle pins (CPU)
def test_hand_example():
    # tpb 4; request 0 holds 1 block for 3 tokens and adds 3: one more block;
    # request 1 is empty and adds 5: two blocks; request 2 still fits.
    tables = np.array([[7, -1, -1], [-1, -1, -1], [6, -1, -1]], np.int32)
    free = np.array([0, 1, 2, 3, 4, -9, -9, -9], np.int32)
    slots, granted, t, held, count = kv.reserve([3, 0, 2], [3, 5, 2], tables, np.array([1, 0, 1], np.int32), free, 5,
                                                4, 5)
    assert granted.tolist() == [3, 5, 2] and held.tolist() == [2, 2, 1] and count == 2
    assert t.tolist() == [[7, 4, -1], [3, 2, -1], [6, -1, -1]]
    assert slots.tolist() == [[31, 16, 17, -1, -1], [12, 13, 14, 15, 8], [26, 27, -1, -1, -1]]
    # rejecting everything gives the blocks back in the order they came off
    t2, h2, f2, c2 = kv.release(t, held, [1, 2, 0], free, count)
    assert np.array_equal(t2, tables) and h2.tolist() == [1, 0, 1] and np.array_equal(f2, free) and c2 == 5


def test_dry_stack_serves_a_prefix_of_the_requests():
    tables = np.full((4, 4), -1, np.int32)
    free = np.arange(8, dtype=np.int32)
    slots, granted, t, held, count = kv.reserve([0, 0, 0, 0], [4, 12, 4, 0], tables, np.zeros(4, np.int32), free, 3,
                                                4, 12)
    assert granted.tolist() == [4, -1, -1, 0] and count == 2  # 2 would fit, but 1 came first and did not
    assert (t[1:] == -1).all() and (slots[1:] == -1).all()


def test_masks_hand_example():
    # 0 -> 1 -> 3, 0 -> 2; node 4 on no path
    m = kv.tree_masks(np.array([[[0, 1, 3], [0, 2, -1], [-1, 4, 4]]], np.int32), 5)
    assert m[0, :, 0].tolist() == [1, 0b11, 0b101, 0b1011, 0]
    assert not kv.tree_masks(np.array([[[0, 1, 5], [0, 2, -1]]], np.int32), 5).any()


def test_refusals():
    lib, P = sv.lib(), ctypes.c_void_p
    f = P(16 * 1024)

    def reserve(**o):
        a = dict(seq=f, W=4, tpb=16, B=2, bt=f, cols=3, held=f, fb=f, n=8, fc=f, slots=f, g=f, **o) \
            if not o else {**dict(seq=f, W=4, tpb=16, B=2, bt=f, cols=3, held=f, fb=f, n=8, fc=f, slots=f, g=f), **o}
        return lib.spec_reserve_blocks(a["seq"], None, a["W"], a["tpb"], a["B"], a["bt"], a["cols"], a["held"],
                                       a["fb"], a["n"], a["fc"], a["slots"], a["g"], None)
    for bad in (dict(seq=None), dict(bt=None), dict(held=None), dict(fb=None), dict(fc=None), dict(g=None),
                dict(B=0), dict(B=8193), dict(W=0), dict(W=65537), dict(tpb=0), dict(cols=0), dict(n=0),
                dict(n=1 << 27, tpb=16)):
        assert reserve(**bad) == sv.SPEC_EINVAL, bad
    r = lib.spec_release_blocks
    assert r(None, 2, f, 3, f, f, 8, f, None) == sv.SPEC_EINVAL
    assert r(f, 0, f, 3, f, f, 8, f, None) == sv.SPEC_EINVAL
    m = lib.spec_tree_masks
    assert m(None, 1, 1, 2, 4, f, None) == sv.SPEC_EINVAL
    assert m(f, 1, 1, 65, 4, f, None) == sv.SPEC_EINVAL
    assert m(f, 1, 1, 2, 1025, f, None) == sv.SPEC_EINVAL
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        sv.reserve_blocks(i, i, i, i, i, 16, 4)
    with pytest.raises(ValueError):
        sv.tree_masks(torch.zeros((1, 2, 3), dtype=torch.int32), 3)


# ------------------------------------------------------------------ GPU parity
def _i32(a):
    return torch.from_numpy(np.array(a, dtype=np.int32)).cuda()


def _case(rng, B, W, tpb, hi, short):
    seq = rng.integers(0, hi + 1, B)
    win = rng.integers(0, W + 1, B)
    held = -(-seq // tpb)
    need = -(-(seq + win) // tpb) - held
    cols = int((held + need).max(initial=0)) + 2
    n = int((held + need).sum()) + 4
    perm = rng.permutation(n)
    tables = np.full((B, cols), -1, np.int32)
    at = 0
    for b in range(B):
        tables[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    free = np.full(n, -7, np.int32)
    spare = n - at if not short else int(need.sum() // 2)
    free[:spare] = perm[at:at + spare]
    return seq.astype(np.int32), win.astype(np.int32), tables, held.astype(np.int32), free, spare


@pytest.mark.gpu
@pytest.mark.parametrize("B,W,tpb,hi", [(1, 1, 16, 0), (3, 8, 1, 40), (64, 8, 32, 2048), (33, 61, 16, 100),
                                        (1025, 3, 16, 60), (2500, 2, 7, 40), (8192, 4, 16, 90), (2, 5000, 16, 9)])
@pytest.mark.parametrize("short", [False, True])
def test_reserve_and_release_match_the_oracle(B, W, tpb, hi, short):
    rng = np.random.default_rng(B + W)
    seq, win, tables, held, free, count = _case(rng, B, W, tpb, hi, short)
    if B > 30:  # entries out of range: served with nothing, left as they are
        seq[3], win[5], held[7], win[9], held[11] = -1, W + 1, -2, -1, tables.shape[1] + 1
        seq[13] = np.int32(2 ** 31 - 5)
    d = [_i32(x) for x in (seq, win, tables, held, free, [count])]
    slots, granted = sv.reserve_blocks(d[0], d[2], d[3], d[4], d[5], tpb, W, window_lens=d[1])
    want = kv.reserve(seq, win, tables, held, free, count, tpb, W)
    for name, got, ref in zip(("slots", "granted", "tables", "held", "count"), (slots, granted, d[2], d[3], d[5]), want):
        assert np.array_equal(got.cpu().numpy().reshape(np.shape(ref)), ref), name
    assert np.array_equal(d[4].cpu().numpy(), free)
    give = rng.integers(0, 3, B).astype(np.int32)
    give = np.minimum(give, np.maximum(want[3], 0)).astype(np.int32)
    if B > 30:
        give[1], give[2] = -1, want[3][2] + 1
    sv.release_blocks(d[2], d[3], _i32(give), d[4], d[5])
    ref = kv.release(want[2], want[3], give, free, want[4])
    for name, got, x in zip(("tables", "held", "free", "count"), (d[2], d[3], d[4], d[5]), ref):
        assert np.array_equal(got.cpu().numpy().reshape(np.shape(x)), x), name


@pytest.mark.gpu
def test_release_restores_and_refuses_an_overflow():
    rng = np.random.default_rng(5)
    seq, win, tables, held, free, count = _case(rng, 200, 40, 16, 300, False)
    d = [_i32(x) for x in (seq, win, tables, held, free, [count])]
    sv.reserve_blocks(d[0], d[2], d[3], d[4], d[5], 16, 40, window_lens=d[1], want_slots=False)
    sv.release_blocks(d[2], d[3], d[3] - _i32(held), d[4], d[5])
    for got, want in zip(d[2:], (tables, held, free, [count])):
        assert np.array_equal(got.cpu().numpy(), np.array(want))
    full = _i32([len(free) - 1])  # more would come back than the stack can hold
    sv.release_blocks(d[2], d[3], _i32(np.minimum(held, 2)), d[4], full)
    assert np.array_equal(d[2].cpu().numpy(), tables) and np.array_equal(d[3].cpu().numpy(), held)
    assert full.item() == len(free) - 1
    for bad in (-1, len(free) + 1):  # a count that cannot be: no block is taken
        fc = _i32([bad])
        _, granted = sv.reserve_blocks(d[0], d[2], d[3], d[4], fc, 16, 40, window_lens=d[1])
        need = -(-(seq + win) // 16) > held
        assert np.array_equal(granted.cpu().numpy(), np.where(need, -1, win)) and fc.item() == bad


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,P,L", [(1, 1, 1, 1), (2, 5, 3, 3), (16, 60, 60, 4), (3, 64, 40, 9), (2, 65, 65, 33),
                                     (2, 1000, 300, 64), (4, 1024, 17, 40)])
def test_tree_masks_match_the_oracle(B, N, P, L):
    rng = np.random.default_rng(N + L)
    paths = np.stack([random_paths(rng, N, P, L) for _ in range(B)])
    if P > 2:
        paths[0, 1, 0] = -1                       # an unused path
        paths[-1, 0, min(L - 1, 2):] = -1         # a path that ends early
        if B > 1 and L > 1:
            paths[1, 2, 0], paths[1, 2, 1] = 0, N  # a node that does not exist
    got = sv.tree_masks(_i32(paths), N)
    assert np.array_equal(got.cpu().numpy(), kv.tree_masks(paths, N))
