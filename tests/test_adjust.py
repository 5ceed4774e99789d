"""Penalties, biases and grammar masks on a window's logits: oracle pins and
refusals on the CPU, the CUDA call against the oracle on the GPU.

Tolerance.  A changed logit takes at most one product or quotient, f * c, two
subtractions and a sum with the bias, each rounded by at most 2^-24 of its
result, which is at most M = max(|x|, |x| r, |x| / r) + |f| c + |p| + |bias|;
the bias's own sum of n values adds n roundings of at most their magnitudes'
sum, one entry and none here but where a list repeats an id (its magnitudes are
in M then).  Then the type's rounding, eps / 2 of the value."""
import ctypes

import numpy as np
import pytest
import torch

import speculative_decoding_verification_row_gb300 as sv
from oracle import kv, window
from _kv import random_paths

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ CPU
def test_oracle_hand_example():
    x = np.array([[[2.0, -2.0, 1.0, 0.5], [2.0, -2.0, 1.0, 0.5]]])
    y = window.adjust(x, x, tokens=[[0, 1, 1]], prompt_lens=[1], repetition=[2.0], frequency=[0.25], presence=[1.0],
                      draft_tokens=[[2]], bias_ids=[[3, 3, -1]], bias_values=[[1.0, 2.0, 9.0]])
    # token 0 in the prompt: 2 / 2; token 1 twice in the output: -2 * 2 - 0.5 - 1; token 3: two biases
    assert y[0, 0].tolist() == [1.0, -5.5, 1.0, 3.5]
    # row 1 follows draft 2 as well: 1 / 2 - 0.25 - 1
    assert y[0, 1].tolist() == [1.0, -5.5, -0.75, 3.5]
    z = window.adjust(x, x, allowed=np.array([[0b0101]]), allowed_rows=np.array([[0, -1]]))
    assert z[0, 0].tolist() == [2.0, -np.inf, 1.0, -np.inf] and z[0, 1].tolist() == x[0, 1].tolist()
    assert np.isneginf(window.adjust(x, x, allowed=np.array([[15]]), allowed_rows=np.array([[1, 0]]))[0, 0]).all()


def test_oracle_tree_rows_count_their_ancestors():
    # 0 -> 1 -> 2 and 0 -> 3; node 0 is among the tokens already
    masks = kv.tree_masks(np.array([[[0, 1, 2], [0, 3, -1]]], np.int32), 4)
    x = np.zeros((1, 4, 8))
    y = window.adjust(x, x, tokens=[[5]], frequency=[1.0], draft_tokens=[[5, 6, 6, 7]], masks=masks)
    assert y[0, :, 5].tolist() == [-1] * 4
    assert y[0, :, 6].tolist() == [0, -1, -2, 0]
    assert y[0, :, 7].tolist() == [0, 0, 0, -1]


def _fake(**o):
    f = 16 * 1024
    big = 1 << 40
    a = dict(size=ctypes.sizeof(sv.AdjustParams), logits=f, out=f + big, dtype=sv.SPEC_F32, B=2, R=3, V=100, tokens=f,
             token_lens=f, prompt_lens=f, T=7, draft_tokens=f, masks=None, draft_lens=None, repetition=f, frequency=f,
             presence=f, bias_ids=f, bias_values=f, num_bias=4, allowed=f, allowed_rows=f, num_allowed=5)
    a.update(o)
    return sv.AdjustParams(*[a[n] for n, _ in sv.AdjustParams._fields_])


BAD = [dict(size=8), dict(logits=None), dict(out=None), dict(dtype=sv.SPEC_F16), dict(dtype=7), dict(B=0), dict(B=8193),
       dict(R=0), dict(R=1025), dict(V=1), dict(V=2**31 - 1), dict(logits=16 * 1024 + 2), dict(out=16 * 1024 + 64),
       dict(T=0), dict(T=1 << 30), dict(masks=16 * 1024, draft_tokens=None),
       dict(masks=16 * 1024, draft_lens=16 * 1024), dict(bias_values=None), dict(num_bias=0),
       dict(num_bias=sv.SPEC_MAX_BIAS + 1), dict(num_allowed=0), dict(allowed=None),
       dict(allowed_rows=None, num_allowed=5)]


@pytest.mark.parametrize("bad", BAD, ids=lambda b: ",".join(b))
def test_refusals_before_any_launch(bad):
    assert sv.lib().spec_adjust_logits(_fake(**bad), None) == sv.SPEC_EINVAL


def test_null_params_are_refused():
    assert sv.lib().spec_adjust_logits(None, None) == sv.SPEC_EINVAL
    with pytest.raises(ValueError):
        sv.adjust_logits(torch.zeros((1, 1, 8)))  # not on a GPU


def test_param_structs_match_the_header(tmp_path):
    import os
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "spec_verify.h"', "int main(void) {"]
    want = []
    for cname, py in (("spec_adjust_params", sv.AdjustParams), ("spec_rotate_params", sv.RotateParams),
                      ("spec_weigh_params", sv.WeighParams), ("spec_evict_params", sv.EvictParams)):
        lines.append(f'  printf("%zu\\n", sizeof({cname}));')
        want.append(ctypes.sizeof(py))
        for name, _ in py._fields_:
            lines.append(f'  printf("%zu\\n", offsetof({cname}, {name}));')
            want.append(getattr(py, name).offset)
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["  return 0;", "}"]))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", inc, str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == want


# ------------------------------------------------------------------ GPU
def _case(rng, B, R, V, T=40, tree=False, bias=5, grammars=3, drafts=True, wild=False):
    """Inputs as numpy arrays; tokens from a small set, so that lists overlap and repeat."""
    few = rng.integers(0, V, 12)
    few[:3] = 0, V - 1, min(V - 1, 4096)  # the ends, and a segment's first token

    def ids(shape):
        t = np.where(rng.random(shape) < 0.7, rng.choice(few, shape), rng.integers(0, V, shape))
        if wild:  # outside the vocabulary: ignored
            t = np.where(rng.random(shape) < 0.1, rng.choice([-1, V, V + 5, -2**31, 2**31 - 1], shape), t)
        return t.astype(np.int32)
    a = dict(logits=rng.normal(0, 3, (B, R, V)))
    a["tokens"] = ids((B, T)) if T else None
    if T:
        a["token_lens"] = rng.integers(0, T + 1, B).astype(np.int32)
        a["prompt_lens"] = rng.integers(0, T + 1, B).astype(np.int32)
        if wild:
            a["token_lens"][0], a["prompt_lens"][-1] = 2**31 - 1, -5
    a["repetition"], a["frequency"], a["presence"] = (rng.uniform(lo, hi, B).astype(np.float32)
                                                      for lo, hi in ((0.7, 1.6), (-0.5, 1), (-1, 1)))
    if drafts and tree:
        a["draft_tokens"] = ids((B, R))
        a["masks"] = kv.tree_masks(np.stack([random_paths(rng, R, R, min(R + 1, 9)) for _ in range(B)]), R)
    elif drafts and R > 1:
        a["draft_tokens"] = ids((B, R - 1))
    if bias:
        a["bias_ids"] = ids((B, bias))
        a["bias_ids"][:, bias // 2:][rng.random((B, bias - bias // 2)) < 0.3] = -1
        a["bias_values"] = rng.normal(0, 4, (B, bias)).astype(np.float32)
        a["bias_values"][rng.random((B, bias)) < 0.1] = -np.inf
    if grammars:
        a["allowed"] = rng.integers(-2**31, 2**31, (grammars, -(-V // 32))).astype(np.int32)
        a["allowed"][0] = -1
        a["allowed_rows"] = rng.integers(-1, grammars, (B, R)).astype(np.int32)
        if wild:
            a["allowed_rows"][0, 0], a["allowed_rows"][-1, -1] = grammars, -77
    return {k: v for k, v in a.items() if v is not None}


def _dev(a, dtype, at=0):
    """Tensors of a case; the logits `at` elements behind a 16-byte boundary."""
    d = {k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in a.items() if k != "logits"}
    d["logits"] = _placed(torch.from_numpy(a["logits"]).to(TYPES[dtype]).cuda(), at)
    return d


def _placed(x, at):
    buf = torch.empty(x.numel() + at, dtype=x.dtype, device="cuda")
    y = buf[at:].view(x.shape)
    y.copy_(x)
    return y


def _bound(a, stored, want, dtype):
    """The header's bound, [B, R, V]."""
    B, R, V = stored.shape
    x = np.abs(stored)
    r = a["repetition"][:, None, None].astype(np.float64) if "repetition" in a else 1.0
    M = np.maximum(x * r, x / r)
    T = (a["tokens"].shape[1] if "tokens" in a else 0) + (a["draft_tokens"].shape[1] if "draft_tokens" in a else 0)
    for k, times in (("frequency", T), ("presence", 1)):
        if k in a:
            M = M + times * np.abs(a[k].astype(np.float64))[:, None, None]
    n = 4
    if "bias_ids" in a:
        finite = np.where(np.isfinite(a["bias_values"]), np.abs(a["bias_values"]), 0).astype(np.float64)
        M = M + finite.sum(1)[:, None, None]
        n += a["bias_ids"].shape[1]
    half = torch.finfo(TYPES[dtype]).eps / 2 if dtype == "bf16" else 0.0
    return n * 2.0 ** -24 * M * (1 + half) + half * np.abs(np.where(np.isfinite(want), want, 0))


def check(a, dtype, at=(0, 0), inplace=False, **call):
    d = _dev(a, dtype, at[0])
    stored = d["logits"].double().cpu().numpy()
    mark = torch.full_like(d["logits"], 7.0) if not inplace else d["logits"]
    out = mark if inplace else _placed(mark, at[1])
    before = out.double().cpu().numpy()
    got = sv.adjust_logits(**{**d, **call}, out=out)
    assert got is out
    got = got.double().cpu().numpy()
    ref = {k: v for k, v in a.items() if k != "logits"}
    if "draft_lens" in call:
        ref["draft_lens"] = call["draft_lens"].cpu().numpy()
    with np.errstate(invalid="ignore"):
        want = window.adjust(stored, before, **ref)
        # what has to be equal: banned, NaN and untouched logits
        assert np.array_equal(np.isneginf(got), np.isneginf(want))
        assert np.array_equal(np.isnan(got), np.isnan(want))
        fine = np.isfinite(want)
        err = np.abs(got - want)[fine]
        assert (err <= _bound(a, np.where(np.isfinite(stored), stored, 0), want, dtype)[fine]).all(), err.max()
    return got, want


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,R,V,tree", [(1, 1, 2, False), (3, 1, 31, False), (2, 5, 1000, False), (2, 9, 4097, False),
                                        (1, 3, 8192, False), (2, 4, 12295, True), (1, 33, 4096, True),
                                        (5, 2, 257, False), (1, 70, 500, True)])
def test_adjust_matches_oracle(dtype, B, R, V, tree):
    a = _case(np.random.default_rng(V + R), B, R, V, tree=tree, wild=True)
    check(a, dtype)
    check(a, dtype, inplace=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("at", [(1, 1), (3, 3), (0, 1), (5, 2), (7, 7)])
def test_rows_that_begin_anywhere(dtype, at):
    a = _case(np.random.default_rng(3), 2, 5, 4099)
    check(a, dtype, at=at)
    check(a, dtype, at=(at[0], at[0]), inplace=True)


@pytest.mark.gpu
@pytest.mark.parametrize("leave", [("repetition",), ("frequency", "presence"), ("repetition", "frequency", "presence"),
                                   ("tokens", "token_lens", "prompt_lens"), ("draft_tokens",),
                                   ("bias_ids", "bias_values"), ("allowed", "allowed_rows"), ("prompt_lens",),
                                   ("token_lens",),
                                   ("tokens", "token_lens", "prompt_lens", "draft_tokens", "bias_ids", "bias_values",
                                    "allowed", "allowed_rows", "repetition", "frequency", "presence")])
def test_each_part_alone(leave):
    a = _case(np.random.default_rng(5), 3, 4, 2050)
    for k in leave:
        a.pop(k)
    check(a, "bf16")
    check(a, "bf16", inplace=True)


@pytest.mark.gpu
@pytest.mark.parametrize("inplace", [False, True])
def test_rows_behind_the_last_draft_are_left(inplace):
    a = _case(np.random.default_rng(7), 5, 4, 999)
    lens = np.array([0, 3, 1, -1, 4], np.int32)  # the last two: none of the rows
    got, want = check(a, "bf16", inplace=inplace, draft_lens=torch.from_numpy(lens).cuda())
    if not inplace:
        assert (got[0, 1:] == 7).all() and (got[3:] == 7).all()


@pytest.mark.gpu
def test_masks_for_each_row_and_banned_nan():
    a = _case(np.random.default_rng(9), 2, 3, 300, bias=0)
    a["logits"][0, 0, 5], a["logits"][1, 2, 6], a["logits"][0, 1, 7] = np.nan, np.inf, -np.inf
    a["allowed"] = np.random.default_rng(1).integers(-2**31, 2**31, (6, 10)).astype(np.int32)
    for row, t in ((0, 5), (5, 6)):
        a["allowed"][row, 0] &= ~(1 << t)
    a.pop("allowed_rows")
    got, _ = check(a, "f32")
    assert np.isneginf(got[0, 0, 5]) and np.isneginf(got[1, 2, 6]) and np.isneginf(got[0, 1, 7])
    d = _dev(a, "f32")
    d["allowed"] = d["allowed"].view(2, 3, 10)  # one mask per row, in the rows' shape
    assert np.array_equal(sv.adjust_logits(**d).double().cpu().numpy(), got, equal_nan=True)


@pytest.mark.gpu
def test_a_draft_counts_as_often_as_it_stands_in_the_window():
    V, k = 5000, 64
    x = torch.zeros((1, k + 1, V), device="cuda")
    y = sv.adjust_logits(x, draft_tokens=torch.full((1, k), 4500, dtype=torch.int32, device="cuda"),
                         frequency=torch.ones(1, device="cuda"))
    assert y[0, :, 4500].tolist() == [-float(i) for i in range(k + 1)]
    y[0, :, 4500] = 0
    assert not y.any()
    tree = torch.full((1, 1024), -1, dtype=torch.int32, device="cuda")  # every bit: all nodes precede all
    y = sv.adjust_logits(torch.zeros((1, 1024, 64), device="cuda"), frequency=torch.ones(1, device="cuda"),
                         draft_tokens=torch.full((1, 1024), 63, dtype=torch.int32, device="cuda"),
                         masks=tree.view(1, 1024, 1).expand(1, 1024, 32).contiguous())
    assert (y[0, :, 63] == -1023).all()


@pytest.mark.gpu
def test_longest_lists():
    rng = np.random.default_rng(11)
    a = _case(rng, 2, 2, 3000, T=60000, bias=sv.SPEC_MAX_BIAS)
    check(a, "f32")


@pytest.mark.gpu
def test_offsets_past_32_bits():
    V, R, B = 151936, 60, 260  # 2.37e9 elements, 4.7 GB of bfloat16
    x = torch.zeros((B, R, V), dtype=torch.bfloat16, device="cuda")
    ids = torch.full((B, 1), V - 1, dtype=torch.int32, device="cuda")
    y = sv.adjust_logits(x, bias_ids=ids, bias_values=torch.arange(B, dtype=torch.float32, device="cuda")[:, None])
    assert torch.equal(y[:, :, V - 1].float(), torch.arange(B, device="cuda").bfloat16().float()[:, None].expand(B, R))
    assert not y[:, :, :V - 1].any()
    del y
    sv.adjust_logits(x, bias_ids=ids, bias_values=torch.ones((B, 1), device="cuda"), out=x)
    assert (x[:, :, V - 1] == 1).all() and float(x.sum(dtype=torch.float64)) == B * R


@pytest.mark.gpu
def test_verify_of_penalised_rows_is_the_oracles_choice():
    """Greedy verify over adjusted logits: row i counts the drafts before it."""
    V, k = 700, 3
    x = torch.zeros((1, k + 1, V), device="cuda")
    x[0, :, 10], x[0, :, 20] = 4.0, 3.5
    draft = torch.tensor([[10, 20, 10]], dtype=torch.int32, device="cuda")
    adj = sv.adjust_logits(x, draft_tokens=draft, frequency=torch.ones(1, device="cuda"))
    # 10 (4.0 > 3.5); then 20 (3.0 < 3.5); then 10 (3.0 > 2.5); then 20 (2.0 < 2.5)
    tok, n = sv.verify_greedy(adj, draft)
    assert n.item() == 3 and tok[0].tolist() == [10, 20, 10, 20]
    assert sv.verify_greedy(x, draft)[1].item() == 1


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sampling_verifies_of_penalised_and_masked_rows(dtype):
    """Rows whose adjusted distribution is one token but for e^-20: chain and tree verify by sampling choose it."""
    V, k = 700, 3
    x = torch.full((2, k + 1, V), -1000.0, dtype=TYPES[dtype], device="cuda")
    for t, v in ((10, 0.0), (20, -20.0), (30, -40.0), (40, -60.0)):  # each is next once those before it stand in the output
        x[:, :, t] = v
    draft = torch.tensor([[10, 20, 30]] * 2, dtype=torch.int32, device="cuda")
    q = torch.full((2, k, V), -1000.0, dtype=TYPES[dtype], device="cuda")
    q.scatter_(2, draft.long()[..., None], 0.0)
    u = torch.full((2, k + 1), 0.5, device="cuda")
    allowed = torch.zeros((1, -(-V // 32)), dtype=torch.int32, device="cuda")
    allowed[0, 0] = 1 << 5
    rows = torch.full((2, k + 1), -1, dtype=torch.int32, device="cuda")
    rows[1, 1] = 0  # behind 10 the second request's grammar has token 5 alone
    adj = sv.adjust_logits(x, draft_tokens=draft, frequency=torch.full((2,), 100.0, device="cuda"), allowed=allowed, allowed_rows=rows)
    tok, n, _ = sv.verify_chain(adj, q, draft, u, 1.0)
    assert n.tolist() == [3, 1] and tok[0].tolist() == [10, 20, 30, 40] and tok[1].tolist() == [10, 5, -1, -1]
    assert sv.verify_chain(x, q, draft, u, 1.0)[1].tolist() == [1, 1]
    # 0 -> 1 (10) -> 2 (20) -> 4 (30), and 1 -> 3 (10 again)
    paths = torch.tensor([[[0, 1, 2, 4], [0, 1, 3, -1]]], dtype=torch.int32, device="cuda")
    tree = torch.tensor([[0, 10, 20, 10, 30]], dtype=torch.int32, device="cuda")
    y = x[:1, :1].expand(1, 5, V).contiguous()
    u = torch.full((1, 5), 0.5, device="cuda")
    adj = sv.adjust_logits(y, draft_tokens=tree, masks=sv.tree_masks(paths, 5), frequency=torch.full((1,), 100.0, device="cuda"))
    tok, n, _, nodes = sv.verify_tree_sampled(adj, tree, paths, u, 1.0)
    assert n.tolist() == [3] and nodes[0].tolist() == [0, 1, 2, 4] and tok[0].tolist() == [10, 20, 30, 40]
    assert sv.verify_tree_sampled(y, tree, paths, u, 1.0)[3][0, :3].tolist() == [0, 1, 3]


@pytest.mark.gpu
def test_two_streams_and_a_captured_call():
    rng = np.random.default_rng(13)
    a, b = _case(rng, 4, 4, 20000), _case(rng, 4, 4, 20000)
    da, db = _dev(a, "bf16"), _dev(b, "bf16")
    want = sv.adjust_logits(**da).clone(), sv.adjust_logits(**db).clone()
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [sv.adjust_logits(**d, stream=st) for d, st in zip((da, db), s)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    out = torch.zeros_like(da["logits"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.adjust_logits(**da, out=out)
    for x, w in ((da, want[0]), (db, want[1])):
        for key in da:
            if key != "out" and key in x:
                da[key].copy_(x[key])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)


@pytest.mark.gpu
def test_binding_refusals():
    x = torch.zeros((2, 3, 64), device="cuda")
    i = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    one = torch.ones(2, device="cuda")
    for bad in (dict(token_lens=i[:, 0]), dict(prompt_lens=i[:, 0]), dict(masks=torch.zeros((2, 3, 1), dtype=torch.int32, device="cuda")),
                dict(draft_tokens=i, masks=torch.zeros((2, 3, 1), dtype=torch.int32, device="cuda")),
                dict(draft_tokens=torch.zeros((2, 3), dtype=torch.int32, device="cuda")),
                dict(bias_ids=i), dict(bias_values=torch.zeros((2, 2), device="cuda")), dict(allowed_rows=i),
                dict(allowed=torch.zeros((2, 2), dtype=torch.int32, device="cuda")),
                dict(allowed=torch.zeros((5, 3), dtype=torch.int32, device="cuda"),
                     allowed_rows=torch.zeros((2, 3), dtype=torch.int32, device="cuda")),
                dict(repetition=torch.ones(3, device="cuda")), dict(frequency=one.double()),
                dict(presence=one.cpu()), dict(tokens=i.long()), dict(out=x.bfloat16()), dict(out=x[:, :2]),
                dict(draft_lens=i)):
        with pytest.raises(ValueError):
            sv.adjust_logits(x, **bad)
    for bad in (x[0], x.half(), x.transpose(1, 2)):
        with pytest.raises(ValueError):
            sv.adjust_logits(bad)
    with pytest.raises(sv.SpecError):
        sv.adjust_logits(torch.zeros((1, 1, 1), device="cuda"))
    flat = torch.zeros(2 * 3 * 64 + 8, device="cuda")
    with pytest.raises(sv.SpecError):  # overlapping, not in place
        sv.adjust_logits(flat[:384].view(2, 3, 64), out=flat[8:].view(2, 3, 64))
    none = torch.zeros((2, 0), dtype=torch.int32, device="cuda")
    y = sv.adjust_logits(x + 1, tokens=none, bias_ids=none, bias_values=none.float(), frequency=one)
    assert (y == 1).all()
