"""GB300-native speculative-decoding verification row.

A thin ctypes binding over ``libspecverify.so`` (C ABI in
``include/spec_verify.h``).  The functions here only check and marshal
arguments: every step of verification runs in the library's CUDA kernels.
PyTorch supplies device memory and the current stream.  If the library has
not been built the first call raises; there is no CPU fallback.

Calls (same names as the C ABI):
  verify_chain     chain rejection-sampling verify (vLLM anatomy page,
                   "Speculative Decoding")
  verify_greedy    greedy chain verify (Kestrel article 32, section 3.3)
  verify_tree      greedy EAGLE tree verify (TensorRT-LLM deployment page,
                   "Eagle-2" section)
  rollback_lengths KV cursor rollback (TensorRT-LLM walkthrough,
                   update_requests / rewind_cache)

The paged 8-bit KV cache a step runs on:
  reserve_blocks / release_blocks  blocks for the windows, block tables and
                   slot maps, and the blocks given back
  tree_masks       ancestor masks of a tree's nodes, from its paths
  store_kv         a window's K and V rows into the cache
  attend_kv        attention of the window's rows over the cache
  relocate_quantised_kv  the accepted nodes' rows behind the prefix

Around them:
  adjust_logits    penalties, biases and grammar masks on a window's logits
  rotate_qk        rotary positions of a window's queries and keys;
                   rotary_frequencies gives the angles per position
  rotate_store_kv  the same, keys and values going into the cache
  weigh_kv         the attention each cached position drew from a window
  evict_kv         the positions of least weight dropped from the cache
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import threading

import torch

from .rotary import rotary_frequencies  # noqa: F401  (host arithmetic)
from .stats import acceptance_stats, anchored_emitted  # noqa: F401  (host bookkeeping)

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libspecverify.so")

SPEC_OK, SPEC_EINVAL, SPEC_EBADINDEX, SPEC_ECUDA, SPEC_EWORKSPACE, SPEC_ETIMEOUT = 0, -1, -2, -3, -4, -5
SPEC_ELIMIT = -6
SPEC_F32, SPEC_BF16, SPEC_F16 = 0, 1, 2
SPEC_MAX_DRAFT = 64
SPEC_MAX_BATCH = 8192
SPEC_MAX_TREE_NODES = 1024
SPEC_MAX_PATH_LEN = 64
SPEC_MAX_TOPK = 256
SPEC_MAX_WINDOW = 65536
SPEC_MAX_BIAS = 1024

# Every entry point the header declares.
SYMBOLS = ("spec_workspace_size", "spec_workspace_init", "spec_verify_chain",
           "spec_verify_greedy", "spec_verify_tree", "spec_rollback_lengths",
           "spec_last_error", "spec_status_string", "spec_verify_chain_noalloc",
           "spec_relocate_accepted_kv", "spec_verify_chain_philox", "spec_philox_uniforms",
           "spec_verify_chain_ex", "spec_verify_greedy_ex", "spec_rollback_paged",
           "spec_workspace_size_filtered", "spec_test_timeout_chain", "spec_test_timeout_greedy",
           "spec_verify_tree_sampled", "spec_reserve_blocks", "spec_release_blocks", "spec_tree_masks",
           "spec_store_kv", "spec_attend_kv", "spec_attend_scratch_size", "spec_relocate_quantised_kv",
           "spec_adjust_logits", "spec_rotate_qk", "spec_rotate_store_kv", "spec_rotate_store_scratch_size",
           "spec_weigh_kv", "spec_weigh_scratch_size",
           "spec_evict_kv", "spec_evict_scratch_size")
SPEC_NOALLOC_SCRATCH_BYTES = 4 << 20

class ChainParams(ctypes.Structure):
    """spec_chain_params (include/spec_verify.h), field for field."""
    _fields_ = [("size", ctypes.c_size_t), ("target_logits", ctypes.c_void_p),
                ("draft_logits", ctypes.c_void_p), ("dtype", ctypes.c_int),
                ("draft_tokens", ctypes.c_void_p), ("draft_lens", ctypes.c_void_p),
                ("uniforms", ctypes.c_void_p), ("seeds", ctypes.c_void_p),
                ("offsets", ctypes.c_void_p), ("temperature", ctypes.c_float),
                ("B", ctypes.c_int), ("k", ctypes.c_int), ("V", ctypes.c_int),
                ("out_tokens", ctypes.c_void_p), ("out_num_accepted", ctypes.c_void_p),
                ("out_probs", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("top_k", ctypes.c_int), ("top_p", ctypes.c_float), ("min_p", ctypes.c_float)]


class GreedyParams(ctypes.Structure):
    """spec_greedy_params (include/spec_verify.h), field for field."""
    _fields_ = [("size", ctypes.c_size_t), ("target_logits", ctypes.c_void_p),
                ("dtype", ctypes.c_int), ("draft_tokens", ctypes.c_void_p),
                ("draft_lens", ctypes.c_void_p), ("B", ctypes.c_int), ("k", ctypes.c_int),
                ("V", ctypes.c_int), ("out_tokens", ctypes.c_void_p),
                ("out_num_accepted", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p)]


class KvCache(ctypes.Structure):
    """spec_kv_cache (include/spec_verify.h), field for field."""
    _fields_ = [("size", ctypes.c_size_t), ("pool", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("block_tables", ctypes.c_void_p), ("num_blocks", ctypes.c_int),
                ("max_blocks", ctypes.c_int), ("tokens_per_block", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int)]


class AttendParams(ctypes.Structure):
    """spec_attend_params (include/spec_verify.h), field for field."""
    _fields_ = [("size", ctypes.c_size_t), ("q", ctypes.c_void_p), ("q_strides", ctypes.c_int64 * 3),
                ("dtype", ctypes.c_int), ("B", ctypes.c_int), ("W", ctypes.c_int),
                ("q_heads", ctypes.c_int), ("seq_lens", ctypes.c_void_p),
                ("window_lens", ctypes.c_void_p), ("masks", ctypes.c_void_p),
                ("scale", ctypes.c_float), ("out", ctypes.c_void_p), ("out_lse", ctypes.c_void_p)]


class AdjustParams(ctypes.Structure):
    """spec_adjust_params (include/spec_verify.h), field for field."""
    _fields_ = [("size", ctypes.c_size_t), ("logits", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("dtype", ctypes.c_int), ("B", ctypes.c_int), ("R", ctypes.c_int), ("V", ctypes.c_int),
                ("tokens", ctypes.c_void_p), ("token_lens", ctypes.c_void_p), ("prompt_lens", ctypes.c_void_p),
                ("T", ctypes.c_int), ("draft_tokens", ctypes.c_void_p), ("masks", ctypes.c_void_p),
                ("draft_lens", ctypes.c_void_p), ("repetition", ctypes.c_void_p), ("frequency", ctypes.c_void_p),
                ("presence", ctypes.c_void_p), ("bias_ids", ctypes.c_void_p), ("bias_values", ctypes.c_void_p),
                ("num_bias", ctypes.c_int), ("allowed", ctypes.c_void_p), ("allowed_rows", ctypes.c_void_p),
                ("num_allowed", ctypes.c_int)]


class RotateParams(ctypes.Structure):
    """spec_rotate_params (include/spec_verify.h), field for field."""
    _fields_ = [("size", ctypes.c_size_t), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
                ("out_q", ctypes.c_void_p), ("out_k", ctypes.c_void_p), ("q_strides", ctypes.c_int64 * 3),
                ("k_strides", ctypes.c_int64 * 3), ("out_q_strides", ctypes.c_int64 * 3),
                ("out_k_strides", ctypes.c_int64 * 3), ("dtype", ctypes.c_int), ("B", ctypes.c_int),
                ("W", ctypes.c_int), ("q_heads", ctypes.c_int), ("k_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("starts", ctypes.c_void_p), ("window_lens", ctypes.c_void_p),
                ("masks", ctypes.c_void_p), ("inv_freq", ctypes.c_void_p), ("pairs", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("gain", ctypes.c_float)]


class WeighParams(ctypes.Structure):
    """spec_weigh_params (include/spec_verify.h), field for field."""
    _fields_ = [("size", ctypes.c_size_t), ("q", ctypes.c_void_p), ("q_strides", ctypes.c_int64 * 3),
                ("dtype", ctypes.c_int), ("B", ctypes.c_int), ("W", ctypes.c_int), ("q_heads", ctypes.c_int),
                ("seq_lens", ctypes.c_void_p), ("window_lens", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("scale", ctypes.c_float), ("weights", ctypes.c_void_p), ("decay", ctypes.c_float),
                ("out", ctypes.c_void_p), ("T", ctypes.c_int)]


class EvictParams(ctypes.Structure):
    """spec_evict_params (include/spec_verify.h), field for field."""
    _fields_ = [("size", ctypes.c_size_t), ("weights", ctypes.c_void_p), ("T", ctypes.c_int), ("B", ctypes.c_int),
                ("seq_lens", ctypes.c_void_p), ("keep", ctypes.c_int), ("first", ctypes.c_int),
                ("recent", ctypes.c_int), ("new_lens", ctypes.c_void_p), ("kept", ctypes.c_void_p),
                ("out_weights", ctypes.c_void_p), ("T_out", ctypes.c_int), ("blocks_held", ctypes.c_void_p),
                ("free_blocks", ctypes.c_void_p)]


_lock = threading.Lock()
_lib = None


class SpecError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        super().__init__(f"{fn} failed: {status_string(code)} ({code})")


def _bind(lib):
    P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.spec_workspace_size.argtypes = [I, I, I]
    lib.spec_workspace_size.restype = S
    lib.spec_workspace_init.argtypes = [P, S, P]
    lib.spec_workspace_size_filtered.argtypes = [I, I, I, I]
    lib.spec_workspace_size_filtered.restype = S
    lib.spec_verify_chain.argtypes = [P, P, I, P, P, ctypes.c_float, I, I, I, P, P, P, P, P, S, P]
    lib.spec_verify_greedy.argtypes = [P, I, P, I, I, I, P, P, P, P, S, P]
    lib.spec_verify_tree.argtypes = [P, I, P, P, I, I, I, I, I, P, P, P, P, P, P, S, P]
    lib.spec_verify_tree_sampled.argtypes = [P, I, P, P, P, ctypes.c_float, I, I, I, I, I, P, P, P, P, P,
                                             P, S, P]
    lib.spec_rollback_lengths.argtypes = [P, P, I, I, P, P, P]
    lib.spec_verify_chain_noalloc.argtypes = [P, P, I, P, P, ctypes.c_float, I, I, I, P, P, P, P, P]
    lib.spec_last_error.argtypes = [P, S, P, ctypes.POINTER(ctypes.c_int)]
    lib.spec_relocate_accepted_kv.argtypes = [P, S, I, I, P, I, P, P, P, I, I, P]
    lib.spec_verify_chain_philox.argtypes = [P, P, I, P, P, P, ctypes.c_float, I, I, I, P, P, P, P, P, S, P]
    lib.spec_philox_uniforms.argtypes = [P, P, I, I, P, P]
    lib.spec_verify_chain_ex.argtypes = [ctypes.POINTER(ChainParams), P, S, P]
    lib.spec_verify_greedy_ex.argtypes = [ctypes.POINTER(GreedyParams), P, S, P]
    lib.spec_rollback_paged.argtypes = [P, P, P, I, P, I, I, P, P, P, P]
    lib.spec_test_timeout_chain.argtypes = [ctypes.POINTER(ChainParams), ctypes.c_longlong, P, S, P]
    lib.spec_test_timeout_greedy.argtypes = [ctypes.POINTER(GreedyParams), ctypes.c_longlong, P, S, P]
    lib.spec_reserve_blocks.argtypes = [P, P, I, I, I, P, I, P, P, I, P, P, P, P]
    lib.spec_release_blocks.argtypes = [P, I, P, I, P, P, I, P, P]
    lib.spec_tree_masks.argtypes = [P, I, I, I, I, P, P]
    S3 = ctypes.POINTER(ctypes.c_int64)
    lib.spec_store_kv.argtypes = [ctypes.POINTER(KvCache), P, S3, P, S3, I, P, P, I, I, P]
    lib.spec_attend_kv.argtypes = [ctypes.POINTER(KvCache), ctypes.POINTER(AttendParams), P, S, P]
    lib.spec_attend_scratch_size.argtypes = [I, I, I, I, I]
    lib.spec_attend_scratch_size.restype = S
    lib.spec_relocate_quantised_kv.argtypes = [ctypes.POINTER(KvCache), P, P, P, I, I, P]
    lib.spec_adjust_logits.argtypes = [ctypes.POINTER(AdjustParams), P]
    lib.spec_rotate_qk.argtypes = [ctypes.POINTER(RotateParams), P]
    lib.spec_rotate_store_kv.argtypes = [ctypes.POINTER(KvCache), ctypes.POINTER(RotateParams), P, S3, P, P, S, P]
    lib.spec_rotate_store_scratch_size.argtypes = [I, I, I, I, I]
    lib.spec_rotate_store_scratch_size.restype = S
    lib.spec_weigh_kv.argtypes = [ctypes.POINTER(KvCache), ctypes.POINTER(WeighParams), P, S, P]
    lib.spec_weigh_scratch_size.argtypes = [I, I, I, I, I]
    lib.spec_weigh_scratch_size.restype = S
    lib.spec_evict_kv.argtypes = [ctypes.POINTER(KvCache), ctypes.POINTER(EvictParams), P, S, P]
    lib.spec_evict_scratch_size.argtypes = [I, I, I, I]
    lib.spec_evict_scratch_size.restype = S
    lib.spec_status_string.argtypes = [I]
    lib.spec_status_string.restype = ctypes.c_char_p
    for f in ("spec_workspace_init", "spec_verify_chain", "spec_verify_greedy", "spec_verify_tree",
              "spec_rollback_lengths", "spec_last_error", "spec_verify_chain_noalloc",
              "spec_relocate_accepted_kv", "spec_verify_chain_philox", "spec_philox_uniforms",
              "spec_verify_chain_ex", "spec_verify_greedy_ex", "spec_rollback_paged",
              "spec_test_timeout_chain", "spec_test_timeout_greedy", "spec_verify_tree_sampled",
              "spec_reserve_blocks", "spec_release_blocks", "spec_tree_masks", "spec_store_kv",
              "spec_attend_kv", "spec_relocate_quantised_kv", "spec_adjust_logits", "spec_rotate_qk",
              "spec_rotate_store_kv", "spec_weigh_kv", "spec_evict_kv"):
        getattr(lib, f).restype = I
    return lib


def lib():
    """The loaded C library; raises if it has not been built."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise RuntimeError(
                        f"{LIB_PATH} is missing: build it with `python -c \"import __graft_entry__ as g; g.build()\"`")
                _lib = _bind(ctypes.CDLL(LIB_PATH))
    return _lib


def status_string(code: int) -> str:
    return lib().spec_status_string(int(code)).decode()


# ---------------------------------------------------------------- marshalling helpers
def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _on(device):
    """The C calls run on the current device: make the arrays' device current
    for the duration of a call."""
    return torch.cuda.device(device)


def _stream_handle(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream), stream
    return ctypes.c_void_p(int(stream)), None


def _dev(t: torch.Tensor, name: str, dtype=None, shape=None) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _logit_code(t: torch.Tensor, name: str) -> int:
    if t.dtype == torch.bfloat16:
        return SPEC_BF16
    if t.dtype == torch.float32:
        return SPEC_F32
    raise ValueError(f"{name} must be bfloat16 or float32, got {t.dtype}")


def _out(t, name, shape, dtype, device):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return _dev(t, name, dtype, shape)


class Workspace:
    """Device scratch for verify calls on one stream (grown on demand).

    A workspace must not be shared by calls that may overlap on the GPU."""

    def __init__(self, device=None):
        self.device = torch.device(device if device is not None else "cuda")
        self.buf = None

    def ensure(self, B: int, rows: int, V: int, stream_handle, need: int | None = None) -> torch.Tensor:
        """Grow to spec_workspace_size(B, rows, V) bytes, or to `need` bytes."""
        if need is None:
            need = lib().spec_workspace_size(B, rows, V)
        if need == 0:
            raise SpecError("spec_workspace_size", SPEC_EINVAL)
        if self.buf is None or self.buf.numel() < need:
            self.buf = torch.empty(need, dtype=torch.uint8, device=self.device)
            with _on(self.buf.device):
                rc = lib().spec_workspace_init(_ptr(self.buf), self.buf.numel(), stream_handle)
            if rc != SPEC_OK:
                raise SpecError("spec_workspace_init", rc)
        return self.buf

    @property
    def nbytes(self) -> int:
        return 0 if self.buf is None else self.buf.numel()


_default_ws: dict = {}


def default_workspace(device, stream_handle) -> Workspace:
    key = (torch.device(device).index, int(stream_handle.value or 0))
    ws = _default_ws.get(key)
    if ws is None:
        ws = _default_ws[key] = Workspace(device)
    return ws


# ---------------------------------------------------------------- calls
def verify_chain(target_logits, draft_logits, draft_tokens, uniforms, temperature: float, *,
                 out_tokens=None, out_num_accepted=None, out_probs=None, want_probs=False,
                 seq_lens=None, workspace: Workspace | None = None, stream=None,
                 seeds=None, offsets=None, draft_lens=None, top_k: int = 0, top_p: float = 1.0,
                 min_p: float = 0.0):
    """Chain rejection-sampling verify; returns (tokens [B,k+1], num_accepted [B], probs [B,k,2] or None).

    seq_lens (int32 [B], optional) is advanced in place by n_acc + 1.  With
    uniforms=None, seeds and offsets (int64 [B]) select each request's Philox
    stream and the uniforms are drawn inside the kernel.  draft_lens (int32
    [B], optional): each request's real draft length (ragged verify).
    top_k > 0, top_p < 1 or min_p > 0: verify on the top-k / top-p / min_p
    filtered target and draft distributions (spec_chain_params.top_k /
    top_p / min_p; top_k = 0 ranks no top-k set)."""
    t = _dev(target_logits, "target_logits")
    if t.dim() != 3:
        raise ValueError("target_logits must be [B, k+1, V]")
    B, k1, V = t.shape
    k = k1 - 1
    code = _logit_code(t, "target_logits")
    d = _dev(draft_logits, "draft_logits", t.dtype, (B, k, V))
    x = _dev(draft_tokens, "draft_tokens", torch.int32, (B, k))
    if uniforms is not None:
        u = _dev(uniforms, "uniforms", torch.float32, (B, k + 1))
    else:
        sd = _dev(seeds, "seeds", torch.int64, (B,))
        of = _dev(offsets, "offsets", torch.int64, (B,))
    dev = t.device
    tok = _out(out_tokens, "out_tokens", (B, k + 1), torch.int32, dev)
    n = _out(out_num_accepted, "out_num_accepted", (B,), torch.int32, dev)
    probs = None
    if out_probs is not None or want_probs:
        probs = _out(out_probs, "out_probs", (B, k, 2), torch.float32, dev)
    if seq_lens is not None:
        _dev(seq_lens, "seq_lens", torch.int32, (B,))
    sh, _ = _stream_handle(stream, dev)
    ws = workspace or default_workspace(dev, sh)
    filtered = top_k != 0 or top_p != 1.0 or min_p != 0.0
    need = lib().spec_workspace_size_filtered(B, k, V, int(top_k)) if filtered else None
    buf = ws.ensure(B, 2 * k + 1, V, sh, need)
    if draft_lens is not None or filtered:
        lens = None if draft_lens is None else _dev(draft_lens, "draft_lens", torch.int32, (B,))
        prm = ChainParams(ctypes.sizeof(ChainParams), _ptr(t), _ptr(d), code, _ptr(x), _ptr(lens),
                          _ptr(u) if uniforms is not None else None,
                          None if uniforms is not None else _ptr(sd),
                          None if uniforms is not None else _ptr(of), float(temperature), B, k, V,
                          _ptr(tok), _ptr(n), _ptr(probs), _ptr(seq_lens), int(top_k),
                          float(top_p), float(min_p))
        with _on(dev):
            rc = lib().spec_verify_chain_ex(ctypes.byref(prm), _ptr(buf), buf.numel(), sh)
        name = "spec_verify_chain_ex"
    elif uniforms is not None:
        with _on(dev):
            rc = lib().spec_verify_chain(_ptr(t), _ptr(d), code, _ptr(x), _ptr(u), float(temperature),
                                         B, k, V, _ptr(tok), _ptr(n), _ptr(probs), _ptr(seq_lens),
                                         _ptr(buf), buf.numel(), sh)
        name = "spec_verify_chain"
    else:
        with _on(dev):
            rc = lib().spec_verify_chain_philox(_ptr(t), _ptr(d), code, _ptr(x), _ptr(sd), _ptr(of),
                                                float(temperature), B, k, V, _ptr(tok), _ptr(n),
                                                _ptr(probs), _ptr(seq_lens), _ptr(buf), buf.numel(), sh)
        name = "spec_verify_chain_philox"
    if rc != SPEC_OK:
        raise SpecError(name, rc)
    return tok, n, probs


def verify_chain_noalloc(target_logits, draft_logits, draft_tokens, uniforms, temperature: float, *,
                         out_tokens=None, out_num_accepted=None, out_probs=None, want_probs=False,
                         seq_lens=None, stream=None):
    """verify_chain without a workspace: for callers that cannot allocate device
    scratch.  The library's fixed device array serves as scratch (problems up to
    SPEC_NOALLOC_SCRATCH_BYTES of scratch); calls that overlap on the GPU race.
    Output tensors are allocated here unless passed in."""
    t = _dev(target_logits, "target_logits")
    if t.dim() != 3:
        raise ValueError("target_logits must be [B, k+1, V]")
    B, k1, V = t.shape
    k = k1 - 1
    code = _logit_code(t, "target_logits")
    d = _dev(draft_logits, "draft_logits", t.dtype, (B, k, V))
    x = _dev(draft_tokens, "draft_tokens", torch.int32, (B, k))
    u = _dev(uniforms, "uniforms", torch.float32, (B, k + 1))
    dev = t.device
    tok = _out(out_tokens, "out_tokens", (B, k + 1), torch.int32, dev)
    n = _out(out_num_accepted, "out_num_accepted", (B,), torch.int32, dev)
    probs = None
    if out_probs is not None or want_probs:
        probs = _out(out_probs, "out_probs", (B, k, 2), torch.float32, dev)
    if seq_lens is not None:
        _dev(seq_lens, "seq_lens", torch.int32, (B,))
    sh, _ = _stream_handle(stream, dev)
    with _on(dev):
        rc = lib().spec_verify_chain_noalloc(_ptr(t), _ptr(d), code, _ptr(x), _ptr(u), float(temperature),
                                             B, k, V, _ptr(tok), _ptr(n), _ptr(probs), _ptr(seq_lens), sh)
    if rc != SPEC_OK:
        raise SpecError("spec_verify_chain_noalloc", rc)
    return tok, n, probs


def verify_greedy(target_logits, draft_tokens, *, out_tokens=None, out_num_accepted=None,
                  seq_lens=None, workspace: Workspace | None = None, stream=None,
                  draft_lens=None):
    """Greedy chain verify; returns (tokens [B,k+1], num_accepted [B]).
    draft_lens (int32 [B], optional): each request's real draft length."""
    t = _dev(target_logits, "target_logits")
    if t.dim() != 3:
        raise ValueError("target_logits must be [B, k+1, V]")
    B, k1, V = t.shape
    k = k1 - 1
    code = _logit_code(t, "target_logits")
    x = _dev(draft_tokens, "draft_tokens", torch.int32, (B, k))
    dev = t.device
    tok = _out(out_tokens, "out_tokens", (B, k + 1), torch.int32, dev)
    n = _out(out_num_accepted, "out_num_accepted", (B,), torch.int32, dev)
    if seq_lens is not None:
        _dev(seq_lens, "seq_lens", torch.int32, (B,))
    sh, _ = _stream_handle(stream, dev)
    ws = workspace or default_workspace(dev, sh)
    buf = ws.ensure(B, k + 1, V, sh)
    if draft_lens is not None:
        lens = _dev(draft_lens, "draft_lens", torch.int32, (B,))
        prm = GreedyParams(ctypes.sizeof(GreedyParams), _ptr(t), code, _ptr(x), _ptr(lens), B, k, V,
                           _ptr(tok), _ptr(n), _ptr(seq_lens))
        with _on(dev):
            rc = lib().spec_verify_greedy_ex(ctypes.byref(prm), _ptr(buf), buf.numel(), sh)
    else:
        with _on(dev):
            rc = lib().spec_verify_greedy(_ptr(t), code, _ptr(x), B, k, V, _ptr(tok), _ptr(n),
                                          _ptr(seq_lens), _ptr(buf), buf.numel(), sh)
    if rc != SPEC_OK:
        raise SpecError("spec_verify_greedy", rc)
    return tok, n


def verify_tree(target_logits, tree_tokens, paths, *, out_tokens=None, out_num_accepted=None,
                out_best_path=None, out_accepted_nodes=None, seq_lens=None,
                workspace: Workspace | None = None, stream=None):
    """Greedy tree verify; returns (tokens [B,L], num_accepted [B], best_path [B], accepted_nodes [B,L])."""
    t = _dev(target_logits, "target_logits")
    if t.dim() != 3:
        raise ValueError("target_logits must be [B, N, V]")
    B, N, V = t.shape
    code = _logit_code(t, "target_logits")
    tt = _dev(tree_tokens, "tree_tokens", torch.int32, (B, N))
    p = _dev(paths, "paths", torch.int32)
    if p.dim() != 3 or p.shape[0] != B:
        raise ValueError("paths must be [B, P, L]")
    P, L = p.shape[1], p.shape[2]
    dev = t.device
    tok = _out(out_tokens, "out_tokens", (B, L), torch.int32, dev)
    n = _out(out_num_accepted, "out_num_accepted", (B,), torch.int32, dev)
    best = _out(out_best_path, "out_best_path", (B,), torch.int32, dev)
    nodes = _out(out_accepted_nodes, "out_accepted_nodes", (B, L), torch.int32, dev)
    if seq_lens is not None:
        _dev(seq_lens, "seq_lens", torch.int32, (B,))
    sh, _ = _stream_handle(stream, dev)
    ws = workspace or default_workspace(dev, sh)
    buf = ws.ensure(B, N, V, sh)
    with _on(dev):
        rc = lib().spec_verify_tree(_ptr(t), code, _ptr(tt), _ptr(p), B, N, P, L, V, _ptr(tok),
                                    _ptr(n), _ptr(best), _ptr(nodes), _ptr(seq_lens), _ptr(buf),
                                    buf.numel(), sh)
    if rc != SPEC_OK:
        raise SpecError("spec_verify_tree", rc)
    return tok, n, best, nodes


def verify_tree_sampled(target_logits, tree_tokens, paths, uniforms, temperature: float, *,
                        out_tokens=None, out_num_accepted=None, out_best_path=None,
                        out_accepted_nodes=None, seq_lens=None, workspace: Workspace | None = None,
                        stream=None):
    """Stochastic tree verify (chosen children as point-mass proposals);
    uniforms float32 [B, N] (column n >= 1: node n's accept test, column 0:
    the final draw).  Returns (tokens [B,L], num_accepted [B], best_path [B],
    accepted_nodes [B,L])."""
    t = _dev(target_logits, "target_logits")
    if t.dim() != 3:
        raise ValueError("target_logits must be [B, N, V]")
    B, N, V = t.shape
    code = _logit_code(t, "target_logits")
    tt = _dev(tree_tokens, "tree_tokens", torch.int32, (B, N))
    p = _dev(paths, "paths", torch.int32)
    if p.dim() != 3 or p.shape[0] != B:
        raise ValueError("paths must be [B, P, L]")
    P, L = p.shape[1], p.shape[2]
    u = _dev(uniforms, "uniforms", torch.float32, (B, N))
    dev = t.device
    tok = _out(out_tokens, "out_tokens", (B, L), torch.int32, dev)
    n = _out(out_num_accepted, "out_num_accepted", (B,), torch.int32, dev)
    best = _out(out_best_path, "out_best_path", (B,), torch.int32, dev)
    nodes = _out(out_accepted_nodes, "out_accepted_nodes", (B, L), torch.int32, dev)
    if seq_lens is not None:
        _dev(seq_lens, "seq_lens", torch.int32, (B,))
    sh, _ = _stream_handle(stream, dev)
    ws = workspace or default_workspace(dev, sh)
    buf = ws.ensure(B, N, V, sh)
    with _on(dev):
        rc = lib().spec_verify_tree_sampled(_ptr(t), code, _ptr(tt), _ptr(p), _ptr(u), float(temperature),
                                            B, N, P, L, V, _ptr(tok), _ptr(n), _ptr(best), _ptr(nodes),
                                            _ptr(seq_lens), _ptr(buf), buf.numel(), sh)
    if rc != SPEC_OK:
        raise SpecError("spec_verify_tree_sampled", rc)
    return tok, n, best, nodes


def rollback_lengths(old_lens, num_accepted, k: int, *, new_lens=None, rewind_lens=None,
                     stream=None):
    """KV cursor rollback lengths; returns (new_lens [B], rewind_lens [B])."""
    o = _dev(old_lens, "old_lens", torch.int32)
    B = o.shape[0]
    n = _dev(num_accepted, "num_accepted", torch.int32, (B,))
    new = _out(new_lens, "new_lens", (B,), torch.int32, o.device)
    rew = _out(rewind_lens, "rewind_lens", (B,), torch.int32, o.device)
    sh, _ = _stream_handle(stream, o.device)
    with _on(o.device):
        rc = lib().spec_rollback_lengths(_ptr(o), _ptr(n), int(k), B, _ptr(new), _ptr(rew), sh)
    if rc != SPEC_OK:
        raise SpecError("spec_rollback_lengths", rc)
    return new, rew


def relocate_accepted_kv(kv_pool, block_tables, base_lens, accepted_nodes, num_accepted,
                         tokens_per_block: int, *, stream=None):
    """Gather the accepted tree nodes' KV rows to consecutive positions after
    each request's prefix, in place.  kv_pool: [num_blocks * tokens_per_block,
    ...] (any dtype; a token's row is its trailing dims), block_tables
    [B, max_blocks] int32, base_lens [B], accepted_nodes [B, L], num_accepted [B]."""
    if not isinstance(kv_pool, torch.Tensor) or not kv_pool.is_cuda or not kv_pool.is_contiguous():
        raise ValueError("kv_pool must be a contiguous CUDA tensor")
    rows = kv_pool.shape[0]
    if rows % tokens_per_block:
        raise ValueError("kv_pool rows must be num_blocks * tokens_per_block")
    row_bytes = kv_pool.numel() * kv_pool.element_size() // max(rows, 1)
    bt = _dev(block_tables, "block_tables", torch.int32)
    B = bt.shape[0]
    base = _dev(base_lens, "base_lens", torch.int32, (B,))
    nodes = _dev(accepted_nodes, "accepted_nodes", torch.int32)
    n = _dev(num_accepted, "num_accepted", torch.int32, (B,))
    sh, _ = _stream_handle(stream, kv_pool.device)
    with _on(kv_pool.device):
        rc = lib().spec_relocate_accepted_kv(_ptr(kv_pool), ctypes.c_size_t(row_bytes),
                                             int(tokens_per_block), rows // tokens_per_block, _ptr(bt),
                                             bt.shape[1], _ptr(base), _ptr(nodes), _ptr(n), B,
                                             nodes.shape[1], sh)
    if rc != SPEC_OK:
        raise SpecError("spec_relocate_accepted_kv", rc)
    return kv_pool


def rollback_paged(old_lens, num_accepted, k: int, tokens_per_block: int, *, draft_lens=None,
                   blocks_held=None, new_lens=None, rewind_lens=None, free_blocks=None,
                   stream=None):
    """Rollback with ragged draft lengths and paged block accounting; returns
    (new_lens [B], rewind_lens [B], free_blocks [B])."""
    o = _dev(old_lens, "old_lens", torch.int32)
    B = o.shape[0]
    n = _dev(num_accepted, "num_accepted", torch.int32, (B,))
    lens = None if draft_lens is None else _dev(draft_lens, "draft_lens", torch.int32, (B,))
    held = None if blocks_held is None else _dev(blocks_held, "blocks_held", torch.int32, (B,))
    new = _out(new_lens, "new_lens", (B,), torch.int32, o.device)
    rew = _out(rewind_lens, "rewind_lens", (B,), torch.int32, o.device)
    fre = _out(free_blocks, "free_blocks", (B,), torch.int32, o.device)
    sh, _ = _stream_handle(stream, o.device)
    with _on(o.device):
        rc = lib().spec_rollback_paged(_ptr(o), _ptr(n), _ptr(lens), int(k), _ptr(held),
                                       int(tokens_per_block), B, _ptr(new), _ptr(rew), _ptr(fre), sh)
    if rc != SPEC_OK:
        raise SpecError("spec_rollback_paged", rc)
    return new, rew, fre


def philox_uniforms(seeds, offsets, n: int, *, stream=None):
    """[B, n] float32: the uniforms verify_chain draws for each request's
    (seed, offset) Philox stream when called without uniforms."""
    sd = _dev(seeds, "seeds", torch.int64)
    B = sd.shape[0]
    of = _dev(offsets, "offsets", torch.int64, (B,))
    out = torch.empty((B, n), dtype=torch.float32, device=sd.device)
    sh, _ = _stream_handle(stream, sd.device)
    with _on(sd.device):
        rc = lib().spec_philox_uniforms(_ptr(sd), _ptr(of), B, int(n), _ptr(out), sh)
    if rc != SPEC_OK:
        raise SpecError("spec_philox_uniforms", rc)
    return out


# ---------------------------------------------------------------- the paged 8-bit KV cache
# These calls are a few microseconds of GPU work each, so their checks are kept
# short: one combined test per tensor, spelled out only when it fails.
_I32, _F32 = torch.int32, torch.float32
_NOTHING = contextlib.nullcontext()


def _on_stream(stream, dev):
    """Handle of `stream` and a context that makes it and its device current
    if they are not (so what torch allocates inside belongs to the stream and,
    while a graph is captured, to that graph)."""
    if stream is None:
        ctx = _NOTHING if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)
        return torch._C._cuda_getCurrentRawStream(dev.index), ctx
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(getattr(stream, "value", stream) or 0)
        stream = torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)
    if stream.device != dev:
        raise ValueError(f"stream belongs to {stream.device}, the tensors to {dev}")
    return stream.cuda_stream, torch.cuda.stream(stream)


def _at(t, name, dev, dtype, shape) -> int:
    """Address of a dense tensor of this type and shape on this device."""
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != dev.index
            or t.shape != shape or not t.is_contiguous()):
        _dev(t, name, dtype, shape)
        raise ValueError(f"{name} must be on {dev}, is on {t.device}")
    return t.data_ptr()


def _cuda(t, name, dims) -> torch.device:
    """Device of the CUDA tensor that sets where a call runs."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != len(dims):
        raise ValueError(f"{name} must be [{', '.join(dims)}]")
    return t.device


def _apart(*addresses):
    """An array that a call writes must not be another of its arrays."""
    if len(set(addresses)) != len(addresses):
        real = [p for p in addresses if p]
        if len(set(real)) != len(real):
            raise ValueError("two of the call's arrays are the same memory")


def _rows(t, name, dev, shape, dtype):
    """Address and first three strides of a [B, W, heads, D] tensor whose rows
    along D are dense and 16-byte aligned."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev.index:
        raise ValueError(f"{name} must be a CUDA tensor on {dev}")
    if t.dtype is not dtype or (dtype is not torch.bfloat16 and dtype is not torch.float16):
        raise ValueError(f"{name} must be bfloat16 or float16, all of one type, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    b, w, h, d = t.stride()
    # the stride of an axis of one element is never used
    if shape[0] == 1:
        b = 0
    if shape[1] == 1:
        w = 0
    if shape[2] == 1:
        h = 0
    p = t.data_ptr()
    if d != 1 or (b | w | h) % 8 or p % 16:
        raise ValueError(f"{name} must be dense along D with 16-byte aligned rows (strides {tuple(t.stride())})")
    return p, _Strides(b, w, h)


_Strides = ctypes.c_int64 * 3


def _cache(kv_pool, kv_scales, block_tables):
    """The spec_kv_cache of a pool [num_blocks, 2, Hkv, tokens_per_block, D]
    (float8_e4m3fn or uint8), its scales [num_blocks, 2, Hkv] and the block
    tables [B, max_blocks]; also B and the device."""
    dev = _cuda(kv_pool, "kv_pool", ("num_blocks", "2", "Hkv", "tokens_per_block", "D"))
    n, two, H, tpb, D = kv_pool.shape
    if kv_pool.dtype is not torch.uint8 and kv_pool.dtype is not torch.float8_e4m3fn:
        raise ValueError(f"kv_pool must be float8_e4m3fn or uint8, got {kv_pool.dtype}")
    if two != 2 or not kv_pool.is_contiguous():
        raise ValueError("kv_pool must be a contiguous [num_blocks, 2, Hkv, tokens_per_block, D]")
    if D not in (64, 128) or tpb % 16 or not 16 <= tpb <= 1024:
        raise ValueError("kv_pool: D must be 64 or 128 and tokens_per_block a multiple of 16 up to 1024")
    _cuda(block_tables, "block_tables", ("B", "max_blocks"))
    B, cols = block_tables.shape
    return KvCache(_CACHE_BYTES, kv_pool.data_ptr(), _at(kv_scales, "kv_scales", dev, _F32, (n, 2, H)),
                   _at(block_tables, "block_tables", dev, _I32, (B, cols)), n, cols, tpb, H, D), B, dev


_CACHE_BYTES, _ATTEND_BYTES = ctypes.sizeof(KvCache), ctypes.sizeof(AttendParams)


def reserve_blocks(seq_lens, block_tables, blocks_held, free_blocks, free_count, tokens_per_block: int,
                   window: int, *, window_lens=None, want_slots=True, out_slots=None, out_granted=None,
                   stream=None):
    """Blocks for every request's window off the free stack; returns (slots
    [B, window] or None, granted [B]).

    block_tables [B, max_blocks], blocks_held [B] and free_count [1] are
    updated in place; free_blocks [num_blocks] is the stack, its top at
    free_count - 1.  granted is the window length (window_lens, or `window`),
    -1 for a request left without the blocks it needs; slots are the pool
    rows of the window's tokens, -1 where there is none."""
    dev = _cuda(block_tables, "block_tables", ("B", "max_blocks"))
    B, cols = block_tables.shape
    W = int(window)
    sh, ctx = _on_stream(stream, dev)
    with ctx:
        slots, granted = out_slots, out_granted
        if slots is None and want_slots:
            slots = torch.empty((B, W), dtype=_I32, device=dev)
        if granted is None:
            granted = torch.empty((B,), dtype=_I32, device=dev)
        _cuda(free_blocks, "free_blocks", ("num_blocks",))
        n = free_blocks.shape[0]
        a = (_at(seq_lens, "seq_lens", dev, _I32, (B,)),
             None if window_lens is None else _at(window_lens, "window_lens", dev, _I32, (B,)),
             _at(block_tables, "block_tables", dev, _I32, (B, cols)),
             _at(blocks_held, "blocks_held", dev, _I32, (B,)), _at(free_blocks, "free_blocks", dev, _I32, (n,)),
             _at(free_count, "free_count", dev, _I32, (1,)),
             None if slots is None else _at(slots, "out_slots", dev, _I32, (B, W)),
             _at(granted, "out_granted", dev, _I32, (B,)))
        _apart(*a)
        rc = lib().spec_reserve_blocks(a[0], a[1], W, int(tokens_per_block), B, a[2], cols, a[3], a[4], n, a[5],
                                       a[6], a[7], sh)
    if rc != SPEC_OK:
        raise SpecError("spec_reserve_blocks", rc)
    return slots, granted


def release_blocks(block_tables, blocks_held, counts, free_blocks, free_count, *, stream=None):
    """Gives back the last counts[b] blocks of every request (rollback_paged's
    free counts): block_tables, blocks_held, free_blocks and free_count are
    updated in place."""
    dev = _cuda(block_tables, "block_tables", ("B", "max_blocks"))
    B, cols = block_tables.shape
    _cuda(free_blocks, "free_blocks", ("num_blocks",))
    n = free_blocks.shape[0]
    a = (_at(counts, "counts", dev, _I32, (B,)), _at(block_tables, "block_tables", dev, _I32, (B, cols)),
         _at(blocks_held, "blocks_held", dev, _I32, (B,)), _at(free_blocks, "free_blocks", dev, _I32, (n,)),
         _at(free_count, "free_count", dev, _I32, (1,)))
    _apart(*a)
    sh, ctx = _on_stream(stream, dev)
    with ctx:
        rc = lib().spec_release_blocks(a[0], B, a[1], cols, a[2], a[3], n, a[4], sh)
    if rc != SPEC_OK:
        raise SpecError("spec_release_blocks", rc)


def tree_masks(paths, num_nodes: int, *, out=None, stream=None):
    """[B, num_nodes, ceil(num_nodes / 32)] int32: the bits of each node's
    ancestors and itself, from the paths [B, P, L] of verify_tree."""
    dev = _cuda(paths, "paths", ("B", "P", "L"))
    B, P, L = paths.shape
    N = int(num_nodes)
    sh, ctx = _on_stream(stream, dev)
    with ctx:
        if out is None:
            out = torch.empty((B, N, -(-N // 32)), dtype=_I32, device=dev)
        src, dst = _at(paths, "paths", dev, _I32, (B, P, L)), _at(out, "out", dev, _I32, (B, N, -(-N // 32)))
        _apart(src, dst)
        rc = lib().spec_tree_masks(src, B, P, L, N, dst, sh)
    if rc != SPEC_OK:
        raise SpecError("spec_tree_masks", rc)
    return out


def store_kv(k, v, kv_pool, kv_scales, block_tables, seq_lens, *, window_lens=None, stream=None):
    """Writes a window's rows k, v [B, W, Hkv, D] (bfloat16 or float16, any
    16-byte aligned strides) at logical positions seq_lens[b] + i of the
    paged cache: kv_pool [num_blocks, 2, Hkv, tokens_per_block, D]
    (float8_e4m3fn or uint8) and kv_scales [num_blocks, 2, Hkv] in place."""
    cache, B, dev = _cache(kv_pool, kv_scales, block_tables)
    _cuda(k, "k", ("B", "W", "Hkv", "D"))
    shape = (B, k.shape[1], cache.kv_heads, cache.head_dim)
    kp, ks = _rows(k, "k", dev, shape, k.dtype)
    vp, vs = _rows(v, "v", dev, shape, k.dtype)
    seq = _at(seq_lens, "seq_lens", dev, _I32, (B,))
    win = None if window_lens is None else _at(window_lens, "window_lens", dev, _I32, (B,))
    sh, ctx = _on_stream(stream, dev)
    with ctx:
        rc = lib().spec_store_kv(cache, kp, ks, vp, vs, SPEC_BF16 if k.dtype is torch.bfloat16 else SPEC_F16, seq, win,
                                 B, shape[1], sh)
    if rc != SPEC_OK:
        raise SpecError("spec_store_kv", rc)


def attend_kv(q, kv_pool, kv_scales, block_tables, seq_lens, *, window_lens=None, masks=None,
              scale: float | None = None, out=None, out_lse=None, want_lse=False, scratch=None, stream=None):
    """Attention of the window's rows q [B, W, Hq, D] (bfloat16 or float16)
    over each request's cached prefix and its window; returns (out [B, W, Hq,
    D], lse [B, W, Hq] float32 or None).

    masks [B, W, ceil(W / 32)] int32 (tree_masks) replace the chain's j <= i
    inside the window; scale defaults to D ** -0.5.  Rows behind a window's
    end are left as they are in `out` and `out_lse` (zeros in tensors made
    here).  scratch: a uint8 tensor of spec_attend_scratch_size bytes; made
    for the call by default."""
    cache, B, dev = _cache(kv_pool, kv_scales, block_tables)
    _cuda(q, "q", ("B", "W", "Hq", "D"))
    W, Hq, D = q.shape[1], q.shape[2], cache.head_dim
    if Hq % cache.kv_heads:
        raise ValueError(f"q must have a multiple of {cache.kv_heads} heads, got {Hq}")
    qp, qs = _rows(q, "q", dev, (B, W, Hq, D), q.dtype)
    seq = _at(seq_lens, "seq_lens", dev, _I32, (B,))
    win = None if window_lens is None else _at(window_lens, "window_lens", dev, _I32, (B,))
    mp = None if masks is None else _at(masks, "masks", dev, _I32, (B, W, -(-W // 32)))
    need = lib().spec_attend_scratch_size(B, W, Hq, cache.kv_heads, D)
    if need == 0:
        raise SpecError("spec_attend_scratch_size", SPEC_EINVAL)
    sh, ctx = _on_stream(stream, dev)
    with ctx:
        make = torch.empty if win is None else torch.zeros
        if out is None:
            out = make((B, W, Hq, D), dtype=q.dtype, device=dev)
        if out_lse is None and want_lse:
            out_lse = make((B, W, Hq), dtype=_F32, device=dev)
        if scratch is None:
            scratch = torch.empty(need, dtype=torch.uint8, device=dev)
        op = _at(out, "out", dev, q.dtype, (B, W, Hq, D))
        lp = None if out_lse is None else _at(out_lse, "out_lse", dev, _F32, (B, W, Hq))
        sp = _at(scratch, "scratch", dev, torch.uint8, (scratch.numel(),))
        _apart(qp, cache.pool, mp, op, lp, sp)
        prm = AttendParams(_ATTEND_BYTES, qp, qs, SPEC_BF16 if q.dtype is torch.bfloat16 else SPEC_F16, B, W, Hq, seq,
                           win, mp, D ** -0.5 if scale is None else scale, op, lp)
        rc = lib().spec_attend_kv(cache, prm, sp, scratch.numel(), sh)
    if rc != SPEC_OK:
        raise SpecError("spec_attend_kv", rc)
    return out, out_lse


def relocate_quantised_kv(kv_pool, kv_scales, block_tables, base_lens, accepted_nodes, num_accepted, *,
                          stream=None):
    """relocate_accepted_kv for the 8-bit cache, in place: the accepted nodes'
    K and V rows move behind each request's prefix, their codes re-rounded
    where a block's scale changes."""
    cache, B, dev = _cache(kv_pool, kv_scales, block_tables)
    _cuda(accepted_nodes, "accepted_nodes", ("B", "L"))
    L = accepted_nodes.shape[1]
    base = _at(base_lens, "base_lens", dev, _I32, (B,))
    nodes = _at(accepted_nodes, "accepted_nodes", dev, _I32, (B, L))
    n = _at(num_accepted, "num_accepted", dev, _I32, (B,))
    sh, ctx = _on_stream(stream, dev)
    with ctx:
        rc = lib().spec_relocate_quantised_kv(cache, base, nodes, n, B, L, sh)
    if rc != SPEC_OK:
        raise SpecError("spec_relocate_quantised_kv", rc)
    return kv_pool


# ---------------------------------------------------------------- around the verify and the cache
_ADJUST_BYTES, _ROTATE_BYTES = ctypes.sizeof(AdjustParams), ctypes.sizeof(RotateParams)
_WEIGH_BYTES, _EVICT_BYTES = ctypes.sizeof(WeighParams), ctypes.sizeof(EvictParams)


def adjust_logits(logits, *, tokens=None, token_lens=None, prompt_lens=None, repetition=None, frequency=None,
                  presence=None, bias_ids=None, bias_values=None, allowed=None, allowed_rows=None,
                  draft_tokens=None, draft_lens=None, masks=None, out=None, stream=None):
    """Penalties for repeated tokens, biases and grammar masks on the logits
    [B, R, V] (float32 or bfloat16) of a window's rows, before verify_chain,
    verify_greedy (R = k + 1) or verify_tree (R = N); returns out [B, R, V].
    out=logits changes them in place and touches only what changes.

    tokens [B, T] int32: the request's tokens so far, token_lens [B] of them
    real (T by default), the first prompt_lens [B] of these its prompt (none
    by default).  draft_tokens: the window's tokens, counted as output by the
    rows behind them: [B, R - 1] of a chain, or [B, R] (verify_tree's
    tree_tokens) with masks [B, R, ceil(R / 32)] (tree_masks).  draft_lens [B]:
    rows past it are left as they are in `out` (zeros in a tensor made here).
    repetition, frequency, presence [B] float32: penalties; with none of them
    the tokens change nothing.  bias_ids [B, M] int32 (-1: none), bias_values
    [B, M] float32.  allowed [n, ceil(V / 32)] int32: token masks, and
    allowed_rows [B, R] int32 each row's (below 0: none); by default one for
    each row, [B, R, ceil(V / 32)] or [B * R, ...]."""
    dev = _cuda(logits, "logits", ("B", "R", "V"))
    B, R, V = logits.shape
    code = _logit_code(logits, "logits")
    words = -(-V // 32)
    src = _at(logits, "logits", dev, logits.dtype, (B, R, V))

    def optional(t, name, dtype, shape):
        return None if t is None else _at(t, name, dev, dtype, shape)
    # the arguments keep their names, so that a tensor made for the call lives until the launch
    T = M = n = 0
    if tokens is not None:
        _cuda(tokens, "tokens", ("B", "T"))
        T = tokens.shape[1]
    elif token_lens is not None or prompt_lens is not None:
        raise ValueError("token_lens and prompt_lens go with tokens")
    if masks is not None and draft_tokens is None:
        raise ValueError("masks go with draft_tokens")
    if masks is not None and draft_lens is not None:
        raise ValueError("draft_lens are a chain's: a tree has masks")
    if (bias_ids is None) != (bias_values is None):
        raise ValueError("bias_ids and bias_values go together")
    if bias_ids is not None:
        _cuda(bias_ids, "bias_ids", ("B", "M"))
        M = bias_ids.shape[1]
    if allowed is None and allowed_rows is not None:
        raise ValueError("allowed_rows go with allowed")
    mask_shape = None
    if allowed is not None:
        if allowed_rows is None:
            n = B * R
            mask_shape = (B, R, words) if isinstance(allowed, torch.Tensor) and allowed.dim() == 3 else (n, words)
        else:
            _cuda(allowed, "allowed", ("n", "ceil(V / 32)"))
            n = allowed.shape[0]
            mask_shape = (n, words)
    said = optional(tokens, "tokens", _I32, (B, T))
    lists = (optional(token_lens, "token_lens", _I32, (B,)), optional(prompt_lens, "prompt_lens", _I32, (B,)))
    window = (optional(draft_tokens, "draft_tokens", _I32, (B, R if masks is not None else R - 1)),
              optional(masks, "masks", _I32, (B, R, -(-R // 32))), optional(draft_lens, "draft_lens", _I32, (B,)))
    penalties = (optional(repetition, "repetition", _F32, (B,)), optional(frequency, "frequency", _F32, (B,)),
                 optional(presence, "presence", _F32, (B,)))
    bias = optional(bias_ids, "bias_ids", _I32, (B, M)), optional(bias_values, "bias_values", _F32, (B, M))
    grammar = optional(allowed, "allowed", _I32, mask_shape), optional(allowed_rows, "allowed_rows", _I32, (B, R))
    if T == 0:  # no token: nothing to count
        said = None
    if M == 0:
        bias = None, None
    sh, ctx = _on_stream(stream, dev)
    with ctx:
        if out is None:
            out = (torch.empty if draft_lens is None else torch.zeros)((B, R, V), dtype=logits.dtype, device=dev)
        dst = _at(out, "out", dev, logits.dtype, (B, R, V))
        prm = AdjustParams(_ADJUST_BYTES, src, dst, code, B, R, V, said, *lists, T, *window, *penalties, *bias, M, *grammar,
                           n)
        rc = lib().spec_adjust_logits(prm, sh)
    if rc != SPEC_OK:
        raise SpecError("spec_adjust_logits", rc)
    return out


@functools.lru_cache(maxsize=1024)
def _scratch_bytes(call: str, *sizes) -> int:
    """spec_<call>_scratch_size of these sizes."""
    need = getattr(lib(), f"spec_{call}_scratch_size")(*sizes)
    if need == 0:
        raise SpecError(f"spec_{call}_scratch_size", SPEC_EINVAL)
    return need


_NO_STRIDES = _Strides(0, 0, 0)


def _rotation(q, k, starts, inv_freq, interleaved, gain, window_lens, masks, out_q, dev, B, W, D, dtype):
    """A RotateParams of everything but where the keys go."""
    _cuda(inv_freq, "inv_freq", ("pairs",))
    pairs = inv_freq.shape[0]
    if pairs < 8 or pairs % 8 or 2 * pairs > D:
        raise ValueError(f"inv_freq must have a multiple of 8 elements, at most {D // 2}, got {pairs}")
    if masks is not None and W > SPEC_MAX_TREE_NODES:
        raise ValueError(f"masks are for windows of at most {SPEC_MAX_TREE_NODES} tokens")
    qp = kp = oq = None
    qs = ks = os = _NO_STRIDES
    Hq = Hk = 0
    if q is not None:
        _cuda(q, "q", ("B", "W", "Hq", "D"))
        Hq = q.shape[2]
        qp, qs = _rows(q, "q", dev, (B, W, Hq, D), dtype)
        oq, os = _rows(out_q, "out_q", dev, (B, W, Hq, D), dtype)
    if k is not None:
        _cuda(k, "k", ("B", "W", "Hkv", "D"))
        Hk = k.shape[2]
        kp, ks = _rows(k, "k", dev, (B, W, Hk, D), dtype)
    return RotateParams(_ROTATE_BYTES, qp, kp, oq, None, qs, ks, os, _NO_STRIDES,
                        SPEC_BF16 if dtype is torch.bfloat16 else SPEC_F16, B, W, Hq, Hk, D,
                        _at(starts, "starts", dev, _I32, (B,)),
                        None if window_lens is None else _at(window_lens, "window_lens", dev, _I32, (B,)),
                        None if masks is None else _at(masks, "masks", dev, _I32, (B, W, -(-W // 32))),
                        _at(inv_freq, "inv_freq", dev, torch.float64, (pairs,)), pairs, int(bool(interleaved)), gain)


def _outside(t, out, name):
    """Names what the C call refused: an output that is its input's memory in
    another order, or has no place for each element."""
    if t.data_ptr() == out.data_ptr() and any(n > 1 and x != y for n, x, y in zip(t.shape, t.stride(), out.stride())):
        raise ValueError(f"{name} is its input's memory with other strides")
    if 0 in out.stride() and any(n > 1 and st == 0 for n, st in zip(out.shape, out.stride())):
        raise ValueError(f"{name} has several elements in one place")


def rotate_qk(q, k, starts, inv_freq, *, interleaved=False, gain: float = 1.0, window_lens=None, masks=None,
              out_q=None, out_k=None, stream=None):
    """Rotary positions of a window's rows q [B, W, Hq, D] and k [B, W, Hkv, D]
    (bfloat16 or float16, any 16-byte aligned strides; k or q may be None);
    returns (q, k) rotated.  out_q=q and out_k=k rotate in place.

    starts [B] int32: the position of token 0.  Token i of a chain has
    position starts + i, a tree's node (masks [B, W, ceil(W / 32)], tree_masks)
    starts + its depth.  inv_freq [pairs] float64 (finite) and gain: rotary_frequencies.
    The first 2 * pairs elements turn, as pairs (i, i + pairs) or, interleaved,
    (2 i, 2 i + 1).  Rows behind a window's end are left as they are in the
    outputs (zeros in tensors made here)."""
    x = q if q is not None else k
    dev = _cuda(x, "q" if q is not None else "k", ("B", "W", "heads", "D"))
    B, W, _, D = x.shape
    sh, ctx = _on_stream(stream, dev)
    with ctx:
        make = torch.empty if window_lens is None else torch.zeros
        if q is not None and out_q is None:
            out_q = make(q.shape, dtype=x.dtype, device=dev)
        if k is not None and out_k is None:
            out_k = make(k.shape, dtype=x.dtype, device=dev)
        if (q is None and out_q is not None) or (k is None and out_k is not None):
            raise ValueError("an output without its input")
        prm = _rotation(q, k, starts, inv_freq, interleaved, gain, window_lens, masks, out_q, dev, B, W, D, x.dtype)
        if k is not None:
            prm.out_k, prm.out_k_strides = _rows(out_k, "out_k", dev, k.shape, x.dtype)
        rc = lib().spec_rotate_qk(prm, sh)
    if rc != SPEC_OK:
        if rc == SPEC_EINVAL:  # say why, where it is one of these
            if k is not None:
                _outside(k, out_k, "out_k")
            if q is not None:
                _outside(q, out_q, "out_q")
            _apart(prm.out_q, prm.out_k)
            _apart(prm.q, prm.out_k)
            _apart(prm.out_q, prm.k)
        raise SpecError("spec_rotate_qk", rc)
    return out_q, out_k


def rotate_store_kv(q, k, v, inv_freq, kv_pool, kv_scales, block_tables, seq_lens, *, starts=None,
                    interleaved=False, gain: float = 1.0, window_lens=None, masks=None, out_q=None, scratch=None,
                    stream=None):
    """rotate_qk and store_kv in one call, with their results: returns q
    [B, W, Hq, D] rotated, and writes the rotated k and v [B, W, Hkv, D] at
    logical positions seq_lens[b] + i of the paged cache.  starts defaults to
    seq_lens: pass the text's own positions once evict_kv has dropped some.
    scratch: a uint8 tensor of spec_rotate_store_scratch_size bytes; made for the
    call by default."""
    cache, B, dev = _cache(kv_pool, kv_scales, block_tables)
    _cuda(k, "k", ("B", "W", "Hkv", "D"))
    W, H, D = k.shape[1], cache.kv_heads, cache.head_dim
    _cuda(q, "q", ("B", "W", "Hq", "D"))
    if k.shape != (B, W, H, D):
        raise ValueError(f"k must have shape {(B, W, H, D)}, got {tuple(k.shape)}")
    vp, vs = _rows(v, "v", dev, k.shape, k.dtype)
    seq = _at(seq_lens, "seq_lens", dev, _I32, (B,))
    sh, ctx = _on_stream(stream, dev)
    with ctx:
        if out_q is None:
            out_q = (torch.empty if window_lens is None else torch.zeros)(q.shape, dtype=k.dtype, device=dev)
        prm = _rotation(q, k, seq_lens if starts is None else starts, inv_freq, interleaved, gain, window_lens, masks,
                        out_q, dev, B, W, D, k.dtype)
        if scratch is None:
            scratch = torch.empty(_scratch_bytes("rotate_store", B, W, H, D, cache.tokens_per_block), dtype=torch.uint8,
                                  device=dev)
        sp = _at(scratch, "scratch", dev, torch.uint8, (scratch.numel(),))
        rc = lib().spec_rotate_store_kv(cache, prm, vp, vs, seq, sp, scratch.numel(), sh)
    if rc != SPEC_OK:
        if rc == SPEC_EINVAL:  # say why, where it is one of these (k and v may be one array: both are only read)
            _outside(q, out_q, "out_q")
            _apart(prm.out_q, prm.k, cache.pool, sp, vp if vp != prm.k else 0)
        raise SpecError("spec_rotate_store_kv", rc)
    return out_q


def weigh_kv(q, lse, kv_pool, kv_scales, block_tables, seq_lens, *, window_lens=None, scale: float | None = None,
             weights=None, decay: float = 1.0, out=None, scratch=None, stream=None):
    """The attention that each cached position drew from a window's rows: q
    [B, W, Hq, D] and lse [B, W, Hq] float32 of attend_kv; returns out
    [B, Hkv, T] float32, decay * weights (before seq_lens[b]; none without
    weights) plus the window's probabilities, summed over its tokens and the
    query heads of each KV head.

    The window is a chain; of a tree, pass the accepted path's rows of q and lse
    with window_lens = num_accepted + 1 after relocate_quantised_kv.  T is that
    of weights or out, else the cache's max_blocks * tokens_per_block; positions
    behind a request's end are left as they are in `out` (zeros in a tensor made
    here).  out=weights updates in place.  scratch: a uint8 tensor of
    spec_weigh_scratch_size bytes; made for the call by default."""
    cache, B, dev = _cache(kv_pool, kv_scales, block_tables)
    _cuda(q, "q", ("B", "W", "Hq", "D"))
    W, Hq, D, H = q.shape[1], q.shape[2], cache.head_dim, cache.kv_heads
    if Hq % H:
        raise ValueError(f"q must have a multiple of {H} heads, got {Hq}")
    qp, qs = _rows(q, "q", dev, (B, W, Hq, D), q.dtype)
    T = cache.max_blocks * cache.tokens_per_block
    for t, name in ((weights, "weights"), (out, "out")):
        if t is not None:
            _cuda(t, name, ("B", "Hkv", "T"))
            T = t.shape[2]
    seq = _at(seq_lens, "seq_lens", dev, _I32, (B,))
    win = None if window_lens is None else _at(window_lens, "window_lens", dev, _I32, (B,))
    lp = _at(lse, "lse", dev, _F32, (B, W, Hq))
    wp = None if weights is None else _at(weights, "weights", dev, _F32, (B, H, T))
    need = _scratch_bytes("weigh", B, W, Hq, H, D)
    sh, ctx = _on_stream(stream, dev)
    with ctx:
        if out is None:
            out = torch.zeros((B, H, T), dtype=_F32, device=dev)
        if scratch is None:
            scratch = torch.empty(need, dtype=torch.uint8, device=dev)
        op = _at(out, "out", dev, _F32, (B, H, T))
        sp = _at(scratch, "scratch", dev, torch.uint8, (scratch.numel(),))
        prm = WeighParams(_WEIGH_BYTES, qp, qs, SPEC_BF16 if q.dtype is torch.bfloat16 else SPEC_F16, B, W, Hq, seq, win,
                          lp, D ** -0.5 if scale is None else scale, wp, decay, op, T)
        rc = lib().spec_weigh_kv(cache, prm, sp, scratch.numel(), sh)
    if rc != SPEC_OK:
        if rc == SPEC_EINVAL:  # say why, where it is this
            _apart(op, lp, qp, cache.pool, sp)
        raise SpecError("spec_weigh_kv", rc)
    return out


def evict_kv(weights, kv_pool, kv_scales, block_tables, seq_lens, keep: int, *, first: int = 0, recent: int = 0,
             blocks_held=None, out_lens=None, out_kept=None, out_weights=None, out_free=None, scratch=None,
             stream=None):
    """Drops cached positions, head by head, down to `keep` of them: the first
    `first`, the last `recent` and, between, those of largest weight (weights
    [B, Hkv, T] float32, weigh_kv; the lowest position among equals) stay and
    move together, in place.

    Returns (new_lens [B], kept [B, Hkv, keep] int32 with -1 behind a request's
    end, their weights [B, Hkv, keep], and with blocks_held [B] the whole blocks
    that are free now, for release_blocks, else None).  out_lens=seq_lens and
    out_weights=weights update in place.  Rotated keys keep their rotation: new
    tokens go on from the text's positions (starts in rotate_store_kv), not from
    new_lens.  scratch: a uint8 tensor of spec_evict_scratch_size bytes; made for
    the call by default."""
    cache, B, dev = _cache(kv_pool, kv_scales, block_tables)
    H, keep = cache.kv_heads, int(keep)
    _cuda(weights, "weights", ("B", "Hkv", "T"))
    T = weights.shape[2]
    if keep < 1 or first < 0 or recent < 0 or first + recent > keep:
        raise ValueError(f"keep must be at least 1 and first + recent, got {keep}, {first} and {recent}")
    wp = _at(weights, "weights", dev, _F32, (B, H, T))
    seq = _at(seq_lens, "seq_lens", dev, _I32, (B,))
    held = None if blocks_held is None else _at(blocks_held, "blocks_held", dev, _I32, (B,))
    if held is None and out_free is not None:
        raise ValueError("out_free goes with blocks_held")
    need = _scratch_bytes("evict", B, H, keep, cache.tokens_per_block)
    sh, ctx = _on_stream(stream, dev)
    with ctx:
        if out_lens is None:
            out_lens = torch.empty((B,), dtype=_I32, device=dev)
        if out_kept is None:
            out_kept = torch.empty((B, H, keep), dtype=_I32, device=dev)
        if out_weights is None:
            out_weights = torch.zeros((B, H, keep), dtype=_F32, device=dev)
        if held is not None and out_free is None:
            out_free = torch.empty((B,), dtype=_I32, device=dev)
        _cuda(out_weights, "out_weights", ("B", "Hkv", "T_out"))
        T_out = out_weights.shape[2]
        if T_out < keep:
            raise ValueError(f"out_weights must hold {keep} positions, got {T_out}")
        lp, kp = _at(out_lens, "out_lens", dev, _I32, (B,)), _at(out_kept, "out_kept", dev, _I32, (B, H, keep))
        op = _at(out_weights, "out_weights", dev, _F32, (B, H, T_out))
        fp = None if held is None else _at(out_free, "out_free", dev, _I32, (B,))
        if scratch is None:
            scratch = torch.empty(need, dtype=torch.uint8, device=dev)
        sp = _at(scratch, "scratch", dev, torch.uint8, (scratch.numel(),))
        prm = EvictParams(_EVICT_BYTES, wp, T, B, seq, keep, int(first), int(recent), lp, kp, op, T_out, held, fp)
        rc = lib().spec_evict_kv(cache, prm, sp, scratch.numel(), sh)
    if rc != SPEC_OK:
        if rc == SPEC_EINVAL:  # say why, where it is this: op may be wp, and lp seq
            _apart(kp, fp, held, sp, cache.pool, cache.scales, cache.block_tables, *{wp, op}, *{seq, lp})
        raise SpecError("spec_evict_kv", rc)
    return out_lens, out_kept, out_weights, out_free


def last_error(workspace: Workspace, stream=None) -> int:
    """Synchronise, read and clear the workspace's data-dependent status."""
    if workspace.buf is None:
        return SPEC_OK
    sh, _ = _stream_handle(stream, workspace.buf.device)
    out = ctypes.c_int(0)
    with _on(workspace.buf.device):
        rc = lib().spec_last_error(_ptr(workspace.buf), workspace.buf.numel(), sh, ctypes.byref(out))
    if rc != SPEC_OK:
        raise SpecError("spec_last_error", rc)
    return out.value
