"""Angles per position of rotary embeddings, on the host in 64 bits."""
from __future__ import annotations

import math

import torch


def rotary_frequencies(rot_dim: int, base: float = 10000.0, *, scaling: str | None = None, factor: float = 1.0,
                       original_len: int | None = None, fast: float = 32.0, slow: float = 1.0, device=None):
    """(inv_freq [rot_dim / 2] float64, gain) for rotate_qk and rotate_store_kv.

    inv_freq[i] = base ** (-2 i / rot_dim) radians per position, and for
    contexts `factor` times the trained length (`original_len`):
      None      as trained, gain 1
      "linear"  every frequency divided by factor (position interpolation)
      "base"    base times factor ** (rot_dim / (rot_dim - 2)): the slowest pair
                is divided by factor, the fastest kept
      "ramp"    pairs that turn at least `fast` times within original_len kept,
                those that turn at most `slow` times divided by factor, a linear
                blend over the number of turns between; gain 0.1 ln(factor) + 1.
                (Model code often blends over the pair's index instead, between the
                pairs of `fast` and `slow` turns: the ends are the same, the blended
                pairs' frequencies differ, and a model trained so needs its own.)
      "smooth"  the same blend with gain 1; models that use it are published with
                fast=4 and slow=1, which have to be given: `fast` is 32 by default
    """
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError(f"rot_dim must be even and positive, got {rot_dim}")
    if not (base > 0 and math.isfinite(base)) or not (factor >= 1 and math.isfinite(factor)):
        raise ValueError("base must be positive and factor at least 1")
    if scaling not in (None, "linear", "base", "ramp", "smooth"):
        raise ValueError(f"scaling must be None, 'linear', 'base', 'ramp' or 'smooth', got {scaling!r}")
    gain = 1.0
    if scaling == "base":
        if rot_dim < 4:
            raise ValueError("scaling 'base' needs rot_dim of 4 or more")
        base = base * factor ** (rot_dim / (rot_dim - 2))
    freq = [base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)]
    if scaling == "linear":
        freq = [f / factor for f in freq]
    if scaling in ("ramp", "smooth"):
        if not original_len or original_len < 1 or not fast > slow > 0:
            raise ValueError("scaling 'ramp' and 'smooth' need original_len, and fast > slow > 0")
        kept = [min(1.0, max(0.0, (original_len * f / (2 * math.pi) - slow) / (fast - slow))) for f in freq]
        freq = [f / factor * (1 - k) + f * k for f, k in zip(freq, kept)]
        if scaling == "ramp":
            gain = 0.1 * math.log(factor) + 1.0
    return torch.tensor(freq, dtype=torch.float64, device=device), gain
