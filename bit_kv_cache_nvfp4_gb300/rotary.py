"""Rotary positions of queries and keys (``kv4_rotary``, C ABI in
``include/kv4mla.h``), and the frequencies they turn by.

Works for the grouped caches' heads (all of a head, or a part of it) and for the
rope part of latent attention: q [T, H, 576] from element 512 on, and the key's
rope row as [T, 1, 64].
"""
from __future__ import annotations

import math

import torch

from . import Kv4Error
from .gqa8 import _extension

_ext = None


def _load():
    global _ext
    _ext = _extension()
    return _ext


def rotary(q: torch.Tensor | None, k: torch.Tensor | None, positions: torch.Tensor,
           inv_freq: torch.Tensor, interleaved: bool = False, q_offset: int = 0,
           k_offset: int = 0, factor: float = 1.0, q_out: torch.Tensor | None = None,
           k_out: torch.Tensor | None = None):
    """q and k with their rotary positions (kv4_rotary).

    q, k bf16 or f16 [T, heads, D], strided, either may be None; positions int32
    or int64 [T], magnitudes up to 2^31; inv_freq fp32 [n] in radians a position, n up
    to 512, magnitudes up to 4 (beyond, and at farther positions, angles lose bits;
    one that is not finite makes its pair NaN).  2 n elements of each head turn, from
    the offset on: neighbours (2i, 2i + 1) where `interleaved`, else halves (i, n + i).
    Turned elements are multiplied by `factor` (a stretched context's attention factor,
    for instance), the others copied.  Returns (q, k), new tensors unless q_out or k_out
    is given, which may be the input itself and else shares no element with q, k or the
    other output; its own rows share none either.  No gradients are computed; that of
    a rotation is the rotation by -positions of the outputs' gradients."""
    r = (_ext or _load()).rotary(q, k, positions, inv_freq, interleaved, q_offset, k_offset, factor, q_out, k_out)
    if type(r) is int:
        raise Kv4Error("kv4_rotary", r)
    return r


def rotary_frequencies(dim: int, base: float = 10000.0, scaling: str | None = None,
                       stretch: float = 1.0, original_length: int = 8192, slow: float = 1.0,
                       fast: float = 32.0, device=None) -> torch.Tensor:
    """inv_freq fp32 [dim / 2] = base^(-2i / dim), scaled for contexts `stretch`
    times as long as `original_length` tokens, computed in 64 bits:

      None      as they are
      "linear"  all divided by stretch
      "base"    base * stretch^(dim / (dim - 2)): the slowest is divided by
                stretch, the fastest kept
      "ramp"    those of fewer than `slow` turns over original_length divided by
                stretch, those of more than `fast` kept, linear in the turns
                between
      "index_ramp"  the same ends, linear in the pair's index between: from the
                index at which a frequency makes `fast` turns, rounded down, to
                that of `slow` turns, rounded up.  In between it is several times
                the other (4.3 at a stretch of 40): take the one that a model was
                trained with"""
    if dim < 2 or dim % 2:
        raise ValueError(f"dim must be even and at least 2, got {dim}")
    if not (base > 0 and math.isfinite(base)) or not (stretch > 0 and math.isfinite(stretch)):
        raise ValueError("base and stretch must be positive and finite")
    i = torch.arange(0, dim, 2, dtype=torch.float64) / dim
    if scaling == "base":
        if dim < 4:
            raise ValueError('scaling "base" needs a dim of 4 or more')
        base = base * stretch ** (dim / (dim - 2))
    f = float(base) ** -i
    if scaling == "linear":
        f = f / stretch
    elif scaling == "ramp":
        if not fast > slow:
            raise ValueError("fast must be above slow")
        keep = ((original_length * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        f = f * (keep + (1 - keep) / stretch)
    elif scaling == "index_ramp":
        if not (math.inf > fast > slow > 0 and base > 1 and math.inf > original_length > 0):
            raise ValueError("fast must be above slow, slow and original_length above 0, base above 1, all finite")
        # base^(-2 at / dim) * original_length = 2 pi turns
        low, high = (dim * math.log(original_length / (2 * math.pi * turns)) / (2 * math.log(base)) for turns in (fast, slow))
        low, high = max(math.floor(low), 0), min(math.ceil(high), dim - 1)
        # (a step where both are one index)
        keep = 1 - ((torch.arange(dim // 2, dtype=torch.float64) - low) / max(high - low, 1e-3)).clamp(0, 1)
        f = f * (keep + (1 - keep) / stretch)
    elif scaling not in (None, "base"):
        raise ValueError(f'scaling must be None, "linear", "base", "ramp" or "index_ramp", got {scaling!r}')
    return f.float().to(device if device is not None else "cpu")
