"""The 4-bit grouped-query cache: append, read-back and attention.

Bindings of ``kv4_append_gqa4``, ``kv4_read_gqa4`` and ``kv4_attention_gqa4``
(C ABI in ``include/kv4mla.h``, which defines the layout, the rounding and the
masks).  The cache is two tensors:

    pool    uint8 [num_pages, Hkv, 2, 64, D / 2]   E2M1 codes of K and V, element 2j
                                                   in a byte's low half
    scales  uint8 [num_pages, Hkv, 2, 64, D / 16]  E4M3: value = code * scale

and a page table int32 [B, stride] as for the other caches of this package.  The
calls are those of the 8-bit cache (gqa8.py), with its rules for devices,
streams and gradients, at 0.5625 of its bytes; a row depends on its token alone,
so an append changes no other.
"""
from __future__ import annotations

import ctypes

import torch

from . import Kv4Error, _check, load_library
from .gqa8 import _extension

_ext = None


def _load():
    global _ext
    _ext = _extension()
    return _ext


def append_gqa4(k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                page_table: torch.Tensor, seq_lens: torch.Tensor, pool: torch.Tensor,
                scales: torch.Tensor, dev_err: torch.Tensor | None = None) -> None:
    """Quantize new tokens into the cache (kv4_append_gqa4).

    k, v bf16 or f16 [T, Hkv, D] (strided: slices of a fused projection are
    fine); cu_seqlens int32 [B + 1]: request b's rows; seq_lens int32 [B]:
    tokens of each request, these included, so request b's rows go to positions
    seq_lens[b] - n .. seq_lens[b] - 1."""
    st = (_ext or _load()).append4(k, v, cu_seqlens, page_table, seq_lens, pool, scales, dev_err)
    if st:
        raise Kv4Error("kv4_append_gqa4", st)


def read_gqa4(pool: torch.Tensor, scales: torch.Tensor, page_table: torch.Tensor,
              starts: torch.Tensor, cu_seqlens: torch.Tensor, total: int,
              dtype: torch.dtype = torch.bfloat16, k_out: torch.Tensor | None = None,
              v_out: torch.Tensor | None = None, dev_err: torch.Tensor | None = None):
    """The values of a range of each request's tokens (kv4_read_gqa4), exact.

    Request b's positions starts[b] .. starts[b] + n - 1 go to rows
    cu_seqlens[b] .. cu_seqlens[b+1] - 1 of k and v [total, Hkv, D], n being
    their number; other rows are left as they are.  Returns (k, v)."""
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise TypeError(f"dtype must be bfloat16 or float16, got {dtype}")
    r = (_ext or _load()).read4(pool, scales, page_table, starts, cu_seqlens, total,
                                dtype is torch.float16, k_out, v_out, dev_err)
    if type(r) is int:
        raise Kv4Error("kv4_read_gqa4", r)
    return r


def attention_gqa4_workspace(B: int, max_new: int, total: int, hq: int, hkv: int, d: int,
                             device=None) -> int:
    """Workspace bytes of attention_gqa4 for `total` new tokens of B requests,
    at most max_new each."""
    n = ctypes.c_size_t(0)
    with torch.cuda.device(device):
        _check("kv4_attention_gqa4_plan", load_library().kv4_attention_gqa4_plan(
            B, max_new, total, hq, hkv, d, ctypes.byref(n)))
    return n.value


def attention_gqa4(q: torch.Tensor, pool: torch.Tensor, scales: torch.Tensor,
                   page_table: torch.Tensor, seq_lens: torch.Tensor, cu_seqlens: torch.Tensor,
                   max_new: int, sm_scale: float, window: int = 0,
                   out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, dev_err: torch.Tensor | None = None):
    """Causal attention of the new tokens over the cache (kv4_attention_gqa4).

    q bf16 or f16 [T, Hq, D] (strided), Hq a multiple of the cache's Hkv;
    cu_seqlens int32 [B + 1]: request b's rows; seq_lens int32 [B]: tokens of
    each request, these included (append them first); max_new: the most rows of
    any request; window > 0: a row sees only that many keys, its own the last.
    Returns (out [T, Hq, D] of q's type, lse fp32 [T, Hq]); a row without a key
    gives 0 and -inf, rows from cu_seqlens[B] on are left as they are.  Without
    `workspace` each call takes its own from PyTorch's allocator."""
    r = (_ext or _load()).attention4(q, pool, scales, page_table, seq_lens, cu_seqlens, max_new,
                                     sm_scale, window, out, lse, workspace, dev_err)
    if type(r) is int:
        raise Kv4Error("kv4_attention_gqa4", r)
    return r
