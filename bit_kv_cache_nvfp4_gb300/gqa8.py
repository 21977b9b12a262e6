"""The 8-bit grouped-query cache: append, read-back and attention.

Bindings of ``kv4_append_gqa8``, ``kv4_read_gqa8`` and ``kv4_attention_gqa8``
(C ABI in ``include/kv4mla.h``, which defines the layout, the exponents and the
masks).  The cache is two tensors:

    pool    uint8 [num_pages, Hkv, 2, 64, D]   E4M3 codes of K and V
    scales  uint8 [num_pages, Hkv, 2]          E8M0: value = code * 2^(byte - 127)

and a page table int32 [B, stride] as for the other caches of this package.
Tensors of one call are on one device, which need not be the current one; work
goes to that device's current stream.  No gradients are computed: the results of
inputs that require one carry none, and tensors that a call writes into count it
as a change in place.  The argument checks and the calls are in
the extension module ``_kv4torch`` (``csrc/kv4_torch.cpp``): these calls are
short enough for a binding in Python to be what they take.
"""
from __future__ import annotations

import ctypes
import importlib.util
import threading

import torch

from . import Kv4Error, _check, load_library

_ext = None
_ext_lock = threading.Lock()


def _extension():
    """The module _kv4torch, built if its sources are newer."""
    global _ext
    load_library()
    with _ext_lock:
        if _ext is None:
            from . import build as _build
            spec = importlib.util.spec_from_file_location("_kv4torch", _build.build_extension())
            mod = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(mod)
            _ext = mod
    return _ext


def append_gqa8(k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                page_table: torch.Tensor, seq_lens: torch.Tensor, pool: torch.Tensor,
                scales: torch.Tensor, dev_err: torch.Tensor | None = None) -> None:
    """Quantize new tokens into the cache (kv4_append_gqa8).

    k, v bf16 or f16 [T, Hkv, D] (strided: slices of a fused projection are
    fine); cu_seqlens int32 [B + 1]: request b's rows; seq_lens int32 [B]:
    tokens of each request, these included, so request b's rows go to positions
    seq_lens[b] - n .. seq_lens[b] - 1.  A page that already holds earlier
    tokens of the request keeps them; a page that receives tokens belongs to
    one request."""
    st = (_ext or _extension()).append(k, v, cu_seqlens, page_table, seq_lens, pool, scales, dev_err)
    if st:
        raise Kv4Error("kv4_append_gqa8", st)


def read_gqa8(pool: torch.Tensor, scales: torch.Tensor, page_table: torch.Tensor,
              starts: torch.Tensor, cu_seqlens: torch.Tensor, total: int,
              dtype: torch.dtype = torch.bfloat16, k_out: torch.Tensor | None = None,
              v_out: torch.Tensor | None = None, dev_err: torch.Tensor | None = None):
    """The values of a range of each request's tokens (kv4_read_gqa8).

    Request b's positions starts[b] .. starts[b] + n - 1 go to rows
    cu_seqlens[b] .. cu_seqlens[b+1] - 1 of k and v [total, Hkv, D], n being
    their number; other rows are left as they are.  Returns (k, v)."""
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise TypeError(f"dtype must be bfloat16 or float16, got {dtype}")
    r = (_ext or _extension()).read(pool, scales, page_table, starts, cu_seqlens, total,
                                    dtype is torch.float16, k_out, v_out, dev_err)
    if type(r) is int:
        raise Kv4Error("kv4_read_gqa8", r)
    return r


def attention_gqa8_workspace(B: int, max_new: int, total: int, hq: int, hkv: int, d: int,
                             device=None) -> int:
    """Workspace bytes of attention_gqa8 for `total` new tokens of B requests,
    at most max_new each."""
    n = ctypes.c_size_t(0)
    with torch.cuda.device(device):
        _check("kv4_attention_gqa8_plan", load_library().kv4_attention_gqa8_plan(
            B, max_new, total, hq, hkv, d, ctypes.byref(n)))
    return n.value


def attention_gqa8(q: torch.Tensor, pool: torch.Tensor, scales: torch.Tensor,
                   page_table: torch.Tensor, seq_lens: torch.Tensor, cu_seqlens: torch.Tensor,
                   max_new: int, sm_scale: float, window: int = 0,
                   out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, dev_err: torch.Tensor | None = None):
    """Causal attention of the new tokens over the cache (kv4_attention_gqa8).

    q bf16 or f16 [T, Hq, D] (strided), Hq a multiple of the cache's Hkv;
    cu_seqlens int32 [B + 1]: request b's rows; seq_lens int32 [B]: tokens of
    each request, these included (append them first); max_new: the most rows of
    any request; window > 0: a row sees only that many keys, its own the last.
    Returns (out [T, Hq, D] of q's type, lse fp32 [T, Hq]); a row without a key
    gives 0 and -inf, rows from cu_seqlens[B] on are left as they are.  Without
    `workspace` each call takes its own from PyTorch's allocator."""
    r = (_ext or _extension()).attention(q, pool, scales, page_table, seq_lens, cu_seqlens, max_new,
                                         sm_scale, window, out, lse, workspace, dev_err)
    if type(r) is int:
        raise Kv4Error("kv4_attention_gqa8", r)
    return r
