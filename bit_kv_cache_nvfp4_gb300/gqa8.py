"""The 8-bit grouped-query cache: append, read-back and attention.

Bindings of ``kv4_append_gqa8``, ``kv4_read_gqa8`` and ``kv4_attention_gqa8``
(C ABI in ``include/kv4mla.h``, which defines the layout, the exponents and the
masks).  The cache is two tensors:

    pool    uint8 [num_pages, Hkv, 2, 64, D]   E4M3 codes of K and V
    scales  uint8 [num_pages, Hkv, 2]          E8M0: value = code * 2^(byte - 127)

and a page table int32 [B, stride] as for the other caches of this package.
Tensors of one call are on one device, which need not be the current one; work
goes to that device's current stream.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import PAGE, _check, load_library

_DTYPES = {torch.bfloat16: 0, torch.float16: 1}
_stream_of = torch._C._cuda_getCurrentRawStream


def _tensor(t, name: str, dtype, dim: int, device):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, got {t.dim()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the pool on {device}")
    return t.data_ptr()


def _strided(t, name: str, dtype, device):
    """Pointer and (token, head) strides of a [T, heads, D] input."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the pool on {device}")
    s0, s1, s2 = t.stride()
    if s2 != 1 or s0 % 8 or s1 % 8 or t.data_ptr() % 16:
        raise ValueError(f"{name}: the last dimension must be contiguous, the other strides "
                         "multiples of 8 elements and the data 16-byte aligned")
    return t.data_ptr(), s0, s1


def _cache(pool, scales, page_table):
    """(device, num_pages, Hkv, D) of a cache, and the three pointers."""
    if not isinstance(pool, torch.Tensor) or not pool.is_cuda:
        raise TypeError("pool must be a CUDA tensor")
    if pool.dim() != 5 or pool.shape[2] != 2 or pool.shape[3] != PAGE:
        raise ValueError("pool must be [num_pages, Hkv, 2, 64, D]")
    num_pages, hkv, _, _, d = pool.shape
    if hkv < 1:
        raise ValueError("the cache needs at least one head")
    dev = pool.device
    p = _tensor(pool, "pool", torch.uint8, 5, dev)
    s = _tensor(scales, "scales", torch.uint8, 3, dev)
    if scales.shape != (num_pages, hkv, 2):
        raise ValueError(f"scales must be [{num_pages}, {hkv}, 2]")
    return dev, num_pages, hkv, d, p, s, _tensor(page_table, "page_table", torch.int32, 2, dev)


def _ragged(cu_seqlens, lens, lens_name, page_table, device):
    """Pointers of cu_seqlens [B + 1] and a per-request int32 [B]; B."""
    B = page_table.shape[0]
    c = _tensor(cu_seqlens, "cu_seqlens", torch.int32, 1, device)
    n = _tensor(lens, lens_name, torch.int32, 1, device)
    if cu_seqlens.shape[0] != B + 1 or lens.shape[0] != B:
        raise ValueError(f"page_table [B, *], cu_seqlens [B + 1] and {lens_name} [B] must agree")
    return c, n, B


def _err(dev_err, device):
    return None if dev_err is None else _tensor(dev_err, "dev_err", torch.int32, 1, device)


def _call(fn: str, device, *args):
    """The library's function on `device` and its current stream."""
    f = getattr(load_library(), fn)
    index = device.index
    if index == torch.cuda.current_device():
        _check(fn, f(*args, _stream_of(index)))
    else:
        with torch.cuda.device(index):
            _check(fn, f(*args, _stream_of(index)))


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
    dev, num_pages, hkv, d, pool_p, scales_p, pt_p = _cache(pool, scales, page_table)
    if k.dtype not in _DTYPES:
        raise TypeError(f"k must be bfloat16 or float16, got {k.dtype}")
    if k.dim() != 3 or k.shape != v.shape or k.shape[1] != hkv or k.shape[2] != d:
        raise ValueError(f"k and v must be [T, {hkv}, {d}]")
    kp, ks0, ks1 = _strided(k, "k", k.dtype, dev)
    vp, vs0, vs1 = _strided(v, "v", k.dtype, dev)
    cu_p, len_p, B = _ragged(cu_seqlens, seq_lens, "seq_lens", page_table, dev)
    _call("kv4_append_gqa8", dev, kp, ks0, ks1, vp, vs0, vs1, _DTYPES[k.dtype], k.shape[0], cu_p,
          pt_p, page_table.shape[1], PAGE, len_p, B, hkv, d, pool_p, scales_p, num_pages,
          _err(dev_err, dev))


def read_gqa8(pool: torch.Tensor, scales: torch.Tensor, page_table: torch.Tensor,
              starts: torch.Tensor, cu_seqlens: torch.Tensor, total: int,
              dtype: torch.dtype = torch.bfloat16, k_out: torch.Tensor | None = None,
              v_out: torch.Tensor | None = None, dev_err: torch.Tensor | None = None):
    """The values of a range of each request's tokens (kv4_read_gqa8).

    Request b's positions starts[b] .. starts[b] + n - 1 go to rows
    cu_seqlens[b] .. cu_seqlens[b+1] - 1 of k and v [total, Hkv, D], n being
    their number; other rows are left as they are.  Returns (k, v)."""
    dev, num_pages, hkv, d, pool_p, scales_p, pt_p = _cache(pool, scales, page_table)
    if dtype not in _DTYPES:
        raise TypeError(f"dtype must be bfloat16 or float16, got {dtype}")
    if total < 0:
        raise ValueError("total must not be negative")
    shape = (total, hkv, d)
    if k_out is None:
        k_out = torch.empty(shape, dtype=dtype, device=dev)
    if v_out is None:
        v_out = torch.empty(shape, dtype=dtype, device=dev)
    if k_out.shape != shape or v_out.shape != shape:
        raise ValueError(f"k_out and v_out must be [{total}, {hkv}, {d}]")
    cu_p, start_p, B = _ragged(cu_seqlens, starts, "starts", page_table, dev)
    _call("kv4_read_gqa8", dev, pool_p, scales_p, num_pages, pt_p, page_table.shape[1], PAGE,
          start_p, cu_p, total, B, hkv, d, _DTYPES[dtype], _tensor(k_out, "k_out", dtype, 3, dev),
          _tensor(v_out, "v_out", dtype, 3, dev), _err(dev_err, dev))
    return k_out, v_out


@functools.lru_cache(maxsize=1024)
def _plan(index: int, B: int, max_new: int, total: int, hq: int, hkv: int, d: int) -> int:
    n = ctypes.c_size_t(0)
    with torch.cuda.device(index):
        _check("kv4_attention_gqa8_plan", load_library().kv4_attention_gqa8_plan(
            B, max_new, total, hq, hkv, d, ctypes.byref(n)))
    return n.value


def attention_gqa8_workspace(B: int, max_new: int, total: int, hq: int, hkv: int, d: int,
                             device=None) -> int:
    """Workspace bytes of attention_gqa8 for `total` new tokens of B requests,
    at most max_new each."""
    index = torch.device("cuda" if device is None else device).index
    return _plan(torch.cuda.current_device() if index is None else index, B, max_new, total, hq,
                 hkv, d)


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
    dev, num_pages, hkv, d, pool_p, scales_p, pt_p = _cache(pool, scales, page_table)
    dt = q.dtype
    if dt not in _DTYPES:
        raise TypeError(f"q must be bfloat16 or float16, got {dt}")
    if q.dim() != 3 or q.shape[2] != d or q.shape[1] % hkv:
        raise ValueError(f"q must be [T, Hq, {d}] with Hq a multiple of {hkv}")
    t, hq, _ = q.shape
    qp, qs0, qs1 = _strided(q, "q", dt, dev)
    cu_p, len_p, B = _ragged(cu_seqlens, seq_lens, "seq_lens", page_table, dev)
    if out is None:
        out = torch.empty((t, hq, d), dtype=dt, device=dev)
    elif out.shape != q.shape:
        raise ValueError(f"out must be [{t}, {hq}, {d}]")
    if lse is None:
        lse = torch.empty((t, hq), dtype=torch.float32, device=dev)
    elif lse.shape != (t, hq):
        raise ValueError(f"lse must be [{t}, {hq}]")
    ws_p, ws_n = None, 0
    if workspace is None:
        ws_n = _plan(dev.index, B, max_new, t, hq, hkv, d)
        if ws_n:
            workspace = torch.empty(ws_n, dtype=torch.uint8, device=dev)
            ws_p = workspace.data_ptr()
    else:
        ws_p = _tensor(workspace, "workspace", torch.uint8, 1, dev)
        ws_n = workspace.numel()
    _call("kv4_attention_gqa8", dev, qp, qs0, qs1, _DTYPES[dt], t, cu_p, max_new, pool_p, scales_p,
          num_pages, pt_p, page_table.shape[1], PAGE, len_p, B, hq, hkv, d, window, sm_scale,
          _tensor(out, "out", dt, 3, dev), _tensor(lse, "lse", torch.float32, 2, dev), ws_p, ws_n,
          _err(dev_err, dev))
    return out, lse
