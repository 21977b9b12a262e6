// kv4_gqa_pages.cuh -- what the writes and read-backs of the grouped-query caches
// share: which page of which request a thread block stands for, the page table,
// 16-bit inputs, and the launch.
#pragma once

#include "kv4_gqa8_device.cuh"

namespace kv4 {

// The page of request `b` that a block of the grid stands for.  Blocks are
// laid out over page indices g(b) + p with g(b) = cu[b] / 64 + 2 b: a
// request's n tokens touch at most ceil(n / 64) + 1 <= g(b + 1) - g(b) pages,
// so no prefix sum over the requests is needed (at most two blocks per
// request find nothing to do).
struct PageItem {
  int b;
  int64_t row0;        // flat row of the first token at or after position 0 (cu[b] + skipped)
  int64_t start, end;  // token positions [start, end) of the request, start >= 0
  int64_t page;        // logical page
};
__device__ __forceinline__ int clamp_cu(int32_t v, int64_t n_tokens) {
  return v < 0 ? 0 : (v > n_tokens ? static_cast<int>(n_tokens) : v);
}

// starts: first position of each request's range, or null: the range ends at
// seq_lens (an append).  A warp looks for the request among 32 at a time, and
// reads what it needs of the last 32 in the same round (of 32 requests or
// fewer: one round of loads).
__device__ __forceinline__ bool find_page(const Gqa8Args& a, int w, PageItem& it) {
  const int lane = threadIdx.x & 31;
  int base = 0, n = a.B;                          // candidates base .. base + n - 1
  while (true) {
    const int step = (n + 31) / 32, b = base + lane * step;
    const bool in = lane * step < n;
    int c0 = 0, c1 = 0, at = 0;
    if (in) {
      c0 = load(a.cu + b);
      if (step == 1) {
        c1 = load(a.cu + b + 1);
        at = load((a.starts != nullptr ? a.starts : a.lens) + b);
      }
    }
    c0 = clamp_cu(c0, a.n_tokens);
    // the largest b with g(b) <= w
    const uint32_t below = __ballot_sync(0xFFFFFFFFu, in && (c0 >> 6) + 2 * b <= w);
    const int l = 31 - __clz(static_cast<int>(below | 1u));
    if (step > 1) {
      n = min(step, n - l * step);
      base += l * step;
      continue;
    }
    c0 = __shfl_sync(0xFFFFFFFFu, c0, l);
    c1 = clamp_cu(__shfl_sync(0xFFFFFFFFu, c1, l), a.n_tokens);
    at = __shfl_sync(0xFFFFFFFFu, at, l);
    it.b = base + l;
    const int p = w - (c0 >> 6) - 2 * it.b;
    const int64_t rows = c1 - c0;
    if (rows <= 0 || p < 0) return false;
    int64_t start = a.starts != nullptr ? static_cast<int64_t>(at) : static_cast<int64_t>(at) - rows;
    it.end = start + rows;
    it.row0 = c0;
    if (start < 0) {                              // tokens before position 0 have no place
      it.row0 -= start;
      start = 0;
    }
    it.start = start;
    it.page = (start >> 6) + p;
    return (it.page << 6) < it.end;
  }
}

// The request of flat row t and the row's position; false where it has none (rows
// behind the last request, positions below 0).
__device__ __forceinline__ bool find_token(const Gqa8Args& a, int t, int& b, int64_t& pos) {
  const int lane = threadIdx.x & 31;
  int base = 0, n = a.B;
  if (n > 32 && t < n) {
    // (a token each, as in a decode step: request t's)
    const int c0 = clamp_cu(load(a.cu + t), a.n_tokens), c1 = clamp_cu(load(a.cu + t + 1), a.n_tokens);
    const int len = load(a.lens + t);
    if (c0 <= t && t < c1) {
      b = t;
      pos = static_cast<int64_t>(len) - (c1 - t);
      return pos >= 0;
    }
  }
  while (true) {
    const int step = (n + 31) / 32, at = base + lane * step;
    const bool in = lane * step < n;
    int c0 = 0, c1 = 0, len = 0;
    if (in) {
      c0 = load(a.cu + at);
      if (step == 1) {
        c1 = load(a.cu + at + 1);
        len = load(a.lens + at);
      }
    }
    c0 = clamp_cu(c0, a.n_tokens);
    // the last request that begins at or before t (empty ones before it do too)
    const int l = 31 - __clz(static_cast<int>(__ballot_sync(0xFFFFFFFFu, in && c0 <= t) | 1u));
    if (step > 1) {
      n = min(step, n - l * step);
      base += l * step;
      continue;
    }
    c0 = __shfl_sync(0xFFFFFFFFu, c0, l);
    c1 = clamp_cu(__shfl_sync(0xFFFFFFFFu, c1, l), a.n_tokens);
    len = __shfl_sync(0xFFFFFFFFu, len, l);
    b = base + l;
    pos = static_cast<int64_t>(len) - (c1 - t);
    return t >= c0 && t < c1 && pos >= 0;
  }
}

// The table's entry, -1 where it has none; and the physical page of an entry, or
// -1 (flagged) where there is none.  (Apart, so that what does not depend on the
// page can be loaded before the entry is looked at: one round of latency less.)
__device__ __forceinline__ int table_entry(const Gqa8Args& a, const PageItem& it) {
  return it.page < a.pt_stride ? load(a.page_table + it.b * a.pt_stride + it.page) : -1;
}
__device__ __forceinline__ int64_t physical_page(const Gqa8Args& a, int64_t pg) {
  if (pg < 0 || pg >= a.num_pages) {
    if ((threadIdx.x & 31) == 0) flag_error(a.dev_err, kDevBadPage);
    return -1;
  }
  return pg;
}

// 8 values of 16 bits as floats.
template <bool F16>
__device__ __forceinline__ void widen8(const uint4& v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F16) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    } else {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}

// Largest magnitudes of two pairs of 16-bit values, pair by pair, a NaN where
// there is one; then that of a pair, as fp32 bits (which order like the
// values).
template <bool F16>
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t x) {
  uint32_t r;
  x &= 0x7FFF7FFFu;
  if constexpr (F16) asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(x));
  else asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(x));
  return r;
}
template <bool F16>
__device__ __forceinline__ uint32_t largest_bits(uint32_t m) {
  float lo, hi;
  if constexpr (F16) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&m));
    lo = f.x;
    hi = f.y;
  } else {
    lo = __uint_as_float(m << 16);
    hi = __uint_as_float(m & 0xFFFF0000u);
  }
  return max(__float_as_uint(lo) & 0x7FFFFFFFu, __float_as_uint(hi) & 0x7FFFFFFFu);
}

inline int64_t page_items(const Gqa8Args& a) { return a.n_tokens / kPage + 2 * static_cast<int64_t>(a.B); }

template <typename K>
cudaError_t launch_grid(K kernel, const Gqa8Args& a, dim3 grid, unsigned threads, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}
// A block for each `each` neighbouring pages (x) and what else there is of them (y).
template <typename K>
cudaError_t launch_pages(K kernel, const Gqa8Args& args, int each, unsigned y, unsigned threads,
                         cudaStream_t stream) {
  Gqa8Args a = args;
  a.each = each;
  return launch_grid(kernel, a, dim3(static_cast<unsigned>((page_items(a) + each - 1) / each), y), threads, stream);
}

}  // namespace kv4
