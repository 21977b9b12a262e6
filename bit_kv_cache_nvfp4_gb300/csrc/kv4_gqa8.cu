// kv4_gqa8.cu -- write and read-back of the 8-bit grouped-query cache
// (kv4_append_gqa8, kv4_read_gqa8).
//
// A page holds 64 tokens of one request; the block of a (page, kv head, side)
// is 64 x D E4M3 codes with one E8M0 exponent byte, value = code * 2^(byte -
// 127).  The exponent is the least e with amax <= 448 * 2^e, kept in
// [-48, 48].  E4M3 is itself a floating-point code, so a power-of-two scale
// costs it no precision (only where in its 15 octaves a block sits), x * 2^-e
// is exact, and a page whose exponent has to rise when tokens join it keeps
// its codes exactly but for those that fall into the code's subnormal range.
//
// The write gives a thread block to one (page of a request, kv head, side),
// the unit whose maximum it needs: its 64 x D values (16 KB of inputs at
// D = 128) stay in the threads' registers between the maximum and the codes, so
// the inputs are read once.  The read-back gives a block to a page and head.
// Both are bound by HBM in large calls (9 prompts, 171 MB: 27.3 us, 6.3 TB/s; 12
// prefixes read back, 431 MB: 71 us, 6.0 TB/s) and by three dependent loads
// (request, page, block) in small ones (one token: 2.6 us).
#include "kv4_gqa8_device.cuh"

namespace kv4 {
namespace {

constexpr int kThreads = 256;         // of a block of the read-back
constexpr int kAppendThreads = 128;   // and of the write

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

__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float hi, float lo) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint4 encode16(const float* x, float f) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = f32x2_to_e4m3x2(x[4 * i + 1] * f, x[4 * i] * f) |
           (f32x2_to_e4m3x2(x[4 * i + 3] * f, x[4 * i + 2] * f) << 16);
  return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ void decode16(const uint4& c, float* x) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t h = e4m3x2_to_f16x2((w[i] >> (16 * j)) & 0xFFFFu);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      x[4 * i + 2 * j] = f.x;
      x[4 * i + 2 * j + 1] = f.y;
    }
  }
}

// Least e with amax <= 448 * 2^e = 1.75 * 2^(e + 8), from the bits of a finite
// fp32 amax; [-48, 48].
__device__ __forceinline__ int block_exponent(uint32_t amax_bits) {
  const int e = static_cast<int>(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return e < kGqa8ExpMin ? kGqa8ExpMin : (e > kGqa8ExpMax ? kGqa8ExpMax : e);
}

template <int D, bool F16>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(Gqa8Args a) {
  constexpr int TPR = D / 16;                      // threads per token row
  constexpr int RPP = kAppendThreads / TPR;        // rows per pass
  constexpr int PASSES = kPage / RPP;
  grid_dependency_wait();
  grid_launch_dependents();
  __shared__ uint32_t red[kAppendThreads / 32];
  PageItem it;
  if (!find_page(a, blockIdx.x, it)) return;
  const int entry = table_entry(a, it);
  const int h = blockIdx.y >> 1, s = blockIdx.y & 1, tid = threadIdx.x;
  const int lo = it.start > (it.page << 6) ? static_cast<int>(it.start & 63) : 0;
  const int hi = it.end - (it.page << 6) < kPage ? static_cast<int>(it.end - (it.page << 6)) : kPage;
  const int64_t row_of_0 = it.row0 + (it.page << 6) - it.start;     // flat row of the page's row 0
  const int col = (tid % TPR) * 16, r0 = tid / TPR;
  const int64_t ts = s == 0 ? a.k_token_stride : a.v_token_stride;
  const uint16_t* src = (s == 0 ? static_cast<const uint16_t*>(a.k) + h * a.k_head_stride
                                : static_cast<const uint16_t*>(a.v) + h * a.v_head_stride) + col;
  uint4 x[PASSES][2];
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int r = r0 + p * RPP;
    x[p][0] = x[p][1] = make_uint4(0, 0, 0, 0);
    if (r >= lo && r < hi) {
      const uint4* g = reinterpret_cast<const uint4*>(src + (row_of_0 + r) * ts);
      x[p][0] = load(g);
      x[p][1] = load(g + 1);
    }
  }
  const int64_t pg = physical_page(a, entry);
  if (pg < 0) return;
  uint8_t* const scale = a.scales + (pg * a.Hkv + h) * 2 + s;
  uint32_t m2 = 0;
#pragma unroll
  for (int p = 0; p < PASSES; ++p)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      m2 = max_abs2<F16>(max_abs2<F16>(m2, x[p][j].x), x[p][j].y);
      m2 = max_abs2<F16>(max_abs2<F16>(m2, x[p][j].z), x[p][j].w);
    }
  uint32_t m = largest_bits<F16>(m2);
  // (nearly always none:) a NaN or an infinity does not count and is flagged,
  // and a NaN gives code 0
  const bool odd = m >= 0x7F800000u;
  if (odd) {
    flag_error(a.dev_err, kDevNonFinite);
    m = 0;
#pragma unroll
    for (int p = 0; p < PASSES; ++p)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float f[8];
        widen8<F16>(x[p][j], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t u = __float_as_uint(f[i]) & 0x7FFFFFFFu;
          if (u < 0x7F800000u) m = max(m, u);
        }
      }
  }
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if ((tid & 31) == 0) red[tid >> 5] = m;
  int old = kGqa8ExpMin;
  if (lo > 0) old = min(max(static_cast<int>(*scale) - 127, kGqa8ExpMin), kGqa8ExpMax);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kAppendThreads / 32; ++i) m = max(m, red[i]);
  const int e = max(block_exponent(m), old);
  if (tid == 0) *scale = static_cast<uint8_t>(e + 127);
  uint8_t* const blk = a.pool + ((pg * a.Hkv + h) * 2 + s) * (kPage * D) + col;
  const float f = pow2f(-e);
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int r = r0 + p * RPP;
    if (r >= lo && r < hi) {
      float v[16];
      widen8<F16>(x[p][0], v);
      widen8<F16>(x[p][1], v + 8);
      if (odd) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = v[i] == v[i] ? v[i] : 0.0f;
      }
      *reinterpret_cast<uint4*>(blk + r * D) = encode16(v, f);
    } else if (r < lo && e > old) {
      uint4* c = reinterpret_cast<uint4*>(blk + r * D);
      float v[16];
      decode16(*c, v);
      *c = encode16(v, pow2f(old - e));
    }
  }
}

// The same with a warp for each (page, head, side): where most pages get a
// token or two (a decode step), a block a page would leave most of its threads
// without a row.  The few rows are read twice, the second time from cache.
template <int D, bool F16>
__global__ void __launch_bounds__(128) append_rows_kernel(Gqa8Args a) {
  constexpr int TPR = D / 16, RPP = 32 / TPR;
  grid_dependency_wait();
  grid_launch_dependents();
  PageItem it;
  if (!find_page(a, blockIdx.x, it)) return;
  const int entry = table_entry(a, it);
  const int lane = threadIdx.x & 31, unit = blockIdx.y * 4 + (threadIdx.x >> 5), h = unit >> 1, s = unit & 1;
  if (h >= a.Hkv) return;
  const int lo = it.start > (it.page << 6) ? static_cast<int>(it.start & 63) : 0;
  const int hi = it.end - (it.page << 6) < kPage ? static_cast<int>(it.end - (it.page << 6)) : kPage;
  const int64_t row_of_0 = it.row0 + (it.page << 6) - it.start;
  const int col = (lane % TPR) * 16, r0 = lane / TPR;
  const int64_t ts = s == 0 ? a.k_token_stride : a.v_token_stride;
  const uint16_t* src = (s == 0 ? static_cast<const uint16_t*>(a.k) + h * a.k_head_stride
                                : static_cast<const uint16_t*>(a.v) + h * a.v_head_stride) + col;
  uint32_t m = 0;
  bool odd = false;
  auto row_in = [&](int r, float (&v)[16]) {
    const uint4* g = reinterpret_cast<const uint4*>(src + (row_of_0 + r) * ts);
    const uint4 x0 = load(g), x1 = load(g + 1);
    widen8<F16>(x0, v);
    widen8<F16>(x1, v + 8);
  };
  for (int r = lo + r0; r < hi; r += RPP) {
    float v[16];
    row_in(r, v);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t u = __float_as_uint(v[i]) & 0x7FFFFFFFu;
      if (u >= 0x7F800000u) odd = true; else m = max(m, u);
    }
  }
  const int64_t pg = physical_page(a, entry);
  if (pg < 0) return;
  if (odd) flag_error(a.dev_err, kDevNonFinite);
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  uint8_t* const scale = a.scales + (pg * a.Hkv + h) * 2 + s;
  int old = kGqa8ExpMin;
  if (lo > 0) old = min(max(static_cast<int>(*scale) - 127, kGqa8ExpMin), kGqa8ExpMax);
  const int e = max(block_exponent(m), old);
  __syncwarp();
  if (lane == 0) *scale = static_cast<uint8_t>(e + 127);
  uint8_t* const blk = a.pool + ((pg * a.Hkv + h) * 2 + s) * (kPage * D) + col;
  if (e > old && lo > 0) {
    for (int r = r0; r < lo; r += RPP) {
      uint4* c = reinterpret_cast<uint4*>(blk + r * D);
      float v[16];
      decode16(*c, v);
      *c = encode16(v, pow2f(old - e));
    }
  }
  for (int r = lo + r0; r < hi; r += RPP) {
    float v[16];
    row_in(r, v);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = v[i] == v[i] ? v[i] : 0.0f;
    *reinterpret_cast<uint4*>(blk + r * D) = encode16(v, pow2f(-e));
  }
}

// Two floats -> 16-bit pair (first in the low half), round half to even; f16
// saturates at 65504 (what rounds to an infinity becomes that), and a NaN stays
// one.
template <bool F16>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
  if constexpr (F16) {
    const __half2 top = __float2half2_rn(65504.0f);
    const __half2 h = __hmax2_nan(__hmin2_nan(__floats2half2_rn(lo, hi), top), __hneg2(top));
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// A block reads a.each neighbouring pages of its head: one where there are
// fewer blocks than the SMs hold, kReadEach where there are several times as
// many (12 prefixes, 431 MB: 74.5 us with 1, 70.8 with 2; 3 prefixes, 0.9 MB:
// 3.1 and 4.1).  Five blocks an SM (48 registers a thread): with the four that
// 64 registers leave, the 128 single pages of a decode step take 0.7 us more.
constexpr int kReadEach = 2;
template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 5) read_kernel(Gqa8Args a) {
  constexpr int TPR = D / 16, RPP = kThreads / TPR, PASSES = kPage / RPP;
  grid_dependency_wait();
  grid_launch_dependents();
  const int h = blockIdx.y, tid = threadIdx.x;
  const int col = (tid % TPR) * 16, r0 = tid / TPR;
#pragma unroll 1
  for (int w = a.each * static_cast<int>(blockIdx.x); w < a.each * (static_cast<int>(blockIdx.x) + 1); ++w) {
    PageItem it;
    if (!find_page(a, w, it)) continue;
    const int64_t pg = physical_page(a, table_entry(a, it));
    const int lo = it.start > (it.page << 6) ? static_cast<int>(it.start & 63) : 0;
    const int hi = it.end - (it.page << 6) < kPage ? static_cast<int>(it.end - (it.page << 6)) : kPage;
    const int64_t row_of_0 = it.row0 + (it.page << 6) - it.start;
    uint4 c[2][PASSES];
    float f[2] = {0.0f, 0.0f};
    bool twice[2] = {false, false};
    if (pg >= 0) {
      const uint8_t* blk = a.pool + (pg * a.Hkv + h) * 2 * (kPage * D) + col;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        // 2^(byte - 127): fp32's exponent field as it is, but for 2^-127, which is
        // subnormal, and 2^128, which goes in as 2^127 and a factor of two
        const uint32_t byte = load(a.scales + (pg * a.Hkv + h) * 2 + s);
        f[s] = byte == 0 ? 0x1p-127f : __uint_as_float(min(byte, 254u) << 23);
        twice[s] = byte == 255;
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
          const int r = r0 + p * RPP;
          c[s][p] = r >= lo && r < hi ? load(reinterpret_cast<const uint4*>(blk + (s * kPage + r) * D))
                                      : make_uint4(0, 0, 0, 0);
        }
      }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int r = r0 + p * RPP;
        if (r < lo || r >= hi) continue;
        uint4 o[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        if (pg >= 0) {
          float v[16];
          decode16(c[s][p], v);
          if (twice[s]) {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] *= 2.0f;
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float* u = v + 8 * j;
            o[j] = make_uint4(narrow2<F16>(u[0] * f[s], u[1] * f[s]), narrow2<F16>(u[2] * f[s], u[3] * f[s]),
                              narrow2<F16>(u[4] * f[s], u[5] * f[s]), narrow2<F16>(u[6] * f[s], u[7] * f[s]));
          }
        }
        uint16_t* dst = static_cast<uint16_t*>(s == 0 ? a.k_out : a.v_out) +
                        ((row_of_0 + r) * a.Hkv + h) * D + col;
        reinterpret_cast<uint4*>(dst)[0] = o[0];
        reinterpret_cast<uint4*>(dst)[1] = o[1];
      }
  }
}

int64_t page_items(const Gqa8Args& a) { return a.n_tokens / kPage + 2 * static_cast<int64_t>(a.B); }

template <typename K>
cudaError_t launch_pages(K kernel, const Gqa8Args& args, int each, unsigned y, unsigned threads,
                         cudaStream_t stream) {
  Gqa8Args a = args;
  a.each = each;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((page_items(a) + each - 1) / each), y);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int D, bool F16>
cudaError_t launch_append(const Gqa8Args& a, cudaStream_t stream) {
  // fewer than 8 tokens a request on average: a warp for each block of codes
  if (a.n_tokens < 8 * static_cast<int64_t>(a.B))
    return launch_pages(append_rows_kernel<D, F16>, a, 1, (2 * a.Hkv + 3) / 4, 128, stream);
  return launch_pages(append_kernel<D, F16>, a, 1, 2 * a.Hkv, kAppendThreads, stream);
}

}  // namespace

cudaError_t launch_append_gqa8(const Gqa8Args& a, cudaStream_t stream) {
  if (a.D == 64) return a.f16 ? launch_append<64, true>(a, stream) : launch_append<64, false>(a, stream);
  return a.f16 ? launch_append<128, true>(a, stream) : launch_append<128, false>(a, stream);
}

cudaError_t launch_read_gqa8(const Gqa8Args& a, cudaStream_t stream) {
  // 8 blocks of 256 threads an SM
  const int each = page_items(a) * a.Hkv >= 3 * 8 * static_cast<int64_t>(a.num_sms) ? kReadEach : 1;
  if (a.D == 64)
    return a.f16 ? launch_pages(read_kernel<64, true>, a, each, a.Hkv, kThreads, stream)
                 : launch_pages(read_kernel<64, false>, a, each, a.Hkv, kThreads, stream);
  return a.f16 ? launch_pages(read_kernel<128, true>, a, each, a.Hkv, kThreads, stream)
               : launch_pages(read_kernel<128, false>, a, each, a.Hkv, kThreads, stream);
}

}  // namespace kv4
