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
#include "kv4_gqa_pages.cuh"

namespace kv4 {
namespace {

constexpr int kThreads = 256;         // of a block of the read-back
constexpr int kAppendThreads = 128;   // and of the write

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
