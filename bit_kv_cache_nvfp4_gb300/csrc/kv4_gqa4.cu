// kv4_gqa4.cu -- write and read-back of the 4-bit grouped-query cache
// (kv4_append_gqa4, kv4_read_gqa4).
//
// A page holds 64 tokens of one request; the block of a (page, kv head, side)
// is 64 rows of D / 2 bytes of E2M1 codes and, in a second tensor, 64 rows of
// D / 16 E4M3 scales, value = code * scale.  A row depends on its token alone:
//   scale = E4M3(amax / 6),  code = E2M1(x / scale)   of 16 elements
// both rounded half to even and saturating, so rows that are there stay as
// they are.
//
// Both are bound by HBM in large calls: 9 prompts of 28,000 tokens written, 147 MB, in
// 26.5 us, 5.5 TB/s (2.9 instructions a clock and SM: the rounding is what is near its
// limit too), 12 prefixes read back, 368 MB, in 59 us, 6.2 TB/s.  In small ones they are
// bound by their dependent loads: the write of a token each of 128 requests takes 1.8
// us (request, page, with the inputs on their way), the read-back of their pages 6.7.
#include "kv4_gqa_pages.cuh"

namespace kv4 {
namespace {

constexpr int kThreads = 256;         // of a block of the read-back
constexpr int kAppendThreads = 128;   // and of the write

// Eight values -> eight E2M1 codes, the first in the lowest bits.
__device__ __forceinline__ uint32_t e2m1x8_of_f32(const float* y) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return r;
}
// The larger magnitude of each pair (under any sign), a NaN where there is one.
template <bool F16>
__device__ __forceinline__ uint32_t max_magnitude2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (F16) asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// One block: 16 values of 16 bits -> 8 bytes of codes and the scale's byte.
// x / s is taken as x * r, r = 1 / s to 2 ulp, rounded to a multiple of 2^-14 by adding
// and taking off 768 (the product of the first addition is exact): x has at most 11
// bits, s 4 and a border between two codes 3, so x / s is either a border exactly,
// which the product is within 2^-19 of (borders are 5 at most, r is within 2^-22 of
// itself) and that rounding makes exact again, or at least 2^-13 away from it (borders
// lie at 2^-2 and above), which neither can bridge.  The conversion then decides every
// code as the quotient itself would.  amax / 6 becomes the scale in the same way: amax *
// fl(1 / 6) is rounded to 16 significant bits, and then decides as the quotient would.
// A NaN counts as 0 and an infinity saturates; neither counts for amax, and `odd` is set.
template <bool F16>
__device__ __forceinline__ uint2 quantize16(const uint4& a, const uint4& b, uint32_t& scale, bool& odd) {
  float x[16];
  widen8<F16>(a, x);
  widen8<F16>(b, x + 8);
  const uint32_t m0 = max_magnitude2<F16>(max_magnitude2<F16>(a.x, a.y), max_magnitude2<F16>(a.z, a.w));
  const uint32_t m1 = max_magnitude2<F16>(max_magnitude2<F16>(b.x, b.y), max_magnitude2<F16>(b.z, b.w));
  uint32_t m = largest_bits<F16>(max_magnitude2<F16>(m0, m1));
  if (m >= 0x7F800000u) {
    odd = true;
    m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t u = __float_as_uint(x[i]) & 0x7FFFFFFFu;
      if (u < 0x7F800000u) m = max(m, u);
      if (u > 0x7F800000u) x[i] = 0.0f;
    }
  }
  const float sixth = __uint_as_float((__float_as_uint(__uint_as_float(m) * (1.0f / 6.0f)) + 0x80u) & 0xFFFFFF00u);
  uint16_t s2;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s2) : "f"(0.0f), "f"(sixth));
  scale = s2;
  const float r = __fdividef(1.0f, fmaxf(e4m3_to_float(scale), 0x1p-9f));
  float y[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) y[i] = copysignf(__fadd_rn(__fmaf_rn(x[i], r, 768.0f), -768.0f), x[i]);
  return scale != 0 ? make_uint2(e2m1x8_of_f32(y), e2m1x8_of_f32(y + 8)) : make_uint2(0, 0);
}

// Row r of a (page, head, side) block, column block c.
template <int D>
__device__ __forceinline__ void store_block(const Gqa8Args& a, int64_t blk, int r, int c, const uint2& codes,
                                            uint32_t scale) {
  const int64_t row = blk * kPage + r;
  *reinterpret_cast<uint2*>(a.pool + row * (D / 2) + c * 8) = codes;
  a.scales[row * (D / 16) + c] = static_cast<uint8_t>(scale);
}

// A block for each (page, kv head, side): a thread takes 16 elements of a row, so
// that a warp reads whole rows and writes 256 contiguous bytes of codes and one
// sector of scales.
template <int D, bool F16>
__global__ void __launch_bounds__(kAppendThreads) append4_kernel(Gqa8Args a) {
  constexpr int TPR = D / 16, RPP = kAppendThreads / TPR, PASSES = kPage / RPP;
  grid_dependency_wait();
  grid_launch_dependents();
  PageItem it;
  if (!find_page(a, blockIdx.x, it)) return;
  const int entry = table_entry(a, it);
  const int h = blockIdx.y >> 1, s = blockIdx.y & 1, tid = threadIdx.x;
  const int lo = it.start > (it.page << 6) ? static_cast<int>(it.start & 63) : 0;
  const int hi = it.end - (it.page << 6) < kPage ? static_cast<int>(it.end - (it.page << 6)) : kPage;
  const int64_t row_of_0 = it.row0 + (it.page << 6) - it.start;     // flat row of the page's row 0
  const int c = tid % TPR, r0 = tid / TPR;
  const int64_t ts = s == 0 ? a.k_token_stride : a.v_token_stride;
  const uint16_t* src = (s == 0 ? static_cast<const uint16_t*>(a.k) + h * a.k_head_stride
                                : static_cast<const uint16_t*>(a.v) + h * a.v_head_stride) + c * 16;
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
  bool odd = false;
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int r = r0 + p * RPP;
    uint32_t scale;
    const uint2 codes = quantize16<F16>(x[p][0], x[p][1], scale, odd);
    if (r >= lo && r < hi) store_block<D>(a, (pg * a.Hkv + h) * 2 + s, r, c, codes, scale);
  }
  if (odd) flag_error(a.dev_err, kDevNonFinite);
}

// The same with a warp's threads on the blocks of one token, all heads and both
// sides: where most pages get a token or two (a decode step), a block a page
// would leave most of its threads without a row.
template <int D, bool F16>
__global__ void __launch_bounds__(kAppendThreads) append4_rows_kernel(Gqa8Args a) {
  constexpr int TPR = D / 16;
  grid_dependency_wait();
  grid_launch_dependents();
  // (the inputs' place is known before the page's: their loads go first)
  const int t = blockIdx.x, u = blockIdx.y * kAppendThreads + threadIdx.x;
  const int c = u % TPR, hs = u / TPR, s = hs >= a.Hkv ? 1 : 0, h = hs - s * a.Hkv;
  const bool mine = hs < 2 * a.Hkv;
  uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
  if (mine) {
    const uint16_t* src = s == 0 ? static_cast<const uint16_t*>(a.k) + t * a.k_token_stride + h * a.k_head_stride
                                 : static_cast<const uint16_t*>(a.v) + t * a.v_token_stride + h * a.v_head_stride;
    const uint4* g = reinterpret_cast<const uint4*>(src + c * 16);
    x0 = load(g);
    x1 = load(g + 1);
  }
  int b, entry = -1;
  int64_t pos;
  if (!find_token(a, t, b, pos)) return;
  if ((pos >> 6) < a.pt_stride) entry = load(a.page_table + b * a.pt_stride + (pos >> 6));
  const int64_t pg = physical_page(a, entry);
  if (pg < 0 || !mine) return;
  bool odd = false;
  uint32_t scale;
  const uint2 codes = quantize16<F16>(x0, x1, scale, odd);
  store_block<D>(a, (pg * a.Hkv + h) * 2 + s, static_cast<int>(pos & 63), c, codes, scale);
  if (odd) flag_error(a.dev_err, kDevNonFinite);
}

// 8 codes times a scale, as 8 values of 16 bits: exact in both types (at most 6
// significant bits, magnitudes from 2^-10 to 2688; a NaN scale gives NaNs).
template <bool F16>
__device__ __forceinline__ uint4 values8(uint32_t codes, uint32_t scale) {
  const __half2 s = bits_h2(e4m3x2_to_f16x2(scale));
  uint32_t h[4];
  e2m1x8_to_f16x8(codes, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 v = __hmul2(bits_h2(h[i]), __low2half2(s));
    h[i] = h2_bits(v);
    if constexpr (!F16) {
      const float2 f = __half22float2(v);
      h[i] = pack16<false>(f.x, f.y);
    }
  }
  return make_uint4(h[0], h[1], h[2], h[3]);
}

// A block for a page and a.each of its heads; a thread takes 8 elements of a row, so
// that a warp writes 512 contiguous bytes at once (with 16, of which each store takes
// every other half sector: 70.4 us for 12 prefixes, 59.2 so).
template <int D, bool F16>
__global__ void __launch_bounds__(kThreads) read4_kernel(Gqa8Args a) {
  constexpr int TPR = D / 8, RPP = kThreads / TPR, PASSES = kPage / RPP;
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x, c = tid % TPR, r0 = tid / TPR;
  PageItem it;
  if (!find_page(a, blockIdx.x, it)) return;
  const int64_t pg = physical_page(a, table_entry(a, it));
  const int lo = it.start > (it.page << 6) ? static_cast<int>(it.start & 63) : 0;
  const int hi = it.end - (it.page << 6) < kPage ? static_cast<int>(it.end - (it.page << 6)) : kPage;
  const int64_t row_of_0 = it.row0 + (it.page << 6) - it.start;
#pragma unroll 1
  for (int h = blockIdx.y * a.each; h < min(a.Hkv, static_cast<int>(blockIdx.y + 1) * a.each); ++h) {
    uint32_t codes[2][PASSES], scale[2][PASSES];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int r = r0 + p * RPP;
        codes[s][p] = scale[s][p] = 0;
        if (pg >= 0 && r >= lo && r < hi) {
          const int64_t row = ((pg * a.Hkv + h) * 2 + s) * kPage + r;
          codes[s][p] = load(reinterpret_cast<const uint32_t*>(a.pool + row * (D / 2)) + c);
          scale[s][p] = load(a.scales + row * (D / 16) + c / 2);
        }
      }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int r = r0 + p * RPP;
        if (r < lo || r >= hi) continue;
        uint16_t* dst = static_cast<uint16_t*>(s == 0 ? a.k_out : a.v_out) + ((row_of_0 + r) * a.Hkv + h) * D;
        reinterpret_cast<uint4*>(dst)[c] = values8<F16>(codes[s][p], scale[s][p]);
      }
  }
}

template <int D, bool F16>
cudaError_t launch_append(const Gqa8Args& a, cudaStream_t stream) {
  // fewer than 8 tokens a request on average: a block for each token
  if (a.n_tokens < 8 * static_cast<int64_t>(a.B)) {
    const int units = 2 * a.Hkv * (D / 16);
    return launch_grid(append4_rows_kernel<D, F16>, a,
                       dim3(static_cast<unsigned>(a.n_tokens), (units + kAppendThreads - 1) / kAppendThreads),
                       kAppendThreads, stream);
  }
  return launch_pages(append4_kernel<D, F16>, a, 1, 2 * a.Hkv, kAppendThreads, stream);
}

}  // namespace

cudaError_t launch_append_gqa4(const Gqa8Args& a, cudaStream_t stream) {
  if (a.D == 64) return a.f16 ? launch_append<64, true>(a, stream) : launch_append<64, false>(a, stream);
  return a.f16 ? launch_append<128, true>(a, stream) : launch_append<128, false>(a, stream);
}

cudaError_t launch_read_gqa4(const Gqa8Args& args, cudaStream_t stream) {
  // Two heads a block where that saves a second or third round of blocks, of which the
  // SMs hold 8 each and which begin with three dependent loads (128 requests of 32
  // tokens 7.5 us with one, 6.7 with two, 9.0 with four; 9 prompts, where there are
  // more rounds, 25.6, 26.3, 27.5).
  Gqa8Args a = args;
  const int64_t blocks = page_items(a) * a.Hkv, most = 8 * static_cast<int64_t>(a.num_sms);
  a.each = blocks > most && blocks <= 3 * most ? 2 : 1;
  const dim3 grid(static_cast<unsigned>(page_items(a)), static_cast<unsigned>((a.Hkv + a.each - 1) / a.each));
  if (a.D == 64)
    return a.f16 ? launch_grid(read4_kernel<64, true>, a, grid, kThreads, stream)
                 : launch_grid(read4_kernel<64, false>, a, grid, kThreads, stream);
  return a.f16 ? launch_grid(read4_kernel<128, true>, a, grid, kThreads, stream)
               : launch_grid(read4_kernel<128, false>, a, grid, kThreads, stream);
}

}  // namespace kv4
