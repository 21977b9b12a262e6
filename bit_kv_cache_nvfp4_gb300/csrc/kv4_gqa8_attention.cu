// kv4_gqa8_attention.cu -- causal attention of new tokens over the 8-bit
// grouped-query cache (kv4_attention_gqa8).
//
// Row (t, h): query head h of flat token t; token i of request b's n new ones
// stands at position seq_lens[b] - n + i and sees the keys j <= its position,
// j > position - window where there is a window.  Scores, the running maximum
// and sum and the output are held in fp32:
//   s_j = sm_scale q.k_j,  o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),
//   lse = m + log sum_j exp(s_j - m);  a row without a key: 0 and -inf.
//
// One warp per row, D / 32 columns per lane, one key at a time.
#include "kv4_device.cuh"
#include "kv4_launch.h"

#include <math.h>

namespace kv4 {
namespace {

__device__ __forceinline__ float pow2f(int e) {
  return __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}

template <int D, bool F16>
__global__ void __launch_bounds__(128) attention_kernel(Gqa8AttnArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  constexpr int C = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (row >= a.n_tokens * a.Hq) return;
  const int64_t t = row / a.Hq;
  const int h = static_cast<int>(row % a.Hq), hk = h / (a.Hq / a.Hkv);
  int lo = 0, hi = a.B - 1;                       // largest b with cu[b] <= t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(a.cu + mid) <= t) lo = mid; else hi = mid - 1;
  }
  const int c0 = __ldg(a.cu + lo), c1 = __ldg(a.cu + lo + 1);
  if (t < c0 || t >= c1) return;                  // behind the last request: left as it was
  if (c1 - c0 > a.max_new) {
    if (lane == 0) flag_error(a.dev_err, kDevBadLength);
    return;
  }
  const int64_t pos = static_cast<int64_t>(__ldg(a.lens + lo)) - c1 + t;
  const int64_t first = a.window > 0 && pos - a.window + 1 > 0 ? pos - a.window + 1 : 0;
  float q[C], o[C], m = -INFINITY, l = 0.0f;
  const uint16_t* qp = static_cast<const uint16_t*>(a.q) + t * a.q_token_stride + h * a.q_head_stride + lane * C;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    q[i] = F16 ? __half2float(reinterpret_cast<const __half*>(qp)[i])
               : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(qp)[i]);
    o[i] = 0.0f;
  }
  const float c = a.sm_scale * 1.4426950408889634f;
  const int64_t held = a.pt_stride << 6;          // what the table can name
  if (pos >= held && lane == 0) flag_error(a.dev_err, kDevBadPage);
  for (int64_t j = first; j <= pos && j < held; ++j) {
    const int64_t pg = __ldg(a.page_table + lo * a.pt_stride + (j >> 6));
    if (pg < 0 || pg >= a.num_pages) {
      if (lane == 0) flag_error(a.dev_err, kDevBadPage);
      j |= 63;                                    // the rest of the page is masked too
      continue;
    }
    const int64_t blk = (pg * a.Hkv + hk) * 2;
    const uint8_t* kp = a.pool + blk * (kPage * D) + (j & 63) * D + lane * C;
    const uint8_t* vp = kp + kPage * D;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i) s = fmaf(q[i], e4m3_to_float(kp[i]), s);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
    s *= c * pow2f(static_cast<int>(__ldg(a.scales + blk)) - 127);
    const float mn = fmaxf(m, s);
    const float corr = exp2f(m - mn), p = exp2f(s - mn);
    const float pv = p * pow2f(static_cast<int>(__ldg(a.scales + blk + 1)) - 127);
    l = l * corr + p;
    m = mn;
#pragma unroll
    for (int i = 0; i < C; ++i) o[i] = o[i] * corr + pv * e4m3_to_float(vp[i]);
  }
  uint16_t* op = static_cast<uint16_t*>(a.out) + row * D + lane * C;
  const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const float v = o[i] * inv;
    if (F16) reinterpret_cast<__half*>(op)[i] = __float2half_rn(v);
    else reinterpret_cast<__nv_bfloat16*>(op)[i] = __float2bfloat16_rn(v);
  }
  if (lane == 0) a.lse[row] = l == 0.0f ? -INFINITY : 0.6931471805599453f * (m + log2f(l));
}

}  // namespace

cudaError_t launch_attention_gqa8(const Gqa8AttnArgs& a, cudaStream_t stream) {
  const int64_t rows = a.n_tokens * a.Hq;
  const unsigned grid = static_cast<unsigned>((rows + 3) / 4);
  if (a.D == 64)
    return a.f16 ? launch_pdl(attention_kernel<64, true>, grid, 128, 0, stream, 1, a)
                 : launch_pdl(attention_kernel<64, false>, grid, 128, 0, stream, 1, a);
  return a.f16 ? launch_pdl(attention_kernel<128, true>, grid, 128, 0, stream, 1, a)
               : launch_pdl(attention_kernel<128, false>, grid, 128, 0, stream, 1, a);
}

size_t attention_gqa8_workspace(int, int, int64_t, int, int, int, int) { return 0; }

}  // namespace kv4
