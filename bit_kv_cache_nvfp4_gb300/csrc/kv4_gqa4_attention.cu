// kv4_gqa4_attention.cu -- causal attention of new tokens over the 4-bit
// grouped-query cache (kv4_attention_gqa4).
//
// Row (t, h): query head h of flat token t; token i of request b's n new ones
// stands at position seq_lens[b] - n + i and sees the keys j <= its position,
// j > position - window where there is a window.  Scores, the running maximum
// and sum and the output are held in fp32:
//   s_j = sm_scale q.k_j,  o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),
//   lse = m + log sum_j exp(s_j - m);  a row without a key: 0 and -inf.
#include "kv4_gqa_merge.cuh"

namespace kv4 {
namespace {

// The plain kernel: a block for each row, a key for each warp at a time, D / 32
// elements a lane.
template <int D, bool F16>
__global__ void __launch_bounds__(128) row_kernel(const Gqa8AttnArgs a) {
  constexpr int E = D / 32;
  grid_dependency_wait();
  grid_launch_dependents();
  __shared__ float part_o[4][D], part_m[4], part_l[4];
  const int t = blockIdx.x, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.Hq / a.Hkv, hk = h / G;
  int b = 0;
  for (; b < a.B; ++b)
    if (load(a.cu + b) <= t && t < load(a.cu + b + 1)) break;
  if (b == a.B) return;
  const Gqa8Request r = gqa8_request(a, b, 1, 0x7FFFFFFF, h == 0 && t == min(max(load(a.cu + b), 0), static_cast<int>(a.n_tokens)));
  if (r.n == 0) return;
  const int pos = r.pos0 + (t - r.cu0);
  const int lo = a.window > 0 ? max(pos - a.window + 1, 0) : 0, hi = min(pos + 1, r.held);
  const uint16_t* q = static_cast<const uint16_t*>(a.q) + t * a.q_token_stride + h * a.q_head_stride + lane * E;
  float x[E], o[E];
  bool odd = false;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    x[e] = F16 ? __half2float(__ushort_as_half(load(q + e))) : __uint_as_float(static_cast<uint32_t>(load(q + e)) << 16);
    odd |= !isfinite(x[e]);
    o[e] = 0.0f;
  }
  odd = __any_sync(0xFFFFFFFFu, odd);
  float m = -INFINITY, l = 0.0f;
  for (int64_t j = lo + warp; j < hi; j += 4) {
    const int pg = load(a.page_table + b * a.pt_stride + (j >> 6));
    if (pg < 0 || pg >= a.num_pages) {
      if (lane == 0) flag_error(a.dev_err, kDevBadPage);
      continue;
    }
    auto values = [&](int side, float (&v)[E]) {
      const int64_t row = ((static_cast<int64_t>(pg) * a.Hkv + hk) * 2 + side) * kPage + (j & 63);
      const float s = e4m3_to_float(load(a.scales + row * (D / 16) + lane * E / 16));
      uint32_t w = 0;
      for (int i = 0; i < E / 2; ++i) w |= static_cast<uint32_t>(load(a.pool + row * (D / 2) + lane * (E / 2) + i)) << (8 * i);
      uint32_t f[4];
      e2m1x8_to_f16x8(w, f);
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        const float2 p = __half22float2(bits_h2(f[i]));
        v[2 * i] = p.x * s;
        v[2 * i + 1] = p.y * s;
      }
    };
    float k[E], v[E];
    values(0, k);
    values(1, v);
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(x[e], k[e], s);
    s = warp_sum(s) * a.sm_scale;
    const float to = fmaxf(m, s), by = expf(m - to), p = expf(s - to);
    m = to;
    l = l * by + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * by + p * v[e];
  }
#pragma unroll
  for (int e = 0; e < E; ++e) part_o[warp][lane * E + e] = o[e];
  if (lane == 0) {
    part_m[warp] = m;
    part_l[warp] = l;
  }
  __syncthreads();
  const float top = fmaxf(fmaxf(part_m[0], part_m[1]), fmaxf(part_m[2], part_m[3]));
  float sum = 0.0f, w[4];
  for (int i = 0; i < 4; ++i) {
    w[i] = part_l[i] > 0.0f ? expf(part_m[i] - top) : 0.0f;
    sum += part_l[i] * w[i];
  }
  const bool nan = odd && hi > lo;
  const int64_t row = static_cast<int64_t>(t) * a.Hq + h;
  for (int d = threadIdx.x; d < D; d += 128) {
    float y = 0.0f;
    for (int i = 0; i < 4; ++i) y += part_o[i][d] * w[i];
    y = nan ? __uint_as_float(0x7FC00000u) : sum > 0.0f ? y / sum : 0.0f;
    if constexpr (F16) static_cast<__half*>(a.out)[row * D + d] = __float2half_rn(y);
    else static_cast<__nv_bfloat16*>(a.out)[row * D + d] = __float2bfloat16_rn(y);
  }
  if (threadIdx.x == 0)
    a.lse[row] = nan ? __uint_as_float(0x7FC00000u) : sum > 0.0f ? top + logf(sum) : -INFINITY;
}

}  // namespace

cudaError_t launch_attention_gqa4(const Gqa8AttnArgs& a, cudaStream_t stream) {
  auto launch = [&](auto kernel) {
    kernel<<<dim3(static_cast<unsigned>(a.n_tokens), a.Hq), 128, 0, stream>>>(a);
    return cudaGetLastError();
  };
  if (a.D == 64) return a.f16 ? launch(row_kernel<64, true>) : launch(row_kernel<64, false>);
  return a.f16 ? launch(row_kernel<128, true>) : launch(row_kernel<128, false>);
}

size_t attention_gqa4_workspace(int, int, int, int, int) { return 0; }

}  // namespace kv4
