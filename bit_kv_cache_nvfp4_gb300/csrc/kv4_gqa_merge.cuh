// kv4_gqa_merge.cuh -- what the attention kernels of the grouped-query caches
// share around the kernels themselves: the workspace of items that were cut, the
// kernels that join their pieces, and launches.
#pragma once

#include <math.h>

#include <mutex>
#include <type_traits>

#include "kv4_gqa8_device.cuh"

namespace kv4 {
namespace {

// ---------------------------------------------------------------------------
// The pieces of items that were cut: block (c, y) joins rows of the item that
// began in block c of the attention kernel, by log-sum-exp over its pieces in
// their order: one kernel for items of few rows, where a long context has many
// pieces, one for items of up to 256 rows, where a warp takes 4 rows at once and
// their pieces in turn.  Those of a prompt or a chunk are
// two or three; but a single short one of few heads over a long context is cut
// over all blocks (40 rows of one head over 200000 tokens: 97 us, where one row,
// in the kernels of few rows, takes 28).
// ---------------------------------------------------------------------------
// Block (c, y) takes EACH rows: 8, a warp each, 8 pieces at a time with the next 8 on
// their way, where requests and heads are many, whose items are cut in two or three; or 1,
// whose pieces its 8 warps share, where few items are cut over all blocks.  Both add up
// pieces 0, 8, 16, .., pieces 1, 9, .. and so on by themselves, and then those sums.  (A
// block for every row: drafts of 35 rows 34.6 us for 28.8, 64 sessions' decode step 227 for
// 223, of the 4-bit cache.  Among many requests one may be cut over all blocks as well, which
// only the device knows: 63 padded slots and a session of 200000 tokens, 8 heads a group,
// take 76 us from the 8-bit cache, 75 with a block for every row, 90 with a block's 8 warps
// on its 8 rows in turns.  Two blocks an SM are enough, and leave the registers for 16
// pieces: 200 of them, one K/V head's, in 5 us less than with three.)
template <int D, int EACH>
__global__ void __launch_bounds__(256, 2) merge_few_kernel(const Gqa8AttnArgs a, const int rows,
                                                        const Gqa8Tail* tails, const float* ws_lse,
                                                        const float* ws_o) {
  grid_dependency_wait();
  grid_launch_dependents();
  constexpr int C = D / 32, W = 8;                        // columns a lane; warps, and sums of a row
  using Vec = std::conditional_t<C == 4, float4, float2>;
  const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Gqa8Tail t = tails[c];
  const int r = blockIdx.y * EACH + (EACH == 1 ? 0 : warp);
  if (t.parts == 0 || r >= t.nrows) return;               // (whole blocks of one row)
  // piece i is slot 2c + 1 for i = 0, else 2 (c + i)
  auto row_of = [&](int i) { return static_cast<int64_t>(i == 0 ? 2 * c + 1 : 2 * (c + i)) * rows + r; };
  auto piece = [&](int i) { return load(reinterpret_cast<const Vec*>(ws_o + row_of(i) * D) + lane); };
  float x = lane < t.parts ? load(ws_lse + row_of(lane)) : -INFINITY;
  // (the first 8 pieces on their way with it)
  Vec v[W];
  if constexpr (EACH > 1)
#pragma unroll
    for (int j = 0; j < W; ++j)
      if (j < t.parts) v[j] = piece(j);
  float m = x, s = 0.0f, o[W][C];                         // (of one row a block o[0] alone, the warp's)
#pragma unroll
  for (int j = 0; j < W; ++j)
#pragma unroll
    for (int k = 0; k < C; ++k) o[j][k] = 0.0f;
  bool odd = x != x;
  for (int i = 32 + lane; i < t.parts; i += 32) {
    const float y = load(ws_lse + row_of(i));
    odd |= y != y;
    m = fmaxf(m, y);
  }
  m = warp_max(m);
  odd = __any_sync(0xFFFFFFFFu, odd);
#pragma unroll 1
  for (int i0 = 0; i0 < t.parts; i0 += 32) {
    if (i0 > 0) x = i0 + lane < t.parts ? load(ws_lse + row_of(i0 + lane)) : -INFINITY;
    const float w = m > -INFINITY ? fast_exp2(x - m) : 0.0f;
    s += w;
    const int n = min(32, t.parts - i0);
    auto add = [&](int i, const Vec& y, float (&to)[C]) {
      const float wt = __shfl_sync(0xFFFFFFFFu, w, i);
      const float* f = reinterpret_cast<const float*>(&y);
#pragma unroll
      for (int k = 0; k < C; ++k) to[k] = fmaf(wt, f[k], to[k]);
    };
    if constexpr (EACH == 1) {
#pragma unroll 4
      for (int i = warp; i < n; i += W) add(i, piece(i0 + i), o[0]);
    } else {
#pragma unroll 1
      for (int i = 0; i < n; i += W)
#pragma unroll
        for (int j = 0; j < W; ++j) {
          if (i + j < n) add(i + j, v[j], o[j]);
          if (i0 + i + j + W < t.parts) v[j] = piece(i0 + i + j + W);
        }
    }
  }
  s = warp_sum(s);
  if (odd) s = __uint_as_float(0x7FC00000u);
  if constexpr (EACH == 1) {
    __shared__ Vec part[W][32];
    part[warp][lane] = *reinterpret_cast<const Vec*>(o[0]);
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int j = 1; j < W; ++j) *reinterpret_cast<Vec*>(o[j]) = part[j][lane];
  }
#pragma unroll
  for (int j = 1; j < W; ++j)
#pragma unroll
    for (int k = 0; k < C; ++k) o[0][k] += o[j][k];
  const int G = a.Hq / a.Hkv, rr = t.r0 + r;
  const int64_t row = static_cast<int64_t>(t.cu0 + rr / G) * a.Hq + t.h * G + rr % G;
  const float inv = s == 0.0f ? 0.0f : 1.0f / s;
  uint32_t u[C / 2];
#pragma unroll
  for (int k = 0; k < C / 2; ++k) {
    const float y0 = o[0][2 * k] * inv, y1 = o[0][2 * k + 1] * inv;
    u[k] = a.f16 ? pack16<true>(y0, y1) : pack16<false>(y0, y1);
  }
  uint32_t* const dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + row * D) + lane * (C / 2);
  if constexpr (C == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(u[0], u[1]);
  else *dst = u[0];
  if (lane == 0) a.lse[row] = s == 0.0f ? -INFINITY : (m + log2f(s)) * 0.6931471805599453f;
}

template <int D>
__global__ void __launch_bounds__(256) merge_many_kernel(const Gqa8AttnArgs a, const int rows,
                                                         const Gqa8Tail* tails, const float* ws_lse,
                                                         const float* ws_o) {
  grid_dependency_wait();
  grid_launch_dependents();
  constexpr int C = D / 32, R = 4;
  using Vec = std::conditional_t<C == 4, float4, float2>;
  const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Gqa8Tail t = tails[c];
  const int r0 = (blockIdx.y * 8 + warp) * R;
  if (t.parts == 0 || r0 >= t.nrows) return;
  auto row_of = [&](int i, int r) { return static_cast<int64_t>(i == 0 ? 2 * c + 1 : 2 * (c + i)) * rows + r; };
  // lane 8 k + i: row r0 + k, piece i of 8 at a time
  const int k8 = lane >> 3, i8 = lane & 7, mine = min(r0 + k8, t.nrows - 1);
  float m = -INFINITY;
  bool odd = false;
  for (int i = i8; i < t.parts; i += 8) {
    const float x = load(ws_lse + row_of(i, mine));
    odd |= x != x;
    m = fmaxf(m, x);
  }
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) {
    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
    odd |= __shfl_xor_sync(0xFFFFFFFFu, static_cast<int>(odd), off) != 0;
  }
  float s = 0.0f, o[R][C];
#pragma unroll
  for (int k = 0; k < R; ++k)
#pragma unroll
    for (int j = 0; j < C; ++j) o[k][j] = 0.0f;
  for (int i0 = 0; i0 < t.parts; i0 += 8) {
    const bool in = i0 + i8 < t.parts && m > -INFINITY;
    const float w = in ? fast_exp2(load(ws_lse + row_of(i0 + i8, mine)) - m) : 0.0f;
    s += w;
    const int n = min(8, t.parts - i0);
#pragma unroll 2
    for (int i = 0; i < n; ++i)
#pragma unroll
      for (int k = 0; k < R; ++k) {
        const float wk = __shfl_sync(0xFFFFFFFFu, w, k * 8 + i);
        const Vec v = load(reinterpret_cast<const Vec*>(ws_o + row_of(i0 + i, min(r0 + k, t.nrows - 1)) * D) + lane);
        const float* f = reinterpret_cast<const float*>(&v);
#pragma unroll
        for (int j = 0; j < C; ++j) o[k][j] = fmaf(wk, f[j], o[k][j]);
      }
  }
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
  if (odd) s = __uint_as_float(0x7FC00000u);
  const int G = a.Hq / a.Hkv;
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const float sk = __shfl_sync(0xFFFFFFFFu, s, k * 8), mk = __shfl_sync(0xFFFFFFFFu, m, k * 8);
    if (r0 + k >= t.nrows) break;
    const int rr = t.r0 + r0 + k;
    const int64_t row = static_cast<int64_t>(t.cu0 + rr / G) * a.Hq + t.h * G + rr % G;
    const float inv = sk == 0.0f ? 0.0f : 1.0f / sk;
    uint32_t u[C / 2];
#pragma unroll
    for (int j = 0; j < C / 2; ++j)
      u[j] = a.f16 ? pack16<true>(o[k][2 * j] * inv, o[k][2 * j + 1] * inv)
                   : pack16<false>(o[k][2 * j] * inv, o[k][2 * j + 1] * inv);
    uint32_t* const dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + row * D) + lane * (C / 2);
    if constexpr (C == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(u[0], u[1]);
    else *dst = u[0];
    if (lane == 0) a.lse[row] = sk == 0.0f ? -INFINITY : (mk + log2f(sk)) * 0.6931471805599453f;
  }
}

// Workspace of one attention kernel: a tail for each of its blocks, then two
// slots of partial rows for each block.
inline size_t part_bytes(int blocks, int rows, int D) {
  return static_cast<size_t>(blocks) * (sizeof(Gqa8Tail) + 2ull * rows * (D + 1) * sizeof(float));
}
struct Parts {
  Gqa8Tail* tails;
  float *lse, *o;
};
inline Parts parts_at(void* ws, int blocks, int rows, int D) {
  Parts p;
  p.tails = static_cast<Gqa8Tail*>(ws);
  p.o = reinterpret_cast<float*>(p.tails + blocks);
  p.lse = p.o + 2ull * blocks * rows * D;
  return p;
}
template <typename... Args>
cudaError_t launch_merge(void (*kernel)(Gqa8AttnArgs, Args...), const Gqa8AttnArgs& a, dim3 grid, cudaStream_t stream,
                         Args... args) {
  if ((a.pt_stride + 1) / 2 <= kWhole) return cudaSuccess;                 // nothing is ever cut
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, args...);
}
template <int D>
cudaError_t launch_merge_few(const Gqa8AttnArgs& a, int blocks, int rows, const Parts& p, cudaStream_t stream) {
  // (of fewer items an average one may have more than 8 pieces)
  if (static_cast<int64_t>(a.B) * a.Hkv * 8 >= blocks)
    return launch_merge<int, const Gqa8Tail*, const float*, const float*>(
        merge_few_kernel<D, 8>, a, dim3(blocks, (rows + 7) / 8), stream, rows, p.tails, p.lse, p.o);
  return launch_merge<int, const Gqa8Tail*, const float*, const float*>(
      merge_few_kernel<D, 1>, a, dim3(blocks, rows), stream, rows, p.tails, p.lse, p.o);
}
template <int D>
cudaError_t launch_merge_many(const Gqa8AttnArgs& a, int blocks, int rows, const Parts& p, cudaStream_t stream) {
  return launch_merge<int, const Gqa8Tail*, const float*, const float*>(
      merge_many_kernel<D>, a, dim3(blocks, (rows + 31) / 32), stream, rows, p.tails, p.lse, p.o);
}

// Once per device and kernel: its shared memory, and, where it splits its
// registers among its warps, that its launch has as many as the split takes.
template <auto kKernel>
cudaError_t prepare_kernel(int smem, int min_regs) {
  static std::once_flag once[64];
  static cudaError_t ready[64];
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::call_once(once[dev], [&] {
    ready[dev] = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    cudaFuncAttributes f;
    if (ready[dev] == cudaSuccess) ready[dev] = cudaFuncGetAttributes(&f, kKernel);
    if (ready[dev] == cudaSuccess && f.numRegs < min_regs) ready[dev] = cudaErrorInvalidConfiguration;
  });
  return ready[dev];
}

}  // namespace
}  // namespace kv4
