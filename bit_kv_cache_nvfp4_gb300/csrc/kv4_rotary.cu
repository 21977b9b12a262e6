// kv4_rotary.cu -- rotary positions of queries and keys (kv4_rotary).
//
// Pair i of a head turns by the angle a = position * inv_freq[i]:
//   (x, y) -> f (x cos a - y sin a, x sin a + y cos a)
// the pairs being neighbours (offset + 2i, offset + 2i + 1) or halves
// (offset + i, offset + i + n).  Products and sums are in fp32, rounded once.
//
// The angle.  A position of 200000 times a frequency of 1 is 2^17.6 radians, of
// which an fp32 product keeps 2^-7: too little.  So the angle is reduced before
// it is rounded, in turns and in integers: F = inv_freq / 2 pi as a 64-bit
// fraction of a turn (to 2^-63 for frequencies up to 1), and position *
// F modulo 2^64 drops the whole turns by itself.  Its top 32 bits are the angle in
// units of pi / 2^31, good to 2^-32 of a turn, for sincospi.
//
// Bound by HBM in large calls and by three dependent loads in small ones.  A thread
// block turns one token (several where their heads are few): it computes the
// token's n pairs of sine and cosine once, for all heads, while the first of its
// rows are on their way.
#include <algorithm>
#include <type_traits>

#include "kv4_gqa8_device.cuh"

namespace kv4 {
namespace {

constexpr int kBlock = 256;

// inv_freq / 2 pi modulo 1, in units of 2^-64: m * 2^(E - 150) times the fraction
// 1 / 2 pi = 0x0.28BE60DB9391054A.. of a turn.
__device__ __forceinline__ uint64_t turn_fraction(float inv_freq) {
  const uint32_t u = __float_as_uint(inv_freq), e = (u >> 23) & 255u;
  if (e == 0 || e == 255) return 0;                       // 0 and subnormals: no turn at all
  const uint64_t m = static_cast<uint64_t>((u & 0x7FFFFFu) | 0x800000u) << 40;
  const uint64_t p = __umul64hi(m, 0x28BE60DB9391054Aull);                 // m / 2 pi, of 2^(e - 126)
  const uint64_t f = e <= 126 ? (e >= 63 ? p >> (126 - e) : 0) : (e < 190 ? p << (e - 126) : 0);
  return (u >> 31) ? 0 - f : f;
}

template <int V>
struct alignas(2 * V) Vec {
  uint16_t x[V];
};
template <int V>
__device__ __forceinline__ Vec<V> load_vec(const uint16_t* p) {
  Vec<V> v;
  if constexpr (V == 8) *reinterpret_cast<uint4*>(v.x) = load(reinterpret_cast<const uint4*>(p));
  else if constexpr (V == 4) *reinterpret_cast<uint2*>(v.x) = load(reinterpret_cast<const uint2*>(p));
  else if constexpr (V == 2) *reinterpret_cast<uint32_t*>(v.x) = load(reinterpret_cast<const uint32_t*>(p));
  else v.x[0] = load(p);
  return v;
}
template <int V>
__device__ __forceinline__ void store_vec(uint16_t* p, const Vec<V>& v) {
  if constexpr (V == 8) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(v.x);
  else if constexpr (V == 4) *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(v.x);
  else if constexpr (V == 2) *reinterpret_cast<uint32_t*>(p) = *reinterpret_cast<const uint32_t*>(v.x);
  else *p = v.x[0];
}
template <bool F16>
__device__ __forceinline__ float wide(uint16_t x) {
  if constexpr (F16) return __half2float(__ushort_as_half(x));
  return __uint_as_float(static_cast<uint32_t>(x) << 16);
}
template <bool F16>
__device__ __forceinline__ uint16_t narrow(float x) {
  if constexpr (F16) return __half_as_ushort(__float2half_rn(x));
  return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

// Threads: vector i of the turned part (n / V of a head), head slot, token slot.
template <int V, bool NEAR, bool F16>
__global__ void __launch_bounds__(2 * kBlock) rotary_kernel(const RotaryArgs a) {
  __shared__ alignas(16) float cosine[kBlock * 8], sine[kBlock * 8];
  grid_dependency_wait();
  grid_launch_dependents();
  const int R = a.n / V, tid = threadIdx.x;
  const int i = tid % R, slot = tid / R, hs = slot % a.heads_at_once, ts = slot / a.heads_at_once;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tokens;
  const int64_t t = t0 + ts;
  const int heads = a.side[0].heads + a.side[1].heads;
  const bool in = t < a.n_tokens && ts < a.tokens;
  const int h_end = min(heads, static_cast<int>(blockIdx.y + 1) * a.heads);
  int h = blockIdx.y * a.heads + hs;
  auto at = [&](int head, bool out) -> uint16_t* {
    const int k = head >= a.side[0].heads;
    const RotarySide& s = a.side[k];
    const int64_t j = head - k * a.side[0].heads;
    return (out ? static_cast<uint16_t*>(s.out) + t * s.out_token + j * s.out_head
                : static_cast<uint16_t*>(const_cast<void*>(s.in)) + t * s.in_token + j * s.in_head) + s.offset;
  };
  const int first = NEAR ? 2 * i * V : i * V, second = NEAR ? first + V : first + a.n;
  Vec<V> x, y;
  if (in && h < h_end) {
    const uint16_t* const p = at(h, false);
    x = load_vec<V>(p + first);
    y = load_vec<V>(p + second);
  }
  for (int k = tid; k < a.tokens * a.n; k += blockDim.x) {
    const int64_t tk = t0 + k / a.n;
    if (tk < a.n_tokens) {
      const int64_t pos = a.wide_positions ? load(static_cast<const int64_t*>(a.positions) + tk)
                                           : load(static_cast<const int32_t*>(a.positions) + tk);
      const uint64_t turn = static_cast<uint64_t>(pos) * turn_fraction(load(a.inv_freq + k % a.n));
      float s, c;
      sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &s, &c);
      cosine[k] = c * a.factor;
      sine[k] = s * a.factor;
    }
  }
  __syncthreads();
  if (in && h < h_end) {
    alignas(16) float c[V], z[V];
    const int k0 = ts * a.n + i * V;
    if constexpr (V % 4 == 0) {
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        *reinterpret_cast<float4*>(c + j) = *reinterpret_cast<const float4*>(cosine + k0 + j);
        *reinterpret_cast<float4*>(z + j) = *reinterpret_cast<const float4*>(sine + k0 + j);
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        c[j] = cosine[k0 + j];
        z[j] = sine[k0 + j];
      }
    }
    while (true) {
      // (the next head's row first)
      const int next = h + a.heads_at_once;
      Vec<V> nx, ny;
      if (next < h_end) {
        const uint16_t* const p = at(next, false);
        nx = load_vec<V>(p + first);
        ny = load_vec<V>(p + second);
      }
      Vec<V> ox, oy;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        // pair j: elements j of both vectors, or 2j and 2j + 1 of the two in a row
        constexpr bool kNear = NEAR;
        const int e0 = 2 * j, e1 = 2 * j + 1;
        const float u = wide<F16>(kNear ? (e0 < V ? x.x[e0 % V] : y.x[e0 % V]) : x.x[j]);
        const float v = wide<F16>(kNear ? (e1 < V ? x.x[e1 % V] : y.x[e1 % V]) : y.x[j]);
        const uint16_t p0 = narrow<F16>(u * c[j] - v * z[j]), p1 = narrow<F16>(u * z[j] + v * c[j]);
        if constexpr (kNear) {
          (e0 < V ? ox : oy).x[e0 % V] = p0;
          (e1 < V ? ox : oy).x[e1 % V] = p1;
        } else {
          ox.x[j] = p0;
          oy.x[j] = p1;
        }
      }
      uint16_t* const o = at(h, true);
      store_vec<V>(o + first, ox);
      store_vec<V>(o + second, oy);
      if (next >= h_end) break;
      h = next;
      x = nx;
      y = ny;
    }
  }
  // the elements that do not turn, where the outputs are not the inputs
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const RotarySide& s = a.side[k];
    const int rest = (s.D - 2 * a.n) / V;                 // vectors of a head
    if (rest == 0 || s.out == s.in) continue;
    const int h0 = max(static_cast<int>(blockIdx.y) * a.heads - k * a.side[0].heads, 0);
    const int h1 = min(h_end - k * a.side[0].heads, s.heads);
    const int per = (h1 - h0) * rest;                     // of a token
    for (int u = tid; u < per * a.tokens; u += blockDim.x) {
      const int64_t tk = t0 + u / per;
      if (tk >= a.n_tokens) break;
      const int w = u % per, j = h0 + w / rest;
      int e = w % rest * V;
      if (e >= s.offset) e += 2 * a.n;
      store_vec<V>(static_cast<uint16_t*>(s.out) + tk * s.out_token + j * s.out_head + e,
                   load_vec<V>(static_cast<const uint16_t*>(s.in) + tk * s.in_token + j * s.in_head + e));
    }
  }
}

template <int V, bool F16>
cudaError_t launch_v(const RotaryArgs& a, dim3 grid, unsigned threads, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return a.interleaved ? cudaLaunchKernelEx(&cfg, rotary_kernel<V, true, F16>, a)
                       : cudaLaunchKernelEx(&cfg, rotary_kernel<V, false, F16>, a);
}

// The widest vectors that every row and part begins and ends at.
int vector_width(const RotaryArgs& a) {
  uint64_t bits = static_cast<uint64_t>(a.n);
  for (const RotarySide& s : a.side) {
    if (s.heads == 0) continue;
    bits |= (reinterpret_cast<uintptr_t>(s.in) | reinterpret_cast<uintptr_t>(s.out)) >> 1;
    bits |= static_cast<uint64_t>(s.D) | static_cast<uint64_t>(s.offset);
    if (a.n_tokens > 1) bits |= static_cast<uint64_t>(s.in_token | s.out_token);
    if (s.heads > 1) bits |= static_cast<uint64_t>(s.in_head | s.out_head);
  }
  return bits % 8 == 0 ? 8 : bits % 4 == 0 ? 4 : bits % 2 == 0 ? 2 : 1;
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& args, cudaStream_t stream) {
  RotaryArgs a = args;
  const int V = vector_width(a), R = a.n / V, heads = a.side[0].heads + a.side[1].heads;
  // (n <= kRotaryPairs, so that R threads are a block at most)
  a.heads_at_once = std::max(1, std::min(heads, kBlock / R));
  a.heads = heads;
  const int64_t sms = a.num_sms;
  // all heads of a token by one block, unless the blocks would not fill the SMs
  if (a.n_tokens < 4 * sms) a.heads = a.heads_at_once;
  a.tokens = a.heads_at_once < heads ? 1 : std::max(1, std::min(kBlock / (R * heads), 16));
  while (a.tokens > 1 && a.n_tokens < 2 * sms * a.tokens) --a.tokens;
  const dim3 grid(static_cast<unsigned>((a.n_tokens + a.tokens - 1) / a.tokens),
                  static_cast<unsigned>((heads + a.heads - 1) / a.heads));
  const unsigned threads = (static_cast<unsigned>(R * a.heads_at_once * a.tokens) + 31) / 32 * 32;
  auto launch = [&](auto v) {
    constexpr int W = decltype(v)::value;
    return a.f16 ? launch_v<W, true>(a, grid, threads, stream) : launch_v<W, false>(a, grid, threads, stream);
  };
  switch (V) {
    case 8: return launch(std::integral_constant<int, 8>{});
    case 4: return launch(std::integral_constant<int, 4>{});
    case 2: return launch(std::integral_constant<int, 2>{});
  }
  return launch(std::integral_constant<int, 1>{});
}

}  // namespace kv4
