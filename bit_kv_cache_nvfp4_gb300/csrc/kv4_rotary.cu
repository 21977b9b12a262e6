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
// units of pi / 2^31, good to 2^-32 of a turn at positions up to 2^31 (to 2^-29 at
// frequencies of 4), which fp32 rounds for sincospi: off by 2^-26 of a turn at most.
//
// Bound by HBM in large calls: 16381 tokens of 40 heads of 128, 336 MB, in 60 us whole and
// 61 with a quarter of each head copied, 5.5 TB/s, where a copy of the same tensors takes
// 54 us.  A thread block turns a few tokens: it computes their n pairs of sine and cosine
// once, for all heads, while the first of its rows are on their way (4 to 6 tokens, as
// many as give every thread an angle; with one a block 94 us).  In small calls it is
// bound by two dependent loads, and their heads go to more blocks: 64 tokens of 72 heads
// take 2.0 us in replays of a graph.  Where n is odd, or rows begin at odd elements, the
// halves lie at odd elements and move by single ones (2.0 TB/s).
#include <algorithm>
#include <type_traits>

#include "kv4_gqa8_device.cuh"

namespace kv4 {
namespace {

constexpr int kBlock = 256, kTable = 2048;                // threads; angles of a block

// inv_freq / 2 pi modulo 1, in units of 2^-64: m * 2^(E - 150) times the fraction
// 1 / 2 pi = 0x0.28BE60DB9391054A.. of a turn.
__device__ __forceinline__ uint64_t turn_fraction(float inv_freq) {
  const uint32_t u = __float_as_uint(inv_freq), e = (u >> 23) & 255u;
  if (e == 0 || e == 255) return 0;                       // 0 and subnormals: no turn; not finite: see below
  const uint64_t m = static_cast<uint64_t>((u & 0x7FFFFFu) | 0x800000u) << 40;
  const uint64_t p = __umul64hi(m, 0x28BE60DB9391054Aull);                 // m / 2 pi, of 2^(e - 126)
  const uint64_t f = e <= 126 ? (e >= 63 ? p >> (126 - e) : 0) : (e < 190 ? p << (e - 126) : 0);
  return (u >> 31) ? 0 - f : f;
}

// V elements in 32-bit words (one alone in the low half).
template <int V>
struct Vec {
  static constexpr int kWords = (V + 1) / 2;
  uint32_t w[kWords];
};
template <int V>
__device__ __forceinline__ Vec<V> load_vec(const uint16_t* p) {
  Vec<V> v;
  if constexpr (V == 8) {
    const uint4 u = load(reinterpret_cast<const uint4*>(p));
    v.w[0] = u.x, v.w[1] = u.y, v.w[2] = u.z, v.w[3] = u.w;
  } else if constexpr (V == 4) {
    const uint2 u = load(reinterpret_cast<const uint2*>(p));
    v.w[0] = u.x, v.w[1] = u.y;
  } else if constexpr (V == 2) {
    v.w[0] = load(reinterpret_cast<const uint32_t*>(p));
  } else {
    v.w[0] = load(p);
  }
  return v;
}
template <int V>
__device__ __forceinline__ void store_vec(uint16_t* p, const Vec<V>& v) {
  if constexpr (V == 8) *reinterpret_cast<uint4*>(p) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
  else if constexpr (V == 4) *reinterpret_cast<uint2*>(p) = make_uint2(v.w[0], v.w[1]);
  else if constexpr (V == 2) *reinterpret_cast<uint32_t*>(p) = v.w[0];
  else *p = static_cast<uint16_t>(v.w[0]);
}
template <bool F16>
__device__ __forceinline__ float2 wide2(uint32_t w) {
  if constexpr (F16) return __half22float2(bits_h2(w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
// The pairs (u.x, v.x), (u.y, v.y), turned.
__device__ __forceinline__ void turn2(const float2& u, const float2& v, const float* c, const float* z, float2& p,
                                      float2& q) {
  p = make_float2(u.x * c[0] - v.x * z[0], u.y * c[1] - v.y * z[1]);
  q = make_float2(u.x * z[0] + v.x * c[0], u.y * z[1] + v.y * c[1]);
}

// Threads: vector i of the turned part (n / V of a head) and a slot; the slots take
// the block's rows (token, head) in turns, with the next row's elements on their way.
template <int V, bool NEAR, bool F16>
__global__ void __launch_bounds__(V == 1 ? 2 * kBlock : kBlock) rotary_kernel(const RotaryArgs a) {
  constexpr int W = Vec<V>::kWords;
  __shared__ alignas(16) float cosine[kTable], sine[kTable];
  grid_dependency_wait();
  grid_launch_dependents();
  const int R = a.n / V, tid = threadIdx.x;
  const int slot = tid / R, i = tid - slot * R;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tokens;
  const int tokens = static_cast<int>(min(static_cast<int64_t>(a.tokens), a.n_tokens - t0));
  const int q_heads = a.side[0].heads, h0 = blockIdx.y * a.heads;
  const int h_end = min(q_heads + a.side[1].heads, h0 + a.heads), heads = h_end - h0;
  const int step_tk = a.slots / heads, step_h = a.slots - step_tk * heads;
  auto row_in = [&](int tk, int h) {
    const int k = h >= q_heads;
    const RotarySide& s = a.side[k];
    return static_cast<const uint16_t*>(s.in) + (t0 + tk) * s.in_token + (h - k * q_heads) * s.in_head + s.offset;
  };
  auto row_out = [&](int tk, int h) {
    const int k = h >= q_heads;
    const RotarySide& s = a.side[k];
    return static_cast<uint16_t*>(s.out) + (t0 + tk) * s.out_token + (h - k * q_heads) * s.out_head + s.offset;
  };
  const int first = NEAR ? 2 * i * V : i * V, second = NEAR ? first + V : first + a.n;
  Vec<V> x, y;
  int tk = slot / heads, h = h0 + slot - tk * heads;
  bool in = tk < tokens && slot < a.slots;
  if (in) {
    const uint16_t* const p = row_in(tk, h);
    x = load_vec<V>(p + first);
    y = load_vec<V>(p + second);
  }
  for (int k = tid; k < tokens * a.n; k += blockDim.x) {
    const int kt = k / a.n;
    const int64_t pos = a.wide_positions ? load(static_cast<const int64_t*>(a.positions) + t0 + kt)
                                         : load(static_cast<const int32_t*>(a.positions) + t0 + kt);
    const float freq = load(a.inv_freq + (k - kt * a.n));
    const uint64_t turn = static_cast<uint64_t>(pos) * turn_fraction(freq);
    float s, c;
    // (freq - freq: 0, or NaN of a frequency that is not finite)
    sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f + (freq - freq), &s, &c);
    cosine[k] = c * a.factor;
    sine[k] = s * a.factor;
  }
  __syncthreads();
  alignas(16) float c[V > 1 ? V : 2], z[V > 1 ? V : 2];
  int have = -1;                                          // token whose angles are in c and z
  while (in) {
    if (have != tk) {
      have = tk;
      const int k0 = tk * a.n + i * V;
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
        if constexpr (V == 1) c[1] = z[1] = 0.0f;
      }
    }
    uint16_t* const o = row_out(tk, h);
    h += step_h;
    tk += step_tk;
    if (h >= h_end) {
      h -= heads;
      ++tk;
    }
    in = tk < tokens;
    Vec<V> nx, ny;
    if (in) {
      const uint16_t* const p = row_in(tk, h);
      nx = load_vec<V>(p + first);
      ny = load_vec<V>(p + second);
    }
    if constexpr (!NEAR || V == 1) {
#pragma unroll
      for (int j = 0; j < W; ++j) {
        float2 p, q;
        turn2(wide2<F16>(x.w[j]), wide2<F16>(y.w[j]), c + 2 * j, z + 2 * j, p, q);
        x.w[j] = pack16<F16>(p.x, p.y);
        y.w[j] = pack16<F16>(q.x, q.y);
      }
    } else {
      // a word is a pair
#pragma unroll
      for (int j = 0; j < 2 * W; ++j) {
        uint32_t& w = j < W ? x.w[j % W] : y.w[j % W];
        const float2 u = wide2<F16>(w);
        w = pack16<F16>(u.x * c[j] - u.y * z[j], u.x * z[j] + u.y * c[j]);
      }
    }
    store_vec<V>(o + first, x);
    store_vec<V>(o + second, y);
    x = nx;
    y = ny;
  }
  // the elements that do not turn, where the outputs are not the inputs
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    const RotarySide& s = a.side[k];
    const int rest = (s.D - 2 * a.n) / V;                 // vectors of a head
    if (rest == 0 || s.out == s.in) continue;
    const int ha = max(static_cast<int>(blockIdx.y) * a.heads - k * q_heads, 0);
    const int per = (min(h_end - k * q_heads, s.heads) - ha) * rest;       // of a token
    auto place = [&](int u, const uint16_t*& in_p, uint16_t*& out_p) {
      const int j = u / rest;
      int e = (u - j * rest) * V;
      if (e >= s.offset) e += 2 * a.n;
      in_p = static_cast<const uint16_t*>(s.in) + t0 * s.in_token + (ha + j) * s.in_head + e;
      out_p = static_cast<uint16_t*>(s.out) + t0 * s.out_token + (ha + j) * s.out_head + e;
    };
    // four loads on their way: of neighbouring tokens, or of one token's vectors
    Vec<V> v[4];
    if (tokens >= 4) {
      for (int u = tid; u < per; u += blockDim.x) {
        const uint16_t* in_p;
        uint16_t* out_p;
        place(u, in_p, out_p);
        for (int kt = 0; kt < tokens; kt += 4, in_p += 4 * s.in_token, out_p += 4 * s.out_token) {
#pragma unroll
          for (int m = 0; m < 4; ++m)
            if (kt + m < tokens) v[m] = load_vec<V>(in_p + m * s.in_token);
#pragma unroll
          for (int m = 0; m < 4; ++m)
            if (kt + m < tokens) store_vec<V>(out_p + m * s.out_token, v[m]);
        }
      }
    } else {
      for (int kt = 0; kt < tokens; ++kt)
        for (int u = tid; u < per; u += 4 * blockDim.x) {
          uint16_t* out_p[4];
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const int um = u + m * blockDim.x;
            if (um >= per) continue;
            const uint16_t* in_p;
            place(um, in_p, out_p[m]);
            v[m] = load_vec<V>(in_p + kt * s.in_token);
          }
#pragma unroll
          for (int m = 0; m < 4; ++m)
            if (u + m * static_cast<int>(blockDim.x) < per) store_vec<V>(out_p[m] + kt * s.out_token, v[m]);
        }
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
  a.slots = std::max(1, kBlock / R);
  a.heads = heads;
  a.tokens = 1;
  const int64_t sms = a.num_sms;
  // No more than 2048 angles (kTable) a block: tokens * n <= kBlock + n.
  if (a.n_tokens < 4 * sms) {
    // few tokens: their heads over more blocks, each with the angles for itself
    const int share = static_cast<int>(heads * a.n_tokens / (8 * sms));
    a.heads = std::min({heads, a.slots, std::max(8, share)});
    while (a.tokens * a.heads < a.slots && a.tokens * a.n < kBlock && a.n_tokens >= 2 * sms * (a.tokens + 1)) ++a.tokens;
  } else {
    // several tokens after one another, so that all threads have angles to compute
    while (a.tokens * a.n < kBlock && a.n_tokens >= 16 * sms * a.tokens) ++a.tokens;
  }
  a.slots = std::min(a.slots, a.tokens * a.heads);
  const dim3 grid(static_cast<unsigned>((a.n_tokens + a.tokens - 1) / a.tokens),
                  static_cast<unsigned>((heads + a.heads - 1) / a.heads));
  // (threads beyond the slots' have their part in the angles and the copies)
  int rest = 0;
  for (const RotarySide& s : a.side)
    if (s.heads > 0 && s.out != s.in) rest = std::max(rest, (s.D - 2 * a.n) / V);
  const int copies = static_cast<int>(std::min<int64_t>(static_cast<int64_t>(rest) * a.heads / 4, kBlock));
  const unsigned threads = (static_cast<unsigned>(std::max(R * a.slots, copies)) + 31) / 32 * 32;
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
