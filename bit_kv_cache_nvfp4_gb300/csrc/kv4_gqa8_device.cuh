// kv4_gqa8_device.cuh -- helpers of the attention over the 8-bit grouped-query
// cache: TMA loads of cache pages, the FP8 tensor-core product, and the
// splitting of 16-bit operands into E4M3 terms.
#pragma once

#include <cuda.h>

#include "kv4_device.cuh"
#include "kv4_launch.h"

namespace kv4 {

// Every load of the caller's tensors and of the workspace.  The kernels here may
// begin before the kernel before them has ended (grid_dependency_wait waits for
// it), and that one may have written any of them, so none is read-only while
// they run: a plain load, never the read-only path, which may be served from
// before the wait.
template <typename T>
__device__ __forceinline__ T load(const T* p) {
  return *p;
}

__device__ __forceinline__ float pow2f(int e) {     // e in [-126, 127]
  return __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}

// 64 rows of one (page, head, side) -> shared memory, swizzled; box index
// `block` past the tensor gives zeros.  Completes on the mbarrier.
__device__ __forceinline__ void tma_load_block(uint32_t dst, const CUtensorMap* map, int block,
                                               uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(0), "r"(0), "r"(block), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// Instruction descriptor for kind::f8f6f4: D fp32, A and B E4M3, dense.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, bool a_mn_major, bool b_mn_major) {
  return (1u << 4) | ((a_mn_major ? 1u : 0u) << 15) | ((b_mn_major ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ void mma_f8kind(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// f16x2 -> two E4M3 bytes, round half to even, saturating; and back (exact).
__device__ __forceinline__ uint32_t e4m3x2_of_f16x2(uint32_t h2) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h2));
  return r;
}
__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }

// Two values (f16x2, magnitudes up to 448) as NT E4M3 terms each:
// x = t0 + t1 / 16 + t2 / 256, every term rounded to nearest (4 significant
// bits).  The differences are exact in f16: after t0 at most 7 of the 11 bits
// are left, after t1 at most 3.  Two terms hold 8 bits (all of a bf16 value),
// three hold 11; a value below 2^-6 keeps 2^-10 / 16 (2^-10 / 256) of absolute
// accuracy.
template <int NT>
__device__ __forceinline__ void split_e4m3(uint32_t x, uint32_t (&t)[NT]) {
  t[0] = e4m3x2_of_f16x2(x);
#pragma unroll
  for (int i = 1; i < NT; ++i) {
    const __half2 r = __hsub2(bits_h2(x), bits_h2(e4m3x2_to_f16x2(t[i - 1])));
    x = h2_bits(__hmul2(r, __half2half2(__float2half(16.0f))));
    t[i] = e4m3x2_of_f16x2(x);
  }
}

// The same without the factors: x = t0 + t1 + .., so that the terms' products
// add up in one accumulator; with |x|'s largest near 448, elements below 2^-10 of
// it (two terms, the 8 bits of a bf16 value) or 2^-7 (three, the 11 of an f16)
// keep 2^-18 of it.
template <int NT>
__device__ __forceinline__ void split_e4m3_same(uint32_t x, uint32_t (&t)[NT]) {
  t[0] = e4m3x2_of_f16x2(x);
#pragma unroll
  for (int i = 1; i < NT; ++i) {
    x = h2_bits(__hsub2(bits_h2(x), bits_h2(e4m3x2_to_f16x2(t[i - 1]))));
    t[i] = e4m3x2_of_f16x2(x);
  }
}

// 16 values of q: widened to fp32; returns the bits of the largest magnitude.
template <bool F16>
__device__ __forceinline__ uint32_t widen16(const uint4 (&w)[2], float (&x)[16]) {
  const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (F16) {
      const float2 f = __half22float2(bits_h2(u[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    } else {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
    m = max(m, max(__float_as_uint(x[2 * i]) & 0x7FFFFFFFu, __float_as_uint(x[2 * i + 1]) & 0x7FFFFFFFu));
  }
  return m;
}
// Least e with amax <= 448 * 2^e of a row of q: 120 for the largest bf16.  From
// below it is kept at -118, so that 2^-e and 2^e are normal fp32: a row whose
// largest is under 2^-109 keeps less of itself than other rows do.
__device__ __forceinline__ int q_exponent(uint32_t amax_bits) {
  const int e = static_cast<int>(amax_bits >> 23) - 135 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, -118), 120);
}
// 16 values times f (0 where `zero`) as NT terms of 16 bytes.
template <int NT, bool kSame>
__device__ __forceinline__ void terms16(const float (&x)[16], float f, bool zero, uint32_t (&o)[NT][4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t t[2][NT];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float x0 = zero ? 0.0f : x[4 * i + 2 * k] * f, x1 = zero ? 0.0f : x[4 * i + 2 * k + 1] * f;
      if constexpr (kSame) split_e4m3_same<NT>(h2_bits(__floats2half2_rn(x0, x1)), t[k]);
      else split_e4m3<NT>(h2_bits(__floats2half2_rn(x0, x1)), t[k]);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) o[n][i] = t[0][n] | (t[1][n] << 16);
  }
}

// Two fp32 values -> 16-bit pair (first in the low half), round half to even.
template <bool F16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (F16) return h2_bits(__floats2half2_rn(lo, hi));
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Two fp32 operations in one instruction, each rounded as by itself.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Largest value over the warp (NaN only where every lane holds one).
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
// Sums over the warp of R values of each lane (R a power of two, up to 32):
// every lane gets the sum of value `row`, with R + 3 or so shuffles in place
// of 5 R.
template <int R>
__device__ __forceinline__ float warp_sums(float (&v)[R], int lane, int& row) {
  int off = 16;
  row = 0;
#pragma unroll
  for (int w = R / 2; w >= 1; w /= 2, off /= 2) {
    const bool up = (lane & off) != 0;
    row += up ? w : 0;
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const float give = up ? v[i] : v[i + w], keep = up ? v[i + w] : v[i];
      v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, off);
    }
  }
  float x = v[0];
#pragma unroll
  for (; off > 0; off /= 2) x += __shfl_xor_sync(0xFFFFFFFFu, x, off);
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, off);
  return x;
}

// ---------------------------------------------------------------------------
// The work list.  A request's rows are r = i * G + g (new token i, head g of
// the group); `rows` consecutive ones, of one kv head, are an item, which
// walks its keys in tiles of 128 (tile t: keys 128 t .. 128 t + 127, two
// pages).  Items are ordered by request, row group, kv head; each counts for
// its tiles and `cost` more (what starting and ending an item takes), in units
// of which a tile has one or more, and every block takes an equal share of the
// whole, found from the lengths on the device.  An item that a border between two shares falls into
// is cut there, unless it has few tiles or the cut would leave fewer than
// kLeast to a side: then the border moves to the item's nearer end.  The
// pieces of a cut item are joined by a second kernel.
// ---------------------------------------------------------------------------
struct Gqa8Request {
  int cu0;          // first flat row
  int n;            // new tokens (0: not of this kernel)
  int pos0;         // position of the first one (may be negative)
  int held;         // tokens that the page table can name, of len
};
struct Gqa8Span {
  int klo, khi;     // keys that some row of the item sees
  int t0, nt;       // first tile, tiles
};
__device__ __forceinline__ Gqa8Request gqa8_request(const Gqa8AttnArgs& a, int b, int min_rows,
                                                    int max_rows, bool report) {
  Gqa8Request q{0, 0, 0, 0};
  if (b >= a.B) return q;
  const int T = static_cast<int>(a.n_tokens);
  const int c0 = min(max(load(a.cu + b), 0), T), c1 = min(max(load(a.cu + b + 1), 0), T);
  const int len = max(load(a.lens + b), 0);
  if (c1 <= c0) return q;
  if (c1 - c0 > a.max_new) {
    if (report) flag_error(a.dev_err, kDevBadLength);
    return q;
  }
  const int64_t cap = a.pt_stride << 6;
  if (report && cap < len) flag_error(a.dev_err, kDevBadPage);
  const int64_t rows = static_cast<int64_t>(c1 - c0) * (a.Hq / a.Hkv);
  if (rows < min_rows || rows > max_rows) return q;
  q.cu0 = c0;
  q.n = c1 - c0;
  q.pos0 = len - q.n;
  q.held = len < cap ? len : static_cast<int>(cap);
  return q;
}
// Keys of rows [r0, r1) of a request.
__device__ __forceinline__ Gqa8Span gqa8_span(const Gqa8AttnArgs& a, const Gqa8Request& q, int G,
                                              int r0, int r1) {
  Gqa8Span s;
  const int64_t first = static_cast<int64_t>(q.pos0) + r0 / G, last = static_cast<int64_t>(q.pos0) + (r1 - 1) / G;
  int64_t lo = a.window > 0 ? first - a.window + 1 : 0;
  if (lo < 0) lo = 0;
  int64_t hi = last + 1 < q.held ? last + 1 : q.held;
  if (hi < lo) hi = lo;
  s.klo = static_cast<int>(lo);
  s.khi = static_cast<int>(hi);
  s.t0 = s.klo >> 7;
  s.nt = hi > lo ? ((s.khi - 1) >> 7) + 1 - s.t0 : 0;
  return s;
}
struct Gqa8Kind {     // of requests that one of the kernels takes
  int min_rows, max_rows;
  int rows;           // of an item
  int cost;           // units of an item beyond its tiles
  int half;           // items of at most so many rows: a unit a tile,
  int half_cost;      //   and so many beyond them
  int tile;           // others: so many a tile
  __device__ __forceinline__ int units(int n_rows) const { return n_rows <= half ? 1 : tile; }
  __device__ __forceinline__ int beyond(int n_rows) const { return n_rows <= half ? half_cost : cost; }
};
constexpr int kWhole = 4, kLeast = 2;

// a / b of non-negative integers; nearly always both fit 32 bits, where the
// division is several times as fast.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0)
    return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// Units of the requests of a warp's lanes: a lane by itself where it has few
// row groups, the warp together for the others.
__device__ __forceinline__ int64_t gqa8_units(const Gqa8AttnArgs& a, const Gqa8Request& q,
                                              const Gqa8Kind& kind, int G, int lane) {
  const int R = q.n * G, groups = (R + kind.rows - 1) / kind.rows;
  auto units = [&](const Gqa8Request& r, int i, int n_rows) {
    const int r0 = i * kind.rows, r1 = min(n_rows, r0 + kind.rows);
    return static_cast<int64_t>(gqa8_span(a, r, G, r0, r1).nt) * kind.units(r1 - r0) + kind.beyond(r1 - r0);
  };
  int64_t u = 0;
  if (groups <= 2)
    for (int i = 0; i < groups; ++i) u += units(q, i, R);
  for (uint32_t todo = __ballot_sync(0xFFFFFFFFu, groups > 2); todo != 0; todo &= todo - 1) {
    const int l = __ffs(todo) - 1;
    Gqa8Request r;
    r.cu0 = 0;
    r.n = __shfl_sync(0xFFFFFFFFu, q.n, l);
    r.pos0 = __shfl_sync(0xFFFFFFFFu, q.pos0, l);
    r.held = __shfl_sync(0xFFFFFFFFu, q.held, l);
    const int gr = __shfl_sync(0xFFFFFFFFu, groups, l);
    int64_t v = 0;
    for (int i = lane; i < gr; i += 32) v += units(r, i, r.n * G);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    if (lane == l) u = v;
  }
  return u * a.Hkv;
}
// Sum over all requests, added to *total by every warp of the block.
__device__ __forceinline__ void gqa8_total(const Gqa8AttnArgs& a, const Gqa8Kind& kind, bool report,
                                           unsigned long long* total) {
  const int lane = threadIdx.x & 31;
  int64_t u = 0;
  for (int base = threadIdx.x & ~31; base < a.B; base += blockDim.x)
    u += gqa8_units(a, gqa8_request(a, base + lane, kind.min_rows, kind.max_rows, report), kind,
                    a.Hq / a.Hkv, lane);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) u += __shfl_xor_sync(0xFFFFFFFFu, u, off);
  if (lane == 0 && u > 0) atomicAdd(total, static_cast<unsigned long long>(u));
}

struct Gqa8Item {
  int b;                     // request, -1: no more work
  int h;
  int cu0, pos0;             // of the request
  int r0, nrows;
  int klo, khi;
  int t_begin, t_end;        // tiles that this block walks
  int slot;                  // partial slot, or -1: the rows are finished here
};

// What the merge kernel reads of a block's item that other blocks continue.
struct Gqa8Tail {
  int parts;                 // 0: none; else pieces, in this block and the next parts - 1
  int cu0, h, r0, nrows, pad[3];
};

constexpr int kMasked = 0x7FFF7FFF;
constexpr float kLowest = -3e38f;

// Where the border at unit u cuts an item of nt tiles of `each` units that
// begins at unit `begin`: tiles before the border, 0 .. nt (0 and nt also where
// it is not in the item at all).
__device__ __forceinline__ int gqa8_cut(int64_t u, int64_t begin, int nt, int each, int cost) {
  const int64_t x = u - begin, all = static_cast<int64_t>(nt) * each + cost;
  if (x <= 0) return 0;
  if (x >= all) return nt;
  if (nt <= kWhole) return 2 * x <= all ? 0 : nt;
  const int64_t t = x <= cost ? 0 : quotient(x - cost, each);
  return t < kLeast ? 0 : t > nt - kLeast ? nt : static_cast<int>(t);
}

// The items of this block, in order, to `emit` (whole warp), of `total` units.
// Also leaves this block's tail.
template <typename Emit>
__device__ __forceinline__ void gqa8_walk(const Gqa8AttnArgs& a, const Gqa8Kind& kind, int64_t total,
                                          Gqa8Tail* tails, int lane, Emit&& emit) {
  const int G = a.Hq / a.Hkv, blocks = gridDim.x, me = blockIdx.x;
  // (no share so small that a long item's pieces would cost more to join than
  // they save; where no item is ever cut, as small as one item)
  const int64_t least = (a.pt_stride + 1) / 2 <= kWhole ? 1 : kWhole * kind.tile;
  const int64_t per = max(quotient(total + blocks - 1, blocks), least);
  const int64_t u0 = me * per, u1 = u0 + per;
  bool tail = false;
  int64_t acc = 0;
  for (int base = 0; base < a.B && acc < u1 && u0 < total; base += 32) {
    const Gqa8Request q = gqa8_request(a, base + lane, kind.min_rows, kind.max_rows, false);
    const int64_t units = gqa8_units(a, q, kind, G, lane);
    int64_t end = units;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t v = __shfl_up_sync(0xFFFFFFFFu, end, off);
      if (lane >= off) end += v;
    }
    end += acc;
    acc = __shfl_sync(0xFFFFFFFFu, end, 31);
    uint32_t todo = __ballot_sync(0xFFFFFFFFu, units > 0 && end > u0 && end - units < u1);
    for (; todo != 0; todo &= todo - 1) {
      const int l = __ffs(todo) - 1;
      Gqa8Request r;
      r.cu0 = __shfl_sync(0xFFFFFFFFu, q.cu0, l);
      r.n = __shfl_sync(0xFFFFFFFFu, q.n, l);
      r.pos0 = __shfl_sync(0xFFFFFFFFu, q.pos0, l);
      r.held = __shfl_sync(0xFFFFFFFFu, q.held, l);
      int64_t first = __shfl_sync(0xFFFFFFFFu, end - units, l);
      const int R = r.n * G, groups = (R + kind.rows - 1) / kind.rows;
      for (int g0 = 0; g0 < groups && first < u1; g0 += 32) {
        // a lane's row group, and where its items begin
        const int gi = g0 + lane;
        Gqa8Span sp{0, 0, 0, 0};
        int64_t w = 0;
        if (gi < groups) {
          sp = gqa8_span(a, r, G, gi * kind.rows, min(R, (gi + 1) * kind.rows));
          const int n = min(kind.rows, R - gi * kind.rows);
          w = (static_cast<int64_t>(sp.nt) * kind.units(n) + kind.beyond(n)) * a.Hkv;
        }
        int64_t g_end = w;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int64_t v = __shfl_up_sync(0xFFFFFFFFu, g_end, off);
          if (lane >= off) g_end += v;
        }
        g_end += first;
        uint32_t gtodo = __ballot_sync(0xFFFFFFFFu, w > 0 && g_end > u0 && g_end - w < u1);
        for (; gtodo != 0; gtodo &= gtodo - 1) {
          const int gl = __ffs(gtodo) - 1;
          const int klo = __shfl_sync(0xFFFFFFFFu, sp.klo, gl), khi = __shfl_sync(0xFFFFFFFFu, sp.khi, gl);
          const int t0 = __shfl_sync(0xFFFFFFFFu, sp.t0, gl), nt = __shfl_sync(0xFFFFFFFFu, sp.nt, gl);
          const int64_t at = __shfl_sync(0xFFFFFFFFu, g_end - w, gl);
          const int r0 = (g0 + gl) * kind.rows, nrows = min(kind.rows, R - r0), upt = kind.units(nrows);
          const int cost = kind.beyond(nrows);
          const int64_t each = static_cast<int64_t>(nt) * upt + cost;
          const int h0 = at < u0 ? static_cast<int>(quotient(u0 - at, each)) : 0;
          int64_t begin = at + h0 * each;
          for (int h = h0; h < a.Hkv && begin < u1; ++h, begin += each) {
            const int tb = gqa8_cut(u0, begin, nt, upt, cost), te = gqa8_cut(u1, begin, nt, upt, cost);
            int slot = -1;
            if (nt == 0) {
              // no tile to cut: the block that its first unit falls to
              if (begin < u0) continue;
            } else if (tb == te) {
              continue;
            } else if (tb > 0) {
              slot = 2 * me;
            } else if (te < nt) {
              slot = 2 * me + 1;
              tail = true;
              // the last block that has some of it
              int last = static_cast<int>(quotient(begin + each - 1, per));
              while (gqa8_cut(last * per, begin, nt, upt, cost) == nt) --last;
              if (lane == 0) tails[me] = Gqa8Tail{last - me + 1, r.cu0, h, r0, nrows, {}};
            }
            emit(Gqa8Item{base + l, h, r.cu0, r.pos0, r0, nrows, klo, khi, t0 + tb, t0 + te, slot});
          }
        }
        first = __shfl_sync(0xFFFFFFFFu, g_end, 31);
      }
    }
  }
  if (lane == 0 && !tail) tails[me].parts = 0;
}

// Page `lane` of the 16 tiles from tile t on: its block of the pool (past the
// pool where there is none: TMA gives zeros) and its two exponents, kMasked
// where there is no page.  The append's exponents lie in [-48, 48]; others
// count as the nearer end, so that sums of p over V exponents stay in range.
__device__ __forceinline__ void gqa8_pages(const Gqa8AttnArgs& a, const Gqa8Item& it, int t, int lane,
                                           int& block, int& ex) {
  const int64_t page = 2 * static_cast<int64_t>(t) + lane;
  block = static_cast<int>(a.num_pages) * a.Hkv;
  ex = kMasked;
  if ((page >> 1) < it.t_end && (page << 6) < it.khi && (page << 6) + 64 > it.klo) {
    const int phys = load(a.page_table + it.b * a.pt_stride + page);
    if (phys < 0 || phys >= a.num_pages) {
      flag_error(a.dev_err, kDevBadPage);
    } else {
      block = phys * a.Hkv + it.h;
      const uint32_t e2 = load(reinterpret_cast<const uint16_t*>(a.scales) + block);
      const int ek = min(max(static_cast<int>(e2 & 0xFF) - 127, kGqa8ExpMin), kGqa8ExpMax);
      const int ev = min(max(static_cast<int>(e2 >> 8) - 127, kGqa8ExpMin), kGqa8ExpMax);
      ex = (ek & 0xFFFF) | static_cast<int>(static_cast<uint32_t>(ev) << 16);
    }
  }
}

}  // namespace kv4
