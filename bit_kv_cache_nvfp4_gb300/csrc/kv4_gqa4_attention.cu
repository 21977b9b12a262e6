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

// ---------------------------------------------------------------------------
// Few rows: single tokens and short drafts
// ---------------------------------------------------------------------------
// What bounds this case is reading the cache once, at 9 bits for two elements: 24
// bytes, or 44 elements, a clock and SM.  Every one of them has to become f16 on
// the way to the tensor core (a scale for each 16 elements of a row, along D,
// which no block-scaled product applies to V), so what the kernel is built around
// is that nothing but the codes passes through shared memory: a warp's registers
// are the operands of mma.sync, m16n8k16, straight from the converted codes.
// (Converted tiles in shared memory, for tcgen05, would be written and read again
// at 88 bytes a clock each, beside the codes: the latent cache's decode is bound
// by that.)  Elements along a product's contraction may stand in any order that
// its two operands share, and rows in any order at all, so both products are
// laid out for the loads:
//   S^T[16 keys x 8 rows] += K . q^T     thread (r, t) = (lane / 4, lane % 4) has
//     elements t D/4 .. of keys r, r + 8: whole 16-byte pieces, with their scales
//   O^T[16 d x 8 rows] += V^T . P^T      thread (j, t) has elements j D/8 .. of
//     four keys; the codes of two keys are paired by nibbles, before they are
//     converted, so that each conversion gives a register of the operand.
// P^T comes from S^T by movmatrix, in f16.  A value code * scale has at most 6
// significant bits, in [2^-10, 2688]: exact in f16.  q is exact too (scaled by a
// power of two for each row, see the header for what it can lose), p is rounded
// to 2^-11.
//
// Block: warp 0 finds the block's share of the work list and copies chunks of 2304
// bytes of K and of V into a ring; each other warp takes every W-th chunk, with a
// softmax and an output of its own, and they join at the item's end.  The running
// reference of a row moves, and its output is rescaled, when the maximum rises by
// more than 2^6 (p stays below 2^14).
template <int D_, int RP_>
struct FewCfg {
  static constexpr int D = D_, RP = RP_, NT = RP / 8;
  static constexpr int kKeys = 4096 / D;                  // of a chunk
  static constexpr int kCodes = kKeys * D / 2, kScales = kKeys * D / 16;
  static constexpr int kStage = 2 * (kCodes + kScales);
  static constexpr int kCtas = RP == 8 ? 2 : 1;
  static constexpr int kWarps = RP == 8 ? 7 : 11;         // that compute
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr int kJoin = kWarps * RP * D * 4;
  static constexpr int kSmall = 3072;
  static constexpr int kRoom = kCtas == 2 ? 112 * 1024 : 227 * 1024;
  static constexpr int kStages = (kRoom - kJoin - kSmall) / kStage < 32 ? (kRoom - kJoin - kSmall) / kStage : 32;
  static constexpr int kSmem = kStages * kStage + kJoin + kSmall;
  static constexpr int kCost = 3;                         // what an item takes beyond its tiles, in tiles
};

struct FewSmall {
  uint64_t full[32], empty[32], item_full[4], item_empty[4], never;
  unsigned long long total;
  int dead;
  int gone[32];               // of a stage: its page is not there
  Gqa8Item items[4];
  float top[11][16], sum[11][16];
};
static_assert(sizeof(FewSmall) <= 3072, "FewSmall");

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Lane 4i + j holds elements 2j, 2j + 1 of row i of an 8 x 8 matrix: of its
// transpose afterwards.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// The nibbles of a and b in pairs (a's low): even elements, odd elements.
__device__ __forceinline__ uint32_t pair_even(uint32_t a, uint32_t b) {
  return (a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u);
}
__device__ __forceinline__ uint32_t pair_odd(uint32_t a, uint32_t b) {
  return ((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u);
}
__device__ __forceinline__ void scaled8(uint32_t w, uint32_t s2, uint32_t (&h)[4]) {
  e2m1x8_to_f16x8(w, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = f16x2_mul(h[i], s2);
}

template <int D, int RP, bool F16>
__global__ void __launch_bounds__(FewCfg<D, RP>::kThreads, FewCfg<D, RP>::kCtas)
few4_kernel(const Gqa8AttnArgs a, const int max_rows, Gqa8Tail* tails, float* ws_lse, float* ws_o) {
  using C = FewCfg<D, RP>;
  constexpr int NT = C::NT, ST = C::kStages, W = C::kWarps, CK = C::kKeys, MK = CK / 16, MD = D / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  float* const join = reinterpret_cast<float*>(smem + ST * C::kStage);
  FewSmall& sm = *reinterpret_cast<FewSmall*>(smem + ST * C::kStage + C::kJoin);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.Hq / a.Hkv;

  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(smem_addr(&sm.full[i]), 1);
      mbar_init(smem_addr(&sm.empty[i]), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_addr(&sm.item_full[i]), 1);
      mbar_init(smem_addr(&sm.item_empty[i]), W);
    }
    mbar_init(smem_addr(&sm.never), 1);
    sm.total = 0;
    sm.dead = 0;
    fence_mbar_init();
  }
  grid_dependency_wait();
  grid_launch_dependents();
  __syncthreads();
  // (a block for each item where they suffice and none is ever cut: all items
  // weigh the same)
  const bool one_each = (a.pt_stride + 1) / 2 <= kWhole && static_cast<int64_t>(a.B) * a.Hkv <= gridDim.x;
  const Gqa8Kind kind = one_each ? Gqa8Kind{1, max_rows, RP, 1, 0, 0, 0} : Gqa8Kind{1, max_rows, RP, C::kCost, RP, C::kCost, 1};
  gqa8_total(a, kind, blockIdx.x == 0, &sm.total);
  __syncthreads();
  volatile int* dead = &sm.dead;
  // A wait that gives up ends every later one of the block at once: the roles
  // then run to their ends without new loads, and the outputs are not valid.
  auto wait = [&](uint64_t& bar, uint32_t parity) {
    if (mbar_try_wait(smem_addr(&bar), parity)) return;
    if (*dead) return;
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait_suspend(smem_addr(&bar), parity, 20000u)) {
      if (*dead) return;
      if (global_timer_ns() - t0 > a.timeout_ns) {
        *dead = 1;
        flag_error(a.dev_err, kDevTimeout);
        return;
      }
    }
  };
  // an item's chunks: of its first key on, up to its last
  struct Chunks {
    int first, n;
  };
  auto chunks_of = [](const Gqa8Item& it) {
    const int64_t lo = max(static_cast<int64_t>(it.klo), static_cast<int64_t>(it.t_begin) * kTileKeys);
    const int64_t hi = min(static_cast<int64_t>(it.khi), static_cast<int64_t>(it.t_end) * kTileKeys);
    Chunks c{static_cast<int>(lo / CK), 0};
    if (hi > lo) c.n = static_cast<int>((hi - 1) / CK) + 1 - c.first;
    return c;
  };

  if (warp == 0) {
    // ==== work list and loads ====
    uint32_t n_items = 0, n_chunks = 0, n_loads = 0;      // chunks; up to which copies began
    auto publish = [&](const Gqa8Item& it) {
      const int s = n_items & 3;
      wait(sm.item_empty[s], ((n_items >> 2) & 1) ^ 1);
      // (of a wait that gave up the item before may still be in use)
      if (lane == 0 && !*dead) {
        sm.items[s] = it;
        mbar_arrive(smem_addr(&sm.item_full[s]));
      }
      ++n_items;
    };
    // lanes 0 .. 3 copy codes of K, of V, scales of K, of V
    uint8_t* const base = lane & 2 ? const_cast<uint8_t*>(a.scales) : const_cast<uint8_t*>(a.pool);
    const int row_bytes = lane & 2 ? D / 16 : D / 2;
    const uint32_t bytes = lane & 2 ? C::kScales : C::kCodes;
    const uint32_t dst0 = smem_addr(smem) + (lane & 2 ? 2 * C::kCodes : 0) + (lane & 1) * bytes;
    auto load_item = [&](const Gqa8Item& it) {
      const Chunks c = chunks_of(it);
      constexpr int kEach = kPage / CK;                   // chunks of a page
      int page = 0, page0 = -32;
      for (int i = 0; i < c.n; ++i, ++n_chunks) {
        const int chunk = c.first + i, p = chunk / kEach;
        if (p >= page0 + 32 || i == 0) {
          page0 = p;
          const int64_t at = static_cast<int64_t>(p) + lane;
          page = at * kPage < it.khi && at < a.pt_stride ? load(a.page_table + it.b * a.pt_stride + at) : 0;
          if (page < 0 || page >= a.num_pages) {
            page = -1;
            flag_error(a.dev_err, kDevBadPage);
          }
        }
        const int phys = __shfl_sync(0xFFFFFFFFu, page, p - page0);
        const int s = n_chunks % ST;
        wait(sm.empty[s], ((n_chunks / ST) & 1) ^ 1);
        const bool go = !__any_sync(0xFFFFFFFFu, *dead != 0);
        if (lane == 0 && go) {
          sm.gone[s] = phys < 0;
          if (phys >= 0) mbar_arrive_expect_tx(smem_addr(&sm.full[s]), C::kStage);
          else mbar_arrive(smem_addr(&sm.full[s]));
        }
        __syncwarp();
        if (go) n_loads = n_chunks + 1;
        if (go && phys >= 0 && lane < 4) {
          const int64_t row = ((static_cast<int64_t>(phys) * a.Hkv + it.h) * 2 + (lane & 1)) * kPage + chunk % kEach * CK;
          bulk_copy_g2s(dst0 + s * C::kStage, base + row * row_bytes, bytes, smem_addr(&sm.full[s]));
        }
        __syncwarp();
      }
    };
    gqa8_walk(a, kind, static_cast<int64_t>(sm.total), tails, lane, [&](const Gqa8Item& it) {
      publish(it);
      load_item(it);
    });
    publish(Gqa8Item{-1, 0, 0, 0, 0, 0, 0, 0, 0, 0, -1});
    // every copy lands before the block's shared memory goes away
    for (uint32_t i = n_chunks > ST ? n_chunks - ST : 0; i < n_chunks; ++i)
      wait(sm.empty[i % ST], (i / ST) & 1);
    if (*dead && lane == 0)
      for (uint32_t i = n_loads > ST ? n_loads - ST : 0; i < n_loads; ++i)
        mbar_wait_bounded(smem_addr(&sm.full[i % ST]), (i / ST) & 1, 1000000);
  } else {
    // ==== scores, softmax, output ====
    const int w = warp - 1, r8 = lane >> 2, t4 = lane & 3;
    // key of row m of a 16-key tile: 0, 4, 1, 5, 2, 6, 3, 7 and 8 more for m >= 8, so
    // that a thread's four keys of V are t, t + 4, t + 8, t + 12, whose rows lie in
    // all banks
    const int key_r = (r8 >> 1) + (r8 & 1) * 4;
    uint32_t n_chunks = 0;
    for (uint32_t n_items = 0;; ++n_items) {
      const int si = n_items & 3;
      wait(sm.item_full[si], (n_items >> 2) & 1);
      // (the warps stop together: one that left alone would leave the others at
      // their barrier)
      if (named_sync_or(1, 32 * W, *dead != 0)) break;
      const Gqa8Item it = sm.items[si];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sm.item_empty[si]));
      if (it.b < 0) break;
      const Chunks c = chunks_of(it);

      // q: row n of 8 is threads 4n .. 4n + 3's, D / 4 elements each
      uint32_t q[MD][NT][2];
      float qf[NT][2];
      int pos[NT][2];
      bool odd_col[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int rr = nt * 8 + r8, r = it.r0 + min(rr, it.nrows - 1);
        float x[D / 4];
        uint32_t m = 0;
        const uint4* g = reinterpret_cast<const uint4*>(
            static_cast<const uint16_t*>(a.q) + static_cast<int64_t>(it.cu0 + r / G) * a.q_token_stride +
            static_cast<int64_t>(it.h * G + r % G) * a.q_head_stride + t4 * (D / 4));
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          const uint4 two[2] = {load(g + 2 * i), load(g + 2 * i + 1)};
          m = max(m, widen16<F16>(two, reinterpret_cast<float(&)[16]>(x[16 * i])));
        }
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        const bool odd = m >= 0x7F800000u;                // a NaN or an infinity: NaN in its row
        const int e = q_exponent(m);
        const float f = (a.sm_scale < 0.0f ? -1.0f : 1.0f) * pow2f(-e);
#pragma unroll
        for (int j = 0; j < MD; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            q[j][nt][i] = odd ? 0u : h2_bits(__floats2half2_rn(x[4 * j + 2 * i] * f, x[4 * j + 2 * i + 1] * f));
        // (at least 2^-126, so that a masked -inf stays one where the scale is 0)
        const float mine = fmaxf(fabsf(a.sm_scale) * 1.4426950408889634f * pow2f(e), 0x1p-126f);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int col = 2 * t4 + i;                     // of the 8: its row's threads hold the factor
          qf[nt][i] = __shfl_sync(0xFFFFFFFFu, mine, col * 4);
          odd_col[nt][i] = __shfl_sync(0xFFFFFFFFu, static_cast<int>(odd), col * 4) != 0;
          pos[nt][i] = it.pos0 + (it.r0 + min(nt * 8 + col, it.nrows - 1)) / G;
        }
      }
      const int pos_first = it.pos0 + it.r0 / G, pos_last = it.pos0 + (it.r0 + it.nrows - 1) / G;
      float o[MD][NT][4], l[NT][2], mref[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          l[nt][i] = 0.0f;
          mref[nt][i] = kLowest;
        }
#pragma unroll
        for (int i = 0; i < MD; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[i][nt][k] = 0.0f;
      }

      // chunk i of the item is the block's chunk n_chunks + i: warp (that mod W)'s
      for (int i = (w + W - static_cast<int>(n_chunks % W)) % W; i < c.n; i += W) {
        const uint32_t n = n_chunks + i;
        const int st = n % ST;
        wait(sm.full[st], (n / ST) & 1);
        const int64_t base = static_cast<int64_t>(c.first + i) * CK;
        const uint8_t* const k_s = smem + st * C::kStage;
        const uint8_t* const v_s = k_s + C::kCodes;
        const uint8_t* const ks_s = k_s + 2 * C::kCodes;
        const uint8_t* const vs_s = ks_s + C::kScales;
        if (!sm.gone[st]) {
          const bool edge = base + CK > min(it.khi, pos_first + 1) || base < it.klo ||
                            (a.window > 0 && base <= static_cast<int64_t>(pos_last) - a.window);
          float s[MK][NT][4];
#pragma unroll
          for (int mk = 0; mk < MK; ++mk) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int k = 0; k < 4; ++k) s[mk][nt][k] = 0.0f;
            const int row0 = mk * 16 + key_r;
            uint32_t w0[D / 32], w1[D / 32], s0, s1;      // codes of keys r and r + 8, scales of their blocks
            if constexpr (D == 128) {
              *reinterpret_cast<uint4*>(w0) = *reinterpret_cast<const uint4*>(k_s + row0 * 64 + t4 * 16);
              *reinterpret_cast<uint4*>(w1) = *reinterpret_cast<const uint4*>(k_s + (row0 + 8) * 64 + t4 * 16);
              s0 = *reinterpret_cast<const uint16_t*>(ks_s + row0 * 8 + t4 * 2);
              s1 = *reinterpret_cast<const uint16_t*>(ks_s + (row0 + 8) * 8 + t4 * 2);
            } else {
              *reinterpret_cast<uint2*>(w0) = *reinterpret_cast<const uint2*>(k_s + row0 * 32 + t4 * 8);
              *reinterpret_cast<uint2*>(w1) = *reinterpret_cast<const uint2*>(k_s + (row0 + 8) * 32 + t4 * 8);
              s0 = ks_s[row0 * 4 + t4];
              s1 = ks_s[(row0 + 8) * 4 + t4];
            }
            s0 = e4m3x2_to_f16x2(s0);
            s1 = e4m3x2_to_f16x2(s1);
#pragma unroll
            for (int x = 0; x < D / 32; ++x) {
              // (two words a block of 16)
              const uint32_t f0 = __byte_perm(s0, 0, x / 2 == 0 ? 0x1010 : 0x3232);
              const uint32_t f1 = __byte_perm(s1, 0, x / 2 == 0 ? 0x1010 : 0x3232);
              uint32_t h0[4], h1[4];
              scaled8(w0[x], f0, h0);
              scaled8(w1[x], f1, h1);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma_16816(s[mk][nt], h0[0], h1[0], h0[1], h1[1], q[2 * x][nt][0], q[2 * x][nt][1]);
                mma_16816(s[mk][nt], h0[2], h1[2], h0[3], h1[3], q[2 * x + 1][nt][0], q[2 * x + 1][nt][1]);
              }
            }
          }
          if (edge) {
            // 0 <= position - key < window, of the keys that are there
            const uint32_t win = a.window > 0 ? a.window : 0x80000000u;
#pragma unroll
            for (int mk = 0; mk < MK; ++mk)
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int key = static_cast<int>(base) + mk * 16 + key_r + (k & 2) * 4;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  if (!(static_cast<uint32_t>(pos[nt][k & 1] - key) < win && key < it.khi)) s[mk][nt][k] = -INFINITY;
              }
          }
          float mx[NT][2];
          bool rise = false;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float m = fmaxf(s[0][nt][k], s[0][nt][k + 2]);
#pragma unroll
              for (int mk = 1; mk < MK; ++mk) m = max3(m, s[mk][nt][k], s[mk][nt][k + 2]);
#pragma unroll
              for (int off = 4; off < 32; off *= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
              mx[nt][k] = m * qf[nt][k];
              rise |= mx[nt][k] > mref[nt][k] + 6.0f;
            }
          if (__any_sync(0xFFFFFFFFu, rise)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const float to = fmaxf(mref[nt][k], mx[nt][k]), by = fast_exp2(mref[nt][k] - to);
                mref[nt][k] = to;
                l[nt][k] *= by;
#pragma unroll
                for (int x = 0; x < MD; ++x) {
                  o[x][nt][k] *= by;
                  o[x][nt][k + 2] *= by;
                }
              }
          }
          uint32_t p[MK][NT][2];                          // P^T: keys 2t, 2t + 1 and 8 more, row lane / 4
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float b0 = 8.0f - mref[nt][0], b1 = 8.0f - mref[nt][1];
#pragma unroll
            for (int mk = 0; mk < MK; ++mk)
#pragma unroll
              for (int k = 0; k < 4; k += 2) {
                const float p0 = fast_exp2(fmaf(s[mk][nt][k], qf[nt][0], b0));
                const float p1 = fast_exp2(fmaf(s[mk][nt][k + 1], qf[nt][1], b1));
                l[nt][0] += p0;
                l[nt][1] += p1;
                p[mk][nt][k / 2] = transpose8x8(h2_bits(__floats2half2_rn(p0, p1)));
              }
          }
#pragma unroll
          for (int mk = 0; mk < MK; ++mk) {
            uint32_t v[4][D / 64], sc[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int row = mk * 16 + t4 + 4 * k;
              if constexpr (D == 128) {
                *reinterpret_cast<uint2*>(v[k]) = *reinterpret_cast<const uint2*>(v_s + row * 64 + r8 * 8);
                sc[k] = vs_s[row * 8 + r8];
              } else {
                v[k][0] = *reinterpret_cast<const uint32_t*>(v_s + row * 32 + r8 * 4);
                sc[k] = vs_s[row * 4 + (r8 >> 1)];
              }
              // a key that no row sees may hold a NaN scale, which a weight of zero
              // would not silence
              if (edge) sc[k] = base + row >= it.klo && base + row < it.khi ? sc[k] : 0u;
            }
            const uint32_t s01 = e4m3x2_to_f16x2(sc[0] | (sc[1] << 8)), s23 = e4m3x2_to_f16x2(sc[2] | (sc[3] << 8));
#pragma unroll
            for (int x = 0; x < D / 64; ++x) {
              uint32_t e01[4], o01[4], e23[4], o23[4];
              scaled8(pair_even(v[0][x], v[1][x]), s01, e01);
              scaled8(pair_odd(v[0][x], v[1][x]), s01, o01);
              scaled8(pair_even(v[2][x], v[3][x]), s23, e23);
              scaled8(pair_odd(v[2][x], v[3][x]), s23, o23);
#pragma unroll
              for (int y = 0; y < 4; ++y)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma_16816(o[4 * x + y][nt], e01[y], o01[y], e23[y], o23[y], p[mk][nt][0], p[mk][nt][1]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sm.empty[st]));
      }
      n_chunks += c.n;

      // ---- the warps' outputs, joined relative to the largest reference ----
      // (behind this barrier all have read what the item before left here)
      named_sync(1, 32 * W);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float x = l[nt][k];
#pragma unroll
          for (int off = 4; off < 32; off *= 2) x += __shfl_xor_sync(0xFFFFFFFFu, x, off);
          const int row = nt * 8 + 2 * t4 + k;
          if (r8 == 0) {
            sm.top[w][row] = mref[nt][k];
            sm.sum[w][row] = odd_col[nt][k] && x > 0.0f ? __uint_as_float(0x7FC00000u) : x;
          }
          // d = 2 MD lane / 4 + 2 i and the next
#pragma unroll
          for (int i = 0; i < MD; ++i)
            *reinterpret_cast<float2*>(join + (w * RP + row) * D + r8 * (D / 8) + 2 * i) =
                make_float2(o[i][nt][k], o[i][nt][k + 2]);
        }
      named_sync(1, 32 * W);
      for (int u = tid - 32; u < it.nrows * (D / 4); u += 32 * W) {
        const int row = u / (D / 4), d = u % (D / 4) * 4;
        float top = kLowest;
#pragma unroll
        for (int i = 0; i < W; ++i) top = fmaxf(top, sm.top[i][row]);
        float y[4] = {0.0f, 0.0f, 0.0f, 0.0f}, sum = 0.0f;
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const float f = fast_exp2(sm.top[i][row] - top);
          sum = fmaf(sm.sum[i][row], f, sum);
          const float4 v = *reinterpret_cast<const float4*>(join + (i * RP + row) * D + d);
          y[0] = fmaf(v.x, f, y[0]);
          y[1] = fmaf(v.y, f, y[1]);
          y[2] = fmaf(v.z, f, y[2]);
          y[3] = fmaf(v.w, f, y[3]);
        }
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        const float ls = sum == 0.0f ? -INFINITY : top - 8.0f + log2f(sum);
        if (it.slot >= 0) {
          const int64_t at = static_cast<int64_t>(it.slot) * RP + row;
          *reinterpret_cast<float4*>(ws_o + at * D + d) = make_float4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
          if (d == 0) ws_lse[at] = ls;
        } else {
          const int r = it.r0 + row;
          const int64_t at = static_cast<int64_t>(it.cu0 + r / G) * a.Hq + it.h * G + r % G;
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at * D + d) =
              make_uint2(pack16<F16>(y[0] * inv, y[1] * inv), pack16<F16>(y[2] * inv, y[3] * inv));
          if (d == 0) a.lse[at] = ls * 0.6931471805599453f;
        }
      }
      if (a.fault_site == 1 && w == 0) wait(sm.never, 0);
    }
  }
  __syncthreads();
}

// The plain kernel: a block for each row, a key for each warp at a time, D / 32
// elements a lane.
template <int D, bool F16>
__global__ void __launch_bounds__(128) row_kernel(const Gqa8AttnArgs a, const int min_rows) {
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
  const Gqa8Request r = gqa8_request(a, b, min_rows, 0x7FFFFFFF, min_rows == 1 && h == 0 && t == min(max(load(a.cu + b), 0), static_cast<int>(a.n_tokens)));
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

// ---------------------------------------------------------------------------
// Launch
// ---------------------------------------------------------------------------
// Rows of few4_kernel's items, and of the largest request that it takes: 8 or 16,
// the smaller that holds every request or, where some have more, a single token of
// any; 0: none.
int few_rows(int max_new, int G) {
  const int64_t all = static_cast<int64_t>(max_new) * G, need = all <= 16 ? all : G;
  return need <= 8 ? 8 : need <= 16 ? 16 : 0;
}
constexpr int kFewCtas = 2;                               // blocks an SM at most
size_t few_bytes(int rows, int D, int sms) {
  return rows == 0 ? 0 : (part_bytes(kFewCtas * sms, rows, D) + 255) / 256 * 256;
}

template <int D, int RP, bool F16>
cudaError_t launch_few(const Gqa8AttnArgs& a, int max_rows, void* ws, cudaStream_t stream) {
  using C = FewCfg<D, RP>;
  cudaError_t e = prepare_kernel<few4_kernel<D, RP, F16>>(C::kSmem, 0);
  if (e != cudaSuccess) return e;
  // (no more blocks than there can be tiles, or items where none is ever cut)
  const int64_t tiles = (a.pt_stride + 1) / 2, most = a.B * static_cast<int64_t>(a.Hkv) * (tiles <= kWhole ? 1 : tiles);
  const int blocks = static_cast<int>(std::min<int64_t>(a.num_sms * C::kCtas, most));
  const Parts p = parts_at(ws, blocks, RP, D);
  e = launch_pdl(few4_kernel<D, RP, F16>, blocks, C::kThreads, C::kSmem, stream, 1, a, max_rows, p.tails, p.lse, p.o);
  return e != cudaSuccess ? e : launch_merge(merge_few_kernel<D>, a, blocks, RP, RP, p, stream);
}

template <int D, bool F16>
cudaError_t launch_d(const Gqa8AttnArgs& a, cudaStream_t stream) {
  const int G = a.Hq / a.Hkv, rows = few_rows(a.max_new, G);
  cudaError_t e = cudaSuccess;
  if (rows == 8) e = launch_few<D, 8, F16>(a, rows, a.ws, stream);
  else if (rows == 16) e = launch_few<D, 16, F16>(a, rows, a.ws, stream);
  if (e != cudaSuccess || static_cast<int64_t>(a.max_new) * G <= rows) return e;
  row_kernel<D, F16><<<dim3(static_cast<unsigned>(a.n_tokens), a.Hq), 128, 0, stream>>>(a, rows + 1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention_gqa4(const Gqa8AttnArgs& a, cudaStream_t stream) {
  if (a.D == 64) return a.f16 ? launch_d<64, true>(a, stream) : launch_d<64, false>(a, stream);
  return a.f16 ? launch_d<128, true>(a, stream) : launch_d<128, false>(a, stream);
}

size_t attention_gqa4_workspace(int max_new, int Hq, int Hkv, int D, int num_sms) {
  return few_bytes(few_rows(max_new, Hq / Hkv), D, num_sms);
}

}  // namespace kv4
