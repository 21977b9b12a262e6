// kv4_gqa8_attention.cu -- causal attention of new tokens over the 8-bit
// grouped-query cache (kv4_attention_gqa8).
//
// Row (t, h): query head h of flat token t; token i of request b's n new ones
// stands at position seq_lens[b] - n + i and sees the keys j <= its position,
// j > position - window where there is a window.  Scores, the running maximum
// and sum and the output are held in fp32:
//   s_j = sm_scale q.k_j,  o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),
//   lse = m + log sum_j exp(s_j - m);  a row without a key: 0 and -inf.
#include "kv4_gqa8_device.cuh"

#include <math.h>
#include <stddef.h>

#include <mutex>
#include <type_traits>

namespace kv4 {
namespace {

// ---------------------------------------------------------------------------
// Few rows: single tokens and short drafts
// ---------------------------------------------------------------------------
// What bounds this case is reading the codes once (2 G flops per byte), so the
// codes go from HBM to the tensor core as they are, with no conversion on the
// way: K and V tiles land in shared memory by TMA in the swizzle that
// tcgen05.mma reads, and it is the small operands -- q and the softmax weights
// p -- that are brought to E4M3, as sums of NT terms (split_e4m3), the terms side
// by side as columns of one product:
//   S^T[128 keys x NT RP] = K . [q_0 | q_1 | ..]^T      (M = 128, N = NT RP)
//   O^T[D x NT RP] = V^T . [p_0 | p_1 | ..]^T            (M = D, K = 128 keys)
// s = S_0 + S_1 / 16 + ..., likewise o.  Both accumulate in fp32.  Two terms
// hold p to 2^-8 (half a bf16 step), three, in f16 calls, to f16's 2^-11; and q
// exactly, but for elements below 2^-14 of their row's largest, which keep 2^-22
// of that (f16: 2^-26).  Block exponents are powers of two: K's is a factor of
// the score, V's is added to it in the exponent of p,
//   p_j = 2^(s_j + eV_j - m + 8),   m = max_j (s_j + eV_j) of the row's keys in
// the tile (s in units of log 2), so that what a weight is rounded by is relative
// to what its key can add to the row, however far apart the exponents of the
// tile's pages are, and a page that the row does not see has no part in it.  The
// terms' 2^-10 granularity is 2^-22 of the tile's largest 2^(s + eV) (two terms;
// 2^-26 three), and never meets a maximum from far away; each tile's O is a
// product of its own, joined to the running output in registers.  The softmax's
// sum takes p 2^-eV, in fp32: eV is in [-48, 48], so the key of the largest score
// is at least 2^-88 there, and neither it nor a sum can leave the range.
//
// Block: warp 0 finds the block's share of the work list and issues the loads,
// warp 1 the products, warps 2-3 bring q of the next item to E4M3, and one or
// two warpgroups are the softmax: a thread holds one key of S^T (and one d of
// O^T).  Two blocks share an SM, with one softmax warpgroup each, where they
// fit; else one block has two warpgroups that take every other tile, each with
// a running output of its own, joined at the item's end.
//
// Measured (D = 128, bf16): 64 sessions of up to 32768 tokens, 8 heads a group,
// 2.29 GB of codes: 340 us, 6.7 TB/s, the rate of a copy; 16 heads a group
// (2.08 GB) 355 us; 2 x 204800 tokens cut over 304 blocks 133 us with the joining
// kernel.  In f16, with three terms, 394 us for 2.16 GB, 5.5 TB/s.
template <int D_, int RP_, int NT_>
struct FewCfg {
  static constexpr int D = D_, RP = RP_, NT = NT_;
  static constexpr bool kF16 = NT == 3;                   // f16 calls take three terms, bf16 ones two
  static constexpr int N = (NT * RP + 15) / 16 * 16;      // MMA columns (N % 16 == 0 at M = 128)
  static constexpr int kTile = 2 * kTileKeys * D;         // K and V of a tile
  static constexpr int kQ = (N * D + 1023) / 1024 * 1024; // one of two
  static constexpr int kP = N / 16 * 2048;                // one of two
  static constexpr int kSmall = 6144;                     // barriers, items, factors
  static constexpr int kFixed = 2 * kQ + 2 * kP + kSmall;
  // two blocks of an SM, with half of its 228 KB each, or one with more stages
  static constexpr int kHalf = 113 * 1024 - 1024;
  static constexpr int kCtas = RP == 8 ? 2 : 1;
  static constexpr int kWgs = kCtas == 2 ? 1 : 2;         // softmax warpgroups
  static constexpr int kThreads = 128 + 128 * kWgs;
  // what an item takes beyond its tiles, in tiles (1, 3 | 2, 5 | 3, 8 of the two
  // kinds: decode with 16 heads a group 370, 360, 357 us, with 8 343 all)
  static constexpr int kCost = kWgs == 2 ? 8 : 3;
  static_assert(kWgs == 1 || 2 * kP >= RP * 512, "the joined output goes through P's memory");
  static constexpr int kStages = (kCtas == 2 ? kHalf - kFixed : 163840) / kTile;
  static constexpr int kSmem = kStages * kTile + kFixed + 1024;
  static constexpr uint32_t kTmem = 4 * N <= 64 ? 64 : 4 * N <= 128 ? 128 : 4 * N <= 256 ? 256 : 512;
};

struct FewSmall {
  uint64_t full[12], empty[12], item_full[4], item_empty[4], q_full[2], q_empty[2], s_full[2], p_full[2],
      o_full[2], never;
  unsigned long long total;
  uint32_t tmem;
  int dead;
  int exps[12][2];            // per stage and page: K exponent | V exponent << 16; kMasked
  Gqa8Item items[4];
  float qf[2][32];            // sm_scale log2(e) 2^eq of a row, NaN where q is not finite
  int pos[2][32];             // a row's position, -1 where it is negative
  alignas(16) float red[4][32 * 4];    // read as float4; by warpgroup and parity of its tiles
  alignas(16) float2 stash[4][32];
  float lsum[2][4][32], top[2][32];
};
static_assert(sizeof(FewSmall) <= 6144 && offsetof(FewSmall, red) % 16 == 0 &&
                  offsetof(FewSmall, stash) % 8 == 0,
              "FewSmall");

template <int D, int RP, int NT>
__global__ void __launch_bounds__(FewCfg<D, RP, NT>::kThreads, FewCfg<D, RP, NT>::kCtas)
few_kernel(const __grid_constant__ CUtensorMap map, const Gqa8AttnArgs a, const int max_rows,
           Gqa8Tail* tails, float* ws_lse, float* ws_o) {
  using C = FewCfg<D, RP, NT>;
  constexpr int N = C::N, ST = C::kStages, WGS = C::kWgs;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const q_s = smem + ST * C::kTile;
  uint8_t* const p_s = q_s + 2 * C::kQ;
  FewSmall& sm = *reinterpret_cast<FewSmall*>(p_s + 2 * C::kP);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.Hq / a.Hkv;

  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(smem_addr(&sm.full[i]), 1);
      mbar_init(smem_addr(&sm.empty[i]), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_addr(&sm.item_full[i]), 1);
      mbar_init(smem_addr(&sm.item_empty[i]), 3 + 4 * WGS);      // the product's warp, 2, the softmax's
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&sm.q_full[i]), 2);
      mbar_init(smem_addr(&sm.q_empty[i]), 1 + 4 * WGS);         // the last QK, the softmax's warps
      mbar_init(smem_addr(&sm.s_full[i]), 1);
      mbar_init(smem_addr(&sm.p_full[i]), 4);
      mbar_init(smem_addr(&sm.o_full[i]), 1);
    }
    mbar_init(smem_addr(&sm.never), 1);
    sm.total = 0;
    sm.dead = 0;
    fence_mbar_init();
    tma_prefetch_map(&map);
  }
  if (warp == 1) tmem_alloc(smem_addr(&sm.tmem), C::kTmem);
  // columns past NT * RP stay zero in both operands
  if constexpr (N > NT * RP)
    for (int i = tid; i < (2 * C::kQ + 2 * C::kP) / 16; i += C::kThreads)
      reinterpret_cast<uint4*>(q_s)[i] = make_uint4(0, 0, 0, 0);
  grid_dependency_wait();
  grid_launch_dependents();
  __syncthreads();
  // (a block for each item where they suffice and none is ever cut: all items
  // weigh the same; in replays of a graph 16 requests of 500 tokens over 8 heads
  // 9.3 us, 10.9 with 304 blocks and items by weight, of 1 to 500 tokens 9.7 and
  // 11.0.  The lengths are on the device, so that it is the page table's width, up
  // to 8 columns, that says none is cut.)
  const bool one_each = (a.pt_stride + 1) / 2 <= kWhole && static_cast<int64_t>(a.B) * a.Hkv <= gridDim.x;
  const Gqa8Kind kind = one_each ? Gqa8Kind{1, max_rows, RP, 1, 0, 0, 0} : Gqa8Kind{1, max_rows, RP, C::kCost, RP, C::kCost, 1};
  gqa8_total(a, kind, blockIdx.x == 0, &sm.total);
  fence_async_smem();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = sm.tmem;
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

  if (warp == 0) {
    // ==== work list and loads ====
    uint32_t n_items = 0, n_tiles = 0, n_loads = 0;       // tiles; loads that lane 0 began
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
    auto load = [&](const Gqa8Item& it) {
      for (int t = it.t_begin; t < it.t_end; t += 16) {
        int block, ex;
        gqa8_pages(a, it, t, lane, block, ex);
        const int nt = min(16, it.t_end - t);
        for (int i = 0; i < nt; ++i, ++n_tiles) {
          const int b0 = __shfl_sync(0xFFFFFFFFu, block, 2 * i), b1 = __shfl_sync(0xFFFFFFFFu, block, 2 * i + 1);
          const int e0 = __shfl_sync(0xFFFFFFFFu, ex, 2 * i), e1 = __shfl_sync(0xFFFFFFFFu, ex, 2 * i + 1);
          const int s = n_tiles % ST;
          wait(sm.empty[s], ((n_tiles / ST) & 1) ^ 1);
          if (lane == 0 && !*dead) {
            n_loads = n_tiles + 1;
            sm.exps[s][0] = e0;
            sm.exps[s][1] = e1;
            const uint32_t bar = smem_addr(&sm.full[s]), dst = smem_addr(smem + s * C::kTile);
            mbar_arrive_expect_tx(bar, C::kTile);
            tma_load_block(dst, &map, 2 * b0, bar);
            tma_load_block(dst + 64 * D, &map, 2 * b1, bar);
            tma_load_block(dst + 128 * D, &map, 2 * b0 + 1, bar);
            tma_load_block(dst + 192 * D, &map, 2 * b1 + 1, bar);
          }
          __syncwarp();
        }
      }
    };
    gqa8_walk(a, kind, static_cast<int64_t>(sm.total), tails, lane, [&](const Gqa8Item& it) {
      publish(it);
      load(it);
    });
    publish(Gqa8Item{-1, 0, 0, 0, 0, 0, 0, 0, 0, 0, -1});
    // every load and every product's signal lands before the block's shared
    // memory goes away
    for (uint32_t i = n_tiles > ST ? n_tiles - ST : 0; i < n_tiles; ++i)
      wait(sm.empty[i % ST], (i / ST) & 1);
    if (*dead && lane == 0)
      for (uint32_t i = n_loads > ST ? n_loads - ST : 0; i < n_loads; ++i)
        mbar_wait_bounded(smem_addr(&sm.full[i % ST]), (i / ST) & 1, 1000000);
  } else if (warp == 1) {
    // ==== products (the whole warp; one lane issues) ====
    constexpr uint32_t kSw = D == 128 ? kSwizzle128 : kSwizzle64;
    constexpr uint32_t idesc_qk = idesc_e4m3(128, N, false, false);
    constexpr uint32_t idesc_pv = idesc_e4m3(D, N, true, true);
    const uint64_t dk0 = smem_desc(smem_addr(smem), 16, 8 * D, kSw), dq0 = smem_desc(smem_addr(q_s), 16, 8 * D, kSw);
    const uint64_t dp0 = smem_desc(smem_addr(p_s), 128, 2048, kSwizzleNone);
    uint32_t n_items = 0, n_tiles = 0;
    uint32_t st = 0, st_par = 0, st_last = 0;             // stage of the next tile and of the one before
    // PV of tile j: O^T = V^T . P^T over 128 keys, 32 a step
    auto pv = [&](uint32_t j) {
      wait(sm.p_full[j & 1], (j >> 1) & 1);
      __syncwarp();
      tc_fence_after_sync();
      if (elect_one()) {
        const uint64_t dv = dk0 + ((st_last * C::kTile + kTileKeys * D) >> 4), dp = dp0 + (j & 1) * (C::kP >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f8kind(tmem + 2 * N + (j & 1) * N, dv + ((k * 32 * D) >> 4), dp + ((k * 512) >> 4), idesc_pv, k > 0);
        mma_commit(smem_addr(&sm.o_full[j & 1]));
        mma_commit(smem_addr(&sm.empty[st_last]));
      }
      __syncwarp();
    };
    auto ready = [&](uint64_t& bar, uint32_t parity) {
      return __any_sync(0xFFFFFFFFu, mbar_try_wait(smem_addr(&bar), parity));
    };
    // In a block that gave up nothing else waits for the products that are
    // still queued: they end before its memory goes away.
    auto drain = [&] {
      if (a.fault_site == 1) wait(sm.never, 0);
      __syncwarp();
      if (!__any_sync(0xFFFFFFFFu, *dead != 0)) return;
      if (elect_one()) mma_commit(smem_addr(&sm.never));
      __syncwarp();
      mbar_wait_bounded(smem_addr(&sm.never), 0, 1000000);
    };
    bool pending = false;
    while (true) {
      const int s = n_items & 3;
      if (pending && !ready(sm.item_full[s], (n_items >> 2) & 1)) {
        pv(n_tiles - 1);
        pending = false;
      }
      wait(sm.item_full[s], (n_items >> 2) & 1);
      if (__any_sync(0xFFFFFFFFu, *dead != 0)) break;
      const int b = __shfl_sync(0xFFFFFFFFu, sm.items[s].b, 0);
      const int nt = __shfl_sync(0xFFFFFFFFu, sm.items[s].t_end - sm.items[s].t_begin, 0);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sm.item_empty[s]));
      if (b < 0) break;
      const uint32_t qb = n_items & 1;
      const uint64_t dq = dq0 + qb * (C::kQ >> 4);
      for (int t = 0; t < nt; ++t, ++n_tiles) {
        const uint32_t j = n_tiles;
        // the next scores first, unless their keys are still on the way
        if (pending && !ready(sm.full[st], st_par)) {
          pv(j - 1);
          pending = false;
        }
        if (t == 0) wait(sm.q_full[qb], (n_items >> 1) & 1);
        wait(sm.full[st], st_par);
        __syncwarp();
        tc_fence_after_sync();
        if (elect_one()) {
          const uint64_t dk = dk0 + st * (C::kTile >> 4);
#pragma unroll
          for (int k = 0; k < D / 32; ++k)
            mma_f8kind(tmem + (j & 1) * N, dk + 2 * k, dq + 2 * k, idesc_qk, k > 0);
          mma_commit(smem_addr(&sm.s_full[j & 1]));
          if (t == nt - 1) mma_commit(smem_addr(&sm.q_empty[qb]));
        }
        __syncwarp();
        if (pending) pv(j - 1);
        pending = true;
        st_last = st;
        if (++st == ST) {
          st = 0;
          st_par ^= 1;
        }
      }
      if (nt == 0) {
        // (a product left pending here would keep the softmax from its item,
        // so from the q buffer that the wait after next is for)
        if (pending) pv(n_tiles - 1);
        pending = false;
        wait(sm.q_full[qb], (n_items >> 1) & 1);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sm.q_empty[qb]));
      }
      if (a.fault_site == 1) wait(sm.never, 0);
      ++n_items;
    }
    if (pending) pv(n_tiles - 1);
    drain();
  } else if (warp < 4) {
    // ==== q of the next item, as NT E4M3 terms ====
    constexpr int TPR = D / 16, RPP = 64 / TPR;           // threads a row, rows at once
    const int part = tid % TPR, row_in = (tid - 64) / TPR;
    for (uint32_t n_items = 0;; ++n_items) {
      const int s = n_items & 3, qb = n_items & 1;
      wait(sm.item_full[s], (n_items >> 2) & 1);
      if (__any_sync(0xFFFFFFFFu, *dead != 0)) break;
      const Gqa8Item it = sm.items[s];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sm.item_empty[s]));
      if (it.b < 0) break;
      wait(sm.q_empty[qb], ((n_items >> 1) & 1) ^ 1);
#pragma unroll 1
      for (int rr = row_in; rr < RP; rr += RPP) {
        uint4 w[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        if (rr < it.nrows) {
          const int r = it.r0 + rr;
          const uint4* g = reinterpret_cast<const uint4*>(
              static_cast<const uint16_t*>(a.q) + static_cast<int64_t>(it.cu0 + r / G) * a.q_token_stride +
              static_cast<int64_t>(it.h * G + r % G) * a.q_head_stride + part * 16);
          w[0] = load(g);
          w[1] = load(g + 1);
        }
        float x[16];
        uint32_t m = widen16<C::kF16>(w, x);
#pragma unroll
        for (int off = 1; off < TPR; off <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
        const bool odd = m >= 0x7F800000u;                // a NaN or an infinity: NaN in its row
        const int e = q_exponent(m);
        if (part == 0) {
          sm.pos[qb][rr] = max(it.pos0 + (it.r0 + rr) / G, -1);
          sm.qf[qb][rr] = odd ? __uint_as_float(0x7FC00000u) : a.sm_scale * 1.4426950408889634f * pow2f(e);
        }
        uint32_t o[NT][4];
        terms16<NT, false>(x, pow2f(-e), odd, o);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const uint32_t off = (t * RP + rr) * D + part * 16;
          *reinterpret_cast<uint4*>(q_s + qb * C::kQ + swizzle<D == 128 ? 3 : 2>(off)) =
              make_uint4(o[t][0], o[t][1], o[t][2], o[t][3]);
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sm.q_full[qb]));
    }
  } else {
    // ==== softmax ====
    const int wg = (warp - 4) >> 2;
    const int key = tid & 127;                            // of a tile; and d of O^T
    const int quarter = warp & 3;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const int bar = 1 + wg;
    constexpr int kBarAll = 3;
    uint32_t n_tiles = 0, n_own = 0;                      // tiles of all items, of this warpgroup
    for (uint32_t n_items = 0;; ++n_items) {
      const int s = n_items & 3, qb = n_items & 1;
      wait(sm.item_full[s], (n_items >> 2) & 1);
      // the warps stop together: a warp that left alone would leave the others
      // at their barrier
      if (named_sync_or(kBarAll, 128 * WGS, *dead != 0)) break;
      const Gqa8Item it = sm.items[s];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sm.item_empty[s]));
      if (it.b < 0) break;
      wait(sm.q_full[qb], (n_items >> 1) & 1);
      float o[RP], l[RP], mref[RP], mref_mine = kLowest;
#pragma unroll
      for (int r = 0; r < RP; ++r) {
        o[r] = l[r] = 0.0f;
        mref[r] = kLowest;
      }
      // rows' positions: pos0 + (r0 + r) / G
      const int pos_first = it.pos0 + it.r0 / G, pos_last = it.pos0 + (it.r0 + it.nrows - 1) / G;
      // O of tile j, this warpgroup's i-th, joins the running output
      auto join = [&](uint32_t j, uint32_t i_own) {
        const float2* const stash = sm.stash[2 * wg + (i_own & 1)];
        wait(sm.o_full[j & 1], (j >> 1) & 1);
        tc_fence_after_sync();
#pragma unroll
        for (int c = 0; c < RP; c += 8) {
          uint32_t v[NT][8];
#pragma unroll
          for (int t = 0; t < NT; ++t) tmem_ld8(lanes + 2 * N + (j & 1) * N + t * RP + c, v[t]);
#pragma unroll
          for (int t = 0; t < NT; ++t) tmem_wait_ld8(v[t]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float x = __uint_as_float(v[NT - 1][i]);
#pragma unroll
            for (int t = NT - 2; t >= 0; --t) x = fmaf(x, 0.0625f, __uint_as_float(v[t][i]));
            const float2 f = stash[c + i];
            o[c + i] = fmaf(o[c + i], f.x, x * f.y);
          }
        }
        tc_fence_before_sync();
      };
      // (of two warpgroups, tile j's is the one with its parity, whose S, P and O
      // memory are)
      const int first = it.t_begin + (WGS == 2 ? static_cast<int>((n_tiles ^ wg) & 1) : 0);
      for (int t = first; t < it.t_end; t += WGS, ++n_own) {
        const uint32_t j = n_tiles + (t - it.t_begin);
        const int st = j % ST;
        wait(sm.full[st], (j / ST) & 1);                  // the exponents, and V where it is cleaned
        const int ex = sm.exps[st][key >> 6];
        const int at = t * kTileKeys + key;               // this thread's key
        const bool live = ex != kMasked && at >= it.klo && at < it.khi;
        const int ek = static_cast<int16_t>(ex & 0xFFFF), ev = ex == kMasked ? kGqa8ExpMin : ex >> 16;
        const float kf = live ? pow2f(ek) : 0.0f;
        const float evf = static_cast<float>(ev), vinv = pow2f(-ev);
        const bool edge = (t + 1) * static_cast<int64_t>(kTileKeys) > min(it.khi, pos_first + 1) ||
                          t * kTileKeys < it.klo ||
                          (a.window > 0 && t * static_cast<int64_t>(kTileKeys) <= static_cast<int64_t>(pos_last) - a.window);
        if (!live) {
          // bytes that belong to nobody may be NaN codes, which a weight of
          // zero does not silence: the row of V is cleared
          uint4* row = reinterpret_cast<uint4*>(smem + st * C::kTile + (kTileKeys + key) * D);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) row[i] = make_uint4(0, 0, 0, 0);
        }
        wait(sm.s_full[j & 1], (j >> 1) & 1);
        tc_fence_after_sync();
        float sc[RP];
        float mine = kLowest;
#pragma unroll
        for (int c = 0; c < RP; c += 8) {
          uint32_t v[NT][8];
#pragma unroll
          for (int k = 0; k < NT; ++k) tmem_ld8(lanes + (j & 1) * N + k * RP + c, v[k]);
#pragma unroll
          for (int k = 0; k < NT; ++k) tmem_wait_ld8(v[k]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float x = __uint_as_float(v[NT - 1][i]);
#pragma unroll
            for (int k = NT - 2; k >= 0; --k) x = fmaf(x, 0.0625f, __uint_as_float(v[k][i]));
            sc[c + i] = fmaf(x * kf, sm.qf[qb][c + i], evf);
          }
        }
        if (edge || !live) {
          // 0 <= position - key < window
          const uint32_t win = live ? (a.window > 0 ? a.window : 0x80000000u) : 0u;
#pragma unroll
          for (int r = 0; r < RP; ++r)
            sc[r] = static_cast<uint32_t>(sm.pos[qb][r] - at) < win ? sc[r] : -INFINITY;
        }
#pragma unroll
        for (int r = 0; r < RP; ++r) {
          const float m = warp_max(sc[r]);
          if (lane == r) mine = m;
        }
        if (lane < RP) sm.red[2 * wg + (n_own & 1)][lane * 4 + quarter] = mine;
        tc_fence_before_sync();
        named_sync(bar, 128);
        // (the tile before is done with its O before P of this one is sent)
        if (WGS == 2 && t > first) join(j - 2, n_own - 1);
        // (all loads before any store: the compiler keeps their order, and a
        // load behind each column's store would cost its whole latency there)
        auto top_of = [&](int r) {
          const float4 m4 = *reinterpret_cast<const float4*>(&sm.red[2 * wg + (n_own & 1)][r * 4]);
          return fmaxf(max3(m4.x, m4.y, m4.z), fmaxf(m4.w, kLowest));
        };
        float mt[RP];
#pragma unroll
        for (int r = 0; r < RP; ++r) mt[r] = top_of(r);
        const float mt_mine = top_of(key < RP ? key : 0);
        uint32_t terms[RP / 8 * NT * 2];                  // bytes of the row of P: term, row
#pragma unroll
        for (int r = 0; r < RP; r += 2) {
          float p[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            // the running reference is the largest so far; of the two factors
            // one is 1
            const bool up = mt[r + i] > mref[r + i];
            const float x = fast_exp2(up ? mref[r + i] - mt[r + i] : mt[r + i] - mref[r + i]);
            p[i] = fast_exp2(sc[r + i] - (mt[r + i] - 8.0f));
            const float w = p[i] * vinv;
            l[r + i] = up ? fmaf(l[r + i], x, w) : fmaf(w, x, l[r + i]);
            mref[r + i] = up ? mt[r + i] : mref[r + i];
          }
          uint32_t tt[NT];
          split_e4m3<NT>(h2_bits(__floats2half2_rn(p[0], p[1])), tt);
#pragma unroll
          for (int k = 0; k < NT; ++k) {
            const int byte = k * RP + r;                  // of the key's row
            if (byte % 4 == 0) terms[byte / 4] = tt[k];
            else terms[byte / 4] |= tt[k] << 16;
          }
        }
        uint8_t* const pb = p_s + (j & 1) * C::kP + key * 16;
#pragma unroll
        for (int k = 0; k < N / 16; ++k) {
          uint32_t w4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w4[i] = (k * 4 + i) < RP * NT / 4 ? terms[(k * 4 + i) < RP * NT / 4 ? k * 4 + i : 0] : 0u;
          *reinterpret_cast<uint4*>(pb + k * 2048) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
        }
        if (key < RP) {
          // row `key`'s factors of the running output and of this tile's
          const bool up = mt_mine > mref_mine;
          const float x = fast_exp2(up ? mref_mine - mt_mine : mt_mine - mref_mine);
          sm.stash[2 * wg + (n_own & 1)][key] = make_float2(up ? x : 1.0f, up ? 1.0f : x);
          mref_mine = up ? mt_mine : mref_mine;
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sm.p_full[j & 1]));
        if (WGS == 1 && t > first) join(j - 1, n_own - 1);
      }
      // the factors of the last tile, written by other warps, are visible
      // behind this barrier
      named_sync(bar, 128);
      if (first < it.t_end) join(n_tiles + (it.t_end - it.t_begin - 1 - (it.t_end - 1 - first) % WGS), n_own - 1);
      n_tiles += it.t_end - it.t_begin;
      if constexpr (RP == 24) {
        float a16[16], a8[8];
#pragma unroll
        for (int r = 0; r < 24; ++r) (r < 16 ? a16[r < 16 ? r : 0] : a8[r < 16 ? 0 : r - 16]) = l[r];
        int r;
        const float s16 = warp_sums<16>(a16, lane, r);
        sm.lsum[wg][quarter][r] = s16;
        const float s8 = warp_sums<8>(a8, lane, r);
        sm.lsum[wg][quarter][16 + r] = s8;
      } else {
        int r;
        const float s = warp_sums<RP>(l, lane, r);
        sm.lsum[wg][quarter][r] = s;
      }
      if (key < RP) sm.top[wg][key] = mref_mine;
      if (lane == 0) mbar_arrive(smem_addr(&sm.q_empty[qb]));
      named_sync(kBarAll, 128 * WGS);
      if constexpr (WGS == 2) {
        // the second warpgroup's output goes to the first relative to the larger
        // reference of the two, through P's memory, which no product reads now
        float* const x = reinterpret_cast<float*>(p_s) + key;
#pragma unroll
        for (int r = 0; r < RP; ++r) {
          const float w = fast_exp2(mref[r] - fmaxf(sm.top[0][r], sm.top[1][r]));
          o[r] *= w;
          if (wg == 1) x[r * 128] = o[r];
        }
        named_sync(kBarAll, 256);
        if (wg == 1) continue;
#pragma unroll
        for (int r = 0; r < RP; ++r) o[r] += x[r * 128];
      }
      const bool mine_d = D == 128 || lane < 16;          // M = 64: 16 lanes of each warp
      const int d = D == 128 ? key : quarter * 16 + lane;
      int tok = it.r0 / G, g = it.r0 - tok * G;
#pragma unroll
      for (int r = 0; r < RP; ++r) {
        if (r >= it.nrows) break;
        auto sum_of = [&](int w) { return (sm.lsum[w][0][r] + sm.lsum[w][1][r]) + (sm.lsum[w][2][r] + sm.lsum[w][3][r]); };
        float lt = sum_of(0), ref = mref[r];
        if constexpr (WGS == 2) {
          ref = fmaxf(mref[r], sm.top[1][r]);
          lt = lt * fast_exp2(mref[r] - ref) + sum_of(1) * fast_exp2(sm.top[1][r] - ref);
        }
        const float y = lt == 0.0f ? 0.0f : __fdividef(o[r], lt);
        const float ls = lt == 0.0f ? -INFINITY : ref - 8.0f + fast_log2(lt);
        if (it.slot >= 0) {
          const int64_t row = static_cast<int64_t>(it.slot) * RP + r;
          if (mine_d) ws_o[row * D + d] = y;
          if (key == 0) ws_lse[row] = ls;
        } else {
          const int64_t row = static_cast<int64_t>(it.cu0 + tok) * a.Hq + it.h * G + g;
          if (mine_d) {
            if constexpr (C::kF16) static_cast<__half*>(a.out)[row * D + d] = __float2half_rn(y);
            else static_cast<__nv_bfloat16*>(a.out)[row * D + d] = __float2bfloat16_rn(y);
          }
          if (key == 0) a.lse[row] = ls * 0.6931471805599453f;
        }
        if (++g == G) {
          g = 0;
          ++tok;
        }
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, C::kTmem);
}

// ---------------------------------------------------------------------------
// Many rows: prompt chunks
// ---------------------------------------------------------------------------
// What bounds this case is the tensor core: 4 D flops a pair of row and key.
// An item is 256 rows of one kv head, two M = 128 tiles that take turns: while
// the softmax of one works on its scores, the products of the other run.  Of an
// item with at most 128 rows the two are the same rows over every other tile of
// keys, joined at its end, so that they take turns all the same.
//   S[128 rows x 128 keys] = sum_t Q_t . K^T     kind::f8f6f4, NT terms of q
//   O[128 rows x D] += P . V                     kind::f16, P from TMEM
// K goes in as its codes, against q split into E4M3 terms (bf16: two, f16:
// three; all with the same scale, so that they add up in one accumulator, which
// keeps 2^-18 of a row's largest: split_e4m3_same).  V
// is widened to f16 once per tile by two warps (exact), for P in f16 (2^-11)
// takes one pass where E4M3 terms would take two and twice the instructions
// in the softmax, which has the least room to spare.
// The chain scores -> softmax -> P -> O, next scores of a row tile is what the
// other tile's products have to cover, so two threads share a row, one for each
// page of the tile (64 keys): K's block exponent and the scale of q multiply
// the scores, V's is added to the exponent of p, so that p is relative to a
// running reference of score and V exponent together, which the two halves
// agree on for every tile.  A row's reference only moves, and its O in TMEM is
// only rescaled, when that rises by more than 2^6 (p stays below 2^14, f16's
// top is 2^16).
//
// Measured (D = 128, 32 heads over 8, bf16): 2 x 2048 new tokens over 16384 625
// us, 1.30 PFLOP/s (69 % of the measured bf16 rate; without the softmax the
// products alone took 500); a prompt of 8192 474 us, 1.16.  f16, three terms:
// 808 us for a chunk with 1.27 times the pairs, 1.27 PFLOP/s, and 506 us.  D = 64:
// 578 and 394 us in bf16, 0.80 and 0.70 PFLOP/s: a tile has the same softmax for
// half the products.
template <int D_, int NT_>
struct ManyCfg {
  static constexpr int D = D_, NT = NT_, kRows = 256;
  static constexpr bool kF16 = NT == 3;
  static constexpr int kK = kTileKeys * D;                // K or V codes of a tile
  static constexpr int kV16 = kTileKeys * D * 2;
  static constexpr int kQ = NT * 128 * D;                 // of one of the two row tiles
  static constexpr int kKStages = NT == 2 ? 3 : 2, kVStages = NT == 2 ? 2 : 1;
  static constexpr int kSmall = 9216;
  static constexpr int kSmem = 2 * kQ + kKStages * kK + kVStages * kK + 2 * kV16 + kSmall + 1024;
};
static_assert(ManyCfg<128, 3>::kSmem <= 227 * 1024 && ManyCfg<128, 2>::kSmem <= 227 * 1024, "shared memory");
constexpr int kManyThreads = 640;
constexpr uint32_t kSoftmaxRegs = 104, kOtherRegs = 64, kLaunchRegs = 96;
static_assert(4 * kSoftmaxRegs + kOtherRegs <= 5 * kLaunchRegs, "register shares draw on the launch's");

// What an item takes beyond its tiles (q in, first scores, last product, output),
// in half tiles; of an item of at most 128 rows.  (A whole prompt of 8192: 619
// us with 6, 541 with 8, 486 with 10, 488 with 12, 493 with 16.)
constexpr int kManyCost = 10, kSharedCost = 4;

struct ManySmall {
  uint64_t k_full[3], k_empty[3], v8_full[2], v8_empty[2], v_full[2], v_empty[2], item_full[2], item_empty[2],
      ex_full[8], q_full[2], s_full[2], p_full[2][2], o_full[2], never;
  unsigned long long total;
  uint32_t tmem;
  int dead;
  alignas(16) float4 exps[8][2];    // per tile and page: 2^eK, eV, 2^-eV, 0 where there is no page
  Gqa8Item items[2];
  float qf[2][128];           // sm_scale log2(e) 2^eq of a row, NaN where q is not finite
  float top[2][2][2][128];    // largest score and V exponent of a half row, by row tile and tile parity
  float last[2][3][128];      // at an item's end: sums of both halves, reference
};
static_assert(sizeof(ManySmall) <= 9216 && offsetof(ManySmall, exps) % 16 == 0, "ManySmall");

template <int D, int NT>
__global__ void __launch_bounds__(kManyThreads, 1)
many_kernel(const __grid_constant__ CUtensorMap map, const Gqa8AttnArgs a, const int min_rows,
            Gqa8Tail* tails, float* ws_lse, float* ws_o) {
  using C = ManyCfg<D, NT>;
  constexpr int KS = C::kKStages, VS = C::kVStages;
  constexpr int kSlab = kTileKeys * 128;                  // 64 f16 columns of V
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const q_s = smem;
  uint8_t* const k_s = q_s + 2 * C::kQ;
  uint8_t* const v8_s = k_s + KS * C::kK;
  uint8_t* const v_s = v8_s + VS * C::kK;
  ManySmall& sm = *reinterpret_cast<ManySmall*>(v_s + 2 * C::kV16);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.Hq / a.Hkv;
  constexpr int kAll = 0x7FFFFFFF;

  if (tid == 0) {
    for (int i = 0; i < 3; ++i) {
      mbar_init(smem_addr(&sm.k_full[i]), 1);
      mbar_init(smem_addr(&sm.k_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&sm.v8_full[i]), 1);
      mbar_init(smem_addr(&sm.v8_empty[i]), 2);
      mbar_init(smem_addr(&sm.v_full[i]), 2);
      mbar_init(smem_addr(&sm.v_empty[i]), 1);
      mbar_init(smem_addr(&sm.item_full[i]), 1);
      mbar_init(smem_addr(&sm.item_empty[i]), 19);        // the product's lane, 2 + 16 warps
      mbar_init(smem_addr(&sm.q_full[i]), 8);
      mbar_init(smem_addr(&sm.s_full[i]), 1);
      mbar_init(smem_addr(&sm.p_full[i][0]), 8);
      mbar_init(smem_addr(&sm.p_full[i][1]), 8);
      mbar_init(smem_addr(&sm.o_full[i]), 1);
    }
    for (int i = 0; i < 8; ++i) mbar_init(smem_addr(&sm.ex_full[i]), 1);
    mbar_init(smem_addr(&sm.never), 1);
    sm.total = 0;
    sm.dead = 0;
    fence_mbar_init();
    tma_prefetch_map(&map);
  }
  if (warp == 1) tmem_alloc(smem_addr(&sm.tmem), 512);
  grid_dependency_wait();
  grid_launch_dependents();
  __syncthreads();
  const Gqa8Kind kind{min_rows, kAll, C::kRows, kManyCost, 128, kSharedCost, 2};
  gqa8_total(a, kind, blockIdx.x == 0 && min_rows == 1, &sm.total);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = sm.tmem;                          // S/P of the row tiles, then O
  volatile int* dead = &sm.dead;
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

  if (warp < 4) {
    setmaxnreg_dec<kOtherRegs>();
    if (warp == 0) {
      // ==== work list and loads ====
      uint32_t n_items = 0, n_tiles = 0, n_loads = 0;     // tiles; loads that lane 0 began
      auto publish = [&](const Gqa8Item& it) {
        const int s = n_items & 1;
        wait(sm.item_empty[s], ((n_items >> 1) & 1) ^ 1);
        // (of a wait that gave up the item before may still be in use)
        if (lane == 0 && !*dead) {
          sm.items[s] = it;
          mbar_arrive(smem_addr(&sm.item_full[s]));
        }
        ++n_items;
      };
      auto load = [&](const Gqa8Item& it) {
        for (int t = it.t_begin; t < it.t_end; t += 16) {
          int block, ex;
          gqa8_pages(a, it, t, lane, block, ex);
          const int nt = min(16, it.t_end - t);
          const bool there = ex != kMasked;
          const int ev = there ? ex >> 16 : kGqa8ExpMin;
          const float4 e4 = make_float4(there ? pow2f(static_cast<int16_t>(ex & 0xFFFF)) : 1.0f,
                                        static_cast<float>(ev), pow2f(-ev), there ? 1.0f : 0.0f);
          for (int i = 0; i < nt; ++i, ++n_tiles) {
            const int b0 = __shfl_sync(0xFFFFFFFFu, block, 2 * i), b1 = __shfl_sync(0xFFFFFFFFu, block, 2 * i + 1);
            const int ks = n_tiles % KS, vs = n_tiles % VS;
            wait(sm.k_empty[ks], ((n_tiles / KS) & 1) ^ 1);
            // (the softmax of the tile eight before is done: QK of the tile KS
            // before, which this stage waited for, came after it)
            if ((lane >> 1) == i) sm.exps[n_tiles & 7][lane & 1] = e4;
            __syncwarp();
            if (lane == 0 && !*dead) {
              n_loads = n_tiles + 1;
              mbar_arrive(smem_addr(&sm.ex_full[n_tiles & 7]));
              const uint32_t bar = smem_addr(&sm.k_full[ks]), dst = smem_addr(k_s + ks * C::kK);
              mbar_arrive_expect_tx(bar, C::kK);
              tma_load_block(dst, &map, 2 * b0, bar);
              tma_load_block(dst + 64 * D, &map, 2 * b1, bar);
            }
            __syncwarp();
            wait(sm.v8_empty[vs], ((n_tiles / VS) & 1) ^ 1);
            if (lane == 0 && !*dead) {
              const uint32_t bar = smem_addr(&sm.v8_full[vs]), dst = smem_addr(v8_s + vs * C::kK);
              mbar_arrive_expect_tx(bar, C::kK);
              tma_load_block(dst, &map, 2 * b0 + 1, bar);
              tma_load_block(dst + 64 * D, &map, 2 * b1 + 1, bar);
            }
            __syncwarp();
          }
        }
      };
      gqa8_walk(a, kind, static_cast<int64_t>(sm.total), tails, lane, [&](const Gqa8Item& it) {
        publish(it);
        load(it);
      });
      publish(Gqa8Item{-1, 0, 0, 0, 0, 0, 0, 0, 0, 0, -1});
      // every signal lands before the block's shared memory goes away
      for (uint32_t i = n_tiles > KS ? n_tiles - KS : 0; i < n_tiles; ++i)
        wait(sm.k_empty[i % KS], (i / KS) & 1);
      for (uint32_t i = n_tiles > 2 ? n_tiles - 2 : 0; i < n_tiles; ++i) wait(sm.v_empty[i & 1], (i >> 1) & 1);
      if (*dead && lane == 0) {
        for (uint32_t i = n_loads > KS ? n_loads - KS : 0; i < n_loads; ++i)
          mbar_wait_bounded(smem_addr(&sm.k_full[i % KS]), (i / KS) & 1, 1000000);
        for (uint32_t i = n_loads > VS ? n_loads - VS : 0; i < n_loads; ++i)
          mbar_wait_bounded(smem_addr(&sm.v8_full[i % VS]), (i / VS) & 1, 1000000);
      }
    } else if (warp == 1) {
      // ==== products (the whole warp; one lane issues) ====
      constexpr uint32_t kSw = D == 128 ? kSwizzle128 : kSwizzle64;
      constexpr uint32_t idesc_qk = idesc_e4m3(128, 128, false, false);
      constexpr uint32_t idesc_pv = idesc_f16(128, D, false, true);
      const uint64_t dk0 = smem_desc(smem_addr(k_s), 16, 8 * D, kSw), dq0 = smem_desc(smem_addr(q_s), 16, 8 * D, kSw);
      const uint64_t dv0 = smem_desc(smem_addr(v_s), kSlab, 1024, kSwizzle128);
      uint32_t n_tiles = 0, ks = 0, k_par = 0;            // stage of K and its parity
      uint32_t w0 = 0, w1 = 0, p0 = 0, p1 = 0;            // parities of the row tiles' q and P
      // The queue of products is a few instructions deep, so what keeps this
      // warp between two groups of them has to be short: waits come where a group
      // has just been queued, and a group ends with all its signals.
      auto qk = [&](int qt, uint32_t stage, int q) {                   // of the elected lane
        const uint64_t dk = dk0 + stage * (C::kK >> 4), dq = dq0 + q * (C::kQ >> 4);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int k = 0; k < D / 32; ++k)
            mma_f8kind(tmem + qt * 128, dq + ((t * 128 * D) >> 4) + 2 * k, dk + 2 * k, idesc_qk, t + k > 0);
        mma_commit(smem_addr(&sm.s_full[qt]));
      };
      // PV of tile j, then, with the last products, `more` (P of each page lies
      // over its own half of S; it comes in two parts, the first 32 keys of both
      // pages and the others, so that the first products overlap the rest of
      // the softmax)
      auto pv = [&](int qt, uint32_t j, bool first, uint32_t& par, auto&& more) {
        const uint64_t dv = dv0 + (j & 1) * (C::kV16 >> 4);
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          wait(sm.p_full[qt][part], par);
          __syncwarp();
          tc_fence_after_sync();
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int k = 2 * part + (i & 1) + 4 * (i >> 1);       // 16 keys
              mma_f16_ts(tmem + 256 + qt * 128, tmem + qt * 128 + 64 * (k >> 2) + 8 * (k & 3),
                         dv + ((k * 2048) >> 4), idesc_pv, !first || part + i > 0);
            }
            if (part == 1) more();
          }
          __syncwarp();
        }
        par ^= 1;
      };
      for (uint32_t n_items = 0;; ++n_items) {
        const int s = n_items & 1;
        wait(sm.item_full[s], (n_items >> 1) & 1);
        if (__any_sync(0xFFFFFFFFu, *dead != 0)) break;
        const int b = __shfl_sync(0xFFFFFFFFu, sm.items[s].b, 0);
        const int nt = __shfl_sync(0xFFFFFFFFu, sm.items[s].t_end - sm.items[s].t_begin, 0);
        const bool two = __shfl_sync(0xFFFFFFFFu, sm.items[s].nrows, 0) > 128;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sm.item_empty[s]));
        if (b < 0) break;
        if (nt == 0) continue;
        wait(sm.q_full[0], w0);
        w0 ^= 1;
        if (two) {
          wait(sm.q_full[1], w1);
          w1 ^= 1;
        }
        auto next_k = [&] {
          if (++ks == KS) {
            ks = 0;
            k_par ^= 1;
          }
        };
        // (P of a row tile lies over its S: the products run in order)
        wait(sm.k_full[ks], k_par);
        __syncwarp();
        tc_fence_after_sync();
        if (two) {
          if (elect_one()) {
            qk(0, ks, 0);
            qk(1, ks, 1);
            mma_commit(smem_addr(&sm.k_empty[ks]));
          }
          __syncwarp();
          for (int t = 0; t < nt; ++t) {
            const uint32_t j = n_tiles + t;
            const bool next = t + 1 < nt;
            wait(sm.v_full[j & 1], (j >> 1) & 1);
            next_k();
            if (next && (KS < 3 || t == 0)) wait(sm.k_full[ks], k_par);
            pv(0, j, t == 0, p0, [&] {
              if (next) qk(0, ks, 0);
              else mma_commit(smem_addr(&sm.o_full[0]));
            });
            const uint32_t ks_now = ks;
            if (KS >= 3 && t + 2 < nt) {                  // K of the tile after the next
              const bool wrap = ks + 1 == KS;
              wait(sm.k_full[wrap ? 0 : ks + 1], wrap ? k_par ^ 1 : k_par);
            }
            pv(1, j, t == 0, p1, [&] {
              if (next) {
                qk(1, ks_now, 1);
                mma_commit(smem_addr(&sm.k_empty[ks_now]));
              } else {
                mma_commit(smem_addr(&sm.o_full[1]));
              }
              mma_commit(smem_addr(&sm.v_empty[j & 1]));
            });
          }
        } else {
          // tile t is row tile t & 1's
          if (elect_one()) {
            qk(0, ks, 0);
            mma_commit(smem_addr(&sm.k_empty[ks]));
          }
          __syncwarp();
          next_k();
          if (nt > 1) {
            wait(sm.k_full[ks], k_par);
            __syncwarp();
            tc_fence_after_sync();
            if (elect_one()) {
              qk(1, ks, 0);
              mma_commit(smem_addr(&sm.k_empty[ks]));
            }
            __syncwarp();
            next_k();
          }
          for (int t = 0; t < nt; ++t) {
            const uint32_t j = n_tiles + t;
            const bool next = t + 2 < nt;
            wait(sm.v_full[j & 1], (j >> 1) & 1);
            if (next) wait(sm.k_full[ks], k_par);
            auto more = [&](int qt) {
              if (next) {
                qk(qt, ks, 0);
                mma_commit(smem_addr(&sm.k_empty[ks]));
              } else {
                mma_commit(smem_addr(&sm.o_full[qt]));
              }
              mma_commit(smem_addr(&sm.v_empty[j & 1]));
            };
            if (t & 1) pv(1, j, t == 1, p1, [&] { more(1); });
            else pv(0, j, t == 0, p0, [&] { more(0); });
            if (next) next_k();
          }
        }
        n_tiles += nt;
        if (a.fault_site == 1) wait(sm.never, 0);
      }
      if (a.fault_site == 1) wait(sm.never, 0);
      // in a block that gave up nothing else waits for the products that are
      // still queued: they end before its memory goes away
      __syncwarp();
      if (__any_sync(0xFFFFFFFFu, *dead != 0)) {
        if (elect_one()) mma_commit(smem_addr(&sm.never));
        __syncwarp();
        mbar_wait_bounded(smem_addr(&sm.never), 0, 1000000);
      }
    } else {
      // ==== V to f16 ====
      uint32_t j = 0;
      for (uint32_t n_items = 0;; ++n_items) {
        const int s = n_items & 1;
        wait(sm.item_full[s], (n_items >> 1) & 1);
        if (__any_sync(0xFFFFFFFFu, *dead != 0)) break;
        const Gqa8Item item = sm.items[s];
        const int b = item.b, t0 = item.t_begin, t1 = item.t_end;
        const int klo = item.klo, khi = item.khi;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sm.item_empty[s]));
        if (b < 0) break;
        // the item's rows of q into L2, while the one before is worked on
        {
          const int cu0 = item.cu0, h = item.h, r0 = item.r0, nrows = item.nrows;
          for (int rr = tid - 64; rr < nrows; rr += 64) {
            const uint16_t* row = static_cast<const uint16_t*>(a.q) +
                                  static_cast<int64_t>(cu0 + (r0 + rr) / G) * a.q_token_stride +
                                  static_cast<int64_t>(h * G + (r0 + rr) % G) * a.q_head_stride;
            prefetch_l2_line(row);
            if (D == 128) prefetch_l2_line(row + 64);
          }
        }
        for (int t = t0; t < t1; ++t, ++j) {
          wait(sm.v8_full[j % VS], (j / VS) & 1);
          wait(sm.v_empty[j & 1], ((j >> 1) & 1) ^ 1);
          const uint8_t* const src = v8_s + (j % VS) * C::kK;
          uint8_t* const dst = v_s + (j & 1) * C::kV16;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int row = (warp - 2) * 64 + half * 32 + lane;
            const int at = t * kTileKeys + row;
            // a key that no row sees may hold NaN codes, which a weight of
            // zero would not silence
            const bool live = at >= klo && at < khi;
            const int sw8 = D == 128 ? row & 7 : (row >> 1) & 3;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              uint4 w = make_uint4(0, 0, 0, 0);
              if (live) w = *reinterpret_cast<const uint4*>(src + row * D + ((c ^ sw8) * 16));
              uint8_t* const o = dst + (c / 4) * kSlab + row * 128;
              const int i0 = (c % 4) * 2;
              *reinterpret_cast<uint4*>(o + ((i0 ^ (row & 7)) * 16)) =
                  make_uint4(e4m3x2_to_f16x2(w.x & 0xFFFFu), e4m3x2_to_f16x2(w.x >> 16),
                             e4m3x2_to_f16x2(w.y & 0xFFFFu), e4m3x2_to_f16x2(w.y >> 16));
              *reinterpret_cast<uint4*>(o + (((i0 + 1) ^ (row & 7)) * 16)) =
                  make_uint4(e4m3x2_to_f16x2(w.z & 0xFFFFu), e4m3x2_to_f16x2(w.z >> 16),
                             e4m3x2_to_f16x2(w.w & 0xFFFFu), e4m3x2_to_f16x2(w.w >> 16));
            }
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_addr(&sm.v8_empty[j % VS]));
            mbar_arrive(smem_addr(&sm.v_full[j & 1]));
          }
        }
      }
    }
  } else {
    // ==== softmax: a thread is half a row, 64 keys of a tile ====
    setmaxnreg_inc<kSoftmaxRegs>();
    const int qt = (warp - 4) >> 3, half = ((warp - 4) >> 2) & 1;
    const int bar = 1 + qt * 4 + (warp & 3);              // the two warps of 32 rows
    const int bar_rows = 9 + (warp & 3);                  // and those of the other row tile
    const int wrow = (warp & 3) * 32, row = wrow + lane;  // of the row tile
    const uint32_t lanes = static_cast<uint32_t>(wrow) << 16;
    const uint32_t s_tm = tmem + qt * 128 + half * 64 + lanes;
    const uint32_t o_tm = tmem + 256 + qt * 128 + half * (D / 2) + lanes;
    uint8_t* const q_mine = q_s + qt * C::kQ;
    uint32_t j = 0, n_mine = 0, n_work = 0;               // tiles of all items, of mine; items of mine
    for (uint32_t n_items = 0;; ++n_items) {
      const int s = n_items & 1;
      wait(sm.item_full[s], (n_items >> 1) & 1);
      if (named_sync_or(bar_rows, 128, *dead != 0)) break;     // (together, for they meet at barriers)
      // (read again at its end, so that the loop over the tiles does not hold it)
      const Gqa8Item it = sm.items[s];
      if (it.b < 0) break;
      const int nt = it.t_end - it.t_begin;
      const bool shared = it.nrows <= 128;                // both row tiles are the same rows
      const int base = shared ? 0 : qt * 128;
      const bool mine = base + row < it.nrows;
      // keys at < hi and >= lo are this row's (a row that is not there takes all,
      // so that its warp needs no mask for it; its numbers go nowhere)
      int hi = 0x7FFFFFFF, lo = 0;
      if (mine) {
        const int64_t pos = static_cast<int64_t>(it.pos0) + (it.r0 + base + row) / G;
        hi = static_cast<int>(max(min(pos + 1, static_cast<int64_t>(it.khi)), static_cast<int64_t>(0)));
        if (a.window > 0) lo = static_cast<int>(max(pos - a.window + 1, static_cast<int64_t>(0)));
      }
      if (nt > 0 && !(shared && qt == 1)) {
        // 16 of the warp's rows of q (the other half's warp has the others) as
        // NT E4M3 terms, kTpr threads a row
        constexpr int kTpr = D / 16, kRpp = 32 / kTpr;
        const int part = lane % kTpr;
        const float sign = a.sm_scale < 0.0f ? -1.0f : 1.0f;   // (so that the factor is positive)
        auto fetch = [&](int p, uint4 (&w)[2]) {
          const int rr = wrow + half * 16 + p * kRpp + lane / kTpr, gr = it.r0 + base + rr;
          w[0] = w[1] = make_uint4(0, 0, 0, 0);
          if (p * kRpp < 16 && base + rr < it.nrows) {
            const uint4* g = reinterpret_cast<const uint4*>(
                static_cast<const uint16_t*>(a.q) + static_cast<int64_t>(it.cu0 + gr / G) * a.q_token_stride +
                static_cast<int64_t>(it.h * G + gr % G) * a.q_head_stride + part * 16);
            w[0] = load(g);
            w[1] = load(g + 1);
          }
        };
        // (a loop of little code, two fetches ahead: it runs once an item, so
        // its instructions are as far away as its data)
        uint4 w[2], w_next[2];
        fetch(0, w);
        fetch(1, w_next);
#pragma unroll 1
        for (int p = 0; p < 16 / kRpp; ++p) {
          const int rr = wrow + half * 16 + p * kRpp + lane / kTpr;
          float y[16];
          uint32_t m = widen16<C::kF16>(w, y);
          w[0] = w_next[0];
          w[1] = w_next[1];
          fetch(p + 2, w_next);
#pragma unroll
          for (int off = 1; off < kTpr; off <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
          const int e = q_exponent(m);
          const bool odd = m >= 0x7F800000u;              // a NaN or an infinity: NaN in its row
          if (part == 0)
            sm.qf[qt][rr] = odd ? __uint_as_float(0x7FC00000u) : fabsf(a.sm_scale) * 1.4426950408889634f * pow2f(e);
          uint32_t o[NT][4];
          terms16<NT, true>(y, sign * pow2f(-e), odd, o);
#pragma unroll
          for (int t = 0; t < NT; ++t)
            *reinterpret_cast<uint4*>(q_mine + t * 128 * D + swizzle<D == 128 ? 3 : 2>(rr * D + part * 16)) =
                make_uint4(o[t][0], o[t][1], o[t][2], o[t][3]);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sm.q_full[qt]));
      }
      // qf is there for the warps that read it
      if (shared) named_sync(bar_rows, 128);
      else named_sync(bar, 64);
      float qf = nt > 0 ? sm.qf[shared ? 0 : qt][row] : 0.0f;
      const bool odd = qf != qf;
      if (odd) qf = 0.0f;
      float mref = kLowest, l = 0.0f;
      // pages that begin before `full` and not before `open` are every row's whole
      int full = hi - 63, open = lo;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        full = min(full, __shfl_xor_sync(0xFFFFFFFFu, full, off));
        open = max(open, __shfl_xor_sync(0xFFFFFFFFu, open, off));
      }
      const int first = it.t_begin + (shared ? qt : 0), step = shared ? 2 : 1;
      for (int t = first; t < it.t_end; t += step, ++n_mine) {
        const uint32_t jt = j + (t - it.t_begin);
        const int at = t * kTileKeys + half * 64;
        wait(sm.ex_full[jt & 7], (jt >> 3) & 1);
        const float4 ex = sm.exps[jt & 7][half];
        wait(sm.s_full[qt], n_mine & 1);
        tc_fence_after_sync();
        float x[64];
        tmem_ld32(s_tm, reinterpret_cast<uint32_t(&)[32]>(x[0]));
        tmem_ld32(s_tm + 32, reinterpret_cast<uint32_t(&)[32]>(x[32]));
        float m[4];
        tmem_wait_ld32(reinterpret_cast<uint32_t(&)[32]>(x[0]));
        tmem_wait_ld32(reinterpret_cast<uint32_t(&)[32]>(x[32]));
        if (at >= full || at < open || ex.w == 0.0f) {
          // keys of this row in the page: [a0, a0 + n)
          const int a0 = max(lo - at, 0), n = ex.w == 0.0f ? 0 : max(min(hi - at, 64) - a0, 0);
#pragma unroll
          for (int c = 0; c < 64; ++c)
            x[c] = static_cast<unsigned>(c - a0) < static_cast<unsigned>(n) ? x[c] : -INFINITY;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) m[k] = fmaxf(x[k], x[4 + k]);
#pragma unroll
        for (int c = 8; c < 64; c += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k) m[k] = max3(m[k], x[c + k], x[c + 4 + k]);
        // (at least 2^-126, so that a masked -inf stays one where the scale is 0)
        const float f = fmaxf(qf * ex.x, 0x1p-126f);
        float top = fmaf(max3(m[0], m[1], fmaxf(m[2], m[3])), f, ex.y);
        sm.top[qt][n_mine & 1][half][row] = top;
        named_sync(bar, 64);
        top = fmaxf(top, sm.top[qt][n_mine & 1][half ^ 1][row]);
        if (__any_sync(0xFFFFFFFFu, top > mref + 6.0f)) {
          const float to = fmaxf(top, mref), by = fast_exp2(mref - to);
          mref = to;
          l *= by;
          if (t > first) {
            // s_full came behind the last product into this O; each half takes
            // its columns
#pragma unroll 1
            for (int c = 0; c < D / 2; c += 16) {
              uint32_t v[16];
              tmem_ld16_sync(o_tm + c, v);
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * by);
              tmem_st16(o_tm + c, v);
            }
          }
        }
        const float b = ex.y - mref + 8.0f;
        const float2 f2 = make_float2(f, f), b2 = make_float2(b, b);
        float2 acc[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t p[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            float2 y = fma2(make_float2(x[q * 32 + 2 * c], x[q * 32 + 2 * c + 1]), f2, b2);
            y.x = fast_exp2(y.x);
            y.y = fast_exp2(y.y);
            acc[c & 1] = add2(acc[c & 1], y);
            p[c] = h2_bits(__floats2half2_rn(y.x, y.y));
          }
          tmem_st16(s_tm + 16 * q, p);
          tmem_st_wait();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sm.p_full[qt][q]));
        }
        acc[0] = add2(acc[0], acc[1]);
        l = fmaf(acc[0].x + acc[0].y, ex.z, l);
      }
      j += nt;
      sm.last[qt][half][row] = l;
      if (half == 0) sm.last[qt][2][row] = mref;
      if (first < it.t_end) {
        wait(sm.o_full[qt], n_work & 1);
        ++n_work;
        tc_fence_after_sync();
      }
      if (shared) named_sync(bar_rows, 128);
      else named_sync(bar, 64);
      const Gqa8Item fin = sm.items[s];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sm.item_empty[s]));
      // out = (O_a w_a + O_b w_b) / (l_a w_a + l_b w_b), b the other row tile of
      // the same rows; both halves read the same numbers
      const int ta = shared ? 0 : qt;
      float wa = 1.0f, wb = 0.0f, lb = 0.0f;
      mref = sm.last[ta][2][row];
      l = sm.last[ta][0][row] + sm.last[ta][1][row];
      if (shared) {
        lb = sm.last[1][0][row] + sm.last[1][1][row];
        const float mb = sm.last[1][2][row], to = fmaxf(mref, mb);
        wa = fast_exp2(mref - to);
        wb = fast_exp2(mb - to);
        mref = to;
      }
      const bool has_a = nt > 0 && l != 0.0f, has_b = lb != 0.0f;      // (else O may be anything)
      l = l * wa + lb * wb;
      const float inv = odd && l > 0.0f ? __uint_as_float(0x7FC00000u) : 1.0f / l;
      const bool some = l > 0.0f || l != l;
      wa *= inv;
      wb *= inv;
      const int r = fin.r0 + base + row;
      const int64_t part = static_cast<int64_t>(fin.slot) * C::kRows + base + row;
      const int64_t orow = static_cast<int64_t>(fin.cu0 + r / G) * a.Hq + fin.h * G + r % G;
      // Out through the rows of q's first two terms, which no product reads any
      // more, so that the stores to memory are up to D contiguous bytes: this
      // warp's columns of 16 bits, or half of them in fp32.
      const int cols = shared ? D / 4 : D / 2, col0 = (shared ? 2 * qt + half : half) * cols;
      const uint32_t oa_tm = tmem + 256 + ta * 128 + lanes + col0, ob_tm = tmem + 256 + 128 + lanes + col0;
      auto stage = [&](int rr, int c) {
        return reinterpret_cast<uint4*>(q_mine + half * (128 * D) + swizzle<D == 128 ? 3 : 2>((wrow + rr) * D + c * 16));
      };
      // 16-byte chunks of a row: D / 16, half as many where the columns are
      // shared and of 16 bits
      const bool cut = fin.slot >= 0;
      const int lg = (D == 128 ? 3 : 2) - (shared && !cut ? 1 : 0);
      uint8_t* const to = cut ? reinterpret_cast<uint8_t*>(ws_o) : static_cast<uint8_t*>(a.out);
      const int64_t row_at = cut ? part * (4 * D) : orow * (2 * D);
#pragma unroll 1
      for (int c0 = 0; c0 < cols; c0 += 16) {             // of this warp's columns
        uint32_t v[16];
        float y[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) y[c] = 0.0f;
        if (nt > 0) {
          tmem_ld16_sync(oa_tm + c0, v);
          if (has_a)
#pragma unroll
            for (int c = 0; c < 16; ++c) y[c] = __uint_as_float(v[c]) * wa;
        }
        if (shared && nt > 1) {
          tmem_ld16_sync(ob_tm + c0, v);
          if (has_b)
#pragma unroll
            for (int c = 0; c < 16; ++c) y[c] = fmaf(__uint_as_float(v[c]), wb, y[c]);
        }
        if (cut) {
          const int at = c0 % (D / 4) / 4;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            *stage(lane, at + c) = make_uint4(__float_as_uint(y[4 * c]), __float_as_uint(y[4 * c + 1]),
                                              __float_as_uint(y[4 * c + 2]), __float_as_uint(y[4 * c + 3]));
        } else {
#pragma unroll
          for (int c = 0; c < 2; ++c)
            *stage(lane, c0 / 8 + c) =
                make_uint4(pack16<C::kF16>(y[8 * c], y[8 * c + 1]), pack16<C::kF16>(y[8 * c + 2], y[8 * c + 3]),
                           pack16<C::kF16>(y[8 * c + 4], y[8 * c + 5]), pack16<C::kF16>(y[8 * c + 6], y[8 * c + 7]));
        }
        if (cut ? (c0 + 16) % (D / 4) == 0 : c0 + 16 == cols) {
          const int64_t at = row_at + (cut ? (col0 + c0 + 16 - D / 4) * 4 : col0 * 2);
          __syncwarp();
#pragma unroll 2
          for (int i = lane; i < 32 << lg; i += 32) {
            const int rr = i >> lg, c = i & ((1 << lg) - 1);
            const int64_t dst = __shfl_sync(0xFFFFFFFFu, at, rr);
            const uint4 v4 = *stage(rr, c);
            if (base + wrow + rr < fin.nrows) *reinterpret_cast<uint4*>(to + dst + c * 16) = v4;
          }
          __syncwarp();
        }
      }
      if (mine && half == 0 && base == qt * 128) {
        const float ls = !some ? -INFINITY : odd ? __uint_as_float(0x7FC00000u) : mref - 8.0f + log2f(l);
        if (fin.slot >= 0) ws_lse[part] = ls;
        else a.lse[orow] = ls * 0.6931471805599453f;
      }
      tc_fence_before_sync();
      // (both tiles of O, and `last`, are read before a warp goes on)
      if (shared) named_sync(bar_rows, 128);
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// The pieces of items that were cut: block (c, y) joins rows of the item that
// began in block c of the attention kernel, by log-sum-exp over its pieces in
// their order: one kernel for items of few rows, where a long context has many
// pieces and 8 warps share a row, one for items of up to 256 rows, where a warp
// takes 4 rows at once and their pieces in turn.  Those of a prompt or a chunk are
// two or three; but a single short one of few heads over a long context is cut
// over all blocks (40 rows of one head over 200000 tokens: 97 us, where one row,
// in the kernels of few rows, takes 28).
// ---------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(256) merge_few_kernel(const Gqa8AttnArgs a, const int rows,
                                                    const Gqa8Tail* tails, const float* ws_lse,
                                                    const float* ws_o) {
  grid_dependency_wait();
  grid_launch_dependents();
  constexpr int C = D / 32;                               // columns a lane
  using Vec = std::conditional_t<C == 4, float4, float2>;
  __shared__ Vec part[8][32];
  const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Gqa8Tail t = tails[c];
  constexpr int W = 8;
  const int r = blockIdx.y, wi = warp;
  if (t.parts == 0 || r >= t.nrows) return;               // (whole blocks)
  float o[C], m = -INFINITY, s = 0.0f;
#pragma unroll
  for (int k = 0; k < C; ++k) o[k] = 0.0f;
  bool odd = false;
  {
    // piece i is slot 2c + 1 for i = 0, else 2 (c + i)
    auto row_of = [&](int i) { return static_cast<int64_t>(i == 0 ? 2 * c + 1 : 2 * (c + i)) * rows + r; };
    for (int i = lane; i < t.parts; i += 32) {
      const float x = load(ws_lse + row_of(i));
      odd |= x != x;
      m = fmaxf(m, x);
    }
    m = warp_max(m);
    odd = __any_sync(0xFFFFFFFFu, odd);
    if (m > -INFINITY) {
      for (int i0 = 0; i0 < t.parts; i0 += 32) {
        const float w = i0 + lane < t.parts ? fast_exp2(load(ws_lse + row_of(i0 + lane)) - m) : 0.0f;
        s += w;
        const int n = min(32, t.parts - i0);
#pragma unroll 4
        for (int i = wi; i < n; i += W) {
          const float wt = __shfl_sync(0xFFFFFFFFu, w, i);
          const Vec v = load(reinterpret_cast<const Vec*>(ws_o + row_of(i0 + i) * D) + lane);
          const float* f = reinterpret_cast<const float*>(&v);
#pragma unroll
          for (int k = 0; k < C; ++k) o[k] = fmaf(wt, f[k], o[k]);
        }
      }
      s = warp_sum(s);
    }
    if (odd) s = __uint_as_float(0x7FC00000u);
  }
  part[warp][lane] = *reinterpret_cast<const Vec*>(o);
  __syncthreads();
  if (wi != 0) return;
#pragma unroll
  for (int i = 1; i < W; ++i) {
    const Vec v = part[i][lane];
#pragma unroll
    for (int k = 0; k < C; ++k) o[k] += reinterpret_cast<const float*>(&v)[k];
  }
  const int G = a.Hq / a.Hkv, rr = t.r0 + r;
  const int64_t row = static_cast<int64_t>(t.cu0 + rr / G) * a.Hq + t.h * G + rr % G;
  const float inv = s == 0.0f ? 0.0f : 1.0f / s;
  uint32_t u[C / 2];
#pragma unroll
  for (int k = 0; k < C / 2; ++k) {
    const float y0 = o[2 * k] * inv, y1 = o[2 * k + 1] * inv;
    if (a.f16) {
      u[k] = h2_bits(__floats2half2_rn(y0, y1));
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(y0, y1);
      u[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
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

// ---------------------------------------------------------------------------
// Launch
// ---------------------------------------------------------------------------
typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled() {
  static const EncodeTiled f = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) !=
            cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return f;
}

// The pool as [num_pages * Hkv * 2] blocks of 64 rows of D bytes.
bool pool_map(const Gqa8AttnArgs& a, CUtensorMap* map) {
  const EncodeTiled f = encode_tiled();
  if (f == nullptr) return false;
  const cuuint64_t n = static_cast<cuuint64_t>(a.num_pages) * a.Hkv * 2;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(a.D), 64, n > 0 ? n : 1};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(a.D), 64ull * a.D};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(a.D), 64, 1}, step[3] = {1, 1, 1};
  return f(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(a.pool), dims, strides, box, step,
           CU_TENSOR_MAP_INTERLEAVE_NONE, a.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of few_kernel's items, and of the largest request that it takes: the
// smallest of 8, 16 and 24 that holds every request or, where some have more, a
// single token of any (the others go to many_kernel); 0: none.
int few_rows(int max_new, int G) {
  const int64_t all = static_cast<int64_t>(max_new) * G, need = all <= 24 ? all : G;
  return need <= 8 ? 8 : need <= 16 ? 16 : need <= 24 ? 24 : 0;
}
// Workspace of one attention kernel: a tail for each of its blocks, then two
// slots of partial rows for each block.
size_t part_bytes(int blocks, int rows, int D) {
  return static_cast<size_t>(blocks) * (sizeof(Gqa8Tail) + 2ull * rows * (D + 1) * sizeof(float));
}
struct Parts {
  Gqa8Tail* tails;
  float *lse, *o;
};
Parts parts_at(void* ws, int blocks, int rows, int D) {
  Parts p;
  p.tails = static_cast<Gqa8Tail*>(ws);
  p.o = reinterpret_cast<float*>(p.tails + blocks);
  p.lse = p.o + 2ull * blocks * rows * D;
  return p;
}
constexpr int kFewCtas = 2, kManyRows = 256;      // blocks an SM at most

template <typename K>
cudaError_t launch_merge(K kernel, const Gqa8AttnArgs& a, int blocks, int y, int rows, const Parts& p,
                         cudaStream_t stream) {
  if ((a.pt_stride + 1) / 2 <= kWhole) return cudaSuccess;                 // nothing is ever cut
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, y);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, rows, static_cast<const Gqa8Tail*>(p.tails),
                            static_cast<const float*>(p.lse), static_cast<const float*>(p.o));
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

template <int D, int RP, int NT>
cudaError_t launch_few(const Gqa8AttnArgs& a, const CUtensorMap& map, int max_rows, void* ws,
                       cudaStream_t stream) {
  using C = FewCfg<D, RP, NT>;
  cudaError_t e = prepare_kernel<few_kernel<D, RP, NT>>(C::kSmem, 0);
  if (e != cudaSuccess) return e;
  // (no more blocks than there can be tiles, or items where none is ever cut)
  const int64_t tiles = (a.pt_stride + 1) / 2, most = a.B * static_cast<int64_t>(a.Hkv) * (tiles <= kWhole ? 1 : tiles);
  const int blocks = static_cast<int>(std::min<int64_t>(a.num_sms * C::kCtas, most));
  const Parts p = parts_at(ws, blocks, RP, D);
  e = launch_pdl(few_kernel<D, RP, NT>, blocks, C::kThreads, C::kSmem, stream, 1, map, a, max_rows, p.tails, p.lse, p.o);
  return e != cudaSuccess ? e : launch_merge(merge_few_kernel<D>, a, blocks, RP, RP, p, stream);
}

template <int D, int NT>
cudaError_t launch_many(const Gqa8AttnArgs& a, const CUtensorMap& map, int min_rows, void* ws,
                        cudaStream_t stream) {
  using C = ManyCfg<D, NT>;
  cudaError_t e = prepare_kernel<many_kernel<D, NT>>(C::kSmem, kLaunchRegs);
  if (e != cudaSuccess) return e;
  const Parts p = parts_at(ws, a.num_sms, kManyRows, D);
  e = launch_pdl(many_kernel<D, NT>, a.num_sms, kManyThreads, C::kSmem, stream, 1, map, a, min_rows, p.tails,
                 p.lse, p.o);
  return e != cudaSuccess ? e : launch_merge(merge_many_kernel<D>, a, a.num_sms, kManyRows / 32, kManyRows, p, stream);
}

size_t few_bytes(int rows, int D, int sms) {
  return rows == 0 ? 0 : (part_bytes(kFewCtas * sms, rows, D) + 255) / 256 * 256;
}

template <int D>
cudaError_t launch_d(const Gqa8AttnArgs& a, cudaStream_t stream) {
  CUtensorMap map;
  if (!pool_map(a, &map)) return cudaErrorInvalidValue;
  const int G = a.Hq / a.Hkv;
  const int rows = few_rows(a.max_new, G);
  auto launch = [&](auto rp) {
    constexpr int RP = decltype(rp)::value;
    return a.f16 ? launch_few<D, RP, 3>(a, map, rows, a.ws, stream)
                 : launch_few<D, RP, 2>(a, map, rows, a.ws, stream);
  };
  cudaError_t e = cudaSuccess;
  if (rows == 8) e = launch(std::integral_constant<int, 8>{});
  else if (rows == 16) e = launch(std::integral_constant<int, 16>{});
  else if (rows == 24) e = launch(std::integral_constant<int, 24>{});
  if (e != cudaSuccess || static_cast<int64_t>(a.max_new) * G <= rows) return e;
  void* const ws = static_cast<uint8_t*>(a.ws) + few_bytes(rows, D, a.num_sms);
  return a.f16 ? launch_many<D, 3>(a, map, rows + 1, ws, stream)
               : launch_many<D, 2>(a, map, rows + 1, ws, stream);
}

}  // namespace

cudaError_t launch_attention_gqa8(const Gqa8AttnArgs& a, cudaStream_t stream) {
  return a.D == 64 ? launch_d<64>(a, stream) : launch_d<128>(a, stream);
}

size_t attention_gqa8_workspace(int max_new, int Hq, int Hkv, int D, int num_sms) {
  const int rows = few_rows(max_new, Hq / Hkv);
  const bool many = static_cast<int64_t>(max_new) * (Hq / Hkv) > rows;
  return few_bytes(rows, D, num_sms) + (many ? part_bytes(num_sms, kManyRows, D) : 0);
}

}  // namespace kv4
