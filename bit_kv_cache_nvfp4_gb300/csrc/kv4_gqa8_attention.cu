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

namespace kv4 {
namespace {

constexpr int kWhole = 4;      // items of at most so many tiles are never cut

// ---------------------------------------------------------------------------
// Few rows: single tokens and short drafts
// ---------------------------------------------------------------------------
// What bounds this case is reading the codes once (2 G flops per byte), so the
// codes go from HBM to the tensor core as they are, with no conversion on the
// way: K and V tiles land in shared memory by TMA in the swizzle that
// tcgen05.mma reads, and it is the small operands -- q and the softmax weights
// p -- that are brought to E4M3, as exact sums of NT terms (split_e4m3), the
// terms side by side as columns of one product:
//   S^T[128 keys x NT RP] = K . [q_0 | q_1 | ..]^T      (M = 128, N = NT RP)
//   O^T[D x NT RP] = V^T . [p_0 | p_1 | ..]^T            (M = D, K = 128 keys)
// s = S_0 + S_1 / 16 + ..., likewise o.  Both accumulate in fp32.  Two terms
// hold a bf16 q exactly and p to 2^-8 (half a bf16 step); f16 calls take three
// (q exactly, p to 2^-12).  Block exponents are powers of two: K's is a factor
// of the score, V's is folded into p (relative to the larger of the tile's two
// pages), both exact.  p is relative to the maximum of its own tile, so that
// the codes' 2^-9 granularity (2^-22 of the tile's largest weight with two
// terms) never meets a maximum from far away; each tile's O is a product of
// its own, joined to the running output in registers.
//
// Block: 8 warps.  Warp 0 finds the block's share of the work list and issues
// the loads, warp 1 the products, warps 2-3 bring q of the next item to E4M3,
// warps 4-7 are the softmax: a thread holds one key of S^T (and one d of O^T).
template <int D_, int RP_, int NT_>
struct FewCfg {
  static constexpr int D = D_, RP = RP_, NT = NT_;
  static constexpr int N = (NT * RP + 15) / 16 * 16;      // MMA columns (N % 16 == 0 at M = 128)
  static constexpr int kTile = 2 * kTileKeys * D;         // K and V of a tile
  static constexpr int kQ = (N * D + 1023) / 1024 * 1024; // one of two
  static constexpr int kP = N / 16 * 2048;                // one of two
  static constexpr int kSmall = 4096;                     // barriers, items, factors
  static constexpr int kFixed = 2 * kQ + 2 * kP + kSmall;
  // two blocks of an SM where three stages (96 KB) and the rest fit into half
  // of its 228 KB each, else one block with more stages
  static constexpr int kHalf = 113 * 1024 - 1024;
  static constexpr int kCtas = kFixed + 98304 <= kHalf && RP <= 16 ? 2 : 1;
  static constexpr int kStages = (kCtas == 2 ? 98304 : 163840) / kTile;
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
  alignas(16) float red[2][32 * 4];    // read as float4
  alignas(16) float2 stash[2][32];
  float lsum[4][32];
};
static_assert(sizeof(FewSmall) <= 4096 && offsetof(FewSmall, red) % 16 == 0 &&
                  offsetof(FewSmall, stash) % 8 == 0,
              "FewSmall");
constexpr int kMasked = 0x7FFF7FFF;
constexpr float kLowest = -3e38f;

template <int D, int RP, int NT>
__global__ void __launch_bounds__(256, FewCfg<D, RP, NT>::kCtas)
few_kernel(const __grid_constant__ CUtensorMap map, const Gqa8AttnArgs a, const int max_rows,
           Gqa8Tail* tails, float* ws_lse, float* ws_o) {
  using C = FewCfg<D, RP, NT>;
  constexpr int N = C::N, ST = C::kStages;
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
      mbar_init(smem_addr(&sm.item_empty[i]), 7);      // the product's lane, 2 + 4 warps
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&sm.q_full[i]), 2);
      mbar_init(smem_addr(&sm.q_empty[i]), 5);         // the last QK, 4 warps
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
    for (int i = tid; i < (2 * C::kQ + 2 * C::kP) / 16; i += 256)
      reinterpret_cast<uint4*>(q_s)[i] = make_uint4(0, 0, 0, 0);
  grid_dependency_wait();
  grid_launch_dependents();
  __syncthreads();
  {
    int64_t u = 0;
    for (int b = tid; b < a.B; b += 256)
      u += gqa8_units(a, gqa8_request(a, b, 1, max_rows, blockIdx.x == 0), G, RP);
    if (u > 0) atomicAdd(&sm.total, static_cast<unsigned long long>(u));
  }
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
    const int64_t total = static_cast<int64_t>(sm.total);
    const int blocks = gridDim.x, me = blockIdx.x;
    const int64_t per = max((total + blocks - 1) / blocks, static_cast<int64_t>(kWhole));
    const int64_t u0 = me * per, u1 = min(u0 + per, total);
    uint32_t n_items = 0, n_tiles = 0;
    bool tail = false;
    auto publish = [&](const Gqa8Item& it) {
      const int s = n_items & 3;
      wait(sm.item_empty[s], ((n_items >> 2) & 1) ^ 1);
      if (lane == 0) {
        sm.items[s] = it;
        mbar_arrive(smem_addr(&sm.item_full[s]));
      }
      ++n_items;
    };
    auto load = [&](const Gqa8Item& it) {
      for (int t = it.t_begin; t < it.t_end; t += 16) {
        // lane l: page l of the next 16 tiles
        const int64_t page = 2 * static_cast<int64_t>(t) + lane;
        int block = -1, ex = kMasked;
        if ((page >> 1) < it.t_end && (page << 6) < it.khi && (page << 6) + 64 > it.klo) {
          const int phys = __ldg(a.page_table + it.b * a.pt_stride + page);
          if (phys < 0 || phys >= a.num_pages) {
            flag_error(a.dev_err, kDevBadPage);
          } else {
            block = phys * a.Hkv + it.h;
            const uint32_t e2 = __ldg(reinterpret_cast<const uint16_t*>(a.scales) + block);
            const int ek = min(max(static_cast<int>(e2 & 0xFF) - 127, -100), 100);
            const int ev = min(max(static_cast<int>(e2 >> 8) - 127, -100), 100);
            ex = (ek & 0xFFFF) | (ev << 16);
          }
        }
        if (block < 0) block = a.num_pages * a.Hkv;           // past the tensor: zeros
        const int nt = min(16, it.t_end - t);
        for (int i = 0; i < nt; ++i, ++n_tiles) {
          const int b0 = __shfl_sync(0xFFFFFFFFu, block, 2 * i), b1 = __shfl_sync(0xFFFFFFFFu, block, 2 * i + 1);
          const int e0 = __shfl_sync(0xFFFFFFFFu, ex, 2 * i), e1 = __shfl_sync(0xFFFFFFFFu, ex, 2 * i + 1);
          const int s = n_tiles % ST;
          wait(sm.empty[s], ((n_tiles / ST) & 1) ^ 1);
          if (lane == 0 && !*dead) {
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
    int64_t acc = 0;
    for (int base = 0; base < a.B && acc < u1 && u0 < u1; base += 32) {
      const Gqa8Request q = gqa8_request(a, base + lane, 1, max_rows, false);
      const int64_t units = gqa8_units(a, q, G, RP);
      int64_t end = units;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, end, off);
        if (lane >= off) end += v;
      }
      end += acc;
      const int64_t chunk_end = __shfl_sync(0xFFFFFFFFu, end, 31);
      uint32_t todo = __ballot_sync(0xFFFFFFFFu, units > 0 && end > u0 && end - units < u1);
      for (; todo != 0; todo &= todo - 1) {
        const int l = __ffs(todo) - 1;
        Gqa8Request r;
        r.cu0 = __shfl_sync(0xFFFFFFFFu, q.cu0, l);
        r.n = __shfl_sync(0xFFFFFFFFu, q.n, l);
        r.pos0 = __shfl_sync(0xFFFFFFFFu, q.pos0, l);
        r.held = __shfl_sync(0xFFFFFFFFu, q.held, l);
        int64_t at = __shfl_sync(0xFFFFFFFFu, end - units, l);
        const int R = r.n * G;
        for (int r0 = 0; r0 < R && at < u1; r0 += RP) {
          const Gqa8Span sp = gqa8_span(a, r, G, r0, min(R, r0 + RP));
          const int64_t w = max(sp.nt, 1);
          if (at + w * a.Hkv <= u0) {
            at += w * a.Hkv;
            continue;
          }
          const int h0 = at < u0 ? static_cast<int>((u0 - at) / w) : 0;
          int64_t begin = at + h0 * w;
          for (int h = h0; h < a.Hkv && begin < u1; ++h, begin += w) {
            int64_t tb = 0, te = sp.nt;
            int slot = -1;
            if (w <= kWhole) {
              if (begin < u0) continue;                       // the block before has it whole
            } else {
              tb = max(u0 - begin, static_cast<int64_t>(0));
              te = min(u1 - begin, w);
              if (tb > 0) {
                slot = 2 * me;
              } else if (te < w) {
                slot = 2 * me + 1;
                tail = true;
                if (lane == 0)
                  tails[me] = Gqa8Tail{static_cast<int>((begin + w - 1) / per) - me + 1, r.cu0, h, r0, min(RP, R - r0), {}};
              }
            }
            const Gqa8Item it{base + l, h, r.cu0, r.pos0, r0, min(RP, R - r0), sp.klo, sp.khi,
                              sp.t0 + static_cast<int>(tb), sp.t0 + static_cast<int>(te), slot};
            publish(it);
            load(it);
          }
          at += w * a.Hkv;
        }
      }
      acc = chunk_end;
    }
    publish(Gqa8Item{-1, 0, 0, 0, 0, 0, 0, 0, 0, 0, -1});
    if (lane == 0 && !tail) tails[me].parts = 0;
    // every load and every product's signal lands before the block's shared
    // memory goes away
    for (uint32_t i = n_tiles > ST ? n_tiles - ST : 0; i < n_tiles; ++i)
      wait(sm.empty[i % ST], (i / ST) & 1);
    if (*dead && lane == 0)
      for (uint32_t i = n_tiles > ST ? n_tiles - ST : 0; i < n_tiles; ++i)
        mbar_wait_bounded(smem_addr(&sm.full[i % ST]), (i / ST) & 1, 1000000);
  } else if (warp == 1) {
    // ==== products ====
    if (lane == 0) {
      constexpr uint32_t kSw = D == 128 ? kSwizzle128 : kSwizzle64;
      constexpr uint32_t idesc_qk = idesc_e4m3(128, N, false, false);
      constexpr uint32_t idesc_pv = idesc_e4m3(D, N, true, true);
      uint32_t n_items = 0, n_tiles = 0;
      // PV of tile j: O^T = V^T . P^T over 128 keys, 32 a step
      auto pv = [&](uint32_t j) {
        wait(sm.p_full[j & 1], (j >> 1) & 1);
        tc_fence_after_sync();
        const uint64_t dv = smem_desc(smem_addr(smem + (j % ST) * C::kTile) + kTileKeys * D, 16, 8 * D, kSw);
        const uint64_t dp = smem_desc(smem_addr(p_s + (j & 1) * C::kP), 128, 2048, kSwizzleNone);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f8kind(tmem + 2 * N + (j & 1) * N, dv + ((k * 32 * D) >> 4), dp + ((k * 512) >> 4), idesc_pv,
                     k > 0);
        mma_commit(smem_addr(&sm.o_full[j & 1]));
        mma_commit(smem_addr(&sm.empty[j % ST]));
      };
      bool pending = false;
      while (true) {
        const int s = n_items & 3;
        if (pending && !mbar_try_wait(smem_addr(&sm.item_full[s]), (n_items >> 2) & 1)) {
          pv(n_tiles - 1);
          pending = false;
        }
        wait(sm.item_full[s], (n_items >> 2) & 1);
        if (*dead) break;
        const int b = sm.items[s].b, nt = sm.items[s].t_end - sm.items[s].t_begin;
        mbar_arrive(smem_addr(&sm.item_empty[s]));
        if (b < 0) break;
        const uint32_t qb = n_items & 1;
        const uint64_t dq = smem_desc(smem_addr(q_s + qb * C::kQ), 16, 8 * D, kSw);
        for (int t = 0; t < nt; ++t, ++n_tiles) {
          const uint32_t j = n_tiles;
          // the next scores first, unless their keys are still on the way
          if (pending && !mbar_try_wait(smem_addr(&sm.full[j % ST]), (j / ST) & 1)) {
            pv(j - 1);
            pending = false;
          }
          if (t == 0) wait(sm.q_full[qb], (n_items >> 1) & 1);
          wait(sm.full[j % ST], (j / ST) & 1);
          tc_fence_after_sync();
          const uint64_t dk = smem_desc(smem_addr(smem + (j % ST) * C::kTile), 16, 8 * D, kSw);
#pragma unroll
          for (int k = 0; k < D / 32; ++k)
            mma_f8kind(tmem + (j & 1) * N, dk + 2 * k, dq + 2 * k, idesc_qk, k > 0);
          mma_commit(smem_addr(&sm.s_full[j & 1]));
          if (t == nt - 1) mma_commit(smem_addr(&sm.q_empty[qb]));
          if (pending) pv(j - 1);
          pending = true;
        }
        if (nt == 0) {
          // (a product left pending here would keep the softmax from its item,
          // so from the q buffer that the wait after next is for)
          if (pending) pv(n_tiles - 1);
          pending = false;
          wait(sm.q_full[qb], (n_items >> 1) & 1);
          mbar_arrive(smem_addr(&sm.q_empty[qb]));
        }
        ++n_items;
      }
      if (pending) pv(n_tiles - 1);
      if (a.fault_site == 1) wait(sm.never, 0);
    }
    __syncwarp();
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
          w[0] = __ldg(g);
          w[1] = __ldg(g + 1);
        }
        float x[16];
        const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (a.f16) {
            const float2 f = __half22float2(bits_h2(u[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
          } else {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
          }
          m = max(m, max(__float_as_uint(x[2 * i]) & 0x7FFFFFFFu, __float_as_uint(x[2 * i + 1]) & 0x7FFFFFFFu));
        }
#pragma unroll
        for (int off = 1; off < TPR; off <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
        const bool odd = m >= 0x7F800000u;                // a NaN or an infinity: NaN in its row
        // least e with amax <= 448 * 2^e, far enough from the ends of fp32
        const int e = min(max(static_cast<int>(m >> 23) - 135 + ((m & 0x7FFFFFu) > 0x600000u ? 1 : 0), -118), 118);
        const float f = odd ? 0.0f : pow2f(-e);
        if (part == 0)
          sm.qf[qb][rr] = odd ? __uint_as_float(0x7FC00000u) : a.sm_scale * 1.4426950408889634f * pow2f(e);
        uint32_t o[NT][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t t0[NT], t1[NT];
          const float x0 = odd ? 0.0f : x[4 * i] * f, x1 = odd ? 0.0f : x[4 * i + 1] * f;
          const float x2 = odd ? 0.0f : x[4 * i + 2] * f, x3 = odd ? 0.0f : x[4 * i + 3] * f;
          split_e4m3<NT>(h2_bits(__floats2half2_rn(x0, x1)), t0);
          split_e4m3<NT>(h2_bits(__floats2half2_rn(x2, x3)), t1);
#pragma unroll
          for (int t = 0; t < NT; ++t) o[t][i] = t0[t] | (t1[t] << 16);
        }
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
    const int key = tid - 128;                            // of a tile; and d of O^T
    const int quarter = warp & 3;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    constexpr int kBar = 1;
    uint32_t n_tiles = 0;
    for (uint32_t n_items = 0;; ++n_items) {
      const int s = n_items & 3, qb = n_items & 1;
      wait(sm.item_full[s], (n_items >> 2) & 1);
      // the four warps stop together: a warp that left alone would leave the
      // others at their barrier
      if (named_sync_or(kBar, 128, *dead != 0)) break;
      const Gqa8Item it = sm.items[s];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sm.item_empty[s]));
      if (it.b < 0) break;
      wait(sm.q_full[qb], (n_items >> 1) & 1);
      float o[RP], l[RP], mref[RP];
#pragma unroll
      for (int r = 0; r < RP; ++r) {
        o[r] = l[r] = 0.0f;
        mref[r] = kLowest;
      }
      // rows' positions: pos0 + (r0 + r) / G
      const int pos_first = it.pos0 + it.r0 / G, pos_last = it.pos0 + (it.r0 + it.nrows - 1) / G;
      // O of tile j joins the running output
      auto join = [&](uint32_t j) {
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
            const float2 f = sm.stash[j & 1][c + i];
            o[c + i] = fmaf(o[c + i], f.x, x * f.y);
          }
        }
        tc_fence_before_sync();
      };
      for (int t = it.t_begin; t < it.t_end; ++t, ++n_tiles) {
        const uint32_t j = n_tiles;
        const int st = j % ST;
        wait(sm.full[st], (j / ST) & 1);                  // the exponents, and V where it is cleaned
        const int ex = sm.exps[st][key >> 6], ex2 = sm.exps[st][(key >> 6) ^ 1];
        const int at = t * kTileKeys + key;               // this thread's key
        const bool live = ex != kMasked && at >= it.klo && at < it.khi;
        const int ek = static_cast<int16_t>(ex & 0xFFFF), ev = ex == kMasked ? -100 : ex >> 16;
        const int evm = max(ev, ex2 == kMasked ? -100 : ex2 >> 16);
        const float kf = live ? pow2f(ek) : 0.0f;
        const int dv = ev - evm + 8;
        const float vf = dv < -126 ? 0.0f : pow2f(dv);
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
            sc[c + i] = x * kf * sm.qf[qb][c + i];
          }
        }
        if (edge || !live) {
          const int64_t win = a.window > 0 ? a.window : (1LL << 40);
#pragma unroll
          for (int r = 0; r < RP; ++r) {
            const int64_t pos = static_cast<int64_t>(it.pos0) + (it.r0 + r) / G;
            if (!live || at > pos || at <= pos - win) sc[r] = -INFINITY;
          }
        }
#pragma unroll
        for (int r = 0; r < RP; ++r) {
          const float m = warp_max(sc[r]);
          if (lane == r) mine = m;
        }
        if (lane < RP) sm.red[j & 1][lane * 4 + quarter] = mine;
        tc_fence_before_sync();
        named_sync(kBar, 128);
        const float vs = pow2f(evm - 8);
        uint32_t terms[RP / 8 * NT * 2];                  // bytes of the row of P: term, row
#pragma unroll
        for (int r = 0; r < RP; r += 2) {
          float p[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float4 m4 = *reinterpret_cast<const float4*>(&sm.red[j & 1][(r + i) * 4]);
            const float mt = fmaxf(fmaxf(fmaxf(m4.x, m4.y), fmaxf(m4.z, m4.w)), kLowest);
            const bool up = mt > mref[r + i];
            const float x = fast_exp2(up ? mref[r + i] - mt : mt - mref[r + i]);
            const float al = up ? x : 1.0f, be = up ? 1.0f : x;
            mref[r + i] = up ? mt : mref[r + i];
            p[i] = fast_exp2(sc[r + i] - mt);
            l[r + i] = fmaf(l[r + i], al, p[i] * be);
            if (key == r + i) sm.stash[j & 1][r + i] = make_float2(al, be * vs);
          }
          uint32_t tt[NT];
          split_e4m3<NT>(h2_bits(__floats2half2_rn(p[0] * vf, p[1] * vf)), tt);
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
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sm.p_full[j & 1]));
        if (t > it.t_begin) join(j - 1);
      }
      // the factors of the last tile, written by other warps, are visible
      // behind this barrier, which also frees lsum
      named_sync(kBar, 128);
      if (it.t_end > it.t_begin) join(n_tiles - 1);
      float mine = 0.0f;
#pragma unroll
      for (int r = 0; r < RP; ++r) {
        const float x = warp_sum(l[r]);
        if (lane == r) mine = x;
      }
      if (lane < RP) sm.lsum[quarter][lane] = mine;
      if (lane == 0) mbar_arrive(smem_addr(&sm.q_empty[qb]));
      named_sync(kBar, 128);
      const bool mine_d = D == 128 || lane < 16;          // M = 64: 16 lanes of each warp
      const int d = D == 128 ? key : quarter * 16 + lane;
#pragma unroll
      for (int r = 0; r < RP; ++r) {
        if (r >= it.nrows) break;
        const float lt = (sm.lsum[0][r] + sm.lsum[1][r]) + (sm.lsum[2][r] + sm.lsum[3][r]);
        const float inv = lt == 0.0f ? 0.0f : 1.0f / lt;
        const float ls = lt == 0.0f ? -INFINITY : mref[r] + log2f(lt);
        if (it.slot >= 0) {
          const int64_t row = static_cast<int64_t>(it.slot) * RP + r;
          if (mine_d) ws_o[row * D + d] = o[r] * inv;
          if (key == 0) ws_lse[row] = ls;
        } else {
          const int rr = it.r0 + r;
          const int64_t row = static_cast<int64_t>(it.cu0 + rr / G) * a.Hq + it.h * G + rr % G;
          if (mine_d) {
            if (a.f16) static_cast<__half*>(a.out)[row * D + d] = __float2half_rn(o[r] * inv);
            else static_cast<__nv_bfloat16*>(a.out)[row * D + d] = __float2bfloat16_rn(o[r] * inv);
          }
          if (key == 0) a.lse[row] = ls * 0.6931471805599453f;
        }
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, C::kTmem);
}

// ---------------------------------------------------------------------------
// The pieces of items that were cut: block (c, r) joins row r of the item that
// began in block c of the attention kernel, by log-sum-exp over its pieces in
// their order.
// ---------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(512) merge_kernel(const Gqa8AttnArgs a, const int RP,
                                                    const Gqa8Tail* tails, const float* ws_lse,
                                                    const float* ws_o) {
  grid_dependency_wait();
  grid_launch_dependents();
  constexpr int kGroups = 512 / D;
  __shared__ float part[kGroups][D];
  __shared__ float top, sum;
  const int c = blockIdx.x, r = blockIdx.y;
  const Gqa8Tail t = tails[c];
  if (t.parts == 0 || r >= t.nrows) return;
  const int tid = threadIdx.x, d = tid % D, g = tid / D;
  // piece i is slot 2c + 1 for i = 0, else 2 (c + i)
  auto row_of = [&](int i) { return static_cast<int64_t>(i == 0 ? 2 * c + 1 : 2 * (c + i)) * RP + r; };
  if (tid < 32) {
    float m = -INFINITY;
    bool odd = false;
    for (int i = tid; i < t.parts; i += 32) {
      const float x = ws_lse[row_of(i)];
      odd |= x != x;
      m = fmaxf(m, x);
    }
    m = warp_max(m);
    odd = __any_sync(0xFFFFFFFFu, odd);
    float s = 0.0f;
    if (m > -INFINITY)
      for (int i = tid; i < t.parts; i += 32) s += fast_exp2(ws_lse[row_of(i)] - m);
    s = warp_sum(s);
    if (tid == 0) {
      top = m;
      sum = odd ? __uint_as_float(0x7FC00000u) : s;
    }
  }
  __syncthreads();
  const float m = top, s = sum;
  float o = 0.0f;
  if (s != 0.0f) {
#pragma unroll 4
    for (int i = g; i < t.parts; i += kGroups) {
      const float w = fast_exp2(ws_lse[row_of(i)] - m);
      if (w != 0.0f) o = fmaf(w, ws_o[row_of(i) * D + d], o);
    }
  }
  part[g][d] = o;
  __syncthreads();
  if (g != 0) return;
#pragma unroll
  for (int i = 1; i < kGroups; ++i) o += part[i][d];
  o = s == 0.0f ? 0.0f : o / s;
  const int G = a.Hq / a.Hkv, rr = t.r0 + r;
  const int64_t row = static_cast<int64_t>(t.cu0 + rr / G) * a.Hq + t.h * G + rr % G;
  if (a.f16) static_cast<__half*>(a.out)[row * D + d] = __float2half_rn(o);
  else static_cast<__nv_bfloat16*>(a.out)[row * D + d] = __float2bfloat16_rn(o);
  if (d == 0) a.lse[row] = s == 0.0f ? -INFINITY : (m + log2f(s)) * 0.6931471805599453f;
}

// ---------------------------------------------------------------------------
// Many rows, one warp per row: one key at a time.
// ---------------------------------------------------------------------------
template <int D, bool F16>
__global__ void __launch_bounds__(128) row_kernel(const Gqa8AttnArgs a, const int min_rows) {
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
  if (c1 - c0 > a.max_new || (c1 - c0) * (a.Hq / a.Hkv) < min_rows) return;   // the other kernel's
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

// Rows of an item and of the largest request that few_kernel takes: the
// smallest of 8, 16 and 32 that holds every request, or a single token of each
// where some have more (these go to the other kernel); 0: none of them.
int few_rows(int max_new, int G) {
  const int64_t most = static_cast<int64_t>(max_new) * G, need = most <= 32 ? most : G;
  return need <= 8 ? 8 : need <= 16 ? 16 : need <= 32 ? 32 : 0;
}
constexpr int kSlotsPerSm = 4;      // two blocks an SM at most, two slots each
size_t few_bytes(int rows, int D, int sms) {
  const size_t slots = static_cast<size_t>(kSlotsPerSm) * sms;
  return slots / 2 * sizeof(Gqa8Tail) + slots * rows * (D + 1) * sizeof(float);
}

template <int D, int RP, int NT>
cudaError_t launch_few(const Gqa8AttnArgs& a, const CUtensorMap& map, cudaStream_t stream) {
  using C = FewCfg<D, RP, NT>;
  static std::once_flag once[64];
  static cudaError_t ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::call_once(once[dev & 63], [&] {
    ready[dev & 63] = cudaFuncSetAttribute(few_kernel<D, RP, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  });
  if (ready[dev & 63] != cudaSuccess) return ready[dev & 63];
  const unsigned grid = static_cast<unsigned>(a.num_sms * C::kCtas);
  const size_t slots = static_cast<size_t>(kSlotsPerSm) * a.num_sms;
  Gqa8Tail* tails = static_cast<Gqa8Tail*>(a.ws);
  float* o = reinterpret_cast<float*>(tails + slots / 2);
  float* lse = o + slots * RP * D;
  e = launch_pdl(few_kernel<D, RP, NT>, grid, 256, C::kSmem, stream, 1, map, a, RP, tails, lse, o);
  if (e != cudaSuccess || (a.pt_stride + 1) / 2 <= kWhole) return e;       // nothing is ever cut
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, RP);
  cfg.blockDim = dim3(512);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, merge_kernel<D>, a, RP, static_cast<const Gqa8Tail*>(tails),
                            static_cast<const float*>(lse), static_cast<const float*>(o));
}

template <int D>
cudaError_t launch_d(const Gqa8AttnArgs& a, cudaStream_t stream) {
  CUtensorMap map;
  if (!pool_map(a, &map)) return cudaErrorInvalidValue;
  const int G = a.Hq / a.Hkv, rows = few_rows(a.max_new, G);
  cudaError_t e = cudaSuccess;
  if (rows == 8) e = a.f16 ? launch_few<D, 8, 3>(a, map, stream) : launch_few<D, 8, 2>(a, map, stream);
  else if (rows == 16) e = a.f16 ? launch_few<D, 16, 3>(a, map, stream) : launch_few<D, 16, 2>(a, map, stream);
  else if (rows == 32) e = a.f16 ? launch_few<D, 32, 3>(a, map, stream) : launch_few<D, 32, 2>(a, map, stream);
  if (e != cudaSuccess || static_cast<int64_t>(a.max_new) * G <= rows) return e;
  const unsigned grid = static_cast<unsigned>((a.n_tokens * a.Hq + 3) / 4);
  return a.f16 ? launch_pdl(row_kernel<D, true>, grid, 128, 0, stream, 1, a, rows + 1)
               : launch_pdl(row_kernel<D, false>, grid, 128, 0, stream, 1, a, rows + 1);
}

}  // namespace

cudaError_t launch_attention_gqa8(const Gqa8AttnArgs& a, cudaStream_t stream) {
  return a.D == 64 ? launch_d<64>(a, stream) : launch_d<128>(a, stream);
}

size_t attention_gqa8_workspace(int, int max_new, int64_t, int Hq, int Hkv, int D, int num_sms) {
  const int rows = few_rows(max_new, Hq / Hkv);
  return rows > 0 ? (few_bytes(rows, D, num_sms) + 255) / 256 * 256 : 0;
}

}  // namespace kv4
