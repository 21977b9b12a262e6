// kv4_gqa4_attention.cu -- causal attention of new tokens over the 4-bit
// grouped-query cache (kv4_attention_gqa4).
//
// Row (t, h): query head h of flat token t; token i of request b's n new ones
// stands at position seq_lens[b] - n + i and sees the keys j <= its position,
// j > position - window where there is a window.  Scores, the running maximum
// and sum and the output are held in fp32:
//   s_j = sm_scale q.k_j,  o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),
//   lse = m + log sum_j exp(s_j - m);  a row without a key: 0 and -inf.
#include <algorithm>

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
// Block: warp 0 finds the block's share of the work list and copies whole pages
// into a ring, K and V by one copy and their scales by another (a copy for each
// side of each half page, 4608 bytes by four of them, left the ring empty: 448 us
// for the decode step below); each other warp takes every W-th 4096 elements of a
// side, a chunk, with a softmax and an output of its own, and they join at the
// item's end.  The running reference of a row moves, and its output is rescaled, when
// the maximum rises by more than 2^6 (p stays below 2^14): each thread looks at its own
// scores, and only where one has risen the row's threads meet.
//
// Measured (D = 128, bf16): 64 sessions of up to 32768 tokens, 8 heads a group, 1.29 GB
// of rows: 222 us, 5.8 TB/s, 86 % of the measured copy rate; the loads alone take 197.
// What is left is instructions: 18 a key and warp, of which the conversions and their
// scales are 8, at 2.4 a clock and SM, half of what the ALU pipe gives (two blocks of
// seven warps a SM; with six 268 us; joining in place, for a ring of 12 pages in place
// of the 9 that it had then, 250 against 244, and of its 8 now, between whose outputs lie
// four floats, a ninth changes nothing; codes of V loaded behind the softmax 243 against
// 240).  2 x 204800 tokens cut over 304 blocks 88 us with the joining kernel, 333 tokens of
// one session 5.7 us.  D = 64, the same sessions: 150 us, 4.4 TB/s (214 before the copies'
// operands were uniform).  Taller items have an SM's registers for one block: drafts of 35 rows
// (D = 64, f16, 24 requests with a window of 4096) 29 us, where the prompt kernel took
// 66; a third of that is the fixed part of the call.
template <int D_, int RP_>
struct FewCfg {
  static constexpr int D = D_, RP = RP_, NT = RP / 8;
  static constexpr int kKeys = D == 64 && RP <= 16 ? 64 : 32;              // of a chunk
  static constexpr int kEach = kPage / kKeys;             // chunks of a page
  static constexpr int kCodes = kPage * D / 2, kScales = kPage * D / 16;   // of a page's side
  static constexpr int kStage = 2 * (kCodes + kScales);   // K, V, scales of K, of V
  // q as operands in registers, or in shared memory where the outputs of more rows
  // take the registers
  static constexpr bool kSharedQ = RP > 16;
  static constexpr int kCtas = RP == 8 ? 2 : 1;
  static constexpr int kWarps = RP == 16 ? 11 : 7;        // that compute
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr int kRowFloats = D + 4;                // of an output that is joined: four rows apart, all banks
  static constexpr int kJoin = kWarps * RP * (kRowFloats + 2) * 4;         // outputs, references, sums
  static constexpr int kQ = kSharedQ ? RP * (D * 2 + 4) : 0;
  static constexpr int kSmall = 2048;
  static constexpr int kRoom = (kCtas == 2 ? 112 * 1024 : 227 * 1024) - kJoin - kQ - kSmall;
  static constexpr int kStages = kRoom / kStage < 40 ? kRoom / kStage : 40;
  static constexpr int kSmem = kStages * kStage + kJoin + kQ + kSmall;
  // what an item takes beyond its tiles, in tiles (2, 3, 5 of them: the decode step
  // below 247, 244, 238 us, drafts of 35 rows 47.7, 41.6, 43.6)
  static constexpr int kCost = RP == 8 ? 5 : 3;
};

struct FewSmall {
  uint64_t full[40], empty[40], item_full[4], item_empty[4], never;
  unsigned long long total;
  int dead;
  // The page of the block that a stage is for (its number, from 0), twice, plus 1
  // where the table has none.  Pages go round the ring in order and their copies end
  // in any order, and a warp does not wait for every page of a stage, only for
  // those with a chunk of its own: a barrier tells odd rounds from even ones, so a
  // warp that waits for a round must know that the one before has ended.  It has
  // once the stage is for the page that the warp looks for.
  volatile uint32_t page[40];
  Gqa8Item items[4];
};
static_assert(sizeof(FewSmall) <= 2048, "FewSmall");
static_assert(FewCfg<128, 8>::kStages == 8, "the ring that the decode step's figures are of");

// This block's items.  Of 32 requests or fewer one warp adds up the work, and walks
// what it has in registers; of more the block has added it up (sm_total).  I: int where
// no sum of units can leave it, half the instructions of a chain that a short call waits
// for (8 requests of 3000 tokens 15.8 us against 16.2, in replays).  Not both in one
// kernel: its code comes from memory at a first call, 5 us more than for one of them.
template <typename I, typename Emit>
__device__ __forceinline__ void walk_work(const Gqa8AttnArgs& a, const Gqa8Kind& kind, unsigned long long sm_total,
                                          bool report, Gqa8Tail* tails, int lane, Emit&& emit) {
  Gqa8Request q{};
  I units = 0, total = static_cast<I>(sm_total);
  if (a.B <= 32) total = gqa8_warp_total<I>(a, kind, report, lane, q, units);
  gqa8_walk<I>(a, kind, total, tails, lane, emit, a.B <= 32, q, units);
}
// c = A B, c += A B.
__device__ __forceinline__ void mma_16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
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
__device__ __forceinline__ void scaled8(uint32_t w, __half2 s, uint32_t (&h)[4]) {
  e2m1x8_to_f16x8(w, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = h2_bits(__hmul2(bits_h2(h[i]), s));
}

// 16 values of q, as widen16, by the call's type.
__device__ __forceinline__ uint32_t widen_q(bool f16, const uint4 (&w)[2], float (&x)[16]) {
  return f16 ? widen16<true>(w, x) : widen16<false>(w, x);
}

template <int D, int RP, typename I>
__global__ void __launch_bounds__(FewCfg<D, RP>::kThreads, FewCfg<D, RP>::kCtas)
few4_kernel(const Gqa8AttnArgs a, const int max_rows, Gqa8Tail* tails, float* ws_lse, float* ws_o) {
  using C = FewCfg<D, RP>;
  constexpr int NT = C::NT, ST = C::kStages, W = C::kWarps, CK = C::kKeys, MK = CK / 16, MD = D / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  float* const join = reinterpret_cast<float*>(smem + ST * C::kStage);
  float* const tops = join + W * RP * C::kRowFloats;
  float* const sums = tops + W * RP;
  uint2* const q_s = reinterpret_cast<uint2*>(smem + ST * C::kStage + C::kJoin);
  float* const qf_s = reinterpret_cast<float*>(q_s + (C::kSharedQ ? RP * D / 4 : 0));
  FewSmall& sm = *reinterpret_cast<FewSmall*>(smem + ST * C::kStage + C::kJoin + C::kQ);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.Hq / a.Hkv;

  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(smem_addr(&sm.full[i]), 1);
      mbar_init(smem_addr(&sm.empty[i]), C::kEach);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_addr(&sm.item_full[i]), 1);
      mbar_init(smem_addr(&sm.item_empty[i]), W);
    }
    mbar_init(smem_addr(&sm.never), 1);
    for (int i = 0; i < ST; ++i) sm.page[i] = 0xFFFFFFFFu;
    sm.total = 0;
    sm.dead = 0;
    fence_mbar_init();
  }
  grid_dependency_wait();
  grid_launch_dependents();
  __syncthreads();
  // Where none is ever cut and they suffice, a block for each request and kv head:
  // nothing has to be added up.
  const bool one_each = (a.pt_stride + 1) / 2 <= kWhole && static_cast<int64_t>(a.B) * a.Hkv <= gridDim.x;
  const Gqa8Kind kind{1, max_rows, RP, C::kCost, RP, C::kCost, 1};
  if (!one_each && a.B > 32) {
    gqa8_total(a, kind, blockIdx.x == 0, &sm.total);
    __syncthreads();
  }
  volatile int* dead = &sm.dead;
  // A wait that gives up (false) ends every later one of the block at once: the roles
  // then run to their ends, and the outputs are not valid.  A warp that gave up a page
  // frees no stage any more, so that a free stage never has a copy on its way, and the
  // loading warp begins none behind the first stage that it does not get.
  auto wait = [&](uint64_t& bar, uint32_t parity) {
    if (mbar_try_wait(smem_addr(&bar), parity)) return true;
    if (*dead) return false;
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait_suspend(smem_addr(&bar), parity, 20000u)) {
      if (*dead) return false;
      if (global_timer_ns() - t0 > a.timeout_ns) {
        *dead = 1;
        flag_error(a.dev_err, kDevTimeout);
        return false;
      }
    }
    return true;
  };
  // an item's pages: of its first key on, up to its last
  struct Pages {
    int first, n;
  };
  auto pages_of = [](const Gqa8Item& it) {
    const int64_t lo = max(static_cast<int64_t>(it.klo), static_cast<int64_t>(it.t_begin) * kTileKeys);
    const int64_t hi = min(static_cast<int64_t>(it.khi), static_cast<int64_t>(it.t_end) * kTileKeys);
    Pages p{static_cast<int>(lo / kPage), 0};
    if (hi > lo) p.n = static_cast<int>((hi - 1) / kPage) + 1 - p.first;
    return p;
  };

  if (warp == 0) {
    // ==== work list and loads ====
    uint32_t n_items = 0, n_pages = 0;                    // pages whose copies began
    uint32_t stage = 0, empty_par = 1;                    // of the next page
    bool stopped = false;                                 // no more copies
    auto publish = [&](const Gqa8Item& it) {
      const int s = n_items & 3;
      wait(sm.item_empty[s], ((n_items >> 2) & 1) ^ 1);
      __syncwarp();                                       // (no lane still looks for the round before)
      // (of a wait that gave up the item before may still be in use)
      if (lane == 0 && !*dead) {
        sm.items[s] = it;
        mbar_arrive(smem_addr(&sm.item_full[s]));
      }
      ++n_items;
    };
    auto load_item = [&](const Gqa8Item& it) {
      const Pages c = pages_of(it);
      for (int i = 0; i < c.n && !stopped; i += 32) {
        // a lane's page: its K and V, or -1 where the table has none
        const int64_t at = static_cast<int64_t>(c.first) + i + lane;
        int block = -1;                                   // (2 Hkv num_pages < 2^31)
        if (at * kPage < it.khi) {
          const int phys = load(a.page_table + it.b * a.pt_stride + at);
          if (phys < 0 || phys >= a.num_pages) flag_error(a.dev_err, kDevBadPage);
          else block = phys * a.Hkv + it.h;
        }
        // (the whole warp walks the pages, so that what the copies take but the page
        // itself stays uniform; whether the block gave up is looked at only where a
        // stage is not free yet)
        const int n = min(32, c.n - i);
        for (int k = 0; k < n; ++k) {
          const int64_t blk = __shfl_sync(0xFFFFFFFFu, block, k);
          if (!__all_sync(0xFFFFFFFFu, mbar_try_wait(smem_addr(&sm.empty[stage]), empty_par))) {
            wait(sm.empty[stage], empty_par);
            stopped = __any_sync(0xFFFFFFFFu, *dead != 0);
            if (stopped) break;
          }
          if (elect_one()) {
            const uint32_t bar = smem_addr(&sm.full[stage]), dst = smem_addr(smem) + stage * C::kStage;
            sm.page[stage] = 2 * n_pages + (blk < 0);
            if (blk >= 0) {
              mbar_arrive_expect_tx(bar, C::kStage);
              bulk_copy_g2s(dst, a.pool + blk * (2 * C::kCodes), 2 * C::kCodes, bar);
              bulk_copy_g2s(dst + 2 * C::kCodes, a.scales + blk * (2 * C::kScales), 2 * C::kScales, bar);
            } else {
              mbar_arrive(bar);
            }
          }
          __syncwarp();
          ++n_pages;
          if (++stage == ST) {
            stage = 0;
            empty_par ^= 1;
          }
        }
      }
    };
    auto take = [&](const Gqa8Item& it) {
      publish(it);
      load_item(it);
    };
    if (one_each) {
      const int b = blockIdx.x / a.Hkv, h = blockIdx.x - b * a.Hkv;
      const Gqa8Request r = gqa8_request(a, b, 1, max_rows, h == 0 && lane == 0);
      const Gqa8Span sp = gqa8_span(a, r, G, 0, max(r.n * G, 1));
      if (r.n > 0) take(Gqa8Item{b, h, r.cu0, r.pos0, 0, r.n * G, sp.klo, sp.khi, sp.t0, sp.t0 + sp.nt, -1});
    } else {
      walk_work<I>(a, kind, sm.total, blockIdx.x == 0, tails, lane, take);
    }
    publish(Gqa8Item{-1, 0, 0, 0, 0, 0, 0, 0, 0, 0, -1});
    // every copy lands before the block's shared memory goes away
    for (uint32_t i = n_pages > ST ? n_pages - ST : 0; i < n_pages; ++i)
      wait(sm.empty[i % ST], (i / ST) & 1);
    if (*dead && lane == 0)
      for (uint32_t i = n_pages > ST ? n_pages - ST : 0; i < n_pages; ++i)
        mbar_wait_bounded(smem_addr(&sm.full[i % ST]), (i / ST) & 1, 1000000);
  } else {
    // ==== scores, softmax, output ====
    const int w = warp - 1, r8 = lane >> 2, t4 = lane & 3;
    // key of row m of a 16-key tile: 0, 4, 1, 5, 2, 6, 3, 7 and 8 more for m >= 8, so
    // that a thread's four keys of V are t, t + 4, t + 8, t + 12, whose rows lie in
    // all banks
    const int key_r = (r8 >> 1) + (r8 & 1) * 4;
    // this warp's next chunk of the ring (of kEach * ST), its rounds' parity and its
    // page's number in the block
    uint32_t slot = w, par = 0, turn = 0, chunk = w;      // turn: chunks of the block so far, mod W
    const uint8_t* const k_l = smem + key_r * (D / 2) + t4 * (D / 8);
    const uint8_t* const ks_l = smem + 2 * C::kCodes + key_r * (D / 16) + t4 * (D / 64);
    const uint8_t* const v_l = smem + C::kCodes + t4 * (D / 2) + r8 * (D / 16);
    const uint8_t* const vs_l = smem + 2 * C::kCodes + C::kScales + t4 * (D / 16) + r8 * (D / 16) / 8;
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
      const Pages c = pages_of(it);

      // q: row n of 8 is threads 4n .. 4n + 3's, D / 4 elements each.  Its factor is
      // at least 2^-126, so that a masked -inf stays one where the scale is 0; a row
      // with a NaN or an infinity becomes NaN at the end.
      constexpr int QN = C::kSharedQ ? 1 : NT, QD = C::kSharedQ ? 1 : MD;
      uint32_t q[QD][QN][2];
      float qf[NT][2];
      const float sign = a.sm_scale < 0.0f ? -1.0f : 1.0f, unit = fabsf(a.sm_scale) * 1.4426950408889634f;
      auto row_of = [&](int rr) {
        const int r = it.r0 + min(rr, it.nrows - 1);
        return static_cast<const uint16_t*>(a.q) + static_cast<int64_t>(it.cu0 + r / G) * a.q_token_stride +
               static_cast<int64_t>(it.h * G + r % G) * a.q_head_stride;
      };
      constexpr float kNan = __builtin_nanf("");
      if constexpr (C::kSharedQ) {
        // 16 elements a thread, a row by D / 16 of them
        constexpr int kTpr = D / 16;
        for (int rr = (tid - 32) / kTpr; rr < RP; rr += 32 * W / kTpr) {
          const int part = (tid - 32) % kTpr;
          float x[16];
          const uint4* g = reinterpret_cast<const uint4*>(row_of(rr) + part * 16);
          const uint4 two[2] = {load(g), load(g + 1)};
          uint32_t m = widen_q(a.f16, two, x);
          const uint32_t group = kTpr == 8 ? 0xFFu << (lane & 24) : 0xFu << (lane & 28);
#pragma unroll
          for (int off = 1; off < kTpr; off *= 2) m = max(m, __shfl_xor_sync(group, m, off));
          const bool odd = m >= 0x7F800000u;
          const int e = q_exponent(m);
          const float f = sign * pow2f(-e);
          if (part == 0) qf_s[rr] = odd ? kNan : fmaxf(unit * pow2f(e), 0x1p-126f);
          // element i of thread t's D / 4: product i / 4, half (i % 4) / 2
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int el = part * 16 + 4 * i, t = el / (D / 4), j = el % (D / 4) / 4;
            q_s[(j * NT + rr / 8) * 32 + rr % 8 * 4 + t] =
                odd ? make_uint2(0, 0) : make_uint2(h2_bits(__floats2half2_rn(x[4 * i] * f, x[4 * i + 1] * f)),
                                                    h2_bits(__floats2half2_rn(x[4 * i + 2] * f, x[4 * i + 3] * f)));
          }
        }
        named_sync(1, 32 * W);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) qf[nt][i] = qf_s[nt * 8 + 2 * t4 + i];
      } else {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float x[D / 4];
          uint32_t m = 0;
          const uint4* g = reinterpret_cast<const uint4*>(row_of(nt * 8 + r8) + t4 * (D / 4));
#pragma unroll
          for (int i = 0; i < D / 64; ++i) {
            const uint4 two[2] = {load(g + 2 * i), load(g + 2 * i + 1)};
            m = max(m, widen_q(a.f16, two, reinterpret_cast<float(&)[16]>(x[16 * i])));
          }
          m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
          m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
          const bool odd = m >= 0x7F800000u;
          const int e = q_exponent(m);
          const float f = sign * pow2f(-e);
#pragma unroll
          for (int j = 0; j < MD; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              q[j][nt][i] = odd ? 0u : h2_bits(__floats2half2_rn(x[4 * j + 2 * i] * f, x[4 * j + 2 * i + 1] * f));
          const float mine = odd ? kNan : fmaxf(unit * pow2f(e), 0x1p-126f);
          // (the columns' factors are their rows' threads')
#pragma unroll
          for (int i = 0; i < 2; ++i) qf[nt][i] = __shfl_sync(0xFFFFFFFFu, mine, (2 * t4 + i) * 4);
        }
      }
      uint32_t odd_rows = 0;                              // bit 2 nt + i
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (qf[nt][i] != qf[nt][i]) {
            odd_rows |= 1u << (2 * nt + i);
            qf[nt][i] = 0x1p-126f;
          }
      const int pos_first = it.pos0 + it.r0 / G, pos_last = it.pos0 + (it.r0 + it.nrows - 1) / G;
      // p = 2^(s qf + ref), ref = 8 - (the reference)
      float o[MD][NT][4], l[NT][2], ref[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          l[nt][i] = 0.0f;
          ref[nt][i] = -kLowest;
        }
#pragma unroll
        for (int i = 0; i < MD; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[i][nt][k] = 0.0f;
      }

      // chunks before `open` or from `full` on have keys that some row does not see
      const int64_t last_whole = min(static_cast<int64_t>(it.khi), static_cast<int64_t>(pos_first) + 1) - CK;
      const int full = static_cast<int>(max(last_whole, static_cast<int64_t>(-1)));
      const int open = a.window > 0 ? max(it.klo, static_cast<int>(max(static_cast<int64_t>(pos_last) - a.window + 1, static_cast<int64_t>(0)))) : it.klo;
      // chunk i of the item: warp ((i + the block's chunks before it) mod W)'s
      for (int i = static_cast<int>((w + W - turn) % W); i < c.n * C::kEach; i += W) {
        const uint32_t st = slot / C::kEach, part = slot % C::kEach;
        const uint32_t number = chunk / C::kEach;
        uint32_t there = sm.page[st];
        if (!__all_sync(0xFFFFFFFFu, there / 2 == number && mbar_try_wait(smem_addr(&sm.full[st]), par))) {
          const uint64_t since = global_timer_ns();
          while ((there = sm.page[st]) / 2 != number && !*dead) {
            __nanosleep(40);
            if (global_timer_ns() - since > a.timeout_ns) {
              *dead = 1;
              flag_error(a.dev_err, kDevTimeout);
            }
          }
          // (a page that was given up frees no stage, and its block is at its last item)
          if (!__all_sync(0xFFFFFFFFu, there / 2 == number && wait(sm.full[st], par))) break;
        }
        chunk += W;
        slot += W;
        if (slot >= ST * C::kEach) {
          slot -= ST * C::kEach;
          par ^= 1;
        }
        const int base = c.first * kPage + i * CK;        // (below khi)
        if (there % 2 == 0) {
          const bool edge = base > full || base < open;
          const uint32_t at = st * C::kStage + part * (CK * D / 2), at_s = st * C::kStage + part * (CK * D / 16);
          float s[MK][NT][4];
          alignas(16) uint32_t kw[MK][2][D / 32];         // codes of keys r and r + 8
          uint32_t ks[MK][2];                             // scales of their blocks
#pragma unroll
          for (int mk = 0; mk < MK; ++mk)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int row = mk * 16 + 8 * j;
              if constexpr (D == 128) {
                *reinterpret_cast<uint4*>(kw[mk][j]) = *reinterpret_cast<const uint4*>(k_l + at + row * 64);
                ks[mk][j] = *reinterpret_cast<const uint16_t*>(ks_l + at_s + row * 8);
              } else {
                *reinterpret_cast<uint2*>(kw[mk][j]) = *reinterpret_cast<const uint2*>(k_l + at + row * 32);
                ks[mk][j] = ks_l[at_s + row * 4];
              }
            }
#pragma unroll
          for (int mk = 0; mk < MK; ++mk) {
            ks[mk][0] = e4m3x2_to_f16x2(ks[mk][0]);
            ks[mk][1] = e4m3x2_to_f16x2(ks[mk][1]);
          }
          // (the key tiles in turns: each is a chain of products)
#pragma unroll
          for (int x = 0; x < D / 32; ++x)
#pragma unroll
            for (int mk = 0; mk < MK; ++mk) {
              // (two words a block of 16)
              uint32_t h0[4], h1[4];
              auto scale = [&](uint32_t two) { return x < 2 ? __low2half2(bits_h2(two)) : __high2half2(bits_h2(two)); };
              scaled8(kw[mk][0][x], scale(ks[mk][0]), h0);
              scaled8(kw[mk][1][x], scale(ks[mk][1]), h1);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                uint2 b0, b1;
                if constexpr (C::kSharedQ) {
                  b0 = q_s[(2 * x * NT + nt) * 32 + lane];
                  b1 = q_s[((2 * x + 1) * NT + nt) * 32 + lane];
                } else {
                  b0 = make_uint2(q[2 * x][nt][0], q[2 * x][nt][1]);
                  b1 = make_uint2(q[2 * x + 1][nt][0], q[2 * x + 1][nt][1]);
                }
                if (x == 0) mma_16816_first(s[mk][nt], h0[0], h1[0], h0[1], h1[1], b0.x, b0.y);
                else mma_16816(s[mk][nt], h0[0], h1[0], h0[1], h1[1], b0.x, b0.y);
                mma_16816(s[mk][nt], h0[2], h1[2], h0[3], h1[3], b1.x, b1.y);
              }
            }
          if (edge) {
            // 0 <= position - key < window, of the keys that are there
            const uint32_t win = a.window > 0 ? a.window : 0x80000000u;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int pos = it.pos0 + (it.r0 + min(nt * 8 + 2 * t4 + i, it.nrows - 1)) / G;
#pragma unroll
                for (int mk = 0; mk < MK; ++mk)
#pragma unroll
                  for (int k = i; k < 4; k += 2) {
                    const int key = base + mk * 16 + key_r + (k & 2) * 4;
                    if (!(static_cast<uint32_t>(pos - key) < win && key < it.khi)) s[mk][nt][k] = -INFINITY;
                  }
              }
          }
          // Each thread looks at its own scores; only where one rises too far is
          // a maximum taken over the row's threads.
          struct Vs {
            alignas(8) uint32_t v[4][D / 64];
            uint32_t sc[4];
          };
          auto load_v = [&](int mk, Vs& z) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int row = mk * 16 + 4 * k;
              if constexpr (D == 128) *reinterpret_cast<uint2*>(z.v[k]) = *reinterpret_cast<const uint2*>(v_l + at + row * 64);
              else z.v[k][0] = *reinterpret_cast<const uint32_t*>(v_l + at + row * 32);
              z.sc[k] = vs_l[at_s + row * (D / 16)];
            }
          };
          Vs vs[2];
          load_v(0, vs[0]);
          auto top_of = [&](int nt, int k) {
            float m = fmaxf(s[0][nt][k], s[0][nt][k + 2]);
#pragma unroll
            for (int mk = 1; mk < MK; ++mk) m = max3(m, s[mk][nt][k], s[mk][nt][k + 2]);
            return m;
          };
          bool rise = false;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) rise |= fmaf(top_of(nt, k), qf[nt][k], ref[nt][k]) > 14.0f;
          if (__any_sync(0xFFFFFFFFu, rise)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                float m = top_of(nt, k);
#pragma unroll
                for (int off = 4; off < 32; off *= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
                const float to = fminf(ref[nt][k], 8.0f - m * qf[nt][k]), by = fast_exp2(to - ref[nt][k]);
                ref[nt][k] = to;
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
#pragma unroll
            for (int mk = 0; mk < MK; ++mk)
#pragma unroll
              for (int k = 0; k < 4; k += 2) {
                const float p0 = fast_exp2(fmaf(s[mk][nt][k], qf[nt][0], ref[nt][0]));
                const float p1 = fast_exp2(fmaf(s[mk][nt][k + 1], qf[nt][1], ref[nt][1]));
                l[nt][0] += p0;
                l[nt][1] += p1;
                p[mk][nt][k / 2] = transpose8x8(h2_bits(__floats2half2_rn(p0, p1)));
              }
          }
#pragma unroll
          for (int mk = 0; mk < MK; ++mk) {
            if (mk + 1 < MK) load_v(mk + 1, vs[(mk + 1) & 1]);
            auto& v = vs[mk & 1].v;
            auto& sc = vs[mk & 1].sc;
            // a key that no row sees may hold a NaN scale, which a weight of zero
            // would not silence
            if (edge) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int row = base + mk * 16 + 4 * k + t4;
                sc[k] = row >= it.klo && row < it.khi ? sc[k] : 0u;
              }
            }
            const __half2 s01 = bits_h2(e4m3x2_to_f16x2(sc[0] + sc[1] * 256)), s23 = bits_h2(e4m3x2_to_f16x2(sc[2] + sc[3] * 256));
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
      turn = (turn + c.n * C::kEach) % W;

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
            tops[w * RP + row] = -ref[nt][k];
            sums[w * RP + row] = (odd_rows >> (2 * nt + k) & 1u) != 0 && x > 0.0f ? kNan : x;
          }
          // elements lane / 4 * D / 8 + 2 i and the next, at 16 i + lane / 4 * 2 of the row,
          // where a half warp's lie in all banks
          float* const to = join + (w * RP + row) * C::kRowFloats + r8 * 2;
#pragma unroll
          for (int i = 0; i < MD; ++i) *reinterpret_cast<float2*>(to + 16 * i) = make_float2(o[i][nt][k], o[i][nt][k + 2]);
        }
      named_sync(1, 32 * W);
      for (int u = tid - 32; u < it.nrows * (D / 4); u += 32 * W) {
        const int row = u / (D / 4), at4 = u % (D / 4);
        // two pairs of elements, D / 8 apart
        const int d = at4 % 4 * 2 * (D / 8) + at4 / 4 * 2;
        float top = kLowest;
#pragma unroll
        for (int i = 0; i < W; ++i) top = fmaxf(top, tops[i * RP + row]);
        float y[4] = {0.0f, 0.0f, 0.0f, 0.0f}, sum = 0.0f;
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const float f = fast_exp2(tops[i * RP + row] - top);
          sum = fmaf(sums[i * RP + row], f, sum);
          const float4 v = *reinterpret_cast<const float4*>(join + (i * RP + row) * C::kRowFloats + at4 * 4);
          y[0] = fmaf(v.x, f, y[0]);
          y[1] = fmaf(v.y, f, y[1]);
          y[2] = fmaf(v.z, f, y[2]);
          y[3] = fmaf(v.w, f, y[3]);
        }
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        const float ls = sum == 0.0f ? -INFINITY : top + log2f(sum);
        if (it.slot >= 0) {
          const int64_t at = static_cast<int64_t>(it.slot) * RP + row;
          *reinterpret_cast<float2*>(ws_o + at * D + d) = make_float2(y[0] * inv, y[1] * inv);
          *reinterpret_cast<float2*>(ws_o + at * D + d + D / 8) = make_float2(y[2] * inv, y[3] * inv);
          if (at4 == 0) ws_lse[at] = ls;
        } else {
          const int r = it.r0 + row;
          const int64_t at = static_cast<int64_t>(it.cu0 + r / G) * a.Hq + it.h * G + r % G;
          uint16_t* const to = static_cast<uint16_t*>(a.out) + at * D + d;
          *reinterpret_cast<uint32_t*>(to) = a.f16 ? pack16<true>(y[0] * inv, y[1] * inv) : pack16<false>(y[0] * inv, y[1] * inv);
          *reinterpret_cast<uint32_t*>(to + D / 8) = a.f16 ? pack16<true>(y[2] * inv, y[3] * inv) : pack16<false>(y[2] * inv, y[3] * inv);
          if (at4 == 0) a.lse[at] = ls * 0.6931471805599453f;
        }
      }
      if (a.fault_site == 1 && w == 0) wait(sm.never, 0);
    }
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------
// Many rows: prompt chunks
// ---------------------------------------------------------------------------
// What bounds this case is the tensor core: 4 D flops a pair of row and key.
// An item is 256 rows of one kv head, two M = 128 tiles that take turns: while
// the softmax of one works on its scores, the products of the other run.  Of an
// item with at most 128 rows the two are the same rows over every other tile of
// keys, joined at its end, so that they take turns all the same.
//   S[128 rows x 128 keys] = Q . K^T     kind::f16, both from shared memory
//   O[128 rows x D] += P . V             kind::f16, P from TMEM
// K and V are widened to f16 once per tile by four warps (exact: code * scale has 6
// significant bits), from codes that bulk copies bring, a side of a tile at a time;
// q is exact in f16 but for elements below 2^-22 of its row's largest.  The chain
// scores -> softmax -> P -> O, next scores of a row tile is what the other tile's
// products have to cover, so two threads share a row, one for each page of the
// tile (64 keys).  A row's reference only moves, and its O in TMEM is only
// rescaled, when the maximum rises by more than 2^6 (p stays below 2^14, f16's top
// is 2^16).
//
// Measured (32 heads over 8, D = 128, bf16): 2 x 2048 new tokens over up to 16384 606 us,
// 1.34 PFLOP/s, 71 % of the measured bf16 rate; without the widening, on whatever the
// tiles hold, 563 (of 632 then).  What it costs is the time of its chain (codes, f16, fence, products)
// rather than its instructions: two warps took 1040 us, four 814, a page's pieces at
// fixed places 698, both pages together 674, and the softmax with 96 registers in place
// of 88 645.  A prompt of 8192 477 us, 1.15 PFLOP/s.
template <int D_>
struct ManyCfg {
  static constexpr int D = D_, kRows = 256;
  static constexpr int kTile = kTileKeys * D * 2;         // of K, of V, or of 128 rows of q in f16
  static constexpr int kCodes = kPage * D / 2, kScales = kPage * D / 16;   // of a page's side
  static constexpr int kSide = 2 * (kCodes + kScales);    // of a tile's: codes of both pages, then scales
  static constexpr int kSmall = 6144;
  static constexpr int kRoom = 227 * 1024 - 1024 - 6 * kTile - kSmall;
  static constexpr int kRaw = kRoom / kSide < 8 ? kRoom / kSide : 8;       // sides of tiles on their way
  static constexpr int kSmem = 6 * kTile + kRaw * kSide + kSmall + 1024;
};
static_assert(ManyCfg<128>::kRaw >= 3 && ManyCfg<64>::kRaw <= 8, "more than a tile is on its way, four tiles at most");
constexpr int kManyThreads = 768;
// (One head's 64 rows: 109 us with 40 and 56 registers, 107 with 48 and 48, 103 so; with
// 88 for the softmax chunks take 5 % more.)
constexpr uint32_t kSoftmaxRegs = 96, kIssueRegs = 32, kWidenRegs = 64, kLaunchRegs = 80;
static_assert(4 * kSoftmaxRegs + kIssueRegs + kWidenRegs <= 6 * kLaunchRegs, "register shares draw on the launch's");

// What an item takes beyond its tiles (q in, first scores, last product, output),
// in half tiles; of an item of at most 128 rows.  (A whole prompt of 8192: 532 us with 8,
// 501 with 10, 503 with 13.)
constexpr int kManyCost = 10, kSharedCost = 4;

struct ManySmall {
  uint64_t raw_full[8], raw_empty[8], k_full[2], k_empty[2], v_full[2], v_empty[2], item_full[2], item_empty[2],
      gone_full[8], q_full[2], s_full[2], p_full[2][2], o_full[2], never;
  unsigned long long total;
  uint32_t tmem;
  int dead;
  int gone[8][2];             // per tile and page: not there
  Gqa8Item items[2];
  float qf[2][128];           // sm_scale log2(e) 2^eq of a row, NaN where q is not finite
  float top[2][2][2][128];    // largest score of a half row, by row tile and tile parity;
                              //   at an item's end sums of both halves and reference (last)
  __device__ float& last(int qt, int k, int row) { return top[qt][k >> 1][k & 1][row]; }
};
static_assert(sizeof(ManySmall) <= 6144, "ManySmall");

template <int D, bool F16, typename I>
__global__ void __launch_bounds__(kManyThreads, 1)
many4_kernel(const Gqa8AttnArgs a, const int min_rows,
            Gqa8Tail* tails, float* ws_lse, float* ws_o) {
  using C = ManyCfg<D>;
  constexpr int NR = C::kRaw;
  constexpr int kSlab = kTileKeys * 128;                  // 64 f16 columns of an operand
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const q_s = smem;
  uint8_t* const k_s = q_s + 2 * C::kTile;
  uint8_t* const v_s = k_s + 2 * C::kTile;
  uint8_t* const raw_s = v_s + 2 * C::kTile;
  ManySmall& sm = *reinterpret_cast<ManySmall*>(raw_s + NR * C::kSide);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.Hq / a.Hkv;
  constexpr int kAll = 0x7FFFFFFF;

  if (tid == 0) {
    for (int i = 0; i < NR; ++i) {
      mbar_init(smem_addr(&sm.raw_full[i]), 1);
      mbar_init(smem_addr(&sm.raw_empty[i]), 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&sm.k_full[i]), 4);
      mbar_init(smem_addr(&sm.k_empty[i]), 1);
      mbar_init(smem_addr(&sm.v_full[i]), 4);
      mbar_init(smem_addr(&sm.v_empty[i]), 1);
      mbar_init(smem_addr(&sm.item_full[i]), 1);
      mbar_init(smem_addr(&sm.item_empty[i]), 21);        // the product's lane, 4 + 16 warps
      mbar_init(smem_addr(&sm.q_full[i]), 8);
      mbar_init(smem_addr(&sm.s_full[i]), 1);
      mbar_init(smem_addr(&sm.p_full[i][0]), 8);
      mbar_init(smem_addr(&sm.p_full[i][1]), 8);
      mbar_init(smem_addr(&sm.o_full[i]), 1);
    }
    for (int i = 0; i < 8; ++i) mbar_init(smem_addr(&sm.gone_full[i]), 1);
    mbar_init(smem_addr(&sm.never), 1);
    sm.total = 0;
    sm.dead = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(smem_addr(&sm.tmem), 512);
  grid_dependency_wait();
  grid_launch_dependents();
  __syncthreads();
  const Gqa8Kind kind{min_rows, kAll, C::kRows, kManyCost, 128, kSharedCost, 2};
  if (a.B > 32) gqa8_total(a, kind, blockIdx.x == 0 && min_rows == 1, &sm.total);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = sm.tmem;                          // S/P of the row tiles, then O
  volatile int* dead = &sm.dead;
  // As in few4_kernel: false where it gave up, and a warp that gave up a side of a tile
  // frees no stage any more.
  auto wait = [&](uint64_t& bar, uint32_t parity) {
    if (mbar_try_wait(smem_addr(&bar), parity)) return true;
    if (*dead) return false;
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait_suspend(smem_addr(&bar), parity, 20000u)) {
      if (*dead) return false;
      if (global_timer_ns() - t0 > a.timeout_ns) {
        *dead = 1;
        flag_error(a.dev_err, kDevTimeout);
        return false;
      }
    }
    return true;
  };

  if (warp < 4) {
    setmaxnreg_dec<kIssueRegs>();
    if (warp == 0) {
      // ==== work list and loads ====
      uint32_t n_items = 0, n_tiles = 0;
      uint32_t n_sides = 0;                               // sides of tiles whose copies began
      uint32_t st = 0, st_par = 1;                        // of the next side
      bool stopped = false;                               // no more copies
      auto publish = [&](const Gqa8Item& it) {
        const int s = n_items & 1;
        wait(sm.item_empty[s], ((n_items >> 1) & 1) ^ 1);
        __syncwarp();                                     // (no lane still looks for the round before)
        // (of a wait that gave up the item before may still be in use)
        if (lane == 0 && !*dead) {
          sm.items[s] = it;
          mbar_arrive(smem_addr(&sm.item_full[s]));
        }
        ++n_items;
      };
      auto load_item = [&](const Gqa8Item& it) {
        for (int t = it.t_begin; t < it.t_end && !stopped; t += 16) {
          // page `lane` of 16 tiles: its K and V, or -1 where no key of it is seen
          // or the table has none
          const int64_t page = 2 * static_cast<int64_t>(t) + lane;
          int block = -1;
          if ((page >> 1) < it.t_end && (page << 6) < it.khi && (page << 6) + 64 > it.klo) {
            const int phys = load(a.page_table + it.b * a.pt_stride + page);
            if (phys < 0 || phys >= a.num_pages) flag_error(a.dev_err, kDevBadPage);
            else block = phys * a.Hkv + it.h;             // (2 Hkv num_pages < 2^31)
          }
          const int nt = min(16, it.t_end - t);
          for (int i = 0; i < nt; ++i, ++n_tiles) {
            const int b[2] = {__shfl_sync(0xFFFFFFFFu, block, 2 * i), __shfl_sync(0xFFFFFFFFu, block, 2 * i + 1)};
#pragma unroll
            for (int side = 0; side < 2; ++side) {        // K, V
              // (the whole warp, so that what the copies take but the page itself stays
              // uniform; whether the block gave up is looked at only where a stage is
              // not free yet)
              if (!__all_sync(0xFFFFFFFFu, mbar_try_wait(smem_addr(&sm.raw_empty[st]), st_par))) {
                wait(sm.raw_empty[st], st_par);
                stopped = __any_sync(0xFFFFFFFFu, *dead != 0);
                if (stopped) return;
              }
              if (elect_one()) {
                if (side == 0) {
                  // (the softmax of the tile eight before is done: this stage was, up
                  // to four tiles ago, one of the widening warps', which then had V of
                  // the tile before, so the products of the tile seven before were over)
                  sm.gone[n_tiles & 7][0] = b[0] < 0;
                  sm.gone[n_tiles & 7][1] = b[1] < 0;
                  mbar_arrive(smem_addr(&sm.gone_full[n_tiles & 7]));
                }
                const uint32_t bar = smem_addr(&sm.raw_full[st]), dst = smem_addr(raw_s) + st * C::kSide;
                const uint32_t there = (b[0] >= 0) + (b[1] >= 0);
                if (there > 0) mbar_arrive_expect_tx(bar, there * (C::kCodes + C::kScales));
                else mbar_arrive(bar);
#pragma unroll
                for (int pg = 0; pg < 2; ++pg)
                  if (b[pg] >= 0) {
                    const int64_t blk = 2 * static_cast<int64_t>(b[pg]) + side;
                    bulk_copy_g2s(dst + pg * C::kCodes, a.pool + blk * C::kCodes, C::kCodes, bar);
                    bulk_copy_g2s(dst + 2 * C::kCodes + pg * C::kScales, a.scales + blk * C::kScales, C::kScales, bar);
                  }
              }
              __syncwarp();
              ++n_sides;
              if (++st == NR) {
                st = 0;
                st_par ^= 1;
              }
            }
          }
        }
      };
      walk_work<I>(a, kind, sm.total, blockIdx.x == 0 && min_rows == 1, tails, lane, [&](const Gqa8Item& it) {
        publish(it);
        load_item(it);
      });
      publish(Gqa8Item{-1, 0, 0, 0, 0, 0, 0, 0, 0, 0, -1});
      // every copy and every signal lands before the block's shared memory goes away
      for (uint32_t i = n_sides > NR ? n_sides - NR : 0; i < n_sides; ++i)
        wait(sm.raw_empty[i % NR], (i / NR) & 1);
      for (uint32_t i = n_tiles > 2 ? n_tiles - 2 : 0; i < n_tiles; ++i) {
        wait(sm.k_empty[i & 1], (i >> 1) & 1);
        wait(sm.v_empty[i & 1], (i >> 1) & 1);
      }
      if (*dead && lane == 0)
        for (uint32_t i = n_sides > NR ? n_sides - NR : 0; i < n_sides; ++i)
          mbar_wait_bounded(smem_addr(&sm.raw_full[i % NR]), (i / NR) & 1, 1000000);
    } else if (warp == 1) {
      // ==== products (the whole warp; one lane issues) ====
      constexpr uint32_t idesc_qk = idesc_f16(128, 128, false, false);
      constexpr uint32_t idesc_pv = idesc_f16(128, D, false, true);
      // (descriptors: addresses are in the lower words, which never carry)
      const uint32_t dk0 = smem_desc(smem_addr(k_s), 16, 1024, kSwizzle128), dq0 = smem_desc(smem_addr(q_s), 16, 1024, kSwizzle128);
      const uint32_t dv0 = smem_desc(smem_addr(v_s), kSlab, 1024, kSwizzle128);
      auto desc = [](uint32_t lower) { return (smem_desc(0, 0, 1024, kSwizzle128) & ~0xFFFFFFFFull) | lower; };
      uint32_t n_tiles = 0, ks = 0, k_par = 0;            // stage of K and its parity
      uint32_t w0 = 0, w1 = 0, p0 = 0, p1 = 0;            // parities of the row tiles' q and P
      // The queue of products is a few instructions deep, so what keeps this
      // warp between two groups of them has to be short: waits come where a group
      // has just been queued, and a group ends with all its signals.
      auto qk = [&](int qt, uint32_t stage, int q) {                   // of the elected lane
        const uint32_t dk = dk0 + stage * (C::kTile >> 4), dq = dq0 + q * (C::kTile >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t at = (k / 4 * kSlab + k % 4 * 32) >> 4;
          mma_f16kind(tmem + qt * 128, desc(dq + at), desc(dk + at), idesc_qk, k > 0);
        }
        mma_commit(smem_addr(&sm.s_full[qt]));
      };
      // PV of tile j, then, with the last products, `more` (P of each page lies
      // over its own half of S; it comes in two parts, the first 32 keys of both
      // pages and the others, so that the first products overlap the rest of
      // the softmax)
      auto pv = [&](int qt, uint32_t j, bool first, uint32_t& par, auto&& more) {
        const uint32_t dv = dv0 + (j & 1) * (C::kTile >> 4);
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
                         desc(dv + ((k * 2048) >> 4)), idesc_pv, !first || part + i > 0);
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
          ks ^= 1;
          if (ks == 0) k_par ^= 1;
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
            // (the wait for K of the next tile comes behind the products of this)
            pv(0, j, t == 0, p0, [&] {
              if (next) {
                wait(sm.k_full[ks], k_par);
                tc_fence_after_sync();
                qk(0, ks, 0);
              } else {
                mma_commit(smem_addr(&sm.o_full[0]));
              }
            });
            pv(1, j, t == 0, p1, [&] {
              if (next) {
                qk(1, ks, 1);
                mma_commit(smem_addr(&sm.k_empty[ks]));
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
            auto more = [&](int qt) {
              mma_commit(smem_addr(&sm.v_empty[j & 1]));
              if (next) {
                wait(sm.k_full[ks], k_par);
                tc_fence_after_sync();
                qk(qt, ks, 0);
                mma_commit(smem_addr(&sm.k_empty[ks]));
              } else {
                mma_commit(smem_addr(&sm.o_full[qt]));
              }
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
    }
  } else if (warp < 8) {
    setmaxnreg_dec<kWidenRegs>();
    {
      // ==== K and V to f16: a thread is half a key of each page ====
      const int key = tid & 63, hf = (tid >> 6) & 1;
      // Pieces of 32 elements, which of a row being the thread's own so that the
      // pieces of 8 keys lie in different banks: where they come from and go to.
      constexpr int kPieces = D / 64;
      uint32_t from[kPieces], to[kPieces];
#pragma unroll
      for (int c = 0; c < kPieces; ++c) {
        const int p = D == 128 ? (hf + (key >> 1) + 2 * c) & 3 : (hf + (key >> 2)) & 1;
        from[c] = key * (D / 2) + p * 16;
        to[c] = p / 2 * kSlab + key * 128 + ((p % 2 * 4) ^ (key & 7)) * 16;
      }
      uint32_t j = 0, st = 0, st_par = 0;
      for (uint32_t n_items = 0;; ++n_items) {
        const int s = n_items & 1;
        wait(sm.item_full[s], (n_items >> 1) & 1);
        if (__any_sync(0xFFFFFFFFu, *dead != 0)) break;
        const int b = sm.items[s].b, t0 = sm.items[s].t_begin, t1 = sm.items[s].t_end;
        const int klo = sm.items[s].klo, khi = sm.items[s].khi;
        // the item's rows of q into L2, while the one before is worked on
        if (b >= 0) {
          const int cu0 = sm.items[s].cu0, h = sm.items[s].h, r0 = sm.items[s].r0, nrows = sm.items[s].nrows;
          for (int rr = tid - 128; rr < nrows; rr += 128) {
            const uint16_t* row = static_cast<const uint16_t*>(a.q) +
                                  static_cast<int64_t>(cu0 + (r0 + rr) / G) * a.q_token_stride +
                                  static_cast<int64_t>(h * G + (r0 + rr) % G) * a.q_head_stride;
            prefetch_l2_line(row);
            if (D == 128) prefetch_l2_line(row + 64);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sm.item_empty[s]));
        if (b < 0) break;
        for (int t = t0; t < t1; ++t, ++j) {
          uint8_t* const tile = k_s + (j & 1) * C::kTile;
          // keys of the tile that some row sees: [lo, hi)
          const int lo = klo - t * kTileKeys, hi = khi - t * kTileKeys;
#pragma unroll 1
          for (int side = 0; side < 2; ++side) {          // K, V
            uint4 w[2][kPieces];
            uint32_t sc[2][kPieces];
            // (a side that was given up frees no stage, and its block is at its last item)
            if (!__all_sync(0xFFFFFFFFu, wait(sm.raw_full[st], st_par))) {
              t = t1;
              break;
            }
            const uint8_t* const src = raw_s + st * C::kSide;
#pragma unroll
            for (int pg = 0; pg < 2; ++pg) {
#pragma unroll
              for (int c = 0; c < kPieces; ++c) {
                w[pg][c] = *reinterpret_cast<const uint4*>(src + pg * C::kCodes + from[c]);
                sc[pg][c] = *reinterpret_cast<const uint16_t*>(src + 2 * C::kCodes + pg * C::kScales + from[c] / 8);
              }
              const bool gone = sm.gone[j & 7][pg] != 0;
              if (gone || pg * kPage < lo || pg * kPage + kPage > hi) {
                // a key that no row sees may hold a NaN scale, which a weight of
                // zero would not silence
                const bool live = !gone && pg * kPage + key >= lo && pg * kPage + key < hi;
#pragma unroll
                for (int c = 0; c < kPieces; ++c) sc[pg][c] = live ? sc[pg][c] : 0u;
              }
            }
            // (the stage goes back before its codes are worked on)
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sm.raw_empty[st]));
            if (++st == NR) {
              st = 0;
              st_par ^= 1;
            }
            wait(side == 0 ? sm.k_empty[j & 1] : sm.v_empty[j & 1], ((j >> 1) & 1) ^ 1);
            uint8_t* const o = tile + side * (2 * C::kTile);
#pragma unroll
            for (int pg = 0; pg < 2; ++pg)
#pragma unroll
              for (int c = 0; c < kPieces; ++c) {
                const __half2 s2 = bits_h2(e4m3x2_to_f16x2(sc[pg][c]));
                auto put = [&](int u, uint32_t x, __half2 f) {
                  uint32_t h[4];
                  scaled8(x, f, h);
                  *reinterpret_cast<uint4*>(o + pg * (kPage * 128) + (to[c] ^ (u * 16))) = make_uint4(h[0], h[1], h[2], h[3]);
                };
                put(0, w[pg][c].x, __low2half2(s2));
                put(1, w[pg][c].y, __low2half2(s2));
                put(2, w[pg][c].z, __high2half2(s2));
                put(3, w[pg][c].w, __high2half2(s2));
              }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(side == 0 ? &sm.k_full[j & 1] : &sm.v_full[j & 1]));
          }
        }
      }
    }
  } else {
    // ==== softmax: a thread is half a row, 64 keys of a tile ====
    setmaxnreg_inc<kSoftmaxRegs>();
    const int qt = (warp - 8) >> 3, half = ((warp - 8) >> 2) & 1;
    const int bar = 1 + qt * 4 + (warp & 3);              // the two warps of 32 rows
    const int bar_rows = 9 + (warp & 3);                  // and those of the other row tile
    const int wrow = (warp & 3) * 32, row = wrow + lane;  // of the row tile
    const uint32_t lanes = static_cast<uint32_t>(wrow) << 16;
    const uint32_t s_tm = tmem + qt * 128 + half * 64 + lanes;
    const uint32_t o_tm = tmem + 256 + qt * 128 + half * (D / 2) + lanes;
    uint8_t* const q_mine = q_s + qt * C::kTile;
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
        // 16 of the warp's rows of q (the other half's warp has the others) as f16,
        // kTpr threads a row
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
          uint32_t m = widen16<F16>(w, y);
          w[0] = w_next[0];
          w[1] = w_next[1];
          fetch(p + 2, w_next);
#pragma unroll
          for (int off = 1; off < kTpr; off <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
          const int e = q_exponent(m);
          const bool odd = m >= 0x7F800000u;              // a NaN or an infinity: NaN in its row
          if (part == 0)
            sm.qf[qt][rr] = odd ? __uint_as_float(0x7FC00000u) : fabsf(a.sm_scale) * 1.4426950408889634f * pow2f(e);
          const float f = sign * pow2f(-e);
          uint32_t o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = odd ? 0u : h2_bits(__floats2half2_rn(y[2 * i] * f, y[2 * i + 1] * f));
          uint8_t* const to = q_mine + (part / 4) * kSlab + rr * 128;
#pragma unroll
          for (int i = 0; i < 2; ++i)
            *reinterpret_cast<uint4*>(to + ((part % 4 * 2 + i) ^ (rr & 7)) * 16) =
                make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sm.q_full[qt]));
      }
      // qf is there for the warps that read it
      if (shared) named_sync(bar_rows, 128);
      else named_sync(bar, 64);
      const float qf = nt > 0 ? sm.qf[shared ? 0 : qt][row] : 0.0f;
      const bool odd = qf != qf;
      // (at least 2^-126, so that a masked -inf stays one where the scale is 0)
      const float f = odd ? 0x1p-126f : fmaxf(qf, 0x1p-126f);
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
        wait(sm.gone_full[jt & 7], (jt >> 3) & 1);
        const bool gone = sm.gone[jt & 7][half] != 0;
        wait(sm.s_full[qt], n_mine & 1);
        tc_fence_after_sync();
        float x[64];
        tmem_ld32(s_tm, reinterpret_cast<uint32_t(&)[32]>(x[0]));
        tmem_ld32(s_tm + 32, reinterpret_cast<uint32_t(&)[32]>(x[32]));
        float m[4];
        tmem_wait_ld32(reinterpret_cast<uint32_t(&)[32]>(x[0]));
        tmem_wait_ld32(reinterpret_cast<uint32_t(&)[32]>(x[32]));
        if (at >= full || at < open || gone) {
          // keys of this row in the page: [a0, a0 + n)
          const int a0 = max(lo - at, 0), n = gone ? 0 : max(min(hi - at, 64) - a0, 0);
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
        float top = max3(m[0], m[1], fmaxf(m[2], m[3])) * f;
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
        const float b = 8.0f - mref;
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
        l += acc[0].x + acc[0].y;
      }
      j += nt;
      named_sync(bar, 64);                                // (`last` lies where the other half reads `top`)
      sm.last(qt, half, row) = l;
      if (half == 0) sm.last(qt, 2, row) = mref;
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
      mref = sm.last(ta, 2, row);
      l = sm.last(ta, 0, row) + sm.last(ta, 1, row);
      if (shared) {
        lb = sm.last(1, 0, row) + sm.last(1, 1, row);
        const float mb = sm.last(1, 2, row), to = fmaxf(mref, mb);
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
      // Out through the rows of q that these warps brought in (each half its own slab
      // or half of the rows: another 32 rows' warps may be at the next item's q), which
      // no product reads any more, so that the stores to memory are up to D contiguous
      // bytes: this warp's columns of 16 bits, or half of them in fp32.
      const int cols = shared ? D / 4 : D / 2, col0 = (shared ? 2 * qt + half : half) * cols;
      const uint32_t oa_tm = tmem + 256 + ta * 128 + lanes + col0, ob_tm = tmem + 256 + 128 + lanes + col0;
      auto stage = [&](int rr, int c) {
        return reinterpret_cast<uint4*>(q_mine + swizzle<3>((wrow + rr) * 128 + half * (D == 128 ? kSlab : 64) + c * 16));
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
                make_uint4(pack16<F16>(y[8 * c], y[8 * c + 1]), pack16<F16>(y[8 * c + 2], y[8 * c + 3]),
                           pack16<F16>(y[8 * c + 4], y[8 * c + 5]), pack16<F16>(y[8 * c + 6], y[8 * c + 7]));
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
  if (warp == 1) {
    // In a block that gave up, which any role may have done up to here, nothing has
    // waited for the products that are queued: they end before its memory goes away.
    if (__any_sync(0xFFFFFFFFu, *dead != 0)) {
      if (elect_one()) mma_commit(smem_addr(&sm.never));
      __syncwarp();
      mbar_wait_bounded(smem_addr(&sm.never), 0, 1000000);
      __syncwarp();
    }
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// Launch
// ---------------------------------------------------------------------------
// Rows of few4_kernel's items, and of the largest request that it takes: the
// smallest of its heights that holds every request or, where some have more than
// it can, a single token of any; 0: none.  (Its outputs are in registers: 32 rows
// of 128 or 48 of 64.)
int few_rows(int max_new, int G, int D) {
  const int64_t all = static_cast<int64_t>(max_new) * G, most = D == 64 ? 48 : 32, need = all <= most ? all : G;
  for (const int rows : {8, 16, 24, 32, 40, 48})
    if (need <= rows && rows <= most) return rows;
  return 0;
}
constexpr int kFewCtas = 2;                               // blocks an SM at most
size_t few_bytes(int rows, int D, int sms) {
  return rows == 0 ? 0 : (part_bytes(kFewCtas * sms, rows, D) + 255) / 256 * 256;
}

// Whether the units of a call's items, of so many rows, fit an int whatever the
// lengths on the device are.
bool narrow(const Gqa8AttnArgs& a, int rows, int units_a_tile, int cost) {
  const double tall = static_cast<double>(std::min<int64_t>(a.max_new, a.n_tokens)) * (a.Hq / a.Hkv) / rows + 1;
  const double tiles = static_cast<double>(a.pt_stride) / 2 + 1;
  return a.B * tall * a.Hkv * (tiles * units_a_tile + cost) < (1 << 30);
}

template <int D, int RP, typename I>
cudaError_t launch_few(const Gqa8AttnArgs& a, void* ws, cudaStream_t stream) {
  using C = FewCfg<D, RP>;
  cudaError_t e = prepare_kernel<few4_kernel<D, RP, I>>(C::kSmem, 0);
  if (e != cudaSuccess) return e;
  // (no more blocks than there can be tiles, or items where none is ever cut)
  const int64_t tiles = (a.pt_stride + 1) / 2, most = a.B * static_cast<int64_t>(a.Hkv) * (tiles <= kWhole ? 1 : tiles);
  const int blocks = static_cast<int>(std::min<int64_t>(a.num_sms * C::kCtas, most));
  const Parts p = parts_at(ws, blocks, RP, D);
  e = launch_pdl(few4_kernel<D, RP, I>, blocks, C::kThreads, C::kSmem, stream, 1, a, RP, p.tails, p.lse, p.o);
  return e != cudaSuccess ? e : launch_merge_few<D>(a, blocks, RP, p, stream);
}
template <int D, int RP>
cudaError_t launch_few(const Gqa8AttnArgs& a, cudaStream_t stream) {
  return narrow(a, RP, 1, FewCfg<D, RP>::kCost) ? launch_few<D, RP, int>(a, a.ws, stream)
                                                : launch_few<D, RP, int64_t>(a, a.ws, stream);
}

template <int D, bool F16, typename I>
cudaError_t launch_many(const Gqa8AttnArgs& a, int min_rows, void* ws, cudaStream_t stream) {
  using C = ManyCfg<D>;
  cudaError_t e = prepare_kernel<many4_kernel<D, F16, I>>(C::kSmem, kLaunchRegs);
  if (e != cudaSuccess) return e;
  const Parts p = parts_at(ws, a.num_sms, C::kRows, D);
  e = launch_pdl(many4_kernel<D, F16, I>, a.num_sms, kManyThreads, C::kSmem, stream, 1, a, min_rows, p.tails, p.lse,
                 p.o);
  return e != cudaSuccess ? e : launch_merge_many<D>(a, a.num_sms, C::kRows, p, stream);
}
template <int D, bool F16>
cudaError_t launch_many(const Gqa8AttnArgs& a, int min_rows, void* ws, cudaStream_t stream) {
  return narrow(a, ManyCfg<D>::kRows, 2, kManyCost) ? launch_many<D, F16, int>(a, min_rows, ws, stream)
                                                    : launch_many<D, F16, int64_t>(a, min_rows, ws, stream);
}

template <int D>
cudaError_t launch_d(const Gqa8AttnArgs& a, cudaStream_t stream) {
  const int G = a.Hq / a.Hkv, rows = few_rows(a.max_new, G, D);
  cudaError_t e = cudaSuccess;
  switch (rows) {
    case 8: e = launch_few<D, 8>(a, stream); break;
    case 16: e = launch_few<D, 16>(a, stream); break;
    case 24: e = launch_few<D, 24>(a, stream); break;
    case 32: e = launch_few<D, 32>(a, stream); break;
  }
  if constexpr (D == 64) {
    if (rows == 40) e = launch_few<D, 40>(a, stream);
    else if (rows == 48) e = launch_few<D, 48>(a, stream);
  }
  if (e != cudaSuccess || static_cast<int64_t>(a.max_new) * G <= rows) return e;
  void* const ws = static_cast<uint8_t*>(a.ws) + few_bytes(rows, D, a.num_sms);
  return a.f16 ? launch_many<D, true>(a, rows + 1, ws, stream) : launch_many<D, false>(a, rows + 1, ws, stream);
}

}  // namespace

cudaError_t launch_attention_gqa4(const Gqa8AttnArgs& a, cudaStream_t stream) {
  return a.D == 64 ? launch_d<64>(a, stream) : launch_d<128>(a, stream);
}

size_t attention_gqa4_workspace(int max_new, int Hq, int Hkv, int D, int num_sms) {
  const int rows = few_rows(max_new, Hq / Hkv, D);
  const bool many = static_cast<int64_t>(max_new) * (Hq / Hkv) > rows;
  return few_bytes(rows, D, num_sms) + (many ? part_bytes(num_sms, ManyCfg<128>::kRows, D) : 0);
}

}  // namespace kv4
