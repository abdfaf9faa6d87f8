// Attention weight of every cached token: weights[b, t] += sum over the request's query rows of
// exp(scale * <q, kv_t> - lse).  C entries at the end (declared in mla.h).

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <stdint.h>

#include <cfloat>
#include <cmath>
#include <cstddef>
#include <mutex>

#include "mla_kernels.h"
#include "mla_ptx.cuh"

namespace mla {
namespace {

struct WeightsParams {
  const __nv_bfloat16* q;
  const float* lse;
  const void* kv;
  float kv_scale;
  int64_t num_blocks;
  const int32_t* block_table;
  int max_blocks;
  const int32_t* seqlens;
  int B, s_q, H, rows, causal;
  int slots;                 // largest length: min(64 max_blocks, weights_stride)
  float scale_hi, scale_lo;  // softmax_scale * log2(e) (times kv_scale) as a float pair, both > 0
  float* weights;
  int64_t weights_stride;
  int* status;
  int withhold;              // test hook: every CTA's first page is not loaded
};

// A CTA holds one 128-row block of a request's queries (heads x query positions) in TMEM and streams
// the cached pages past it: S = Q K^T on tcgen05 (TMEM accumulators), then for every row
// p = exp2(S * scale - lse) and for every token the sum over the rows.  A page is 72 KiB (36 KiB in
// FP8) read once, against 9.4 MFLOP.  Measured (GPU time of a call, B = 64, H = 128):
//     bf16, 4096 tokens                       49-50 us  6.3 TB/s, 0.94 of the copy rate: HBM-bound
//     FP8, 4096 tokens                        33 us     4.9 TB/s, 0.73: q is two E4M3 terms, so bf16's MMA time for half
//                                                       the bytes.  27 pages a CTA of 1290 clk (1152 of them the tensor pipe's) are
//                                                       16.8 us at 2.07 GHz, start and end 7; the other 9 have not been traced
//     bf16, two query positions, 8192 tokens  99-106 us 5.9-6.3 TB/s: HBM and the MMAs (81.8 us at the pipe's rate)
// Called for seconds on end, the last two run into the power limit (1.35 kW): 35 to 37 us, and 114 to 124 from board to board.
//  * Rows on the TMEM lanes, tokens on the columns: Q is loaded once per request, and the ring has the
//    whole of shared memory for pages (221 KiB: what is in flight covers HBM latency).  Q comes through the ring
//    too: read from global memory by its threads, 1152 bytes apart, it took 9.5 us instead of 2.4.
//  * One TMA box a page: boxes of three chunks with a barrier pair each refill the ring earlier, but cost more
//    (54 us against 51 at 4096 tokens).
//  * S is read with four of the rows in a lane, so that the sum over the rows is three additions in the
//    lane, a butterfly over eight lanes that halves the columns with every step (7 shuffles; with one row a
//    lane it is 31, whose issue slots the MMA warp misses), and four partial sums in shared memory, which a
//    warp of its own adds to the weights: a fixed order.
//  * More than 128 rows: a cluster of ceil(rows / 128) CTAs walks the same pages, each with its row
//    block; the others hand their 64 sums a page to CTA 0 through distributed shared memory.
//  * Two CTAs whose row blocks share pages make a pair: one MMA of 256 rows (cta_group::2), for which each
//    loads half of a page's tokens.  That halves what a page costs in L2 reads and shared memory: two query positions took 111
//    us where they take 101, each CTA with whole pages.  Three row blocks stay single: padded to two pairs, a third
//    fewer clusters fit (16 requests of 8192 tokens 54.0 us, where single ones took 43.1 on the same board).
//  * bf16, one row block: a page's scores come from three accumulators of 12 MMA steps each (kBlockParts says why).
//  * Work: all requests' pages in a row, with kSwitchPages for each request's start, cut evenly over the
//    clusters that fit the GPU.  Each CTA finds its own piece from the lengths (no schedule, no metadata).
constexpr int kWThreads = 352;                 // warp 0: TMA, 1: MMA, 2..9: exponentials, 10: sums
constexpr int kEpiWarps = 8;
constexpr int kSBufs = 3;                      // S accumulators in TMEM
constexpr int kPartBufs = 4;                   // pages of partial sums between the epilogue and the sum warp
constexpr uint32_t kQCol = 0, kSCol0 = 320;    // TMEM columns: Q [0, 288), S at 320, 384, 448
constexpr int kRecvRows = 12;                  // cluster: 64-token sums in flight towards CTA 0: a slot takes cl - 1
constexpr uint64_t kTimeoutNs = 500ull * 1000 * 1000;

// 16 consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

template <bool F8, bool Pair, int Parts = 1>
struct WCfg {
  static constexpr uint32_t kTokens = Pair ? 32 : 64;           // of a page that a CTA loads
  static constexpr uint32_t kChunk = kTokens * 128;             // 128 bytes of each, 128-byte swizzle
  static constexpr uint32_t kKChunks = F8 ? 5 : 9;
  static constexpr uint32_t kStageBytes = kKChunks * kChunk;    // (FP8: the RoPE codes zero-padded)
  static constexpr int kStages = (F8 ? 5 : 3) * (Pair ? 2 : 1);
  static constexpr int kQItems = (F8 ? 4 : 2) * (Pair ? 2 : 1); // a row block's q in ring items of kQRows rows
  static constexpr int kQRows = 128 / kQItems;
  static constexpr uint32_t kEpiArrivals = kEpiWarps * (Pair ? 2 : 1);   // where a pair's epilogue warps all arrive
  static constexpr uint32_t kQItemBytes = static_cast<uint32_t>(kQRows) * kDimQK * 2;
  // what a switch of requests costs (Q's load and its way into TMEM), in pages: the split charges it.  bf16: 128 requests
  // of up to 400 tokens 12.3 us with 2 and 13.7 with 4 (two query positions 16.5 and 17.1), 64 x 4096 49.0 and 49.5; FP8: 128 of
  // up to 8192 72.8 us with 2, 70.4 with 5, 71.2 with 8, two query positions over 64 of up to 8192 66.8, 64.0 and 64.2
  static constexpr int kSwitchPages = F8 ? 5 : 2;
  static constexpr int kParts = Parts;   // accumulators that a page's scores are added up from, a run of its chunks each
  static_assert(kParts == 1 || kKChunks % kParts == 0, "equal parts");
  static_assert(kQRows * 128 % 1024 == 0 && kStageBytes % 1024 == 0, "swizzled rows start where the swizzle does");
  static constexpr uint32_t kOffShared = kStages * kStageBytes;
  static_assert(kQItemBytes <= kStageBytes && kQItems <= kStages, "a row block's q is resident at once");
};

struct WShared {
  uint64_t full[10], empty[10];                // (a pair's full: in its first CTA, for both halves of a page)
  uint64_t q_item[8];                          // a row block's q has arrived
  uint64_t s_full[kSBufs], s_empty[kSBufs];
  uint64_t part_full[kPartBufs], part_empty[kPartBufs];
  uint64_t q_read;                             // FP8: raw q is in TMEM, and the rows' maxima are in amax
  uint64_t q_taken;                            // FP8: q has left the ring (of both CTAs of a pair)
  uint64_t q_full, drain;
  uint64_t recv_full[kRecvRows];               // CTA 0: the other CTAs' sums have arrived
  uint64_t credit[kRecvRows];                  // the other CTAs: CTA 0 has taken what was in the slot
  uint32_t tmem_base;
  volatile int abort;
  uint32_t items, units;                       // what the MMA warp has given back and filled, when it ends
  int64_t scan[kWThreads / 32 + 1];
  int64_t offset, count;                       // this part's piece: from `offset` positions into request b0 on
  int b0;
  float amax[2][128];                          // FP8: row maxima of the two halves of q
  alignas(16) float part[kPartBufs][4][kPageTokens];   // sums over the rows of one TMEM quadrant
  alignas(16) float recv[kRecvRows][kPageTokens];
};
// pairs of sums are read, written and sent as 8 bytes
static_assert(offsetof(WShared, part) % 16 == 0 && offsetof(WShared, recv) % 16 == 0 && alignof(WShared) == 16, "alignment");
template <bool F8>
constexpr uint32_t weights_smem() { return WCfg<F8, false>::kOffShared + sizeof(WShared); }
static_assert(weights_smem<false>() <= 232448 && weights_smem<true>() <= 232448, "shared memory per CTA");
static_assert(WCfg<false, true>::kOffShared == WCfg<false, false>::kOffShared &&
              WCfg<true, true>::kOffShared == WCfg<true, false>::kOffShared && WCfg<true, true>::kStages == 10 &&
              WCfg<true, true>::kQItems == 8, "a pair's CTAs lay shared memory out as others do");

struct WMaps {
  CUtensorMap kv;     // bf16: [chunk 0..8][row][64 dims]; FP8: [chunk 0..3][row][128 codes]; box: all chunks of 64 rows
  CUtensorMap rope;   // FP8: [row][576 codes], box 128 codes x 64 rows (read at code 512)
  CUtensorMap q;      // [chunk 0..8][q row][64 dims], box kQRows rows
};

// ------------------------------------------------------------------ waits --
__device__ __forceinline__ void w_abort(WShared& sh, int* status, uint32_t cl) {
  atomicCAS(status, 0, MLA_ERR_TIMEOUT);
  for (uint32_t r = 0; r < cl; ++r) st_cluster_u32(map_to_rank(smem_u32(const_cast<int*>(&sh.abort)), r), 1u);
}
__device__ __noinline__ bool w_wait_slow(WShared& sh, uint32_t bar, uint32_t parity, int* status, uint32_t cl) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_test(bar, parity)) {
    if (sh.abort) return false;
    if (global_timer_ns() - t0 > kTimeoutNs) {
      w_abort(sh, status, cl);
      return false;
    }
  }
  return true;
}
// Bounded wait (0.5 s): false once this cluster has given up.
__device__ __forceinline__ bool w_wait(WShared& sh, uint64_t& bar, uint32_t parity, int* status, uint32_t cl) {
  const uint32_t a = smem_u32(&bar);
  if (mbar_test(a, parity)) return true;
  return w_wait_slow(sh, a, parity, status, cl);
}
__device__ __forceinline__ bool w_warp_wait(WShared& sh, uint64_t& bar, uint32_t parity, int* status, uint32_t cl) {
  return __all_sync(0xffffffffu, w_wait(sh, bar, parity, status, cl));
}
// Before a CTA leaves: waits until the phase is complete or the time is `until` (one limit for all the phases that a role
// drains, each looked at once at least); ignores the abort flag.
__device__ __noinline__ void w_drain(uint64_t& bar, uint32_t parity, uint64_t until) {
  const uint32_t a = smem_u32(&bar);
  while (!mbar_test(a, parity))
    if (global_timer_ns() > until) return;
}

// --------------------------------------------------------------- the walk --
__device__ __forceinline__ int length_of(const WeightsParams& p, int b) {   // 0 where it is out of range
  const int n = __ldg(p.seqlens + b);
  return n < 0 || n > p.slots ? 0 : n;
}
__device__ __forceinline__ int pages_of(int n) { return (n + kPageTokens - 1) / kPageTokens; }

// All requests lie on a line, each with kSwitch positions for its start and one for each of its pages; the
// line is cut evenly.  This finds the part's piece.  All threads of the CTA.
template <int kSwitch>
__device__ void find_piece(const WeightsParams& p, WShared& sh, int part, int parts) {
  auto length_on_line = [&](int b) {
    const int nb = pages_of(length_of(p, b));
    return nb ? nb + kSwitch : 0;
  };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int each = (p.B + kWThreads - 1) / kWThreads;
  const int b0 = min(p.B, tid * each), b1 = min(p.B, b0 + each);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = __ldg(p.seqlens + b);
    if ((n < 0 || n > p.slots) && blockIdx.x == 0) atomicCAS(p.status, 0, MLA_ERR_DEVICE_BOUNDS);
    mine += length_on_line(b);
  }
  int64_t s = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  if (lane == 31) sh.scan[warp] = s;
  if (tid == 0) sh.count = 0;
  __syncthreads();
  int64_t before = 0, total = 0;
  for (int w = 0; w < kWThreads / 32; ++w) {
    if (w < warp) before += sh.scan[w];
    total += sh.scan[w];
  }
  int64_t at = before + s - mine;
  const int64_t lo = total * part / parts, hi = total * (part + 1) / parts;
  if (lo < hi && lo >= at && lo < at + mine) {
    int b = b0;
    for (int on; lo >= at + (on = length_on_line(b)); ++b) at += on;
    sh.b0 = b;
    sh.offset = lo - at;
    sh.count = hi - lo;
  }
  __syncthreads();
}

struct WSegment {
  int b, n, k0, k1;   // request, its length, pages [k0, k1)
};
template <int kSwitch>
struct WWalk {
  int64_t left;     // positions of the piece still to walk
  int b, offset;    // from `offset` positions into request b on
  __device__ explicit WWalk(const WShared& sh) : left(sh.count), b(sh.b0), offset(static_cast<int>(sh.offset)) {}
  __device__ bool next(const WeightsParams& p, WSegment& s) {
    while (left > 0 && b < p.B) {
      s.b = b++;
      s.n = length_of(p, s.b);
      const int nb = pages_of(s.n), from = offset;
      if (nb == 0) continue;
      offset = 0;
      const int64_t take = left < nb + kSwitch - from ? left : nb + kSwitch - from;
      left -= take;
      s.k0 = max(0, from - kSwitch);
      s.k1 = from + static_cast<int>(take) - kSwitch;
      if (s.k1 > s.k0) return true;   // (a piece may end in a request's start)
    }
    return false;
  }
};

__device__ __forceinline__ int block_of(const WeightsParams& p, int b, int k) {   // -1 where it is out of range
  const int blk = __ldg(p.block_table + static_cast<int64_t>(b) * p.max_blocks + k);
  return blk >= 0 && blk < p.num_blocks ? blk : -1;
}

// --------------------------------------------------------------- producer --
__device__ __forceinline__ uint64_t l2_policy_evict_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// Loads of a pair: the barrier may be the other CTA's (addresses of the cluster).
__device__ __forceinline__ void pair_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z,
                                             uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;"
      :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(policy) : "memory");
}
__device__ __forceinline__ void pair_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y,
                                             uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint"
      " [%0], [%1, {%3, %4}], [%2], %5;"
      :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "l"(policy) : "memory");
}

// A pair's CTAs load half of each page's tokens each, and the first one's barrier counts both halves.  Neither half can
// be a use of the stage ahead: both CTAs' stages are given back together, once the first one's barrier has completed
// (pages) or both have taken their q.
template <bool F8, bool Pair>
__device__ void w_producer(const WeightsParams& p, const WMaps& maps, WShared& sh, uint32_t smem, uint32_t rank,
                           uint32_t cl) {
  using C = WCfg<F8, Pair>;
  WWalk<C::kSwitchPages> walk(sh);
  WSegment s;
  uint32_t i = 0, seg = 0, q_seg = 0, q_last = 0;   // q_last: the last ring item of the latest q
  int q_flying = 0;                                 // how many items of the latest q have been asked for
  const bool first = !Pair || (rank & 1) == 0;
  // A page that one CTA or pair reads need not stay in L2 (50.5 us against 53.7 for 64 requests of 4096 tokens); one that
  // several read, each by itself, has to until the last of them (145 us against 176 for two CTAs over 64 x 8192 tokens; 163
  // where they shared the loads by multicast).
  const uint64_t policy = cl == (Pair ? 2 : 1) ? l2_policy_evict_first() : l2_policy_evict_normal();
  bool ok = true;
  auto stage_free = [&]() {   // waits for the next ring stage
    const uint32_t st = i % C::kStages;
    ok = w_wait(sh, sh.empty[st], ((i / C::kStages) & 1) ^ 1, p.status, cl);
    if (ok) ++i;
    return st;
  };
  for (; ok && walk.next(p, s); ++seg) {
    // the q before has been taken, so that its items' barriers are free (a stage that has come round again says so, too)
    if (seg > 0 && i <= q_last + C::kStages &&
        !(ok = w_wait(sh, sh.empty[q_last % C::kStages], (q_last / C::kStages) & 1, p.status, cl)))
      break;
    q_flying = 0;
    q_seg = seg;
    for (int j = 0; j < C::kQItems && ok; ++j) {
      const uint32_t st = stage_free();
      if (!ok) break;
      if (first) mbar_arrive(smem_u32(&sh.full[st]));   // (nobody waits for it: the stage's phases go on)
      mbar_arrive_expect_tx(smem_u32(&sh.q_item[j]), C::kQItemBytes);
      tma_load_3d(smem + st * C::kStageBytes, &maps.q, smem_u32(&sh.q_item[j]), 0,
                  s.b * p.rows + static_cast<int>(rank) * kRowsPerPair + C::kQRows * j, 0);
      q_last = i - 1;
      q_flying = j + 1;
    }
    if (!ok) break;
    for (int k = s.k0; k < s.k1 && ok; ++k) {
      int blk = block_of(p, s.b, k);
      if (blk < 0) {   // reported; the box lies past the cache, so TMA fills it with zeros
        atomicCAS(p.status, 0, MLA_ERR_DEVICE_BOUNDS);
        blk = static_cast<int>(p.num_blocks);
      }
      const uint32_t st = stage_free();
      if (!ok) break;
      if (p.withhold && seg == 0 && k == s.k0) continue;   // test hook: this page never arrives
      const uint32_t dst = smem + st * C::kStageBytes;
      if constexpr (Pair) {
        if (first) mbar_arrive_expect_tx(smem_u32(&sh.full[st]), 2 * C::kStageBytes);
        const uint32_t bar = map_to_rank(smem_u32(&sh.full[st]), rank & ~1u);
        const int row = blk * kPageTokens + static_cast<int>(rank & 1) * static_cast<int>(C::kTokens);
        pair_load_3d(dst, &maps.kv, bar, 0, row, 0, policy);
        if constexpr (F8) pair_load_2d(dst + 4 * C::kChunk, &maps.rope, bar, kDimV, row, policy);
      } else {
        const uint32_t bar = smem_u32(&sh.full[st]);
        const int row = blk * kPageTokens;
        mbar_arrive_expect_tx(bar, C::kStageBytes);
        tma_load_3d_hint(dst, &maps.kv, bar, 0, row, 0, policy);
        if constexpr (F8) tma_load_2d_hint(dst + 4 * C::kChunk, &maps.rope, bar, kDimV, row, policy);
      }
    }
  }
  // Loads still in flight land before the CTA may exit (a pair's second CTA sees it by its stages' coming back), and so do
  // the arrivals that give the stages back.
  const uint64_t until = global_timer_ns() + kTimeoutNs;
  const uint32_t flying = i < C::kStages ? i : C::kStages;
  if (first)
    for (uint32_t j = i - flying; j < i; ++j) w_drain(sh.full[j % C::kStages], (j / C::kStages) & 1, until);
  for (int j = 0; j < q_flying; ++j) w_drain(sh.q_item[j], q_seg & 1, until);
  for (uint32_t j = i - flying; j < i; ++j) w_drain(sh.empty[j % C::kStages], (j / C::kStages) & 1, until);
}

// -------------------------------------------------------------------- MMA --
// Whether a phase is complete; unlike a wait it never suspends the thread.
__device__ __forceinline__ bool mbar_peek(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}

// One lane of the warp, the same every time.
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e;
}
// An MMA step by the lane that has `lead`, all lanes with the same operands: A in TMEM, B at shared-memory address
// 16 k_lo, 128-byte swizzle; for a pair, 128 rows of A and half of B's rows in each CTA.  The lane is elected once a
// page, not a step, and a step's address is one 32-bit addition: the issue slots that a step takes are what the
// epilogue warps leave of an SM's quarter (FP8: 33.0 -> 31.6 us; alone beside warps of FMAs, a step every 34 clk where
// it was 55).
template <bool F8, bool Pair>
__device__ __forceinline__ void mma_step(uint32_t d_tmem, uint32_t a_tmem, uint32_t k_lo, uint32_t accumulate,
                                         uint32_t lead) {
  constexpr int M = Pair ? 256 : 128;
  constexpr uint32_t idesc = F8 ? idesc_e4m3_f32(M, 64, 0, 0) : idesc_bf16_f32(M, 64, 0, 0);
  constexpr uint32_t k_hi = (1024u >> 4) | (1u << 14) | (2u << 29);   // 8 rows are 1024 bytes; version 1, 128-byte swizzle
#define MLA_MMA_STEP(GROUP, KIND)                                                                                   \
  asm volatile(                                                                                                     \
      "{\n\t.reg .pred p, e;\n\t.reg .b64 k;\n\tmov.b64 k, {%2, %3};\n\tsetp.ne.b32 p, %5, 0;\n\t"                   \
      "setp.ne.b32 e, %6, 0;\n\t@e tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], [%1], k, %4, p;\n\t}"      \
      :: "r"(d_tmem), "r"(a_tmem), "r"(k_lo), "r"(k_hi), "r"(idesc), "r"(accumulate), "r"(lead) : "memory")
  if constexpr (F8 && Pair) MLA_MMA_STEP("2", "f8f6f4");
  else if constexpr (F8) MLA_MMA_STEP("1", "f8f6f4");
  else if constexpr (Pair) MLA_MMA_STEP("2", "f16");
  else MLA_MMA_STEP("1", "f16");
#undef MLA_MMA_STEP
}
// The barrier (of a pair: in the cluster's CTAs of `mask`, at the same place in their shared memory) gets an arrival once
// all MMAs so far are complete.  Somebody in each of those CTAs has to wait for it before the CTA may leave.
template <bool Pair>
__device__ __forceinline__ void commit_step(uint32_t bar, uint32_t mask) {
  if constexpr (Pair)
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}"
        :: "r"(bar), "h"(static_cast<uint16_t>(mask)) : "memory");
  else
    mma_commit_warp(bar);
}
template <bool Pair>
__device__ __forceinline__ void weights_tmem_alloc(uint32_t dst_smem) {   // whole warp; a pair's two CTAs together
  if constexpr (Pair) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(dst_smem), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc(dst_smem, 512);
  }
}
template <bool Pair>
__device__ __forceinline__ void weights_tmem_dealloc(uint32_t taddr) {
  if constexpr (Pair)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(taddr), "r"(512) : "memory");
  else
    tmem_dealloc(taddr, 512);
}

// (of a pair: in its first CTA)
template <bool F8, bool Pair, int Parts>
__device__ void w_mma(const WeightsParams& p, WShared& sh, uint32_t smem, uint32_t rank, uint32_t cl) {
  using C = WCfg<F8, Pair, Parts>;
  const uint32_t tmem = sh.tmem_base;
  WWalk<C::kSwitchPages> walk(sh);
  WSegment s;
  uint32_t i = 0, T = 0, seg = 0;   // T: S accumulators filled
  bool ok = true;
  while (ok && walk.next(p, s)) {
    if (!(ok = w_warp_wait(sh, F8 ? sh.q_taken : sh.q_full, seg & 1, p.status, cl))) break;
    const uint32_t lane = threadIdx.x & 31;   // the epilogue warps have read the ring's q: an item a lane
    if (lane < C::kQItems) {
      const uint32_t bar = smem_u32(&sh.empty[(i + lane) % C::kStages]);
      mbar_arrive(bar);
      if (Pair) mbar_arrive_other(map_to_rank(bar, rank + 1));
    }
    i += C::kQItems;
    if (F8 && !(ok = w_warp_wait(sh, sh.q_full, seg & 1, p.status, cl))) break;
    ++seg;
    bool ready = false;   // the next part's S buffer (and stage) have been seen free during the part before
    for (int k = s.k0; k < s.k1; ++k, ++i) {
      const uint32_t st = i % C::kStages;
      const uint32_t page = (((smem + st * C::kStageBytes) >> 4) & 0x3FFF) | (1u << 16);   // (16 bytes: unused with a swizzle)
#pragma unroll
      for (int part = 0; part < C::kParts; ++part) {
        const uint32_t sb = T % kSBufs;
        if (!ready) ok = w_warp_wait(sh, sh.s_empty[sb], ((T / kSBufs) & 1) ^ 1, p.status, cl) &&
                         (part > 0 || w_warp_wait(sh, sh.full[st], (i / C::kStages) & 1, p.status, cl));
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + kSCol0 + sb * kPageTokens, lead = elect_lane();
        const int c0 = part * (C::kKChunks / C::kParts), c1 = c0 + C::kKChunks / C::kParts;
        auto chunks = [&](int first, int last) {   // the MMAs of the page's chunks [first, last)
#pragma unroll
          for (int c = first; c < last; ++c)
#pragma unroll
            for (int j = 0; j < (F8 && c == 4 ? 2 : 4); ++j) {
              const uint32_t at = page + (c * C::kChunk + j * 32) / 16;
              if constexpr (F8) {   // chunks of 128 codes, K = 32 a step; the half of q that it lies in holds hi, then lo
                const int step = 4 * c + j, col = 144 * (step / 9) + 8 * (step % 9);
                mma_step<F8, Pair>(d, tmem + kQCol + col, at, (c | j) ? 1u : 0u, lead);
                mma_step<F8, Pair>(d, tmem + kQCol + col + 72, at, 1u, lead);
              } else {
                mma_step<F8, Pair>(d, tmem + kQCol + c * 32 + j * 8, at, c > c0 || j ? 1u : 0u, lead);
              }
            }
        };
        const int look = c1 - (F8 || C::kParts > 1 ? 1 : 2);
        chunks(c0, look);
        // a look at the next part's barriers while MMAs are queued, not between two parts where the pipe would drain
        // (FP8: 31.8 -> 30.9 us)
        const bool more = part + 1 < C::kParts, next_page = k + 1 < s.k1;
        ready = (more || next_page) &&
                __all_sync(0xffffffffu,
                           mbar_peek(smem_u32(&sh.s_empty[(T + 1) % kSBufs]), (((T + 1) / kSBufs) & 1) ^ 1) &&
                               (more || mbar_peek(smem_u32(&sh.full[(i + 1) % C::kStages]), ((i + 1) / C::kStages) & 1)));
        chunks(look, c1);
        if (!more) commit_step<Pair>(smem_u32(&sh.empty[st]), 3u << rank);   // waited for by the producers, at the latest when they end
        commit_step<Pair>(smem_u32(&sh.s_full[sb]), 3u << rank);             // waited for by the epilogue warps
        ++T;
      }
      if (!ok) break;
    }
  }
  if (T > 0) {   // no MMA is in flight when the CTAs free their TMEM: said to this CTA alone, which waits for it
    commit_step<Pair>(smem_u32(&sh.drain), 1u << rank);
    w_drain(sh.drain, 0, global_timer_ns() + kTimeoutNs);
  }
  if (elect_lane()) {   // for w_settle, across the cluster's last barrier
    sh.items = i, sh.units = T;
    if (Pair) {
      st_cluster_u32(map_to_rank(smem_u32(&sh.items), rank + 1), i);
      st_cluster_u32(map_to_rank(smem_u32(&sh.units), rank + 1), T);
    }
  }
  __syncwarp();
}

// Where a wait has given up, the roles no longer wait for one another: after the cluster's last barrier, the commits'
// arrivals on their way to this CTA land (their MMAs are complete), and the other CTAs' sums, for which there is no
// barrier that would complete, get the time that a store in a cluster takes many times over.
template <bool F8, bool Pair>
__device__ __noinline__ void w_settle(WShared& sh) {
  using C = WCfg<F8, Pair>;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t j = sh.items - min(sh.items, static_cast<uint32_t>(C::kStages)); j < sh.items; ++j)
    w_drain(sh.empty[j % C::kStages], (j / C::kStages) & 1, t0 + kTimeoutNs);
  for (uint32_t j = sh.units - min(sh.units, static_cast<uint32_t>(kSBufs)); j < sh.units; ++j)
    w_drain(sh.s_full[j % kSBufs], (j / kSBufs) & 1, t0 + kTimeoutNs);
  while (global_timer_ns() - t0 < 100 * 1000) {}
}

// --------------------------------------------------------------- epilogue --
// A thread's half row of q (288 values, 36 units of 16 bytes) in its ring item: chunks of chunk_bytes, a
// row's units swizzled.
struct QHalf {
  uint32_t row, chunk_bytes;
  int u0, swizzle;
  __device__ __forceinline__ uint4 unit(int j) const {
    const int u = u0 + j;
    return ld_shared_v4(row + (u >> 3) * chunk_bytes + (((u & 7) ^ swizzle) << 4));
  }
  // Into TMEM, two bf16 values a column, from column `col` on.  Returns the largest magnitude, NaN where a value is
  // NaN (asked for by kLargest).
  template <bool kLargest>
  __device__ __forceinline__ float store(uint32_t col) const {
    __nv_bfloat162 top = __float2bfloat162_rn(0.f);
#pragma unroll
    for (int c = 0; c < 9; ++c) {
      uint32_t v[16];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 x = unit(4 * c + j);
        v[4 * j] = x.x, v[4 * j + 1] = x.y, v[4 * j + 2] = x.z, v[4 * j + 3] = x.w;
      }
      tmem_st16(col + c * 16, v);
      if (kLargest)
#pragma unroll
        for (int j = 0; j < 16; ++j) top = __hmax2_nan(top, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&v[j])));
    }
    const float lo = __low2float(top), hi = __high2float(top);
    return isnan(lo) || isnan(hi) ? NAN : fmaxf(lo, hi);
  }
};

// FP8: a thread's half row in TMEM (144 columns of two bf16 values from `col` on), turned in place into two E4M3
// terms of q 2^k, four values a column: hi = e4m3(q 2^k) in the first 72 columns, lo = e4m3(q 2^k - hi) in the
// others.  A bf16 value has 8 significant bits, of which hi holds 4 and lo the rest, so hi + lo is exact for
// values down to 2^-2 after scaling and within 2^-10 below.  It goes through fp16 pairs, two values an
// instruction (conversions of single floats, which bound it, take 3.7 us a row block, these 2.4): with the
// magnitude's exponent rebased (112 = 127 - 15, less k; smaller ones become 0, below 2^-15) a bf16 pattern
// shifted left by three bits is the fp16 one.
__device__ __forceinline__ void split_q(uint32_t col, int k) {
  const uint32_t base = static_cast<uint32_t>(112 - k) << 7, base2 = base | (base << 16);
  auto split = [&](uint32_t w) {   // hi of the pair in bits 0..15, lo in 16..31
    const __nv_bfloat162 m = __hmax2(__habs2(*reinterpret_cast<const __nv_bfloat162*>(&w)),
                                     *reinterpret_cast<const __nv_bfloat162*>(&base2));
    const uint32_t v = ((*reinterpret_cast<const uint32_t*>(&m) - base2) << 3) | (w & 0x80008000u);
    uint32_t both;
    asm("{\n\t.reg .b16 h, l;\n\t.reg .b32 b, d;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 h, %1;\n\tcvt.rn.f16x2.e4m3x2 b, h;\n\tsub.rn.f16x2 d, %1, b;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 l, d;\n\tmov.b32 %0, {h, l};\n\t}"
        : "=r"(both) : "r"(v));
    return both;
  };
  // 16 columns a step: raw columns [16 c, 16 c + 16) give hi and lo columns [8 c, 8 c + 8).  Columns are written
  // once they have been read: hi at once (8 c + 8 <= 16 c + 16), lo from the step on that has read past it.
  uint32_t lo[9][8];
#pragma unroll
  for (int c = 0; c < 9; ++c) {
    uint32_t v[16], hi[8];
    tmem_ld16(col + 16 * c, v);
    tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t a = split(v[2 * j]), b = split(v[2 * j + 1]);
      hi[j] = __byte_perm(a, b, 0x5410);
      lo[c][j] = __byte_perm(a, b, 0x7632);
    }
    tmem_st8(col + 8 * c, hi);
#pragma unroll
    for (int l = 0; l < 9; ++l)   // 72 + 8 l + 8 <= 16 c + 16, and not yet so a step before
      if (2 * c - 8 >= l && 2 * c - 10 < l) tmem_st8(col + 72 + 8 * l, lo[l]);
  }
}

// 32 columns of 16 TMEM lanes: lane l of the warp gets, in r[4 n + 2 h + e], row 8 h + l / 4, column 8 n + 2 (l % 4) + e.
__device__ __forceinline__ void tmem_ld_16x256(uint32_t taddr, float (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
        "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
      : "r"(taddr));
}
// Two floats an instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Sums over the lanes that share l % 4: lane l gets that of v[4 (l / 16) + 2 (l / 8 % 2) + l / 4 % 2].  Each step
// exchanges half of the values a lane still has with the lane `o` away, in a fixed order.
__device__ __forceinline__ float sum_lanes(float (&v)[8], int lane) {
#pragma unroll
  for (int o = 16, half = 4; o >= 4; o >>= 1, half >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int c = 0; c < half; ++c) {
      const float keep = up ? v[c + half] : v[c], give = up ? v[c] : v[c + half];
      v[c] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  return v[0];
}

struct Row {   // of the scores: p = exp2(s scale + c), both as float pairs
  float c_hi, c_lo, scale_hi, scale_lo;
  int vis;     // tokens it sees
};

// Warps 2..9.  Warp quadrant q (TMEM lanes 32 q .. 32 q + 31: the rows), half `half` of the page's columns.
// All waits are on bounded barriers (no bar.sync), so a warp that gives up leaves no other hanging.
template <bool F8, bool Pair, int Parts>
__device__ void w_epilogue(const WeightsParams& p, WShared& sh, uint32_t smem, uint32_t rank, uint32_t cl) {
  using C = WCfg<F8, Pair, Parts>;
  // an arrival for the warp that issues the MMAs: of a pair, in its first CTA.  What it orders is TMEM alone (the
  // tcgen05 fences beside it), so it releases no further than any arrival.
  auto tell_mma = [&](uint64_t& bar) {
    if constexpr (Pair) mbar_arrive_other(map_to_rank(smem_u32(&bar), rank & ~1u));
    else mbar_arrive(smem_u32(&bar));
  };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = warp & 3, half = (warp - 2) >> 2;
  const int r = quad * 32 + lane;                    // row of the block == TMEM lane
  const int g = static_cast<int>(rank) * kRowsPerPair + r;   // row of the request: i * H + h
  const uint32_t lane_base = sh.tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
  const int cb = half * 32;
  // the column whose sum sum_lanes leaves to this lane: 8 n + 2 (lane % 4) + e
  const int column = 16 * (lane >> 4) + 8 * (lane >> 3 & 1) + 2 * (lane & 3) + (lane >> 2 & 1);
  WWalk<C::kSwitchPages> walk(sh);
  WSegment s;
  uint32_t i = 0, T = 0, seg = 0;
  while (walk.next(p, s)) {
    // rows past the request's, and rows that gave no weight, see nothing
    int vis = 0;
    float c_hi = 0.f, c_lo = 0.f, scale_hi = p.scale_hi, scale_lo = p.scale_lo;
    if (g < p.rows) {
      const float lse = __ldg(p.lse + static_cast<int64_t>(s.b) * p.rows + g);
      if (lse != -INFINITY) {
        vis = p.causal ? s.n - p.s_q + g / p.H + 1 : s.n;
        // -lse * log2(e) as a float pair, so that the exponent's rounding is relative to itself
        constexpr float kL2eHi = 1.4426950216293335f, kL2eLo = 1.9259629911266175e-8f;
        c_hi = -lse * kL2eHi;
        if (isfinite(c_hi)) c_lo = fmaf(-lse, kL2eLo, fmaf(-lse, kL2eHi, -c_hi));   // (lse may be finite and c_hi not)
      }
    }
    // Q into TMEM: every MMA of the request before is complete (its last S has been waited for)
    const uint32_t item = i + static_cast<uint32_t>(r / C::kQRows);
    i += C::kQItems + static_cast<uint32_t>(s.k1 - s.k0);
    if (!w_warp_wait(sh, sh.q_item[r / C::kQRows], seg & 1, p.status, cl)) return;
    const int rl = r % C::kQRows;
    const QHalf q{smem + (item % C::kStages) * C::kStageBytes + rl * 128, C::kQRows * 128, 36 * half, rl & 7};
    const uint32_t col = lane_base + kQCol + 144 * half;
    if constexpr (F8) {
      sh.amax[half][r] = q.store<true>(col);
      tmem_wait_st();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.q_read)), tell_mma(sh.q_taken);
      if (!w_warp_wait(sh, sh.q_read, seg & 1, p.status, cl)) return;
      const float a = sh.amax[0][r], b = sh.amax[1][r];   // the row's two halves agree on its scale:
      // 2^e brings the largest magnitude into (224, 448]; a row with an infinity or a NaN gives NaN
      const bool finite = a <= 3.4e38f && b <= 3.4e38f;
      const float top = fmaxf(a, b), t = finite && top > 0.f ? fminf(448.f / top, 0x1p100f) : 1.f;
      const int e = static_cast<int>(__float_as_uint(t) >> 23) - 127;
      split_q(col, e);
      const float inv = finite ? __uint_as_float(static_cast<uint32_t>(127 - e) << 23) : NAN;
      scale_hi *= inv;   // a power of two: exact
      scale_lo *= inv;
    } else {
      q.store<false>(col);
    }
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) tell_mma(sh.q_full);
    ++seg;
    // the constants of the four rows 8 j + lane / 4 whose scores this lane gets
    Row row[4];
    int least = 0x7fffffff;   // of their numbers of visible tokens
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int from = 8 * j + (lane >> 2);
      row[j].c_hi = __shfl_sync(0xffffffffu, c_hi, from);
      row[j].c_lo = __shfl_sync(0xffffffffu, c_lo, from);
      row[j].scale_hi = F8 ? __shfl_sync(0xffffffffu, scale_hi, from) : scale_hi;
      row[j].scale_lo = F8 ? __shfl_sync(0xffffffffu, scale_lo, from) : scale_lo;
      row[j].vis = __shfl_sync(0xffffffffu, vis, from);
      least = min(least, row[j].vis);
    }
    for (int k = s.k0; k < s.k1; ++k, ++T) {
      const uint32_t buf = T % kPartBufs;
      float v[2][16];   // rows 16 h .. 16 h + 15 of the quadrant
#pragma unroll
      for (int part = 0; part < C::kParts; ++part) {
        const uint32_t unit = T * C::kParts + part, sb = unit % kSBufs;
        if (!w_warp_wait(sh, sh.s_full[sb], (unit / kSBufs) & 1, p.status, cl)) return;
        tc_fence_after();
        float x[2][16];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          tmem_ld_16x256(lane_base + (static_cast<uint32_t>(16 * h) << 16) + kSCol0 + sb * kPageTokens + cb, x[h]);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) tell_mma(sh.s_empty[sb]);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const float2 sum = part ? add2({v[h][e], v[h][e + 1]}, {x[h][e], x[h][e + 1]}) : make_float2(x[h][e], x[h][e + 1]);
            v[h][e] = sum.x, v[h][e + 1] = sum.y;
          }
      }
      const int c0 = k * kPageTokens + cb;   // token of the columns' first
      const bool whole = least - c0 >= 32;   // all 32 columns are visible to the four rows
      float total[8];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        float2 e[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x = {v[j >> 1][4 * n + 2 * (j & 1)], v[j >> 1][4 * n + 2 * (j & 1) + 1]};
          const Row& r4 = row[j];
          const float2 y = add2(fma2(x, {r4.scale_hi, r4.scale_hi}, {r4.c_hi, r4.c_hi}),
                                fma2(x, {r4.scale_lo, r4.scale_lo}, {r4.c_lo, r4.c_lo}));
          e[j] = {fast_exp2(y.x), fast_exp2(y.y)};
          if (!whole) {
            const int seen = r4.vis - (c0 + 8 * n + 2 * (lane & 3));
            e[j].x = seen > 0 ? e[j].x : 0.f;
            e[j].y = seen > 1 ? e[j].y : 0.f;
          }
        }
        const float2 sum2 = add2(add2(e[0], e[1]), add2(e[2], e[3]));
        total[2 * n] = sum2.x, total[2 * n + 1] = sum2.y;
      }
      const float sum = sum_lanes(total, lane);
      if (!w_warp_wait(sh, sh.part_empty[buf], ((T / kPartBufs) & 1) ^ 1, p.status, cl)) return;
      sh.part[buf][quad][cb + column] = sum;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.part_full[buf]));
    }
  }
}

// Two floats into another CTA's shared memory; its barrier counts their 8 bytes.
__device__ __forceinline__ void st_async_v2(uint32_t cluster_addr, float a, float b, uint32_t cluster_bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];"
               :: "r"(cluster_addr), "f"(a), "f"(b), "r"(cluster_bar) : "memory");
}
// Warp 10: adds the four quadrants' sums of a page up and takes them to the weights, or, in the other CTAs of a
// cluster, to CTA 0.  Lane l has tokens 2 l and 2 l + 1.
template <bool F8, bool Pair>
__device__ void w_sum(const WeightsParams& p, WShared& sh, uint32_t cl, uint32_t rank) {
  using C = WCfg<F8, Pair>;
  const int lane = threadIdx.x & 31;
  const uint32_t others = cl - 1, slots = cl > 1 ? kRecvRows / others : 1;
  WWalk<C::kSwitchPages> walk(sh);
  WSegment s;
  uint32_t T = 0;
  // CTA 0: each slot's barrier waits for one arrival, here, and the bytes of the other CTAs' sums
  auto expect = [&](uint32_t slot) { mbar_arrive_expect_tx(smem_u32(&sh.recv_full[slot]), others * kPageTokens * 4); };
  if (rank == 0 && static_cast<uint32_t>(lane) < slots && cl > 1) expect(lane);
  while (walk.next(p, s)) {
    for (int k = s.k0; k < s.k1; ++k, ++T) {
      const uint32_t buf = T % kPartBufs, slot = T % slots, ph = (T / slots) & 1;
      const bool page = rank == 0 && block_of(p, s.b, k) >= 0;
      if (!w_warp_wait(sh, sh.part_full[buf], (T / kPartBufs) & 1, p.status, cl)) return;
      float2 sum = {0.f, 0.f};
      float2 q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) q[j] = *reinterpret_cast<const float2*>(&sh.part[buf][j][2 * lane]);
      sum.x = (q[0].x + q[1].x) + (q[2].x + q[3].x);
      sum.y = (q[0].y + q[1].y) + (q[2].y + q[3].y);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.part_empty[buf]));
      if (cl > 1 && rank != 0) {
        if (!w_warp_wait(sh, sh.credit[slot], ph ^ 1, p.status, cl)) return;
        st_async_v2(map_to_rank(smem_u32(&sh.recv[slot * others + rank - 1][2 * lane]), 0), sum.x, sum.y,
                    map_to_rank(smem_u32(&sh.recv_full[slot]), 0));
      } else if (cl > 1) {
        if (!w_warp_wait(sh, sh.recv_full[slot], ph, p.status, cl)) return;
        for (uint32_t o = 0; o < others; ++o) {
          const float2 r = *reinterpret_cast<const float2*>(&sh.recv[slot * others + o][2 * lane]);
          sum.x += r.x, sum.y += r.y;
        }
        __syncwarp();
        if (lane == 0) expect(slot);   // before the other CTAs may send the slot's next sums
        __syncwarp();
        if (lane > 0 && static_cast<uint32_t>(lane) < cl) mbar_arrive_other(map_to_rank(smem_u32(&sh.credit[slot]), lane));
      }
      // One addition a token and call, so the order of the calls alone decides the result; as a reduction at L2 it
      // costs this warp no round trip to memory.
      const int t = k * kPageTokens + 2 * lane;
      float* const w = p.weights + s.b * p.weights_stride + t;
      if (page && t < s.n) atomicAdd(w, sum.x);
      if (page && t + 1 < s.n) atomicAdd(w + 1, sum.y);
    }
  }
  // sums on their way to CTA 0 land before it may leave: it has waited for all of them above; where it gave up, w_settle
  // waits
}

template <bool F8, bool Pair, int Parts>
__global__ void __launch_bounds__(kWThreads, 1)
mla_attn_weights_kernel(const __grid_constant__ WMaps maps, const __grid_constant__ WeightsParams p) {
  using C = WCfg<F8, Pair>;
  extern __shared__ __align__(1024) uint8_t dyn_smem[];
  const uint32_t smem = smem_u32(dyn_smem);
  if (smem & 1023u) {   // the swizzled layout needs it (no static shared memory is declared); every CTA alike
    if (threadIdx.x == 0) atomicCAS(p.status, 0, MLA_ERR_UNSUPPORTED);
    return;
  }
  WShared& sh = *reinterpret_cast<WShared*>(dyn_smem + C::kOffShared);
  const int warp = threadIdx.x >> 5;
  const uint32_t cl = static_cast<uint32_t>((p.rows + kRowsPerPair - 1) / kRowsPerPair);
  const uint32_t rank = cl > 1 ? cluster_ctarank() : 0;
  if (threadIdx.x == 0) {
    prefetch_tensormap(&maps.kv);
    prefetch_tensormap(&maps.q);
    if (F8) prefetch_tensormap(&maps.rope);
    sh.abort = 0;
    sh.items = sh.units = 0;
    for (int j = 0; j < C::kStages; ++j) {
      mbar_init(smem_u32(&sh.full[j]), 1);
      mbar_init(smem_u32(&sh.empty[j]), 1);
    }
    for (int j = 0; j < kSBufs; ++j) {
      mbar_init(smem_u32(&sh.s_full[j]), 1);
      mbar_init(smem_u32(&sh.s_empty[j]), C::kEpiArrivals);
    }
    for (int j = 0; j < kPartBufs; ++j) {
      mbar_init(smem_u32(&sh.part_full[j]), kEpiWarps);
      mbar_init(smem_u32(&sh.part_empty[j]), 1);
    }
    for (int j = 0; j < C::kQItems; ++j) mbar_init(smem_u32(&sh.q_item[j]), 1);
    mbar_init(smem_u32(&sh.q_read), kEpiWarps);
    mbar_init(smem_u32(&sh.q_taken), C::kEpiArrivals);
    mbar_init(smem_u32(&sh.q_full), C::kEpiArrivals);
    mbar_init(smem_u32(&sh.drain), 1);
    for (int j = 0; j < kRecvRows; ++j) {
      mbar_init(smem_u32(&sh.recv_full[j]), 1);
      mbar_init(smem_u32(&sh.credit[j]), 1);
    }
    fence_mbar_init();
  }
  __syncwarp();
  if (warp == 0) weights_tmem_alloc<Pair>(smem_u32(&sh.tmem_base));
  tc_fence_before();
  __syncthreads();
  if (cl > 1) cluster_sync();   // every barrier of the cluster is initialised before any remote use
  tc_fence_after();
  griddep_wait();
  griddep_launch_dependents();
  find_piece<C::kSwitchPages>(p, sh, static_cast<int>(blockIdx.x / cl), static_cast<int>(gridDim.x / cl));
  if (warp == 0) {
    if ((threadIdx.x & 31) == 0) w_producer<F8, Pair>(p, maps, sh, smem, rank, cl);
  } else if (warp == 1) {
    if (!Pair || (rank & 1) == 0) w_mma<F8, Pair, Parts>(p, sh, smem, rank, cl);
  } else if (warp < 2 + kEpiWarps) {
    w_epilogue<F8, Pair, Parts>(p, sh, smem, rank, cl);
  } else {
    w_sum<F8, Pair>(p, sh, cl, rank);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (cl > 1) cluster_sync();   // no CTA leaves while another may still touch its shared memory
  if (warp == 0) {
    tc_fence_after();
    weights_tmem_dealloc<Pair>(sh.tmem_base);
  }
  if (threadIdx.x == 32 && sh.abort) w_settle<F8, Pair>(sh);
}

// ------------------------------------------------------------------- host --
constexpr int kMaxDevices = 64;
struct WeightsDevice {
  bool ready = false;
  int clusters[2][kMaxPairsPerCluster + 1] = {};   // [fp8][CTAs of a cluster]: how many fit the GPU
};
WeightsDevice g_dev[kMaxDevices];
std::mutex g_mutex;
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

using WeightsKernel = void (*)(WMaps, WeightsParams);
// An even number of row blocks pairs up.
bool pairs_up(int cl) { return cl % 2 == 0; }
// bf16: every step that the tensor pipe adds to an accumulator truncates, which leaves a score short in proportion to the
// steps.  One row block adds its scores up from three accumulators of 12 steps (rounded sums).  Error against 64 bits and
// time, N(0, 1) q and k, with three accumulators and with one: 64 requests of 4096 tokens, 128 heads, 1.9e-7 and 5.6e-7,
// 48.9 and 48.1 us; 16 heads 3.7e-7 and 1.1e-6, 48.6 and 47.5 us; 8 requests of 1000 tokens, one head, 1.2e-6 and 3.9e-6, 8.6 and
// 8.5 us.  (Nine: 9.6e-8 and 2.5e-7, but 56 us.)  With more blocks a weight is a sum of more than 128 rows, its error 5e-7 with
// one accumulator, and the epilogue has no time for three: two query positions over 64 x 8192 tokens 116 us and
// 101, three over 16 x 8192 51 and 46.  FP8: an E4M3 product has 8 bits, so that one accumulator leaves out less (2.0e-7; 8.7e-7
// for one head).
constexpr int kBlockParts = 3;
WeightsKernel weights_kernel(bool fp8, int cl) {
  if (fp8) return pairs_up(cl) ? mla_attn_weights_kernel<true, true, 1> : mla_attn_weights_kernel<true, false, 1>;
  if (cl == 1) return mla_attn_weights_kernel<false, false, kBlockParts>;
  return pairs_up(cl) ? mla_attn_weights_kernel<false, true, 1> : mla_attn_weights_kernel<false, false, 1>;
}
cudaLaunchConfig_t weights_config(bool fp8, int clusters, int cl, cudaStream_t stream, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = pdl_config(dim3(static_cast<unsigned>(clusters * cl)), dim3(kWThreads),
                                      fp8 ? weights_smem<true>() : weights_smem<false>(), stream, attr);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cl);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.numAttrs = cl > 1 ? 2 : 1;
  return cfg;
}

// Once per device, with that device current: kernel attributes and how many clusters fit.
mla_status_t weights_setup(WeightsDevice** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return MLA_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_mutex);
  WeightsDevice& d = g_dev[dev];
  if (!d.ready) {
    if (!g_encode) {
      cudaDriverEntryPointQueryResult q;
      void* fn = nullptr;
      if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
          q != cudaDriverEntryPointSuccess || fn == nullptr)
        return MLA_ERR_CUDA;
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return MLA_ERR_CUDA;
    for (int f = 0; f < 2; ++f) {
      for (int cl = 1; cl <= 3; ++cl)   // every kernel
        if (cudaFuncSetAttribute(weights_kernel(f, cl), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(f ? weights_smem<true>() : weights_smem<false>())) != cudaSuccess)
          return MLA_ERR_CUDA;
      d.clusters[f][1] = sms;
      for (int cl = 2; cl <= kMaxPairsPerCluster; ++cl) {
        cudaLaunchAttribute attr[2];
        const cudaLaunchConfig_t cfg = weights_config(f, 1, cl, nullptr, attr);
        cudaLaunchConfig_t query = cfg;
        query.attrs = attr + 1;
        query.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&d.clusters[f][cl], weights_kernel(f, cl), &query) != cudaSuccess ||
            d.clusters[f][cl] < 1) {
          cudaGetLastError();
          return MLA_ERR_CUDA;
        }
      }
    }
    d.ready = true;
  }
  *out = &d;
  return MLA_OK;
}

template <bool F8, bool Pair>
bool encode_maps(WMaps* m, const void* kv, int64_t num_blocks, const void* q, int64_t q_rows) {
  using C = WCfg<F8, Pair>;
  const cuuint32_t es[3] = {1, 1, 1};
  auto encode = [&](CUtensorMap* map, CUtensorMapDataType type, int rank, const void* base, const cuuint64_t* dims,
                    const cuuint64_t* strides, const cuuint32_t* box) {
    return g_encode(map, type, rank, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  const cuuint64_t rows = static_cast<cuuint64_t>(num_blocks) * kPageTokens;
  bool ok;
  if (F8) {
    const cuuint64_t dims[3] = {128, rows, 4}, strides[2] = {kDimQK, 128}, rdims[2] = {kDimQK, rows}, rstrides[1] = {kDimQK};
    const cuuint32_t box[3] = {128, C::kTokens, 4}, rbox[2] = {128, C::kTokens};
    ok = encode(&m->kv, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, kv, dims, strides, box) &&
         encode(&m->rope, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, kv, rdims, rstrides, rbox);
  } else {
    const cuuint64_t dims[3] = {64, rows, 9}, strides[2] = {kDimQK * 2, 128};
    const cuuint32_t box[3] = {64, C::kTokens, 9};
    ok = encode(&m->kv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, kv, dims, strides, box);
  }
  const cuuint64_t qdims[3] = {64, static_cast<cuuint64_t>(q_rows), 9}, qstrides[2] = {kDimQK * 2, 128};
  const cuuint32_t qbox[3] = {64, static_cast<cuuint32_t>(C::kQRows), 9};
  return ok && encode(&m->q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, q, qdims, qstrides, qbox);
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

mla_status_t weights_impl(const mla_bf16_t* q, const float* lse, const void* kv_cache, bool fp8, float kv_scale,
                          int64_t num_blocks, const int32_t* block_table, int max_blocks, const int32_t* seqlens, int B,
                          int s_q, int H, float softmax_scale, int causal_s_q, float* weights, int64_t weights_stride,
                          mla_stream_t stream) {
  if (!q || !lse || !kv_cache || !block_table || !seqlens || !weights) return MLA_ERR_INVALID_ARG;
  if (B < 1 || s_q < 1 || H < 1 || num_blocks < 1 || max_blocks < 1 || weights_stride < 1) return MLA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(lse, 4) || !aligned(block_table, 4) ||
      !aligned(seqlens, 4) || !aligned(weights, 4))
    return MLA_ERR_INVALID_ARG;
  if (!std::isfinite(softmax_scale) || !(softmax_scale > 0.f)) return MLA_ERR_INVALID_ARG;
  if (fp8 && (!std::isfinite(kv_scale) || !(kv_scale > 0.f))) return MLA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(s_q) * H > kRowsPerPair * kMaxPairsPerCluster || B > kScheduleMaxB) return MLA_ERR_UNSUPPORTED;
  if (num_blocks * kPageTokens > (int64_t(1) << 31) - kPageTokens) return MLA_ERR_UNSUPPORTED;
  WeightsParams p = {};
  p.q = reinterpret_cast<const __nv_bfloat16*>(q);
  p.lse = lse;
  p.kv = kv_cache;
  p.kv_scale = kv_scale;
  p.num_blocks = num_blocks;
  p.block_table = block_table;
  p.max_blocks = max_blocks;
  p.seqlens = seqlens;
  p.B = B;
  p.s_q = s_q;
  p.H = H;
  p.rows = s_q * H;
  p.causal = causal_s_q ? 1 : 0;
  int64_t slots = static_cast<int64_t>(max_blocks) * kPageTokens;
  slots = slots < weights_stride ? slots : weights_stride;
  constexpr int64_t kMostSlots = INT32_MAX / kPageTokens * kPageTokens;   // token numbers are ints
  p.slots = static_cast<int>(slots < kMostSlots ? slots : kMostSlots);
  // The scale as it was given: the tensor pipe truncates as it adds up a score's 36 steps (18 over FP8, twice), and what
  // that leaves out depends on the partial sums (nothing, for a score of one product), so no factor makes up for it.
  // The decode's scores, and with them lse, are formed the same way.
  const double scale = static_cast<double>(softmax_scale) * 1.4426950408889634074 * (fp8 ? kv_scale : 1.0);
  // Both floats of the pair are positive: a score of -inf times either is -inf, and its exponential 0 (with a negative
  // or zero low part the sum of the two products would be NaN).
  p.scale_hi = static_cast<float>(scale);
  if (!std::isnormal(p.scale_hi)) return MLA_ERR_INVALID_ARG;
  if (static_cast<double>(p.scale_hi) > scale) p.scale_hi = std::nextafterf(p.scale_hi, 0.f);
  p.scale_lo = static_cast<float>(scale - static_cast<double>(p.scale_hi));
  const float least = p.scale_hi * 0x1p-48f;   // where the residue is (nearly) 0: far below what the pair resolves
  p.scale_lo = std::fmax(p.scale_lo, std::fmax(least, FLT_TRUE_MIN));
  p.weights = weights;
  p.weights_stride = weights_stride;
  p.status = device_status_word();
  WeightsDevice* d = nullptr;
  if (!p.status) return MLA_ERR_CUDA;
  const mla_status_t st = weights_setup(&d);
  if (st != MLA_OK) return st;
  p.withhold = take_withheld_load();
  WMaps maps = {};
  const int cl = (p.rows + kRowsPerPair - 1) / kRowsPerPair;
  const int64_t q_rows = static_cast<int64_t>(B) * p.rows;
  const auto encode = pairs_up(cl) ? (fp8 ? encode_maps<true, true> : encode_maps<false, true>)
                                   : (fp8 ? encode_maps<true, false> : encode_maps<false, false>);
  if (!encode(&maps, kv_cache, num_blocks, q, q_rows)) return MLA_ERR_CUDA;
  // no more clusters than pages there can be
  const int64_t most = static_cast<int64_t>(B) * ((p.slots + kPageTokens - 1) / kPageTokens);
  const int clusters = static_cast<int>(most < d->clusters[fp8][cl] ? most : d->clusters[fp8][cl]);
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = weights_config(fp8, clusters, cl, reinterpret_cast<cudaStream_t>(stream), attr);
  return cudaLaunchKernelEx(&cfg, weights_kernel(fp8, cl), maps, p) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" {

mla_status_t mla_attn_weights(const mla_bf16_t* q, const float* lse, const mla_bf16_t* kv_cache, int64_t num_blocks,
                              const int32_t* block_table, int max_blocks, const int32_t* seqlens, int B, int s_q, int H,
                              float softmax_scale, int causal_s_q, float* weights, int64_t weights_stride,
                              mla_stream_t stream) {
  return weights_impl(q, lse, kv_cache, false, 1.f, num_blocks, block_table, max_blocks, seqlens, B, s_q, H,
                      softmax_scale, causal_s_q, weights, weights_stride, stream);
}

mla_status_t mla_attn_weights_fp8(const mla_bf16_t* q, const float* lse, const uint8_t* kv_cache, float kv_scale,
                                  int64_t num_blocks, const int32_t* block_table, int max_blocks,
                                  const int32_t* seqlens, int B, int s_q, int H, float softmax_scale, int causal_s_q,
                                  float* weights, int64_t weights_stride, mla_stream_t stream) {
  return weights_impl(q, lse, kv_cache, true, kv_scale, num_blocks, block_table, max_blocks, seqlens, B, s_q, H,
                      softmax_scale, causal_s_q, weights, weights_stride, stream);
}

}  // extern "C"
