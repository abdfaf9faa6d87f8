// Absorbed MLA decode over the 4-bit latent cache (mla_fp4.cuh): dense, and over lists of tokens.
// C entries at the end (declared in mla.h).
//
//   s_t = scale * <q, kv_t>,  p_t = exp(s_t - max),  out = sum_t p_t kv_t[0:512] / sum_t p_t,  lse = ln sum_t exp(s_t)
//
// for every query row (head and query position) of a request, whose rows share the cached tokens.  A token is 352 bytes, and
// 2176 FLOP per row: at 128 rows 791 FLOP/B, so the tensor pipes bound it, not HBM.  The codes become fp16 on the
// way to them (code * scale is exact there; kv_scale goes into the scores and the output), and the work of a 128-row block is
// split over a CTA pair, because an output accumulator of 128 x 512 takes all of one SM's TMEM:
//   * the S-CTA (even cluster rank) computes S^T = K Q^T in tiles of 128 tokens (two pages): tokens on the TMEM lanes, so that
//     the converted keys go from the converting threads' registers straight into TMEM as the MMA's A operand (a thread
//     a token) and never through shared memory, whose bandwidth the operands need; Q is the B operand, in
//     shared memory for a whole segment.  An MMA is as wide as there are heads (rounded up to 16), so few heads cost little.
//     S^T is read with four tokens and 16 heads in a thread, which keeps the heads' references and sums in registers;
//     each softmax warp sends its 32 tokens of P^T to the partner with one shared-to-shared bulk copy a tile, and overwrites them
//     once the partner has told its warpgroup that they have landed;
//   * the O-CTA (odd rank) converts the latent part of the pages into shared memory (from L2, where its row finder has them brought)
//     and accumulates O += P V, P^T and V both read by the MMA as they lie (tokens by rows: transposed operands).
// Rows past 128 go to further pairs of the cluster, which walk the same pages.  A cluster is one part of the split schedule.
//
// Measured (GB300, 1.9 GHz; call with its merge, q and cache from HBM): 64 x 4096 tokens, 128 heads 83.9 us (870 TFLOP/s, 0.45 of a
// library's bf16 product), 16 heads 72 us; 64 x 2 x 8192: 267 us (1094 TFLOP/s); 4 x 131072: 136 us (202 us with 1% of the tokens eight
// times as large, whose references move); 64 lists of 2048 tokens: 66 us; 2 x 300 tokens, 16 heads: 16 us.  A tile takes a pair some
// 3900 cycles, of which S's MMAs are 2304 and O's 2048: what is between are the
// waits of chains (keys converted -> MMA -> exponentials -> vote -> copy -> landed -> MMA) whose links take 100 to 300 cycles each however
// little they do (the last packet's landing 400 to 800), with 20 warps on an SM that issue 0.59 of the time; TMEM, where MMAs without gaps
// hold up the others' loads and stores; and the O-CTA's shared memory (V written once and read by the MMAs with P: 2800 cycles at 128
// bytes each).
//
// The softmax is online, with the reference maximum of a head raised only where a score passes it by 2^8: the threads take the
// exponentials against the old reference, and a vote (the barrier that ends a tile) tells whether one overflowed its room;
// only then the tile is done again with new references, and O rescaled.  P is fp16 with an offset of 2^6, so that everything down to
// 2^-20 of the reference keeps 11 bits.
//
// q is bf16 and K fp16, and an MMA takes one type: each row of q is multiplied by a power of two that brings its largest
// element into [2^14, 2^15) and rounded to fp16, which is exact for elements down to 2^-31 of the largest.
//
// Every wait is bounded: a pair without progress for 0.5 s records MLA_ERR_TIMEOUT and tells every CTA of its cluster to leave, which
// they do once what they have in flight has landed.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <stdint.h>

#include <cfloat>
#include <climits>
#include <cstddef>
#include <cmath>
#include <mutex>

#include "mla_fp4.cuh"
#include "mla_kernels.h"
#include "mla_ptx.cuh"

namespace mla {
namespace {

constexpr int kThreads = 640;   // warps 0..3: loads, MMAs, copies; 4..11: softmax or rescale and epilogue; 12..19: conversion
constexpr int kTile = 128;      // tokens of a tile: two pages
constexpr uint32_t kRawPage = kPageTokens * kFp4RowBytes;
constexpr uint32_t kQChunk = 128 * 128;       // 64 dims of the row block's q: up to 128 rows of 128 bytes, swizzled
constexpr uint32_t kVChunk = 64 * 128;        // 64 dims of a page's values
constexpr int kVSlots = 4;                    // half pages (64 tokens x 256 dims) of converted values
constexpr uint32_t kVSlot = 4 * kVChunk;
// converted keys of a tile, in the order of their MMAs: latent chunks (128 tokens x 64 dims, 32 TMEM columns) in pairs, one from
// each converting warpgroup, and the rope chunk before the last pair.  The pairs have slots of their own; the rope chunk goes where the
// first pair's first chunk was, which is done with by the time that it is converted, as the rope chunk is when the next tile's first
// pair comes (a pair earlier the converters waited for the one, 83.7 us instead of 81.4; at the end for the other with 16 heads).
constexpr int kItems = 5, kRopeItem = 3;
// a packet: what one softmax warpgroup (half of the row block's heads) sends to the O-CTA for a tile
constexpr uint32_t kPktAlpha = 128 * 128;     // after P^T (128 tokens x 64 heads): float[64], factors of a rebase
constexpr uint32_t kPktFlag = kPktAlpha + 256;   // whether alpha counts
constexpr uint32_t kPktBytes = kPktFlag + 16;
constexpr uint32_t kPktStride = 17 * 1024;
// O-CTA: segments whose output factors may be there.  The S-CTA has sent at most two tiles that the MMAs are not done with, and these
// wait for the epilogue of the segment before.
constexpr uint32_t kInvSlots = 4;
constexpr uint32_t kRowSlots = 8;             // pages whose rows have been found (16: the same speed)
constexpr uint32_t kRowBytes = 4 * (kPageTokens + 1);
constexpr uint32_t kKCol = 256;               // S-CTA's TMEM columns: S^T of two tiles at 0 and 128, the keys from 256
constexpr float kOffset = 6.f;                // P is taken against 2^-6 of the reference maximum
constexpr float kTop = kOffset + 8.f;         // an exponent past this rebases its head
constexpr uint32_t kTimeoutNs = 500u * 1000 * 1000;
constexpr float kLn2 = 0.69314718055994530942f;
// Registers a thread: the three kinds of warpgroups share what the launch gets (640 x 96).  No loop may spill: with 48 / 136 / 80, where a
// converter spilled 4 to 30 bytes a thread, its loop was up to 25% slower (its fences to the other proxy seem to wait for these too).
constexpr int kRegsMisc = 64, kRegsSoftmax = 120, kRegsConvert = 88;
static_assert(128 * kRegsMisc + 256 * kRegsSoftmax + 256 * kRegsConvert <= kThreads * 96, "more would wait forever");

// shared memory (offsets from a 1024-byte aligned base)
constexpr uint32_t kOffSend = 9 * kQChunk;                   // S-CTA: q first, then a packet of each warpgroup
constexpr uint32_t kOffRaw = kOffSend + 2 * kPktStride;      // S-CTA: the two pages of a tile as cached (lists: the ring of found rows)
constexpr uint32_t kOffV = 4 * kPktStride;                   // O-CTA: the packets of two tiles first, then values
constexpr uint32_t kOffEpi = kOffV + kVSlots * kVSlot;       // O-CTA: 2 KiB transpose buffer per epilogue warp
constexpr uint32_t kOffInvL = kOffEpi + 8 * 2048;            // O-CTA: output factors of segments [kInvSlots][2][64]
constexpr uint32_t kOffRows = kOffInvL + kInvSlots * 512;    // O-CTA: the ring of found rows
constexpr uint32_t kOffShared = kOffRaw + 2 * kRawPage;
static_assert(kOffRows + kRowSlots * kRowBytes <= kOffShared, "O-CTA layout");

constexpr uint32_t kDone = 0xffffffffu;

struct Fp4Params : DecodeParams {
  float unit;  // softmax_scale * kv_scale * log2(e): log2 units of a score of codes (scale_log2 alone may pass float32's range)
  int q_box;   // q rows of a TMA box
};

struct Shared {
  // S-CTA
  uint64_t raw_full[2], raw_empty[2];         // a page of the tile has landed; is in the converters' registers
  uint64_t k_full[kItems], k_empty[kItems];   // an item of keys is in TMEM (eight warps); its MMAs are done
  uint64_t s_full[2], s_empty[2];
  uint64_t q_raw, q_full, q_empty;            // the segment's q has landed; is fp16 (a softmax warp each); is done with
  uint64_t credit[2];                         // the partner's receive slot is free (remote)
  uint64_t sent[2];                           // a warpgroup's last packet has landed, and may be overwritten here (remote)
  // O-CTA
  uint64_t p_full[2][2];                      // a slot's packet of a warpgroup has landed
  uint64_t p_free[2];
  uint64_t rows_full[kRowSlots], rows_empty[kRowSlots];   // (lists: the S-CTA's too)
  uint64_t v_full[kVSlots], v_empty[kVSlots];
  uint64_t o_full, o_free, o_sync, corr_go, corr_done;
  uint64_t inv_full[kInvSlots];               // a segment's output factors have come (64 threads of either softmax warpgroup)
  uint64_t gone;                              // the S-CTA's converters have ended (a warp each, remote)
  uint64_t drain;                             // both
  uint32_t tmem_base;
  uint32_t abort;                             // nonzero: leave
  uint32_t tiles;                             // O-CTA: tiles whose MMAs are issued, kDone at the end
  int cmd, cmd_arg;                           // O-CTA: 1 = rescale (by the packets of slot cmd_arg), 2 = epilogue, 3 = leave
  alignas(16) float q_scale[128];                         // S-CTA: raw score -> log2 units, by column
  alignas(16) float part[2][4][64];                       // a warpgroup's maxima or sums by warp and head
  alignas(16) float ref[2][64];
  uint16_t pos[128];                          // a column's query position
};
static_assert(alignof(Shared) == 16 && kOffShared % 16 == 0, "pairs of floats are read and written as 8 bytes");
constexpr uint32_t kSmemBytes = kOffShared + sizeof(Shared);
static_assert(kSmemBytes <= 232448, "shared memory per CTA");

// ------------------------------------------------------------------ waits --
// Address of a member of Shared (an element of an array of barriers: + 8 i).
#define AT(member) (smem + kOffShared + static_cast<uint32_t>(offsetof(Shared, member)))

// A wait ends when the phase is complete or the CTA has been told to give up, which the watchdog (o_watch) does after 0.5 s without
// a tile: the code around each of some twenty waits has to be short, since 20 warps of ten kinds share the instruction caches
// (64 x 4096, 128 heads: an early form took 220 us with a way out inlined at every wait, 120 with the same ways made short).  What a role does after
// a wait that gave up is harmless -- it touches the CTA's own buffers -- and each looks once a tile whether to leave.
template <bool Cluster = false>
__device__ __forceinline__ void wait(uint32_t smem, uint32_t bar, uint32_t parity) {
  if constexpr (Cluster)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 r;\nAGAIN:\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%0], %1;\n\t@p bra DONE;\n\t"
        "ld.volatile.shared.b32 r, [%2];\n\tsetp.eq.b32 q, r, 0;\n\t@q bra AGAIN;\nDONE:\n\t}"
        :: "r"(bar), "r"(parity), "r"(AT(abort)) : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 r;\nAGAIN:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%0], %1;\n\t@p bra DONE;\n\t"
        "ld.volatile.shared.b32 r, [%2];\n\tsetp.eq.b32 q, r, 0;\n\t@q bra AGAIN;\nDONE:\n\t}"
        :: "r"(bar), "r"(parity), "r"(AT(abort)) : "memory");
}
// The same, and whether the phase is complete.
__device__ __forceinline__ bool wait_done(uint32_t smem, uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b32 r;\nAGAIN:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE;\n\t"
      "ld.volatile.shared.b32 r, [%3];\n\tsetp.eq.b32 q, r, 0;\n\t@q bra AGAIN;\nDONE:\n\tselp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(done) : "r"(bar), "r"(parity), "r"(AT(abort)) : "memory");
  return done != 0;
}
// The same by a warp that goes on together.
template <bool Cluster = false>
__device__ __forceinline__ void warp_wait(uint32_t smem, uint32_t bar, uint32_t parity) {
  wait<Cluster>(smem, bar, parity);
  __syncwarp();
}
__device__ __forceinline__ bool told_to_leave(uint32_t smem) {
  uint32_t r;
  asm volatile("ld.volatile.shared.b32 %0, [%1];" : "=r"(r) : "r"(AT(abort)) : "memory");
  return r != 0;
}
__device__ __forceinline__ bool warp_told_to_leave(uint32_t smem) { return __any_sync(0xffffffffu, told_to_leave(smem)); }
__device__ __forceinline__ uint32_t timer_lo() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
  return t;
}
// Bounded wait that ignores the abort flag: for what is in flight.
__device__ __forceinline__ void drain_bar(uint32_t bar, uint32_t parity) {
  const uint32_t t0 = timer_lo();
  while (!mbar_test(bar, parity))
    if (timer_lo() - t0 > kTimeoutNs) return;
}

// ------------------------------------------------------------ instructions --
template <int R>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(R)); }
template <int R>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(R)); }
// 32 aligned bytes.
__device__ __forceinline__ void load32(const void* at, uint4& a, uint4& b) {
  asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w) : "l"(at));
}
__device__ __forceinline__ void prefetch_line(const void* at) { asm volatile("prefetch.global.L2 [%0];" :: "l"(at) : "memory"); }
// `bytes` (a multiple of 16, both addresses 16-byte aligned) of global memory into shared memory.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               :: "r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}
// 32 (x4) or 16 (x2) columns of 16 TMEM lanes: lane l of the warp gets, in r[4 n + 2 h + e], row 8 h + l / 4, column
// 8 n + 2 (l % 4) + e.
__device__ __forceinline__ void tmem_ld_16x256(uint32_t taddr, float (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
        "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_16x256(uint32_t taddr, float (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
        "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]),
        "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]),
        "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]) : "r"(taddr));
}
// Four 8 x 8 matrices of 16-bit elements: register m of lane l has row l / 4, columns 2 (l % 4) and the next, of matrix m, whose
// row r goes to the 16 bytes at lane 8 m + r's address.
__device__ __forceinline__ void stmatrix4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};"
               :: "r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void st_shared_s32(uint32_t a, int v) { asm volatile("st.shared.b32 [%0], %1;" :: "r"(a), "r"(v) : "memory"); }
__device__ __forceinline__ int ld_shared_s32(uint32_t a) {
  int v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
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
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// kind::f16 with fp16 inputs and fp32 accumulation (the bf16 descriptor without its two type bits).
__device__ __forceinline__ constexpr uint32_t idesc_f16_f32(int M, int N, int a_mn, int b_mn) {
  return idesc_bf16_f32(M, N, a_mn, b_mn) & ~((1u << 7) | (1u << 10));
}
// A value that all lanes have, as one that the compiler knows to be uniform.  An MMA takes its operands from uniform registers: issued
// by a whole warp that elects a lane, with operands known to be uniform, a step takes 50 clk; from one lane's own
// registers 70 to 140 (the pipe takes 64 for 128 x 128 x 16).
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }
// Four steps of an MMA (all lanes call), then the arrival on `bar` when they and all before them are done.
// A from TMEM (8 columns a step), B 32 bytes a step.  accumulate: whether the first step adds to what is in D.
__device__ __forceinline__ void mma4_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred p, t, e;\n\t.reg .b64 b1, b2, b3;\n\t.reg .b32 a1, a2, a3;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
      "add.s32 a1, %1, 8;\n\tadd.s32 a2, %1, 16;\n\tadd.s32 a3, %1, 24;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n\t}"
      :: "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(bar) : "memory");
}
// Eight steps: of the second four, B's chunk follows the first's.
__device__ __forceinline__ void mma8_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred p, t, e;\n\t.reg .b64 b1, b2, b3, b4, b5, b6, b7;\n\t.reg .b32 a1, a2, a3, a4, a5, a6, a7;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
      "add.s64 b4, %2, %6;\n\tadd.s64 b5, %2, %6 + 2;\n\tadd.s64 b6, %2, %6 + 4;\n\tadd.s64 b7, %2, %6 + 6;\n\t"
      "add.s32 a1, %1, 8;\n\tadd.s32 a2, %1, 16;\n\tadd.s32 a3, %1, 24;\n\tadd.s32 a4, %1, 32;\n\tadd.s32 a5, %1, 40;\n\t"
      "add.s32 a6, %1, 48;\n\tadd.s32 a7, %1, 56;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a4], b4, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a5], b5, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a6], b6, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a7], b7, %3, t;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n\t}"
      :: "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(bar), "n"(kQChunk >> 4) : "memory");
}
// Both from shared memory, 16 tokens (2 KiB) of either a step.
__device__ __forceinline__ void mma4_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred p, t, e;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "add.s64 a1, %1, 128;\n\tadd.s64 a2, %1, 256;\n\tadd.s64 a3, %1, 384;\n\t"
      "add.s64 b1, %2, 128;\n\tadd.s64 b2, %2, 256;\n\tadd.s64 b3, %2, 384;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n\t}"
      :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(bar) : "memory");
}
// 16 latent values (two words of codes) as fp16 pairs; `scale` twice in a word.
__device__ __forceinline__ void values16(uint32_t w0, uint32_t w1, uint32_t scale, uint32_t* v) {
  v[0] = mul_f16x2(e2m1x2_to_f16x2<0>(w0), scale);
  v[1] = mul_f16x2(e2m1x2_to_f16x2<1>(w0), scale);
  v[2] = mul_f16x2(e2m1x2_to_f16x2<2>(w0), scale);
  v[3] = mul_f16x2(e2m1x2_to_f16x2<3>(w0), scale);
  v[4] = mul_f16x2(e2m1x2_to_f16x2<0>(w1), scale);
  v[5] = mul_f16x2(e2m1x2_to_f16x2<1>(w1), scale);
  v[6] = mul_f16x2(e2m1x2_to_f16x2<2>(w1), scale);
  v[7] = mul_f16x2(e2m1x2_to_f16x2<3>(w1), scale);
}

// Four E4M3 scales, 0 in place of NaN: a row that sees the token is NaN by its score, and a row that does not (P = 0) stays clean.
__device__ __forceinline__ uint32_t without_nan(uint32_t scales) {
  const uint32_t nan = ((scales & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
  return scales & ~(nan | (nan - (nan >> 7)));
}

// ------------------------------------------------------------------- walk --
struct Segment {
  int b, kb, ke, split;   // request, page range, split index within the request
};

// Walks the segments of one part in order (the same walk in every role).
struct SegmentWalker {
  const Fp4Params* p;
  int b_last, k_end, b, kb, split0;
  bool first, done;
  __device__ void init(const Fp4Params& prm, int part) {
    p = &prm;
    const int* m = prm.meta + part * kMetaInts;
    b = m[0];
    kb = m[1];
    b_last = m[2];
    k_end = m[3];
    split0 = m[4];
    first = true;
    done = b < 0;
    // a record that does not fit this call would send the walk past the caller's buffers: reported, and nothing walked
    if (!done && (b >= prm.B || b_last < b || b_last >= prm.B || kb < 0 || k_end < 0 || split0 < 0)) {
      atomicCAS(prm.status, 0, MLA_ERR_DEVICE_BOUNDS);
      done = true;
    }
  }
  __device__ bool next(Segment& s) {
    while (!done) {
      if (b > b_last) {
        done = true;
        break;
      }
      const int L = __ldg(p->lens + b);
      const int nb = L > 0 ? (L - 1) / kPageTokens + 1 : 0;
      const int k0 = first ? kb : 0;
      const int k1 = b == b_last ? min(k_end, nb) : nb;
      const int sp = first ? split0 : 0;
      first = false;
      const int cur = b++;
      if (k1 > k0) {
        s.b = cur, s.kb = k0, s.ke = k1, s.split = sp;
        return true;
      }
    }
    return false;
  }
};

__device__ __forceinline__ int tiles_of(const Segment& s) { return (s.ke - s.kb + 1) >> 1; }
// Listed tokens of the tile that starts at page k.
__device__ __forceinline__ int tile_tokens(const Fp4Params& p, const Segment& s, int k) {
  return min(min(kTile, (s.ke - k) * kPageTokens), __ldg(p.lens + s.b) - k * kPageTokens);
}

// Walks the pages of one part.
struct PageIter {
  SegmentWalker w;
  Segment s;
  int k, L, L_seq;   // listed tokens and length of the segment's request
  bool valid;
  __device__ void init(const Fp4Params& p, int part) {
    w.init(p, part);
    valid = true;
    s.kb = s.ke = k = 0;
  }
  __device__ bool next(const Fp4Params& p) {   // on to the next page, the first one to begin with; a segment's last tile has two in any case
    ++k;
    if (valid && (k > s.ke || (k == s.ke && ((k - s.kb) & 1) == 0))) {
      valid = w.next(s);
      k = s.kb;
      if (valid) {
        L = __ldg(p.lens + s.b);
        L_seq = __ldg(p.seqlens + s.b);
      }
    }
    return valid;
  }
};

// Whether split slot `slot` lies in the workspace, which holds B + num_parts; one outside (metadata that does not fit the
// call) is reported and not written.
__device__ __forceinline__ bool split_slot_ok(const Fp4Params& p, int slot) {
  if (slot >= 0 && slot < p.B + p.num_parts) return true;
  atomicCAS(p.status, 0, MLA_ERR_DEVICE_BOUNDS);
  return false;
}

// Page number of page k of request b; one that is out of range is reported, and page 0 read in its place.
__device__ __forceinline__ int page_of(const Fp4Params& p, int b, int k) {
  int blk = -1;
  if (k < p.max_blocks) blk = __ldg(p.block_table + static_cast<int64_t>(b) * p.max_blocks + k);
  if (blk >= 0 && blk < p.num_blocks) return blk;
  atomicCAS(p.status, 0, MLA_ERR_DEVICE_BOUNDS);
  return 0;
}

// Finds the cached rows of every page of a part, a warp's work: a lane has rows `lane` and `lane + 32` of the page.  Its loads of a list
// entry, of that token's table entry, and the use of the row are a page apart, so that none waits for the one before.
constexpr int kListAhead = 4 * kPageTokens;   // list entries that are brought into L2 ahead of their loads
template <bool Sparse>
struct RowFinder {
  int row[2], n;   // of the page at hand: cached rows (-1: the page ends before; -2: a list or table entry is out of range), their number
  PageIter it;
  struct { int t[2], n, b, k, L_seq; bool valid; } tok;     // the page whose list entries are being loaded
  struct { int t[2], blk[2], n; bool valid; } tab;   // the one before it, whose table entries are
  int lane;
  __device__ void init(const Fp4Params& p, int part) {
    lane = threadIdx.x & 31;
    it.init(p, part);
    tok.valid = tab.valid = false;
    tok.n = tab.n = 0;
  }
  // On to the next page; false after the last.
  __device__ bool next(const Fp4Params& p) {
    bool have;
    do {
      have = tab.valid;
      if (!have && !tok.valid && !it.valid) return false;
      n = tab.n;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int r = lane + 32 * g;
        row[g] = r >= n ? -1 : tab.blk[g] < 0 || tab.blk[g] >= p.num_blocks ? -2 : tab.blk[g] * kPageTokens + (Sparse ? tab.t[g] % kPageTokens : r);
      }
      tab.valid = tok.valid;
      tab.n = tok.n;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int t = tok.t[g], k = Sparse ? t / kPageTokens : tok.k;
        tab.t[g] = t;
        tab.blk[g] = -1;
        if (lane + 32 * g < tok.n && k < p.max_blocks && (!Sparse || (t >= 0 && t < tok.L_seq)))
          tab.blk[g] = __ldg(p.block_table + static_cast<int64_t>(tok.b) * p.max_blocks + k);
      }
      tok.valid = it.next(p);
      tok.n = 0;
      if (tok.valid) {
        tok.b = it.s.b;
        tok.k = it.k;
        tok.L_seq = it.L_seq;
        if (it.k < it.s.ke) tok.n = min(kPageTokens, it.L - it.k * kPageTokens);
        if constexpr (Sparse) {
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const int r = lane + 32 * g, e = it.k * kPageTokens + r;
            const int32_t* const at = p.indices + static_cast<int64_t>(it.s.b) * p.idx_stride + e;
            tok.t[g] = r < tok.n && e < p.idx_stride ? __ldg(at) : -1;
            if (lane == 0 && e + kListAhead < min(static_cast<int64_t>(it.L), p.idx_stride)) prefetch_line(at + kListAhead);
          }
        }
      }
    } while (!have);
    return true;
  }
};

// A row block's heads: `valid` of its columns are query rows, the MMA has N (a multiple of 16), a softmax warpgroup N / 2.
struct Block {
  int rb, valid, N, half;
  __device__ Block(const Fp4Params& p, int rb_) : rb(rb_) {
    valid = min(kRowsPerPair, p.rows - rb * kRowsPerPair);
    N = (valid + 15) & ~15;
    half = N >> 1;
  }
};

// ------------------------------------------------------------------ S-CTA --
// Where q's 64 dims `c` lie: the warpgroups' chunks (c < 4, and from 4 on) in turn, the rope dims before the last pair.
__device__ __forceinline__ int q_place(int c) {
  const int k = c & 3, at = 2 * k + (c >> 2);
  return c == 8 ? 2 * kRopeItem : at < 2 * kRopeItem ? at : at + 1;
}

// Warp 0, dense: the two pages of every tile, a copy a page as far as the request has tokens (in 16 copies, with
// gaps that would spare the converters bank conflicts, a page took a microsecond longer).
__device__ void s_load(const Fp4Params& p, uint32_t smem, int part) {
  const int lane = threadIdx.x & 31;
  SegmentWalker w;
  w.init(p, part);
  Segment s;
  uint32_t i = 0;                               // pages (two a tile)
  bool withhold = p.withhold_first_load != 0;   // test hook: the first page never arrives
  while (w.next(s)) {
    const int L = __ldg(p.lens + s.b);
    const int end = s.kb + 2 * tiles_of(s);
#pragma unroll 1
    for (int k = s.kb; k < end; ++k, ++i) {
      const uint32_t h = i & 1, full = AT(raw_full) + 8 * h;
      const int n = k < s.ke ? min(kPageTokens, L - k * kPageTokens) : 0;   // rows
      const int64_t row = n > 0 ? static_cast<int64_t>(page_of(p, s.b, k)) * kPageTokens : 0;
      warp_wait(smem, AT(raw_empty) + 8 * h, ((i >> 1) & 1) ^ 1);
      if (warp_told_to_leave(smem)) goto out;
      if (withhold) {
        withhold = false;
        ++i;
        goto out;
      }
      if (lane == 0) {
        const uint32_t bytes = static_cast<uint32_t>(n) * kFp4RowBytes;
        if (n > 0) {
          mbar_arrive_expect_tx(full, bytes);
          bulk_load(smem + kOffRaw + h * kRawPage, reinterpret_cast<const uint8_t*>(p.kv) + row * kFp4RowBytes, bytes, full);
        } else {
          mbar_arrive(full);
        }
      }
      __syncwarp();
    }
  }
out:
  // Loads still in flight land before the CTA may leave: the last two pages' (the phases that their barriers were armed for last; a
  // withheld page's never comes, which costs the limit).
  if (lane == 0) {
    if (i > 0) drain_bar(AT(raw_full) + 8 * ((i - 1) & 1), ((i - 1) >> 1) & 1);
    if (i > 1) drain_bar(AT(raw_full) + 8 * (i & 1), ((i - 2) >> 1) & 1);
  }
  __syncwarp();
}

// Finds the cached rows of every page, kRowSlots pages ahead of the converters at most, and puts their numbers into a ring in shared
// memory (64 of them, and how many count; -1 on either page of a tile after the last).  The O-CTA's warp 0 also has them brought into
// L2; the S-CTA's, for lists, reports what is out of range (row 0 is read in its place, which is always there).
template <bool Sparse, bool IsS>
__device__ void find_rows(const Fp4Params& p, uint32_t smem, int part) {
  const int lane = threadIdx.x & 31;
  RowFinder<Sparse> rows;
  rows.init(p, part);
  int end = 0;
#pragma unroll 1
  for (uint32_t i = 0; end < 2; ++i) {
    if (end > 0 || !rows.next(p)) ++end;
    if (IsS && end == 0 && p.withhold_first_load != 0) break;   // test hook: the first page never arrives
    const uint32_t slot = i % kRowSlots, at = smem + (IsS ? kOffRaw : kOffRows) + slot * kRowBytes;
    warp_wait(smem, AT(rows_empty) + 8 * slot, ((i / kRowSlots) & 1) ^ 1);
    if (warp_told_to_leave(smem)) break;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int row = end > 0 ? -1 : rows.row[g];
      if (IsS && row == -2) atomicCAS(p.status, 0, MLA_ERR_DEVICE_BOUNDS);
      st_shared_s32(at + (lane + 32 * g) * 4, row >= 0 ? row : Sparse ? 0 : lane + 32 * g);
      if (!IsS && row >= 0) {
        const uint8_t* const src = reinterpret_cast<const uint8_t*>(p.kv) + static_cast<int64_t>(row) * kFp4RowBytes;
        if constexpr (Sparse) {   // (a bulk prefetch a row took longer: 104 against 90 us for 64 x 2048 listed tokens at that time)
#pragma unroll
          for (int c = 0; c < kFp4RowBytes + 127; c += 128) prefetch_line(src + min(c, kFp4RowBytes - 1));
        } else if (lane == 0 && g == 0) {
          prefetch_l2(src, rows.n * kFp4RowBytes);
        }
      }
    }
    if (lane == 0) st_shared_s32(at + 256, end > 0 ? -1 : rows.n);
    __syncwarp();
    if (lane == 0) mbar_arrive(AT(rows_full) + 8 * slot);
  }
}

// Warps 12..19: a thread a token; warpgroup c takes latent dims [256 c, 256 c + 256) and half of the rope dims.  Dense: a tile's
// codes are read into registers at once, which frees the page buffers for the next tile's loads.  Lists: a thread loads its row from
// global memory, every part as soon as the same part of the tile before has been converted (by copies of a row each into the page
// buffers 64 x 2048 listed tokens took 122 us; now 66).
template <bool Sparse>
__device__ void s_convert(const Fp4Params& p, Shared& sh, uint32_t smem, int part, int c) {
  const int quad = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  const uint32_t h = quad >> 1;                              // page of the tile
  const int r = (quad & 1) * 32 + lane;                      // row of the page
  const uint32_t raw = smem + kOffRaw + h * kRawPage + r * kFp4RowBytes;
  const uint32_t tm = sh.tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + kKCol;
  constexpr int kRow = Sparse ? 16 : 32;
  uint4 code[8], rope[2], sc;
  // lists: the next tile's row, and loads of its parts
  const uint8_t* src = nullptr;
  int n = 0, n_next = 0;   // rows that count of the thread's page, and of the next tile's (-1: none follows)
  uint32_t i = h;
  auto look_up = [&]() {
    const uint32_t slot = i % kRowSlots, at = smem + kOffRaw + slot * kRowBytes;
    warp_wait(smem, AT(rows_full) + 8 * slot, (i / kRowSlots) & 1);
    n_next = ld_shared_s32(at + 256);
    src = reinterpret_cast<const uint8_t*>(p.kv) + static_cast<int64_t>(ld_shared_s32(at + r * 4)) * kFp4RowBytes;
    __syncwarp();
    if (lane == 0) mbar_arrive(AT(rows_empty) + 8 * slot);
    i += 2;
  };
  // (a row past the page's end is row 0, read and not seen: under a condition a load would be waited for at once)
  auto load = [&](uint4* to, uint32_t offset) { load32(src + offset, to[0], to[1]); };
  auto load_scales = [&]() { sc = __ldg(reinterpret_cast<const uint4*>(src + kFp4Scales + 16 * c)); };
  SegmentWalker w;
  Segment s;
  int t = 0;               // dense: tiles of the segment to come
  if constexpr (Sparse) {
#pragma unroll
    for (int k = 0; k < 8; ++k) code[k] = make_uint4(0, 0, 0, 0);
    rope[0] = rope[1] = sc = make_uint4(0, 0, 0, 0);
    look_up();
    if (warp_told_to_leave(smem)) return;
#pragma unroll
    for (int k = 0; k < 4; ++k) load(&code[2 * k], 128 * c + 32 * k);
    load_scales();
    load(rope, kFp4Rope + 32 * c);
    n = n_next;
  } else {
    w.init(p, part);
  }
#pragma unroll 1
  for (uint32_t T = 0; Sparse ? n >= 0 : true; ++T) {
    if constexpr (Sparse) {
      look_up();
    } else {
      if (t == 0) {
        if (!w.next(s)) break;
        t = tiles_of(s);
      }
      --t;
      warp_wait(smem, AT(raw_full) + 8 * h, T & 1);
    }
    if (warp_told_to_leave(smem)) return;
    if constexpr (!Sparse) {
#pragma unroll
      for (int k = 0; k < 8; ++k) code[k] = ld_shared_v4(raw + 128 * c + 16 * k);
      sc = ld_shared_v4(raw + kFp4Scales + 16 * c);
      rope[0] = ld_shared_v4(raw + kFp4Rope + 32 * c);
      rope[1] = ld_shared_v4(raw + kFp4Rope + 32 * c + 16);
      __syncwarp();
      if (lane == 0) mbar_arrive(AT(raw_empty) + 8 * h);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t item = k < kRopeItem ? k : k + 1;
      const uint32_t empty = AT(k_empty) + 8 * (k > 0 ? item : kRopeItem);   // (the first pair's slots had the rope chunk last)
      const uint32_t sk = k == 0 ? sc.x : k == 1 ? sc.y : k == 2 ? sc.z : sc.w;
      const uint32_t s01 = e4m3x2_to_f16x2<0>(sk), s23 = e4m3x2_to_f16x2<1>(sk);
      uint32_t v[kRow];
      if constexpr (Sparse) {   // (in two halves, or registers run out)
        warp_wait(smem, empty, (T & 1) ^ 1);
        tc_fence_after();
        values16(code[2 * k].x, code[2 * k].y, __byte_perm(s01, 0, 0x1010), v);
        values16(code[2 * k].z, code[2 * k].w, __byte_perm(s01, 0, 0x3232), v + 8);
        tmem_st16(tm + (2 * k + c) * 32, v);
        values16(code[2 * k + 1].x, code[2 * k + 1].y, __byte_perm(s23, 0, 0x1010), v);
        values16(code[2 * k + 1].z, code[2 * k + 1].w, __byte_perm(s23, 0, 0x3232), v + 8);
        load(&code[2 * k], 128 * c + 32 * k);
        if (k == 3) load_scales();
        tmem_st16(tm + (2 * k + c) * 32 + 16, v);
      } else {
        values16(code[2 * k].x, code[2 * k].y, __byte_perm(s01, 0, 0x1010), v);
        values16(code[2 * k].z, code[2 * k].w, __byte_perm(s01, 0, 0x3232), v + 8);
        values16(code[2 * k + 1].x, code[2 * k + 1].y, __byte_perm(s23, 0, 0x1010), v + 16);
        values16(code[2 * k + 1].z, code[2 * k + 1].w, __byte_perm(s23, 0, 0x3232), v + 24);
        warp_wait(smem, empty, (T & 1) ^ 1);
        tc_fence_after();
        tmem_st32(tm + (2 * k + c) * 32, v);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(AT(k_full) + 8 * item);
      if (k == kRopeItem - 1) {
        const uint32_t x[8] = {rope[0].x, rope[0].y, rope[0].z, rope[0].w, rope[1].x, rope[1].y, rope[1].z, rope[1].w};
        uint32_t u[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) u[2 * j] = e4m3x2_to_f16x2<0>(x[j]), u[2 * j + 1] = e4m3x2_to_f16x2<1>(x[j]);
        if constexpr (Sparse) {
          load(rope, kFp4Rope + 32 * c);
        }
        warp_wait(smem, AT(k_empty), T & 1);   // the tile's first pair is done with
        tc_fence_after();
        tmem_st16(tm + 16 * c, u);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(AT(k_full) + 8 * kRopeItem);
      }
    }
    n = n_next;
  }
}

// Warp 1: a segment's q; then S^T = K Q^T, 36 steps of 16 dims a tile.  Its loop is what the tensor pipe waits for: few waits, and q
// lies in the keys' order.
__device__ void s_mma(const Fp4Params& p, const CUtensorMap* q_map, Shared& sh, uint32_t smem, int part, const Block& blk) {
  SegmentWalker w;
  w.init(p, part);
  Segment s;
  uint32_t T = 0, seg = 0;
  const uint32_t tmem = uniform(sh.tmem_base);
  const uint32_t idesc = uniform(idesc_f16_f32(kTile, blk.N, 0, 0));
  const uint64_t q0 = smem_desc_sw128(smem, 16, 1024);
  while (w.next(s)) {
    warp_wait(smem, AT(q_empty), (seg & 1) ^ 1);   // (the MMAs of the segment before are done)
    if (warp_told_to_leave(smem)) goto out;
    if ((threadIdx.x & 31) == 0) {   // 64 dims of the block's rows a box; rows past the request's are another's, or zeros past q's end
      mbar_arrive_expect_tx(AT(q_raw), 9u * static_cast<uint32_t>(p.q_box) * 128u);
#pragma unroll 1
      for (int c = 0; c < 9; ++c) tma_load_3d(smem + q_place(c) * kQChunk, q_map, AT(q_raw), 0, s.b * p.rows + blk.rb * kRowsPerPair, c);
    }
    __syncwarp();
    ++seg;
    warp_wait(smem, AT(q_full), (seg - 1) & 1);
#pragma unroll 1
    for (int t = tiles_of(s); t > 0; --t, ++T) {
      const uint32_t sb = T & 1;
      warp_wait(smem, AT(s_empty) + 8 * sb, ((T >> 1) & 1) ^ 1);
      if (warp_told_to_leave(smem)) goto out;
      const uint32_t d = uniform(tmem + sb * kTile);
#pragma unroll 1
      for (uint32_t it = 0; it < kItems; ++it) {
        warp_wait(smem, AT(k_full) + 8 * it, T & 1);
        tc_fence_after();
        const uint32_t bar = AT(k_empty) + 8 * it;
        if (it == kRopeItem) {
          mma4_ts(d, tmem + kKCol, q0 + 2 * kRopeItem * (kQChunk >> 4), idesc, 1u, bar);
        } else {
          const uint32_t pair = it > kRopeItem ? it - 1 : it, at = it > kRopeItem ? 2 * it - 1 : 2 * it;
          mma8_ts(d, tmem + kKCol + pair * 64, q0 + at * (kQChunk >> 4), idesc, it, bar);
        }
      }
      mma_commit_warp(AT(s_full) + 8 * sb);
    }
    mma_commit_warp(AT(q_empty));
  }
out:
  mma_commit_warp(AT(drain));   // behind everything issued
  drain_bar(AT(drain), 0);
  if (seg > 0) drain_bar(AT(q_raw), (seg - 1) & 1);   // and the last q lands before the CTA may leave
  __syncwarp();
}

// Rows of q of warpgroup w's heads, in place: bf16 as loaded to fp16, and their scores' factors.  A warp takes four rows at a time (a
// segment's first MMA waits for it: 9000 cycles for 128 rows one by one): of each 32 bytes a lane for the latent dims, of the four
// RoPE parts 16 bytes a lane.  The largest element is found in the bits, whose order is that of the absolute values (a NaN's the highest).
__device__ __forceinline__ void s_scale_q(const Fp4Params& p, Shared& sh, uint32_t smem, const Block& blk, int w, int wq, int lane) {
#pragma unroll 1
  for (int j = wq; j < blk.half; j += 16) {
    auto place = [&](int g, int chunk) {   // 16 bytes, lane % 8, of a chunk of row g
      const int n = w * blk.half + min(j + 4 * g, blk.half - 1);
      return smem + chunk * kQChunk + n * 128 + (((lane & 7) ^ (n & 7)) << 4);
    };
    auto largest = [](uint32_t top, const uint4& v) {
      return __vmaxu2(__vmaxu2(top, __vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu)), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
    };
    auto scaled = [](const uint4& v, uint32_t e) {   // (a row with an infinity or a NaN, e = 255, becomes NaN)
      const float sc = __uint_as_float((268u - e) << 23);
      const uint32_t x[4] = {v.x, v.y, v.z, v.w};
      uint32_t y[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) y[q] = e < 255 ? pack_f16x2(bf16_lo(x[q]) * sc, bf16_hi(x[q]) * sc) : 0x7E007E00u;
      return make_uint4(y[0], y[1], y[2], y[3]);
    };
    const int mine = lane >> 3;   // the row whose RoPE part the lane has
    uint4 v[4][2];
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
      for (int u = 0; u < 2; ++u) v[g][u] = ld_shared_v4(place(g, (lane >> 3) + 4 * u));
    const uint4 rope = ld_shared_v4(place(mine, 8));
    const uint32_t rope_top = largest(0u, rope);
    uint32_t e[4], rope_e = 0;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      uint32_t top = largest(largest(mine == g ? rope_top : 0u, v[g][0]), v[g][1]);
      top = __reduce_max_sync(0xffffffffu, max(top & 0xFFFFu, top >> 16));
      e[g] = max(top >> 7, 15u);   // the exponent: a factor of 2^126 at most, whose inverse is a normal number
      if (mine == g) rope_e = e[g];
    }
    __syncwarp();
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      if (j + 4 * g >= blk.half) break;
#pragma unroll
      for (int u = 0; u < 2; ++u) st_shared_v4(place(g, (lane >> 3) + 4 * u), scaled(v[g][u], e[g]));
      // what `scaled` took out of the row, into its scores (never 0 or infinite, so that scores of -inf and 0 stay what they are)
      if (lane == 0) {
        const float back = __uint_as_float(((e[g] < 255u ? e[g] : 141u) - 14u) << 23);
        sh.q_scale[w * blk.half + j + 4 * g] = fminf(fmaxf(p.unit * back, 0x1p-126f), FLT_MAX);
      }
    }
    if (j + 4 * mine < blk.half) st_shared_v4(place(mine, 8), scaled(rope, rope_e));
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(AT(q_full));
}

// Warps 4..11: warpgroup w has heads [w N/2, (w + 1) N/2) of the block.  Thread l of a warp has four of a tile's tokens (rows l / 4
// + 8 {0..3} of the warp's TMEM quadrant) and up to 16 heads (8 i + 2 (l % 4) + {0, 1}).
template <bool Sparse>
__device__ void s_softmax(const Fp4Params& p, Shared& sh, uint32_t smem, int part, const Block& blk, uint32_t peer) {
  const int t = threadIdx.x & 127, w = (threadIdx.x - 128) >> 7, wq = t >> 5, lane = t & 31, tr = lane >> 2, tc = lane & 3;
  const uint32_t bar = 1 + w;                     // named barrier of the warpgroup
  const int units = blk.half >> 3;                // of 8 heads
  const uint32_t tm = sh.tmem_base + (static_cast<uint32_t>(wq * 32) << 16) + w * blk.half;
  const uint32_t pkt = smem + kOffSend + w * kPktStride, dst = map_to_rank(smem + w * kPktStride, peer);
  const uint32_t full = map_to_rank(AT(p_full) + 8 * w, peer);
  // stmatrix: lane 8 m + r has row r of matrix m: unit m / 2 of a pair, rows 8 (m % 2) + r of 16
  const uint32_t st = pkt + (32 * wq + 8 * ((lane >> 3) & 1) + (lane & 7)) * 128, st_unit = (lane >> 4) ^ (lane & 7);
  SegmentWalker walk;
  walk.init(p, part);
  Segment s;
  uint32_t T = 0, seg = 0;
  while (walk.next(s)) {
    const int L = __ldg(p.lens + s.b);
    const int L_seq = Sparse ? __ldg(p.seqlens + s.b) : L;
    wait(smem, AT(q_raw), seg & 1);
    if (named_bar_or(bar, 128, told_to_leave(smem))) break;
    ++seg;
    s_scale_q(p, sh, smem, blk, w, wq, lane);
    if (t < 64) sh.ref[w][t] = -INFINITY;
    named_bar_sync(bar, 128);
    // score factor, offset - reference maximum (log2; -inf: none yet, exponentials are 0), sum over the thread's tokens
    float2 sl[8], nm[8], l[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sl[i] = i < units ? *reinterpret_cast<const float2*>(&sh.q_scale[w * blk.half + 8 * i + 2 * tc]) : make_float2(0.f, 0.f);
      nm[i] = make_float2(-INFINITY, -INFINITY);
      l[i] = make_float2(0.f, 0.f);
    }
    bool unset = true;   // some head of the warpgroup has no reference yet
#pragma unroll 1
    for (int k = s.kb; k < s.ke; k += 2, ++T) {
      const uint32_t sb = T & 1;
      const int ntok = min(min(kTile, (s.ke - k) * kPageTokens), L - k * kPageTokens);
      // Scores that are not seen become -inf where they lie, so that the loop below need not know: lane by token, a few tiles only
      // (with lists and several query positions, all).
      const bool masked = ntok < kTile || (p.causal && (Sparse || k * kPageTokens + kTile > L_seq - p.s_q + 1));
      int key = INT_MAX;   // the token's position; a head sees those below its limit
      if (masked) {
        const int tok = 32 * wq + lane, e = k * kPageTokens + tok;
        if (tok < ntok) key = !Sparse ? e : e < p.idx_stride ? __ldg(p.indices + static_cast<int64_t>(s.b) * p.idx_stride + e) : -1;
      }
      bool leave = !wait_done(smem, AT(s_full) + 8 * sb, (T >> 1) & 1);
      __syncwarp();
      tc_fence_after();
      if (masked) {
        if (Sparse && (key < 0 || key >= L_seq)) key = INT_MAX;   // (a bad entry is reported by the loads; the result is undefined)
#pragma unroll 1
        for (int c = 0; c < blk.half; c += 8) {
          uint32_t x[8];
          tmem_ld8(tm + sb * kTile + c, x);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (key >= (p.causal ? L_seq - p.s_q + 1 + sh.pos[w * blk.half + c + j] : INT_MAX)) x[j] = 0xff800000u;
          tmem_st8(tm + sb * kTile + c, x);
        }
        tmem_wait_st();
      }
      float2 ls[8];
      bool rebased = false;
      while (true) {   // once, or twice where references have to move
        if (!unset || rebased) {
#pragma unroll
          for (int i = 0; i < 8; ++i) ls[i] = make_float2(0.f, 0.f);
#pragma unroll 1
          for (uint32_t hf = 0; hf < 2; ++hf) {
            float x[32];   // [unit][token row 8 of 16][head 2]
            tmem_ld_16x256(tm + sb * kTile + (hf << 20), x);
            tmem_wait_ld();
#pragma unroll
            for (int ii = 0; ii < 4; ++ii) {
              if (2 * ii >= units) break;
              uint32_t pk[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) {   // unit 2 ii + q / 2, token row q % 2
                const int i = 2 * ii + (q >> 1);
                float2 y = fma2(make_float2(x[8 * ii + 2 * q], x[8 * ii + 2 * q + 1]), sl[i], nm[i]);
                y.x = fast_exp2(y.x);
                y.y = fast_exp2(y.y);
                ls[i] = add2(ls[i], y);
                pk[q] = pack_f16x2(y.x, y.y);
              }
              if (hf == 0 && ii == 0) {   // the warpgroup's last packet has landed (waited for behind more exponentials: no gain)
                leave |= !wait_done(smem, AT(sent) + 8 * w, (T & 1) ^ 1);
                __syncwarp();
              }
              stmatrix4(st + hf * (16 * 128) + (((2 * ii) ^ st_unit) << 4), pk[0], pk[1], pk[2], pk[3]);
            }
          }
          if (t == 96) asm volatile("st.shared.u32 [%0], %1;" :: "r"(pkt + kPktFlag), "r"(rebased ? 1 : 0) : "memory");
          fence_proxy_async_smem();
          tc_fence_before();
          // a P past 2^14 (no sum of four shows less): the tile again, with new references
          float top = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) top = fmaxf(top, fmaxf(ls[i].x, ls[i].y));
          leave |= !wait_done(smem, AT(credit) + 8 * sb, ((T >> 1) & 1) ^ 1);   // (most often there long since)
          if (!named_bar_or(bar, 128, (!rebased && top > 0x1p14f) || leave)) break;
        }
        if (named_bar_or(bar, 128, leave)) goto out;
        rebased = true;
#pragma unroll 1
        for (int i0 = 0; i0 < units; i0 += 4) {   // the heads' largest scores over the warp's tokens, four units at a time
          float x[2][16];
          float2 cm[4];
          tmem_ld_16x256(tm + sb * kTile + 8 * i0, x[0]);
          tmem_ld_16x256(tm + sb * kTile + 8 * i0 + (1u << 20), x[1]);
          tmem_wait_ld();
#pragma unroll
          for (int u = 0; u < 4; ++u)
            cm[u] = make_float2(fmaxf(fmaxf(x[0][4 * u], x[0][4 * u + 2]), fmaxf(x[1][4 * u], x[1][4 * u + 2])),
                                fmaxf(fmaxf(x[0][4 * u + 1], x[0][4 * u + 3]), fmaxf(x[1][4 * u + 1], x[1][4 * u + 3])));
#pragma unroll
          for (int o = 4; o <= 16; o <<= 1)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              cm[u].x = fmaxf(cm[u].x, __shfl_xor_sync(0xffffffffu, cm[u].x, o));
              cm[u].y = fmaxf(cm[u].y, __shfl_xor_sync(0xffffffffu, cm[u].y, o));
            }
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (tr == 0) *reinterpret_cast<float2*>(&sh.part[w][wq][8 * (i0 + u) + 2 * tc]) = cm[u];
        }
        named_bar_sync(bar, 128);
        leave |= !wait_done(smem, AT(sent) + 8 * w, (T & 1) ^ 1);   // (the factors below go into the packet too)
        if (t < blk.half) {   // a thread a head: its new reference, and what it makes of the sums so far
          float m = fmaxf(fmaxf(sh.part[w][0][t], sh.part[w][1][t]), fmaxf(sh.part[w][2][t], sh.part[w][3][t])) *
                    sh.q_scale[w * blk.half + t];
          if (m > FLT_MAX) m = FLT_MAX;   // a score past float32's range: its exponential is infinite, and the row NaN (not empty)
          const float old = sh.ref[w][t];
          float alpha = 1.f;
          if (old == -INFINITY ? m > -INFINITY : m + old > kTop) {
            if (old != -INFINITY) alpha = fast_exp2(kOffset - old - m);
            sh.ref[w][t] = kOffset - m;
          }
          asm volatile("st.shared.f32 [%0], %1;" :: "r"(pkt + kPktAlpha + t * 4), "f"(alpha) : "memory");
        }
        named_bar_sync(bar, 128);
        unset = false;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < units) {
            nm[i] = *reinterpret_cast<const float2*>(&sh.ref[w][8 * i + 2 * tc]);
            l[i].x *= ld_shared_f32(pkt + kPktAlpha + (8 * i + 2 * tc) * 4);
            l[i].y *= ld_shared_f32(pkt + kPktAlpha + (8 * i + 2 * tc) * 4 + 4);
            unset = unset || nm[i].x == -INFINITY || nm[i].y == -INFINITY;
          }
        unset = named_bar_or(bar, 128, unset);   // (alike for the warpgroup)
      }
      if (lane == 0) {
        mbar_arrive(AT(s_empty) + 8 * sb);   // S^T has been read
        // the warp's 32 tokens to the partner, the last warp's with the factors behind them
        bulk_copy_to_cluster(dst + sb * 2 * kPktStride + wq * 4096, pkt + wq * 4096, wq == 3 ? kPktBytes - 3 * 4096 : 4096, full + 16 * sb);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) l[i] = add2(l[i], ls[i]);
    }
    // the heads' sums over the warpgroup's threads, and a thread a head: the output's factor to the partner, and the lse
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int o = 4; o <= 16; o <<= 1) {
        l[i].x += __shfl_xor_sync(0xffffffffu, l[i].x, o);
        l[i].y += __shfl_xor_sync(0xffffffffu, l[i].y, o);
      }
      if (tr == 0) *reinterpret_cast<float2*>(&sh.part[w][wq][8 * i + 2 * tc]) = l[i];
    }
    named_bar_sync(bar, 128);
    if (t < 64) {
      const float sum = (sh.part[w][0][t] + sh.part[w][1][t]) + (sh.part[w][2][t] + sh.part[w][3][t]);
      const uint32_t inv = map_to_rank(smem + kOffInvL + ((seg - 1) % kInvSlots) * 512 + w * 256 + t * 4, peer);
      st_cluster_u32(inv, __float_as_uint(sum == 0.f ? 0.f : __fdividef(1.f, sum)));
      mbar_arrive_remote(map_to_rank(AT(inv_full) + 8 * ((seg - 1) % kInvSlots), peer));
      const int n = w * blk.half + t, g = blk.rb * kRowsPerPair + n;
      if (t < blk.half && n < blk.valid) {
        const float lse = sum == 0.f ? -INFINITY : (log2f(sum) - sh.ref[w][t]) * kLn2;
        const int ns0 = __ldg(p.num_splits + s.b), nsplit = __ldg(p.num_splits + s.b + 1) - ns0;
        if (nsplit == 1) p.lse[static_cast<int64_t>(s.b) * p.rows + g] = lse;
        else if (split_slot_ok(p, ns0 + s.split))   // (NaN travels as +inf, whose weight the merge makes NaN)
          p.lse_part[static_cast<int64_t>(ns0 + s.split) * p.rows + g] = isnan(lse) ? INFINITY : lse;
      }
    }
  }
out:
  __syncwarp();   // (the partner, which stays until what is on its way has landed, has this CTA stay as well)
}

// ------------------------------------------------------------------ O-CTA --
// Warps 12..19: the latent dims of every page, from global memory through registers into shared memory as fp16 (64 tokens by
// 64 dims a chunk, 128-byte swizzle).  A warpgroup has a half of the dims, a thread a row of the page (a quarter warp eight rows:
// eight different banks) and two of the half's four chunks; as soon as it has converted one it loads the same one of the next page,
// which it needs a page later.
__device__ void o_convert(const Fp4Params& p, uint32_t smem) {
  const int lane = threadIdx.x & 31, r = 16 * ((threadIdx.x >> 5) & 3) + (lane & 15), half = (threadIdx.x >> 7) - 3;
  const uint32_t chunk = lane >> 4, dims = 128 * half + 32 * chunk, scales = kFp4Scales + 16 * half + 4 * chunk;   // and the chunk two on
  const uint8_t* const kv = reinterpret_cast<const uint8_t*>(p.kv);
  const uint32_t to = smem + kOffV + half * kVSlot + chunk * kVChunk + r * 128;
  uint4 code[2][2];
  uint32_t scale[2];
  const uint8_t* src = kv;
  int n = 0, n_next = 0;   // rows that count, of this page and the next (-1: none follows)
  uint32_t i = 0;          // pages looked up
  auto look_up = [&]() {   // where the next page's row is
    const uint32_t slot = i % kRowSlots, at = smem + kOffRows + slot * kRowBytes;
    warp_wait(smem, AT(rows_full) + 8 * slot, (i / kRowSlots) & 1);
    n_next = ld_shared_s32(at + 256);
    src = kv + static_cast<int64_t>(ld_shared_s32(at + r * 4)) * kFp4RowBytes;
    __syncwarp();
    if (lane == 0) mbar_arrive(AT(rows_empty) + 8 * slot);
    ++i;
  };
  auto load = [&](int c) {
    if (r < n_next) {
      load32(src + dims + 64 * c, code[c][0], code[c][1]);
      scale[c] = __ldg(reinterpret_cast<const uint32_t*>(src + scales + 8 * c));
    }
  };
  look_up();
  if (warp_told_to_leave(smem)) return;
  load(0);
  load(1);
  n = n_next;
#pragma unroll 1
  for (uint32_t page = 0; n >= 0; ++page) {
    look_up();
    if (warp_told_to_leave(smem)) return;
    const uint32_t vs = 2 * (page & 1) + half;
    warp_wait(smem, AT(v_empty) + 8 * vs, ((page >> 1) & 1) ^ 1);
    if (n > 0) {   // (0: a tile's second page that is none)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t x[32];
        if (r < n) {
          const uint32_t sc = without_nan(scale[c]), s01 = e4m3x2_to_f16x2<0>(sc), s23 = e4m3x2_to_f16x2<1>(sc);
          values16(code[c][0].x, code[c][0].y, __byte_perm(s01, 0, 0x1010), x);
          values16(code[c][0].z, code[c][0].w, __byte_perm(s01, 0, 0x3232), x + 8);
          values16(code[c][1].x, code[c][1].y, __byte_perm(s23, 0, 0x1010), x + 16);
          values16(code[c][1].z, code[c][1].w, __byte_perm(s23, 0, 0x3232), x + 24);
        } else {   // P is 0 there, and 0 times what lies in an unused row need not be 0
#pragma unroll
          for (int j = 0; j < 32; ++j) x[j] = 0u;
        }
        load(c);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          st_shared_v4(to + (page & 1) * (2 * kVSlot) + c * (2 * kVChunk) + ((j ^ (r & 7)) << 4),
                       make_uint4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]));
      }
      fence_proxy_async_smem();
    } else {
      load(0);
      load(1);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(AT(v_full) + 8 * vs);
    n = n_next;
  }
}

// Warp 1: O += P V, for every page and 256-column half of O a step per 16 tokens.
__device__ void o_mma(const Fp4Params& p, Shared& sh, uint32_t smem, int part) {
  const int lane = threadIdx.x & 31;
  SegmentWalker w;
  w.init(p, part);
  Segment s;
  uint32_t T = 0, seg = 0, nresc = 0;
  const uint32_t tmem = uniform(sh.tmem_base);
  constexpr uint32_t idesc = idesc_f16_f32(128, 256, 1, 1);
  const uint64_t v0 = smem_desc_sw128(smem + kOffV, kVChunk, 1024);
  // A packet is expected from when the one before it in its slot has come: it completes `p_full` whatever these MMAs are at.
  if (lane < 4) mbar_arrive_expect_tx(AT(p_full) + 8 * lane, kPktBytes);
  __syncwarp();
  while (w.next(s)) {
    if (seg > 0) warp_wait(smem, AT(o_free), (seg - 1) & 1);
#pragma unroll 1
    for (int k = s.kb; k < s.ke; k += 2, ++T) {
      const uint32_t slot = T & 1, pkt = smem + slot * 2 * kPktStride, full = AT(p_full) + 16 * slot;
      const bool last = k + 2 >= s.ke;
      const int ntok = tile_tokens(p, s, k);
      warp_wait(smem, full, (T >> 1) & 1);
      warp_wait(smem, full + 8, (T >> 1) & 1);
      if (warp_told_to_leave(smem)) goto out;
      if (lane < 2) mbar_arrive_expect_tx(full + 8 * lane, kPktBytes);
      __syncwarp();
      if (k != s.kb && (ld_shared_s32(pkt + kPktFlag) | ld_shared_s32(pkt + kPktStride + kPktFlag))) {   // scale O before adding
        mma_commit_warp(AT(o_sync));
        warp_wait(smem, AT(o_sync), nresc & 1);
        if (lane == 0) {
          sh.cmd = 1;
          sh.cmd_arg = static_cast<int>(slot);
          mbar_arrive(AT(corr_go));
        }
        __syncwarp();
        warp_wait(smem, AT(corr_done), nresc & 1);
        ++nresc;
      }
      tc_fence_after();
      const uint64_t a = smem_desc_sw128(uniform(pkt), kPktStride, 1024);
      const uint32_t go_on = uniform(k != s.kb);
#pragma unroll 1
      for (uint32_t ph = 0; ph < 4; ++ph) {   // half ph % 2 of page ph / 2, in slot ph (a tile of one page leaves two slots empty)
        const int steps = (ntok - static_cast<int>(ph >> 1) * kPageTokens + 15) >> 4;
        const uint64_t pa = a + (ph >> 1) * (kPageTokens * 128 >> 4), vb = v0 + ph * (kVSlot >> 4);
        warp_wait(smem, AT(v_full) + 8 * ph, T & 1);
        tc_fence_after();
        if (steps >= 4) {
          mma4_ss(tmem + 256 * (ph & 1), pa, vb, idesc, ph > 1 ? 1u : go_on, AT(v_empty) + 8 * ph);
        } else {
#pragma unroll 1
          for (int j = 0; j < steps; ++j)
            mma_bf16_ss_warp(tmem + 256 * (ph & 1), pa + 128 * j, vb + 128 * j, idesc, j || ph > 1 ? 1u : go_on);
          mma_commit_warp(AT(v_empty) + 8 * ph);
        }
      }
      mma_commit_warp(AT(p_free) + 8 * slot);
      if (last) mma_commit_warp(AT(o_full));
      if (lane == 0) {
        if (last) {
          sh.cmd = 2;
          mbar_arrive(AT(corr_go));
        }
        asm volatile("st.volatile.shared.b32 [%0], %1;" :: "r"(AT(tiles)), "r"(T + 1) : "memory");
      }
      __syncwarp();
    }
    ++seg;
  }
  if (seg > 0) warp_wait(smem, AT(o_free), (seg - 1) & 1);   // the last epilogue has taken its command
out:
  mma_commit_warp(AT(drain));   // behind everything issued
  drain_bar(AT(drain), 0);
  if (warp_told_to_leave(smem)) {   // packets of this tile and the next may be on their way (part of them, which costs the limit)
    const uint32_t t0 = timer_lo();
    for (uint32_t j = 2 * T; j < 2 * T + 4; ++j)
      while (!mbar_test(AT(p_full) + 8 * (j & 3), (j >> 2) & 1) && timer_lo() - t0 <= kTimeoutNs) {}
  }
  __syncwarp();
  if (lane == 0) {
    sh.cmd = 3;
    mbar_arrive(AT(corr_go));
    asm volatile("st.volatile.shared.b32 [%0], %1;" :: "r"(AT(tiles)), "r"(kDone) : "memory");
  }
}

// A lane of warp 2: tells the S-CTA's warpgroups that their packets have landed (a copy to another CTA's shared memory is known to be
// done by that CTA's barrier alone: no bulk group of the sender's counts it), and gives slots back once the MMAs are done with them.
// It polls: one after the other a warpgroup would wait for the other's packet too (64 x 4096: 91.4 against 84.0 us), and its arrivals say
// that something has been read and release nothing to the cluster (with such releases 97 against 91.9 us).
__device__ void o_forward(const Fp4Params& p, uint32_t smem, int part, uint32_t peer) {
  SegmentWalker w;
  w.init(p, part);
  Segment s;
  uint32_t tiles = 0, n0 = 0, n1 = 0, nf = 0;   // tiles in all; landed packets of either warpgroup and free slots told of
  while (w.next(s)) tiles += tiles_of(s);
  const uint32_t sent = map_to_rank(AT(sent), peer), credit = map_to_rank(AT(credit), peer);
  while (n0 < tiles || n1 < tiles || nf < tiles) {
    if (n0 < tiles && mbar_poll(AT(p_full) + 16 * (n0 & 1), (n0 >> 1) & 1)) mbar_arrive_other(sent), ++n0;
    if (n1 < tiles && mbar_poll(AT(p_full) + 16 * (n1 & 1) + 8, (n1 >> 1) & 1)) mbar_arrive_other(sent + 8), ++n1;
    if (nf < tiles && mbar_poll(AT(p_free) + 8 * (nf & 1), (nf >> 1) & 1)) mbar_arrive_other(credit + 8 * (nf & 1)), ++nf;
    if (told_to_leave(smem)) return;
  }
}

// A lane of warp 3: the pair's limit on waiting.  No tile's MMAs for kTimeoutNs (every role's progress is needed for one), or the S-CTA's
// converters, which alone may wait once all tiles are done, still there so long after the last: the status word gets
// MLA_ERR_TIMEOUT, and all CTAs of the cluster are told to leave.
__device__ void o_watch(const Fp4Params& p, uint32_t smem, uint32_t cl) {
  uint32_t seen = 0, since = timer_lo();
  while (true) {
    uint32_t tiles;
    asm volatile("ld.volatile.shared.b32 %0, [%1];" : "=r"(tiles) : "r"(AT(tiles)) : "memory");
    if ((tiles == kDone && mbar_test(AT(gone), 0)) || told_to_leave(smem)) return;
    const uint32_t now = timer_lo();
    if (tiles != seen) {
      seen = tiles;
      since = now;
    } else if (now - since > kTimeoutNs) {
      atomicCAS(p.status, 0, MLA_ERR_TIMEOUT);
      for (uint32_t r = 0; r < cl; ++r) st_cluster_u32(map_to_rank(AT(abort), r), 1u);
      return;
    }
    __nanosleep(500);
  }
}

// Warps 4..11: rescale O's rows, or normalise and store a finished segment.  Warpgroup wg owns O's columns [256 wg, 256 wg + 256).
// TMEM lane m is head (m / 64) N/2 + m % 64 of the block, where m % 64 < N/2.
__device__ void o_epilogue(const Fp4Params& p, Shared& sh, uint32_t smem, int part, const Block& blk) {
  const int t = threadIdx.x - 128, wg = t >> 7, r = t & 127, wq = r >> 5, lane = r & 31;
  const uint32_t tmem_row = sh.tmem_base + (static_cast<uint32_t>(wq * 32) << 16) + wg * 256;
  const int h0 = 32 * (wq & 1), n0 = (wq >> 1) * blk.half + h0;                  // the warp's first head
  const int nrows = max(0, min(min(32, blk.half - h0), blk.valid - n0));         // its heads
  SegmentWalker w;
  w.init(p, part);
  Segment s;
  uint32_t ncmd = 0, seg = 0;
  bool have = w.next(s);
  while (true) {
    warp_wait(smem, AT(corr_go), ncmd & 1);
    if (warp_told_to_leave(smem)) break;
    ++ncmd;
    const int cmd = sh.cmd;
    if (cmd == 3) break;
    if (cmd == 1) {
      const uint32_t pkt = smem + sh.cmd_arg * 2 * kPktStride + (r >> 6) * kPktStride;
      // (a warpgroup that did not rebase sends no factors)
      const float alpha = __float_as_uint(ld_shared_f32(pkt + kPktFlag)) ? ld_shared_f32(pkt + kPktAlpha + (r & 63) * 4) : 1.f;
      tc_fence_after();
      if (__any_sync(0xffffffffu, lane < nrows && alpha != 1.f)) {
#pragma unroll 1
        for (int c = 0; c < 256; c += 32) {
          uint32_t v[32];
          tmem_ld32(tmem_row + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * alpha);
          tmem_st32(tmem_row + c, v);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(AT(corr_done));
      continue;
    }
    if (!have) break;
    warp_wait(smem, AT(o_full), seg & 1);
    tc_fence_after();
    warp_wait<true>(smem, AT(inv_full) + 8 * (seg % kInvSlots), (seg / kInvSlots) & 1);
    const float inv_l = ld_shared_f32(smem + kOffInvL + (seg % kInvSlots) * 512 + r * 4);
    const int ns0 = __ldg(p.num_splits + s.b);
    const bool final_out = __ldg(p.num_splits + s.b + 1) - ns0 == 1;
    const bool slot_ok = final_out || split_slot_ok(p, ns0 + s.split);
    // Through the warp's transpose buffer, so that a store instruction writes 64 bytes of 8 rows.  Buffer row x (64 B) holds
    // 16-byte unit u at ((u ^ ((x >> 1) & 3)) * 16): the 8 rows that a quarter-warp stores (or the 2 it loads) touch 8
    // different bank groups.
    const int64_t head0 = static_cast<int64_t>(s.b) * p.rows + blk.rb * kRowsPerPair + n0;
    __nv_bfloat16* const obase = p.out + head0 * kDimV + wg * 256;
    float* const pbase = p.o_part + (static_cast<int64_t>(ns0 + s.split) * p.rows + blk.rb * kRowsPerPair + n0) * kDimV + wg * 256;
    const uint32_t stg = smem + kOffEpi + ((wg << 2) | wq) * 2048;
    const int tq = lane & 3;                // transposed: 16-byte quad tq of rows 8 j + (lane >> 2)
    auto put = [&](int j, uint4 u) { st_shared_v4(stg + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4), u); };
    auto get = [&](int j) {
      const int x = 8 * j + (lane >> 2);
      return ld_shared_v4(stg + x * 64 + ((tq ^ ((x >> 1) & 3)) << 4));
    };
    // kv_scale by itself: 2^-116 over a sum of up to 2^31 would be a subnormal factor with a bit or two
    auto f = [&](uint32_t v) { return __uint_as_float(v) * inv_l * p.kv_scale; };
    auto emit = [&](int c, const uint32_t (&v)[32]) {
      if (final_out) {   // 32 bf16 columns: 64 B a row
#pragma unroll
        for (int j = 0; j < 4; ++j)
          put(j, make_uint4(pack_bf16x2(f(v[8 * j]), f(v[8 * j + 1])), pack_bf16x2(f(v[8 * j + 2]), f(v[8 * j + 3])),
                            pack_bf16x2(f(v[8 * j + 4]), f(v[8 * j + 5])), pack_bf16x2(f(v[8 * j + 6]), f(v[8 * j + 7]))));
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int x = 8 * j + (lane >> 2);
          const uint4 u = get(j);
          if (x < nrows) *reinterpret_cast<uint4*>(obase + static_cast<int64_t>(x) * kDimV + c + 8 * tq) = u;
        }
        __syncwarp();
      } else {           // fp32 partials: two passes of 16 columns
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int e = 16 * h + 4 * j;
            put(j, make_uint4(__float_as_uint(f(v[e])), __float_as_uint(f(v[e + 1])), __float_as_uint(f(v[e + 2])),
                              __float_as_uint(f(v[e + 3]))));
          }
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int x = 8 * j + (lane >> 2);
            const uint4 u = get(j);
            if (x < nrows && slot_ok) *reinterpret_cast<uint4*>(pbase + static_cast<int64_t>(x) * kDimV + c + 16 * h + 4 * tq) = u;
          }
          __syncwarp();
        }
      }
    };
    // the TMEM load of the next 32 columns is in flight while the current ones are stored
    uint32_t va[32], vb[32];
    tmem_ld32(tmem_row, va);
#pragma unroll 1
    for (int c = 0; c < 256; c += 64) {
      tmem_wait_ld();
      tmem_ld32(tmem_row + c + 32, vb);
      emit(c, va);
      tmem_wait_ld();
      if (c + 64 < 256) {
        tmem_ld32(tmem_row + c + 64, va);
      } else {   // O may be overwritten by the next segment
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(AT(o_free));
      }
      emit(c + 32, vb);
    }
    ++seg;
    have = w.next(s);
  }
}

template <bool Sparse>
__global__ void __launch_bounds__(kThreads, 1) mla_decode_fp4_kernel(const __grid_constant__ CUtensorMap q_map,
                                                                        const __grid_constant__ Fp4Params p) {
  extern __shared__ __align__(1024) uint8_t dyn_smem[];
  const uint32_t smem = smem_u32(dyn_smem);
  if (smem & 1023u) {   // the swizzled layouts need the base aligned (no static shared memory is declared)
    if (threadIdx.x == 0) atomicCAS(p.status, 0, MLA_ERR_UNSUPPORTED);
    return;             // every CTA of the grid takes this branch alike
  }
  Shared& sh = *reinterpret_cast<Shared*>(dyn_smem + kOffShared);
  const int warp = threadIdx.x >> 5;
  const uint32_t rank = cluster_ctarank();
  const uint32_t cl = 2u * static_cast<uint32_t>(p.n_rb);
  const int part = static_cast<int>(blockIdx.x / cl);
  const Block blk(p, static_cast<int>(rank >> 1));
  const bool is_s = (rank & 1u) == 0;
  const uint32_t peer = rank ^ 1u;

  if (threadIdx.x == 0) {
    if (is_s) prefetch_tensormap(&q_map);
    sh.abort = 0;
    sh.tiles = 0;
    sh.cmd = 0;
    auto init = [](uint64_t& b, uint32_t n) { mbar_init(smem_u32(&b), n); };
    for (int i = 0; i < 2; ++i) {
      init(sh.raw_full[i], 1);
      init(sh.raw_empty[i], 4);      // two warps of each converting warpgroup
      init(sh.s_full[i], 1);
      init(sh.s_empty[i], 8);
      init(sh.credit[i], 1);
      init(sh.sent[i], 1);
      init(sh.p_full[i][0], 1);
      init(sh.p_full[i][1], 1);
      init(sh.p_free[i], 1);
    }
    for (int i = 0; i < kItems; ++i) {
      init(sh.k_full[i], 8);
      init(sh.k_empty[i], 1);
    }
    for (uint32_t i = 0; i < kRowSlots; ++i) {
      init(sh.rows_full[i], 1);
      init(sh.rows_empty[i], is_s ? 4 : 8);   // (the S-CTA's pages go to half of the converters)
    }
    for (int i = 0; i < kVSlots; ++i) {
      init(sh.v_full[i], 4);
      init(sh.v_empty[i], 1);
    }
    init(sh.q_raw, 1);
    init(sh.q_full, 8);
    init(sh.q_empty, 1);
    init(sh.o_full, 1);
    init(sh.o_free, 8);
    init(sh.o_sync, 1);
    init(sh.corr_go, 1);
    init(sh.corr_done, 8);
    for (uint32_t i = 0; i < kInvSlots; ++i) init(sh.inv_full[i], 128);
    init(sh.gone, 8);
    init(sh.drain, 1);
    fence_mbar_init();
  }
  if (threadIdx.x < 128) sh.pos[threadIdx.x] = static_cast<uint16_t>(min(blk.rb * kRowsPerPair + static_cast<int>(threadIdx.x), p.rows - 1) / p.H);
  __syncwarp();
  if (warp == 0) tmem_alloc(smem_u32(&sh.tmem_base), 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();        // every barrier of the cluster is initialised before any remote use
  tc_fence_after();
  griddep_wait();        // the metadata, q and the cache are complete from here on

  // Each CTA's hot loops lie together (the roles of an SM share its instruction caches): of eight orders of these branches, 64 x 2 x 8192
  // took from 267 to 276 us, 16 heads of 64 x 4096 70 to 75.
  const bool lane0 = (threadIdx.x & 31) == 0;
  if (is_s && warp >= 12) {
    regs_down<kRegsConvert>();
    s_convert<Sparse>(p, sh, smem, part, (warp - 12) >> 2);
    __syncwarp();
    if (lane0) mbar_arrive_remote(map_to_rank(AT(gone), peer));
  } else if (is_s && warp >= 4 && warp < 12) {
    regs_up<kRegsSoftmax>();
    s_softmax<Sparse>(p, sh, smem, part, blk, peer);
  } else if (is_s && warp < 4) {
    regs_down<kRegsMisc>();
    if (warp == 0) {
      if constexpr (Sparse) find_rows<true, true>(p, smem, part);
      else s_load(p, smem, part);
    } else if (warp == 1) {
      s_mma(p, &q_map, sh, smem, part, blk);
    }
  } else if (!is_s && warp >= 4 && warp < 12) {
    regs_up<kRegsSoftmax>();
    o_epilogue(p, sh, smem, part, blk);
  } else if (!is_s && warp >= 12) {
    regs_down<kRegsConvert>();
    o_convert(p, smem);
  } else {
    regs_down<kRegsMisc>();
    if (warp == 0) find_rows<Sparse, false>(p, smem, part);
    else if (warp == 1) o_mma(p, sh, smem, part);
    else if (lane0 && warp == 2) o_forward(p, smem, part, peer);
    else if (lane0) o_watch(p, smem, cl);
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();        // no CTA leaves while a partner may still touch its shared memory
  __syncwarp();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(sh.tmem_base, 512);
  }
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

// One-time set-up of the kernels on the current device.
bool fp4_ready() {
  static std::mutex mutex;
  static bool ready[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  std::lock_guard<std::mutex> lock(mutex);
  if (ready[dev]) return true;
  if (!g_encode) {
    cudaDriverEntryPointQueryResult found;
    void* fn = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess || fn == nullptr)
      return false;
    g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }
  for (auto kernel : {mla_decode_fp4_kernel<false>, mla_decode_fp4_kernel<true>}) {
    cudaFuncAttributes a;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemBytes)) != cudaSuccess ||
        cudaFuncGetAttributes(&a, kernel) != cudaSuccess)
      return false;
    if (a.numRegs < 96) return false;   // the warpgroups' shares add up to 96 a thread
  }
  return ready[dev] = true;
}

mla_status_t decode_fp4_impl(const void* q, const uint8_t* kv_cache, float kv_scale, int64_t num_blocks,
                             const int32_t* block_table, int max_blocks, const int32_t* seqlens, const int32_t* indices,
                             int64_t index_stride, const int32_t* topk_lens, int B, int s_q, int H, float softmax_scale,
                             int causal_s_q, const void* metadata, int num_sm_parts, void* workspace,
                             size_t workspace_bytes, mla_bf16_t* out, float* lse, mla_stream_t stream) {
  if (!q || !kv_cache || !block_table || !seqlens || !metadata || !out || !lse) return MLA_ERR_INVALID_ARG;
  if (B < 1 || s_q < 1 || H < 1 || num_blocks < 1 || max_blocks < 1 || num_sm_parts < 1) return MLA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(kv_cache, 32) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(block_table, 4) ||
      !aligned(seqlens, 4) || !aligned(metadata, 4))
    return MLA_ERR_INVALID_ARG;
  if (indices && (!topk_lens || index_stride < 1 || !aligned(indices, 4) || !aligned(topk_lens, 4))) return MLA_ERR_INVALID_ARG;
  if (!std::isfinite(softmax_scale) || !(softmax_scale > 0.f)) return MLA_ERR_INVALID_ARG;
  if (!std::isfinite(kv_scale) || !(kv_scale > 0.f) || !fp4_scale_ok(kv_scale)) return MLA_ERR_INVALID_ARG;
  const float unit = static_cast<float>(static_cast<double>(softmax_scale) * 1.4426950408889634074 * kv_scale);
  if (!std::isnormal(unit)) return MLA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(s_q) * H > kMaxPairsPerCluster * kRowsPerPair || B > kScheduleMaxB) return MLA_ERR_UNSUPPORTED;
  if (num_blocks > ((int64_t(1) << 31) - kPageTokens) / kPageTokens) return MLA_ERR_UNSUPPORTED;
  const int rows = s_q * H;
  const size_t need = mla_decode_workspace_size(B, s_q, H, num_sm_parts);
  if (workspace_bytes < need || !workspace) return MLA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return MLA_ERR_INVALID_ARG;
  Fp4Params p = {};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.kv = reinterpret_cast<const __nv_bfloat16*>(kv_cache);
  p.num_blocks = num_blocks;
  p.block_table = block_table;
  p.max_blocks = max_blocks;
  p.seqlens = seqlens;
  p.lens = indices ? topk_lens : seqlens;
  p.indices = indices;
  p.idx_stride = indices ? index_stride : 0;
  p.B = B;
  p.s_q = s_q;
  p.H = H;
  p.rows = rows;
  p.n_rb = (rows + kRowsPerPair - 1) / kRowsPerPair;
  p.unit = unit;
  p.causal = causal_s_q && s_q > 1 ? 1 : 0;   // (a single query position sees every token)
  p.kv_scale = kv_scale;
  p.meta = static_cast<const int32_t*>(metadata);
  p.num_splits = p.meta + kMetaInts * num_sm_parts;
  p.num_parts = num_sm_parts;
  const size_t slots = static_cast<size_t>(B) + static_cast<size_t>(num_sm_parts);   // partial outputs in the workspace
  p.o_part = static_cast<float*>(workspace);
  p.lse_part = p.o_part + slots * rows * kDimV;
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.status = device_status_word();
  if (!p.status || !fp4_ready()) return MLA_ERR_CUDA;
  p.withhold_first_load = take_withheld_load();
  // q as [chunk 0..8][row][64 dims], a box 64 dims of a row block (as many rows as its MMA is wide)
  p.q_box = rows >= kRowsPerPair ? kRowsPerPair : (rows + 15) & ~15;
  CUtensorMap q_map;
  const cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(B) * rows, kDimQK / 64}, strides[2] = {kDimQK * 2, 128};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(p.q_box), 1}, steps[3] = {1, 1, 1};
  if (g_encode(&q_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, steps,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return MLA_ERR_CUDA;
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const unsigned cl = 2u * static_cast<unsigned>(p.n_rb);
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = pdl_config(dim3(static_cast<unsigned>(num_sm_parts) * cl), dim3(kThreads), kSmemBytes, cs, attr);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cl;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.numAttrs = 2;
  if ((indices ? cudaLaunchKernelEx(&cfg, mla_decode_fp4_kernel<true>, q_map, p)
               : cudaLaunchKernelEx(&cfg, mla_decode_fp4_kernel<false>, q_map, p)) != cudaSuccess)
    return MLA_ERR_CUDA;
  return launch_combine(p.o_part, p.lse_part, p.num_splits, B, rows, static_cast<int>(slots), p.out, lse, p.status, cs) ==
                 cudaSuccess
             ? MLA_OK
             : MLA_ERR_CUDA;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" {

mla_status_t mla_decode_fp4(const mla_bf16_t* q, const uint8_t* kv_cache, float kv_scale, int64_t num_blocks,
                            const int32_t* block_table, int max_blocks, const int32_t* seqlens, int B, int s_q, int H,
                            float softmax_scale, int causal_s_q, const void* metadata, int num_sm_parts,
                            void* workspace, size_t workspace_bytes, mla_bf16_t* out, float* lse, mla_stream_t stream) {
  return decode_fp4_impl(q, kv_cache, kv_scale, num_blocks, block_table, max_blocks, seqlens, nullptr, 0, nullptr, B, s_q, H,
                         softmax_scale, causal_s_q, metadata, num_sm_parts, workspace, workspace_bytes, out, lse, stream);
}

mla_status_t mla_decode_sparse_fp4(const mla_bf16_t* q, const uint8_t* kv_cache, float kv_scale, int64_t num_blocks,
                                   const int32_t* block_table, int max_blocks, const int32_t* seqlens,
                                   const int32_t* indices, int64_t index_stride, const int32_t* topk_lens, int B, int s_q,
                                   int H, float softmax_scale, int causal_s_q, const void* metadata, int num_sm_parts,
                                   void* workspace, size_t workspace_bytes, mla_bf16_t* out, float* lse,
                                   mla_stream_t stream) {
  if (!indices) return MLA_ERR_INVALID_ARG;
  return decode_fp4_impl(q, kv_cache, kv_scale, num_blocks, block_table, max_blocks, seqlens, indices, index_stride,
                         topk_lens, B, s_q, H, softmax_scale, causal_s_q, metadata, num_sm_parts, workspace,
                         workspace_bytes, out, lse, stream);
}

}  // extern "C"
