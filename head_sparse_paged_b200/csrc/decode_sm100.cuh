// decode_sm100.cuh -- attention of one new token per sequence over its own stored pages.
//
// For sequence b, KV head k and the G query heads h of its group, at position i = L - 1:
//   s_j = scale q_h . k_j over the visible keys j,  O_h = sum_j softmax(s)_j v_j,  LSE_h = ln sum_j exp(s_j).
// Every visible key and value is read once and used by G heads only, so the call is bound by HBM (for G = 8, 16
// flops per bf16 byte, where mma.sync passes about 60). (A group of more than 16 heads is done in passes of 16, each of which
// reads and converts the tiles again: 32 sequences of 16-32K take 79, 143, 272 and 521 us in e4m3 and 112, 208, 404 and 789
// us in bf16 with 16, 32, 64 and 128 heads a KV head.) What matters is that all SMs load all the time. So:
//   - The work is the list of 128-token tiles of all (sequence, KV head) pairs, cut into one equal run of tiles per
//     CTA (one CTA per SM): a pair's tiles may end in one CTA and go on in the next. Each CTA finds its run by itself
//     from ctx_len and the classes in device memory (a prefix sum over the pairs), so a captured call follows the
//     lengths and there is no host plan. Runs that end inside a pair leave a partial result (O / l, m and l) in
//     the workspace, which decode_combine_kernel joins in tile order: no atomics, no state from call to call, and the
//     rounding depends on the lengths, the size of the table array (see kDecodeWholeTokens) and the grid only.
//   - Two to four helper warps stream the tiles through a ring of shared-memory stages with TMA (page id = coordinate),
//     three to eight tiles deep (as many as fit, see DecodeCfg), across pair boundaries, with the next page ids in flight.
//   - Eight or twelve consumer warps take 32 tokens of every second or third tile, and keep their own
//     running maximum, sum and O in registers. S^T = K Q^T puts the tokens on the 16 rows of mma.m16n8k16 and the heads
//     on its 8 columns, so up to 8 heads cost the same and nothing is padded from 8 to 16; O^T = V^T P^T likewise.
//   - Where a pair ends, a consumer leaves its maxima and sums in shared memory and its O in tensor memory (0.25 us) and
//     goes on; the four helpers, one to each quarter of tensor memory's lanes, join the warps' results. (When the
//     consumers met and joined them themselves, all of them waited for the last one's tile and then for one another: 1.7 us
//     per pair and CTA; 65.5 instead of 63.3 us on 32 sequences of 16-32K in e4m3, 71.0 instead of 65.9 us in int8, 27.5
//     instead of 22.8 us on 64 sequences of 0.1-0.9K.)
//   - tcgen05.mma would need the tile's rows as its 128-row M and TMEM round trips for an S of 128 x 8; the work is a
//     fifth of what mma.sync can do in the time the bytes take, so the legacy path is the shorter one here.
// 8-bit pools: codes become fp16 in registers (exact). Query rows are brought to a largest magnitude of 2^15 by a power
// of two first, so that bf16 queries of any size are exact in fp16 to 2^-29 of the row's largest. The K row's exponent
// scales the logit; the V row's exponent 2^(y - r), r the largest one so far in this warp, multiplies the
// probability, and O is kept in units of 2^(r - 14): the product, at most 2^14, is rounded to fp16 (2^-11 relative
// down to 2^-14, 2^-25 below). While the y of a chunk lie within kDecodeSpread of one another, its most probable key weighs
// 2^3 or more, so that nothing above 2^-28 of a head's largest weight is lost. A chunk whose y lie farther apart (a large V
// row, maybe of no probability at all, beside small ones) is done again in fp32 behind the loop: 32 sequences of 16-32K
// whose chunks are all like that take 927 instead of 62 us. (Units by each head's largest weight instead, in the loop: 88
// instead of 78 us for 16 heads on such sequences in e4m3, by the registers they take, needed or not.)
// bf16 pools: a probability is split into a sum of two bf16 (2^-16 relative), which
// costs a second V product where the tensor pipe idles.
//
// Measured (B200, back-to-back calls; of the 6543 GB/s that a large copy reaches): 32 sequences of 16-32K, 64/8 heads,
// one global head each: bf16 106.7 us, 6.2 TB/s (94 %); e4m3 61.9 us, 5.3 TB/s (82 %); int8 63.8 us. 64 global heads at
// 128K: bf16 614 us, 7.0 TB/s (107 %); e4m3 321 us, 6.7 TB/s (103 %), 337 us after seconds of it, when the power cap
// holds the SMs at 1.6 GHz and the conversions' ALU work (53 % of its pipe at 1.9 GHz) no longer hides. What the short
// calls are made of, on 32 sequences in e4m3: 2.6 us to find the run, 1.2 us to issue the first copies, 1.4 us to the first
// tile, 48 us of tiles, 2 us to the last chunk's results, 1.3 us to the combine kernel's start, 2.6 us in it, and 4 us
// between the median and the last CTA.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "plan.h"
#include "quant_pages.cuh"
#include "quant_rows.cuh"
#include "sm100_ptx.cuh"

namespace segpaged {

constexpr int kDecodeTile = 128;         // tokens of a tile
constexpr int kDecodeMaxWarps = 12;      // most consumer warps
constexpr int kDecodeHelpers = 4;        // warps beside the consumers: one for each quarter of tensor memory's lanes
constexpr int kDecodeMails = 2;          // finished chunks that tensor memory holds
constexpr int kDecodeMaxCtas = 160;      // most CTAs a launch uses (B200 has 148 SMs)
constexpr int kDecodeMostPairCost = 6;   // DecodeCfg's PAIR_COST at most
constexpr int kDecodeGroup = 16;         // most query heads of one pass; larger groups take several
constexpr int kDecodeStatusTimeout = 4;  // SEGPAGED_STATUS_TIMEOUT
// Tries (of 0.2 to some 6 us) that a helper makes in a row without anything to do before it gives up: 1 to 25 s; other roles'
// waits end after 1 s. It looks at that, and at whether another warp has given up, once in SEGPAGED_DECODE_IDLE_CHECK tries
// (a power of two). A test builds the kernels with limits that run out.
#ifndef SEGPAGED_DECODE_IDLE_TRIES
#define SEGPAGED_DECODE_IDLE_TRIES (1 << 22)
#define SEGPAGED_DECODE_IDLE_CHECK 64
#endif
constexpr int kDecodeSpread = 11;        // how far apart the exponent bytes of a chunk's V rows may lie in fp16 weights

struct DecodeParams {
  const __nv_bfloat16* q;      // [B][Hq][D]
  const uint8_t* kv_scale;     // [num_pages][2][P], null for bf16
  const uint8_t* k_pool;       // what the tensor maps stand for, for the 8-bit chunks that are done again
  const uint8_t* v_pool;
  const int32_t* table;
  const int32_t* offs;         // [B*Hkv+1]
  const int32_t* ctx_len;      // [B]
  const int32_t* q_len;        // [B] or null
  const int32_t* cls;          // [B*Hkv][3]
  __nv_bfloat16* o;            // [B][Hq][D]
  float* lse;                  // [Hq][B]
  float* part_o;               // [2 x CTAs][16][D]: O / l of a chunk
  float2* part_sum;            // [2 x CTAs][16]: its maximum m (log2 units) and sum l
  int32_t* part_meta;          // [CTAs][2]: pair and chunk count of the pair whose first chunk is this CTA's last
  int32_t* status;             // nullable
  int64_t table_len;
  int32_t B, Hkv, G, log2_page, num_pages;
  int32_t log2_hg;             // passes of a group: max(1, G / 16)
  int32_t whole;               // no pair is cut: each is done by the CTA whose share its first unit lies in
  float scale_log2;
};

template <int D, int FMT, int NB>
struct DecodeCfg {
  // A warp takes 32 tokens of every second or third tile: two independent chains of products, and one maximum, wait and
  // header for twice the tokens. (16 tokens of every tile: 89.2 instead of 80.5 us with 16 heads on 32 sequences of
  // 16-32K in e4m3.) Twelve consumer warps leave 128 registers a thread, too few for the O and q of 16 heads of 128 columns;
  // for bf16 pools of 128 columns, whose stages are three, a third turn would only hold one more of them (see STAGES). With
  // 64 columns twelve warps against eight take 56.7 instead of 59.2 us on the same sequences with 16 heads in e4m3, and 17.9
  // instead of 19.7 us on 64 of 0.1-0.9K with 4 heads in bf16; with 16 heads in bf16 66.5 instead of 64.3 us.
  static constexpr int MB = 2;
  static constexpr bool BYTES = FMT != kFmtBf16;
  static constexpr int WARPS = (NB == 1 ? BYTES || D == 64 : BYTES && D == 64) ? 12 : 8;  // consumer warps
  static constexpr int TILE_WARPS = kDecodeTile / (16 * MB);     // of which these share a tile
  static constexpr int TURNS = WARPS / TILE_WARPS;
  static constexpr int EB = FMT == kFmtBf16 ? 2 : 1;             // bytes of an element
  static constexpr int ROWB = D * EB < 128 ? D * EB : 128;       // bytes of a row in one column block
  static constexpr int CB = D * EB / ROWB;                       // column blocks
  static constexpr int BLOCK_BYTES = kDecodeTile * ROWB;
  static constexpr int TILE_BYTES = CB * BLOCK_BYTES;            // K or V
  static constexpr int SCALE_BYTES = FMT == kFmtBf16 ? 0 : 2 * kDecodeTile;
  // A query row takes 16 bytes more than it holds, so that the eight rows that a fragment load touches lie in different
  // banks: without them the twelve warps' loads take 1536 cycles of shared memory at the start of each chunk.
  static constexpr int Q_ROW = D * 2 + 16;
  static constexpr int Q_BYTES = NB * 8 * Q_ROW;
  static constexpr int STAGE_BYTES = 2 * TILE_BYTES;
  static constexpr int EXTRA_BYTES = SCALE_BYTES + Q_BYTES;      // beside a stage: exponent bytes, query rows
  static constexpr int MERGE_BYTES = kDecodeHelpers * 8 * D * 4;  // a helper's sum of one column block of O
  static constexpr int MAIL = WARPS * 8 * NB;                     // entries of a mail's arrays
  static constexpr int SMALL_BYTES = MAIL <= 96 ? 3584 : MAIL <= 128 ? 3904 : 4928;  // a DecodeSmall<MAIL>
  static constexpr int FIXED_BYTES = MERGE_BYTES + SMALL_BYTES + 1024;  // 1024: alignment slack
  static constexpr int FIT = (227 * 1024 - FIXED_BYTES) / (STAGE_BYTES + EXTRA_BYTES);
  static constexpr int STAGES = FIT > 8 ? 8 : FIT;
  static constexpr int SMEM_BYTES = FIXED_BYTES + STAGES * (STAGE_BYTES + EXTRA_BYTES);
  static constexpr int PRODUCERS = FMT == kFmtBf16 ? 2 : kDecodeHelpers;  // most helpers that issue copies
  // A producer's wait for a stage looks at one parity bit, so the stage may be at most one use behind it: what it waited
  // for before its last tile, as many tiles ago as there are producers, has to cover the use before the last one,
  // 2 STAGES tiles ago.
  static_assert(STAGES >= 2 && STAGES <= 8 && PRODUCERS <= STAGES, "ring");
  static constexpr int THREADS = 32 * (WARPS + kDecodeHelpers);
  // Tensor-memory columns of one warp's O in its quarter of the lanes, of a chunk, and of all of them.
  static constexpr int OCOLS = NB * D / 4;
  static constexpr int MAIL_COLS = (WARPS + 3) / 4 * OCOLS;
  static constexpr int TMEM_COLS = kDecodeMails * MAIL_COLS <= 64 ? 64 : kDecodeMails * MAIL_COLS <= 128 ? 128 : 256;
  static_assert(kDecodeMails * MAIL_COLS <= TMEM_COLS, "tensor memory");
  static_assert(MAIL <= 192 && WARPS % 4 == 0 && WARPS <= kDecodeMaxWarps, "a mail's arrays, the quarters");
  // What ending a pair costs a CTA, in half tiles. With 3, 5, 6, 7 and 9 for 8-bit pools 32 sequences of 16-32K in e4m3 take
  // 63.5, 62.1, 61.6, 62.1 and 62.3 us and 64 of 0.1-0.9K 22.2, 21.8, 21.8, 22.1 and 22.3 us (D = 128); with 64 columns 44.9,
  // 45.0, 45.4, 45.7, 46.5 and 17.0, 16.4, 16.4, 16.7, 16.7 us. With 1, 2, 3, 4 and 6 for bf16 107.1, 106.6, 106.7, 106.3,
  // 106.6 and 30.6, 25.1, 24.5, 24.2, 24.5 us; with 64 columns 60.5, 60.5, 60.4, 60.3, 60.8 and 18.6, 18.4, 17.6, 17.4, 17.3.
  static constexpr int PAIR_COST = FMT == kFmtBf16 ? 3 : 6;
  static_assert(PAIR_COST <= kDecodeMostPairCost, "the host's check of sizes");
};

template <bool B>
struct Flag {
  static constexpr bool value = B;
};

// What a consumer needs to know of a tile.
struct DecodeTileHeader {
  int32_t rows;     // visible rows [v0, v1) of the tile: v0 | v1 << 16
  int32_t b, h0;    // sequence, first query head
  int32_t flags;    // bit 0: first tile of a chunk, bit 1: last; bits 2..: 1 + partial slot, 0: the whole pair
};

// Tiles of one (sequence, KV head), n of them: the first n_a cover tokens [0, a1), the others those from b0, the start of
// lo's page, of which [lo, L) are visible.
struct DecodeGeom {
  int32_t L, a1, lo, n;
  __device__ __forceinline__ int32_t n_a() const { return (int32_t)(((uint32_t)a1 + kDecodeTile - 1) / kDecodeTile); }
  __device__ __forceinline__ int32_t b0(int32_t log2_page) const { return lo >> log2_page << log2_page; }
};
// A pair: those tiles, the outputs they go to, and the page table: entries [off, off + len), logical page lp at entry lp
// below n_sink and at lp - w0 + n_sink from there on.
struct DecodePair {
  DecodeGeom g;
  int32_t off, len, n_sink, w0, b, h0;
};

// Pair u: (sequence, KV head, pass of 16 query heads), u = (b * Hkv + k) << log2_hg | pass.
__device__ __forceinline__ DecodePair decode_pair(const DecodeParams& p, int32_t u) {
  const int32_t bk = u >> p.log2_hg;
  DecodePair r;
  r.b = bk / p.Hkv;
  r.h0 = (bk - r.b * p.Hkv) * p.G + (u - (bk << p.log2_hg)) * kDecodeGroup;
  const HeadPages hp = head_pages(p.ctx_len, p.q_len, p.cls, r.b, bk, p.log2_page, 1);
  const int32_t L = hp.L, lp = p.log2_page;
  r.off = p.offs[bk];
  r.len = p.offs[bk + 1] - r.off;
  r.n_sink = hp.n_sink;
  r.w0 = hp.w0;
  r.g.L = L;
  r.g.lo = max(L - hp.window, 0);
  r.g.a1 = hp.sink;
  if (hp.global || hp.sink >= r.g.lo) r.g.a1 = r.g.lo = 0;  // one run of visible tokens
  r.g.n = r.g.n_a() + (int32_t)(((uint32_t)(L - r.g.b0(lp)) + kDecodeTile - 1) / kDecodeTile);
  // A table that does not hold exactly these pages: the pair is reported and left out.
  if (L > 0 && (r.len != hp.total || r.off < 0 || r.off > p.table_len - r.len)) {
    report(p.status, 2);
    r.g.n = 0;
  }
  return r;
}

// First token of a tile and its visible tokens [lo, hi).
struct DecodeSpan {
  int32_t t0, lo, hi;
};
__device__ __forceinline__ DecodeSpan decode_span(const DecodeGeom& g, int32_t tile, int32_t log2_page) {
  DecodeSpan s;
  const int32_t n_a = g.n_a();
  const bool in_sink = tile < n_a;
  s.t0 = in_sink ? tile * kDecodeTile : g.b0(log2_page) + (tile - n_a) * kDecodeTile;
  s.lo = max(s.t0, in_sink ? 0 : g.lo);
  s.hi = (int32_t)min((int64_t)s.t0 + kDecodeTile, (int64_t)(in_sink ? g.a1 : g.L));
  return s;
}

// The K and V copies of one box (up to 64 rows of a page): `at`, its first row in the stage's tiles; `row`, its first row in
// the page.
template <typename C>
__device__ __forceinline__ void issue_box(uint8_t* stage, const CUtensorMap& tk, const CUtensorMap& tv, int32_t at, int32_t row,
                                          int32_t page, uint64_t* bar) {
#pragma unroll
  for (int cb = 0; cb < C::CB; ++cb) {
    uint8_t* to = stage + cb * C::BLOCK_BYTES + at * C::ROWB;
    ptx::tma_load_3d(to, &tk, cb * (C::ROWB / C::EB), row, page, bar);
    ptx::tma_load_3d(to + C::TILE_BYTES, &tv, cb * (C::ROWB / C::EB), row, page, bar);
  }
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// 2^e for e <= 127; 0 below the normal range.
__device__ __forceinline__ float exp2_int(int32_t e) { return __uint_as_float((uint32_t)max(e + 127, 0) << 23); }

// Bulk copy of `bytes` (a multiple of 16) contiguous bytes.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   ptx::smem_addr(dst)),
               "l"((uint64_t)__cvta_generic_to_global(src)), "r"(bytes), "r"(ptx::smem_addr(bar))
               : "memory");
}

// A bounded wait of a whole warp, with one answer for all its lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int32_t* status) {
  return __all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, abort, status, kDecodeStatusTimeout));
}

// N (16 or 32) consecutive tensor-memory columns of this warp's lanes, to and from registers.
template <int N>
__device__ __forceinline__ void tmem_put(uint32_t taddr, const uint32_t* r) {
  if constexpr (N == 32) {
    ptx::tmem_st32(taddr, r);
  } else {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
  }
}
template <int N>
__device__ __forceinline__ void tmem_get(uint32_t taddr, uint32_t* r) {
  if constexpr (N == 32) {
    ptx::tmem_ld32(taddr, r);
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
  }
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_addr(dst)),
               "l"((uint64_t)__cvta_generic_to_global(src))
               : "memory");
}
// Arrives on `bar` (one of its expected arrivals) when this thread's earlier cp.async copies have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(ptx::smem_addr(bar)) : "memory");
}

// A finished chunk as the consumers leave it for the helpers: each warp's maxima (log2 units), sums and unit of O, which
// lies in tensor memory.
template <int N>
struct DecodeMail {
  float m[N], l[N];                 // [consumer warp][8 NB heads]
  // 8-bit pools: the largest exponent byte of the V rows it saw, which is r + 127 of the unit 2^(r - 14) of its O, and << 8
  // the smallest (0 and 255 if it saw none).
  int32_t vref[kDecodeMaxWarps];
  int32_t b, h0, slot, final;  // first sequence and head, partial slot or -1, whether it is the run's last chunk
};

// Shared memory beside the ring and the helpers' sums.
template <int N>
struct DecodeSmall {
  uint64_t full[8], empty[8];
  uint64_t mail_full[kDecodeMails], mail_empty[kDecodeMails];
  uint64_t sync;                                // the helpers' meeting point
  DecodeTileHeader hdr[8];
  DecodeMail<N> mail[kDecodeMails];
  int32_t warp_sum[kDecodeMaxWarps + kDecodeHelpers];
  int32_t first_rank, end_rank;                 // this CTA's run in the list of all tiles
  int32_t pair0, tile0;                         // where its first tile lies
  int32_t abort;
  uint32_t tmem;
  int32_t last[8];                              // the last tile that was issued into each stage, -1 if none was
  uint32_t redo;                                // bit c: chunk c of the run is to be done again (31: and those after it)
  DecodePair window[32];                        // pairs pair0 ..
};
static_assert(sizeof(DecodeSmall<192>) <= 4928 && sizeof(DecodeSmall<128>) <= 3904 && sizeof(DecodeSmall<96>) <= 3584,
              "small shared arrays");

// Does the run's chunks named in `redo` again, in fp32 throughout, and replaces what was written for them. For chunks of 8-bit
// pools whose V rows are of too different size for weights in fp16. Called by the whole block, with the ring as `scratch`.
// Four heads at a time; a warp takes batches of 32 tokens, a lane one token's logits, then D / 32 columns of all values.
// (Out of line, behind the loop: inlined it made every other call 1 to 6 % slower.)
constexpr int kRedoHeads = 4;
template <int D>
__host__ __device__ constexpr int redo_scratch(int warps) {  // floats: queries [4][D], weights [warp][32][4], results [4][warp][D + 2]
  return kRedoHeads * (D + warps * (32 + D + 2));
}
template <int D, int FMT>
__device__ __noinline__ void decode_redo(const DecodeParams& p, float* scratch, int32_t u, int32_t tile0, int32_t tiles,
                                         uint32_t redo, int32_t warps) {
  constexpr int E = D / 32, H = kRedoHeads;  // columns of a lane: lane * E ..
  constexpr float kSmall = 0x1p-20f;         // O is summed in units of 2^20: many values near the largest float
  const int32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;
  const int32_t heads = min(p.G, kDecodeGroup), Hq = p.Hkv * p.G, page = 1 << p.log2_page;
  const int32_t pairs = (p.B * p.Hkv) << p.log2_hg;
  float* qs = scratch;
  float4* weights = reinterpret_cast<float4*>(scratch + H * D + warp * 32 * H);
  float* parts = scratch + H * (D + warps * 32);
  uint32_t chunk = 0;
#pragma unroll 1
  for (; tiles > 0 && u < pairs; ++u, tile0 = 0) {
    const DecodePair w = decode_pair(p, u);
    const int32_t end = min(w.g.n, tile0 + tiles);
    if (end <= tile0) continue;
    tiles -= end - tile0;
    if (!(redo >> min(chunk++, 31u) & 1)) continue;
    const int32_t slot = tile0 == 0 && end == w.g.n ? -1 : 2 * cta + (tile0 == 0 ? 1 : 0);
#pragma unroll 1
    for (int32_t h0 = 0; h0 < heads; h0 += H) {
      const int64_t q0 = ((int64_t)w.b * Hq + w.h0 + h0) * D;
      for (int32_t x = threadIdx.x; x < H * D; x += 32 * warps)
        qs[x] = h0 + x / D < heads ? p.scale_log2 * __bfloat162float(p.q[q0 + x]) : 0.f;
      __syncthreads();
      float o[H][E] = {}, m[H], l[H] = {};
#pragma unroll
      for (int h = 0; h < H; ++h) m[h] = -INFINITY;
#pragma unroll 1
      for (int32_t x = warp; x < 4 * (end - tile0); x += warps) {
        const DecodeSpan sp = decode_span(w.g, tile0 + x / 4, p.log2_page);
        const int64_t tok = (int64_t)sp.t0 + x % 4 * 32 + lane;
        const bool in = tok >= sp.lo && tok < sp.hi;
        const uint32_t ins = __ballot_sync(0xffffffffu, in);
        if (ins == 0) continue;
        int64_t row = 0;
        float s[H] = {}, k_scale = 0.f, v_scale = 0.f;
        if (in) {
          const int32_t lp = (int32_t)(tok >> p.log2_page), at = (int32_t)tok & (page - 1);
          int32_t id = p.table[w.off + (lp < w.n_sink ? lp : lp - w.w0 + w.n_sink)];
          if ((uint32_t)id >= (uint32_t)p.num_pages) id = 0;  // (reported when it was loaded)
          row = ((int64_t)id << p.log2_page) + at;
          const uint8_t* y = p.kv_scale + ((int64_t)id << (p.log2_page + 1)) + at;
          k_scale = row_scale(y[0]);
          v_scale = row_scale(y[page]) * kSmall;
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            const uint4 codes = *reinterpret_cast<const uint4*>(p.k_pool + row * D + c);
            const uint32_t in4[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t c2[2];
              codes_to_half2x2<FMT, false>(in4[i], c2[0], c2[1]);
              const float2 k01 = __half22float2(*reinterpret_cast<const __half2*>(&c2[0]));
              const float2 k23 = __half22float2(*reinterpret_cast<const __half2*>(&c2[1]));
#pragma unroll
              for (int h = 0; h < H; ++h) {
                const float4 q = *reinterpret_cast<const float4*>(qs + h * D + c + 4 * i);
                s[h] = fmaf(q.x, k01.x, fmaf(q.y, k01.y, fmaf(q.z, k23.x, fmaf(q.w, k23.y, s[h]))));
              }
            }
          }
        }
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const float y = in ? s[h] * k_scale : -INFINITY;
          float top = y;
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
          top = fmaxf(top, m[h]);
          const float from = top == -INFINITY ? 0.f : top;
          const float c = m[h] == -INFINITY ? 0.f : ptx::ex2(m[h] - from), e = ptx::ex2(y - from);
          l[h] = l[h] * c + e;
          m[h] = top;
#pragma unroll
          for (int i = 0; i < E; ++i) o[h][i] *= c;
          s[h] = e * v_scale;
        }
        weights[lane] = make_float4(s[0], s[1], s[2], s[3]);
        __syncwarp();
#pragma unroll 4
        for (int i = 0; i < 32; ++i) {
          const int64_t from = __shfl_sync(0xffffffffu, row, i);
          if (!(ins >> i & 1)) continue;
          const uint8_t* at = p.v_pool + from * D + lane * E;
          uint32_t codes, c2[2];
          if (E == 4) codes = *reinterpret_cast<const uint32_t*>(at);
          else codes = *reinterpret_cast<const uint16_t*>(at);
          codes_to_half2x2<FMT, false>(codes, c2[0], c2[1]);
          const float4 w4 = weights[i];
          const float ws[H] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
          for (int k = 0; k < E; ++k) {
            const float v = __half2float(reinterpret_cast<const __half*>(c2)[k]);
#pragma unroll
            for (int h = 0; h < H; ++h) o[h][k] = fmaf(ws[h], v, o[h][k]);
          }
        }
        __syncwarp();
      }
#pragma unroll
      for (int h = 0; h < H; ++h) {
        float* mine = parts + (h * warps + warp) * (D + 2);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], d);
#pragma unroll
        for (int i = 0; i < E; ++i) mine[lane * E + i] = o[h][i];
        if (lane == 0) {
          mine[D] = m[h];
          mine[D + 1] = l[h];
        }
      }
      __syncthreads();
      const int32_t head = w.h0 + h0 + warp, own = h0 + warp;  // of the model, of this pass's group
      if (warp < H && own < heads) {
        const float* from = parts + warp * warps * (D + 2);
        float top = -INFINITY, sum = 0.f, acc[E] = {};
#pragma unroll 1
        for (int32_t x = 0; x < warps; ++x) top = fmaxf(top, from[x * (D + 2) + D]);
#pragma unroll 1
        for (int32_t x = 0; x < warps; ++x) {
          const float mx = from[x * (D + 2) + D], c = mx == -INFINITY ? 0.f : ptx::ex2(mx - top);
          sum += c * from[x * (D + 2) + D + 1];
#pragma unroll
          for (int i = 0; i < E; ++i) acc[i] += c * from[x * (D + 2) + lane * E + i];
        }
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const float out = acc[i] / sum * (1.f / kSmall);
          if (slot < 0) p.o[((int64_t)w.b * Hq + head) * D + lane * E + i] = __float2bfloat16_rn(out);
          else p.part_o[((int64_t)slot * kDecodeGroup + own) * D + lane * E + i] = out;
        }
        if (lane == 0) {
          if (slot < 0) p.lse[(int64_t)head * p.B + w.b] = 0.6931471805599453f * (top + log2f(sum));
          else p.part_sum[(int64_t)slot * kDecodeGroup + own] = make_float2(top, sum);
        }
      }
      __syncthreads();
    }
  }
}

template <int D, int FMT, int NB>
__global__ void __launch_bounds__(DecodeCfg<D, FMT, NB>::THREADS, 1)
    decode_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const __grid_constant__ DecodeParams p) {
  using C = DecodeCfg<D, FMT, NB>;
  constexpr bool BF = FMT == kFmtBf16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* extras = ring + C::STAGES * C::STAGE_BYTES;
  float4* merge = reinterpret_cast<float4*>(extras + C::STAGES * C::EXTRA_BYTES);  // [helper][KS][lane]
  DecodeSmall<C::MAIL>& sm = *reinterpret_cast<DecodeSmall<C::MAIL>*>(extras + C::STAGES * C::EXTRA_BYTES + C::MERGE_BYTES);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t cta = blockIdx.x;
  const int32_t pairs = (p.B * p.Hkv) << p.log2_hg;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      ptx::mbar_init(&sm.full[s], BF ? 1 : 33);  // the copies' bytes; for 8-bit pools also each lane's cp.async
      ptx::mbar_init(&sm.empty[s], C::WARPS);
    }
    for (int k = 0; k < kDecodeMails; ++k) {
      ptx::mbar_init(&sm.mail_full[k], C::WARPS);
      ptx::mbar_init(&sm.mail_empty[k], kDecodeHelpers);
    }
    ptx::mbar_init(&sm.sync, kDecodeHelpers);
    ptx::mbar_fence_init();
    sm.abort = 0;
    sm.redo = 0;
    for (int s = 0; s < 8; ++s) sm.last[s] = -1;
    sm.first_rank = sm.end_rank = 0;
    sm.pair0 = sm.tile0 = 0;
    ptx::tma_prefetch_desc(&tk);
    ptx::tma_prefetch_desc(&tv);
  }
  if (warp == C::WARPS) {
    ptx::tmem_alloc(&sm.tmem, C::TMEM_COLS);
    ptx::tmem_relinquish();
  }
  // The launch may start while the one before it ends; nothing it wrote is read, and nothing written, before this.
  early_start();

  // ---- this CTA's run of tiles. The work is counted in half tiles: a pair of n tiles is 2 n + PAIR_COST of them, and
  // a CTA takes the tiles that begin in its equal share of the sum. Thread i adds up pairs [i * per, (i + 1) * per).
  const int32_t per = (pairs + C::THREADS - 1) / C::THREADS;
  const int32_t u_lo = min((int32_t)threadIdx.x * per, pairs), u_hi = min(u_lo + per, pairs);
  DecodePair own = {};
  int32_t mine = 0;  // the tiles are fewer than the entries of the page table
  // (The kernel runs most of its code once per launch, so its size is time: loops over pairs stay rolled.)
#pragma unroll 1
  for (int32_t u = u_lo; u < u_hi; ++u) {
    own = decode_pair(p, u);
    mine += own.g.n;
  }
  int32_t incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int32_t x = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += x;
  }
  if (lane == 31) sm.warp_sum[warp] = incl;
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  int32_t before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < C::WARPS + kDecodeHelpers; ++w) {
    const int32_t x = sm.warp_sum[w];
    if (w < warp) before += x;
    total += x;
  }
  const uint32_t units = 2u * total + (uint32_t)C::PAIR_COST * pairs;
  // every CTA that takes part has two units or more, so one in the middle of a pair has a tile of it
  const uint32_t ctas = min(gridDim.x, max(units / 2, 1u));
  const uint32_t share = units / ctas, spare = units - share * ctas;  // the first `spare` CTAs take one unit more
  const bool takes_part = cta < (int32_t)ctas;
  const uint32_t lo_unit = share * cta + min((uint32_t)cta, spare), hi_unit = lo_unit + share + ((uint32_t)cta < spare);
  const int32_t heads = min(p.G, kDecodeGroup), Hq = p.Hkv * p.G;
  int32_t rank = before;
#pragma unroll 1
  for (int32_t u = u_lo; u < u_hi; ++u) {
    if (per > 1) own = decode_pair(p, u);
    const int32_t n = own.g.n;
    const uint32_t at = 2u * rank + (uint32_t)C::PAIR_COST * u, next = at + 2u * n + C::PAIR_COST;
    if (p.whole) {
      // (the pair after this one is a run's first if the share begins inside this one or at its end)
      if (takes_part && lo_unit > at && lo_unit <= next) {
        sm.pair0 = u + 1;
        sm.first_rank = rank + n;
      }
      if (takes_part && hi_unit > at && hi_unit <= next) sm.end_rank = rank + n;
    } else if (takes_part && lo_unit >= at && lo_unit < next) {
      const int32_t tile = min(n, (int32_t)(lo_unit - at + 1) / 2);
      sm.pair0 = u;
      sm.tile0 = tile;
      sm.first_rank = rank + tile;
      if (tile < n) {  // the run's first page ids will be wanted in a moment
        const int32_t n_a = own.g.n_a();
        const int64_t tok = tile < n_a ? (int64_t)tile * kDecodeTile
                                       : own.g.b0(p.log2_page) + (int64_t)(tile - n_a) * kDecodeTile;
        const int32_t page = (int32_t)(tok >> p.log2_page);
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p.table + own.off + (page < own.n_sink ? page : page - own.w0 + own.n_sink)));
      }
    }
    if (!p.whole && takes_part && hi_unit > at && hi_unit <= next) sm.end_rank = rank + min(n, (int32_t)(hi_unit - at + 1) / 2);
    rank += n;
    // a pair without a visible key (an empty sequence): O = 0, LSE = -inf, written by one CTA
    if (own.g.L == 0 && u % gridDim.x == cta) {
      uint4* o = reinterpret_cast<uint4*>(p.o + ((int64_t)own.b * Hq + own.h0) * D);
#pragma unroll 1
      for (int i = 0; i < heads * D / 8; ++i) o[i] = make_uint4(0, 0, 0, 0);
#pragma unroll 1
      for (int h = 0; h < heads; ++h) p.lse[(int64_t)(own.h0 + h) * p.B + own.b] = -INFINITY;
    }
  }
  if (threadIdx.x == 0) {
    p.part_meta[2 * cta] = 0;
    p.part_meta[2 * cta + 1] = 0;
  }
  __syncthreads();
  const int32_t first_rank = sm.first_rank, tiles = max(sm.end_rank - first_rank, 0);
  const uint32_t tmem = sm.tmem + ((uint32_t)(warp & 3) << 21);  // this warp's quarter of the lanes
  if (per == 1) {
    const int32_t k = (int32_t)threadIdx.x - sm.pair0;
    if (k >= 0 && k < 32) sm.window[k] = own;
    __syncthreads();
  }

  if (warp >= C::WARPS) {
    // ------------------------------------------------------------------------------------- helpers
    // The first n_step helpers issue the copies. Producer j does tiles j, j + n_step, ... of the run: preparing and issuing a
    // tile's copies takes a warp 0.5 us (pages of 64 rows) to 0.9 us (of 16), and is a chain of latencies that several warps
    // overlap. Two do for the tiles of 128 columns in pages of 32 and more; half as large ones, and eight boxes to a
    // tile, go faster with four: 32 sequences of 16-32K in e4m3 with pages of 16 take 69.1 us with two and 63.6 us with
    // four, with 64 columns 46.1 and 45.2 us, with both 63.1 and 46.8 us. Where two do, four cost up to 1 us (64 sequences
    // of 0.1-0.9K: 21.6 and 22.6 us): the helpers join the chunks too. bf16 tiles are twice as large and gain nothing.
    // Each works in batches of 32 boxes (a box: up to 64 rows of one page; 2 to 8 to a tile), one per lane: the lanes find
    // their boxes' pages for the next batch, whose loads are then in flight while this batch's copies are issued.
    // (Looking one tile ahead instead left 0.9 us per tile, the latency of a page id under load: 5.0 TB/s of an
    // all-global layer's 2.2 GB.)
    const int32_t page = 1 << p.log2_page;
    const int32_t log2_box = min(p.log2_page, 6), box = 1 << log2_box;  // rows of one TMA box
    const int32_t boxes = kDecodeTile >> log2_box, batch_tiles = 32 / boxes;
    const int32_t my_tile = lane / boxes, my_row = (lane % boxes) * box;
    const int32_t log2_step = BF ? 1 : D == 64 || p.log2_page == 4 ? 2 : 1;
    const int32_t n_step = 1 << log2_step;
    // Window: lane k holds pair window + k, whose tiles are [w_end - w.g.n, w_end) of this CTA's run.
    int32_t window = sm.pair0 - 32, w_end = -sm.tile0;  // the pairs before the run: to be followed by its first 32
    DecodePair w = {};
    auto load_window = [&](int32_t u0, int32_t at) {  // `at`: where pair u0's tile 0 lies in the run
      window = u0;
      w = DecodePair{};
      if (u0 + lane < pairs) {
        if (per == 1 && u0 == sm.pair0) w = sm.window[lane];
        else w = decode_pair(p, u0 + lane);
      }
      w_end = w.g.n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int32_t x = __shfl_up_sync(0xffffffffu, w_end, d);
        if (lane >= d) w_end += x;
      }
      w_end += at;
    };
    struct Box {
      int32_t id, row;  // page id as the table has it, first row in the page
      bool need;        // a visible token lies in it
      DecodeTileHeader h;
    } cur, nxt;
    // The header (but b and h0) of the run's tile i, which is tile `tile` of pair u's n; the pair ends before tile `pair_end` of
    // the run. `say`: this lane leaves word of a chunk that the CTAs behind this one go on with.
    auto header = [&](int32_t i, int32_t tile, int32_t n, int32_t u, int32_t pair_end, const DecodeSpan& sp, bool say) {
      DecodeTileHeader h;
      const bool last = i + 1 == tiles || tile + 1 == n;
      h.rows = (sp.lo - sp.t0) | (sp.hi - sp.t0) << 16;
      h.flags = (tile == 0 || i == 0 ? 1 : 0) | (last ? 2 : 0);
      if (last) {
        const bool from_start = tile <= i, to_end = tile + 1 == n;  // does the chunk hold the pair's first, last tile
        if (!(from_start && to_end)) h.flags |= (1 + 2 * cta + (from_start ? 1 : 0)) << 2;
        if (say && from_start && !to_end) {
          // the pair goes on in the CTAs after this one, to the CTA that holds its last tile
          const uint32_t at = 2u * (first_rank + pair_end - 1) + (uint32_t)C::PAIR_COST * u;  // that tile's unit
          const uint32_t wide = (share + 1) * spare;  // units of the CTAs that take one more
          const int32_t to = at < wide ? at / (share + 1) : spare + (at - wide) / share;
          p.part_meta[2 * cta] = u;
          p.part_meta[2 * cta + 1] = to - cta + 1;
        }
      }
      return h;
    };
    // The boxes of tiles i0, i0 + n_step, ... into nxt; returns how many tiles that are (0: the run is done).
    auto plan = [&](int32_t i0) -> int32_t {
      nxt.need = false;
      if (i0 >= tiles) return 0;
      int32_t stop = __shfl_sync(0xffffffffu, w_end, 31);
#pragma unroll 1
      while (stop <= i0) {
        if (window + 32 >= pairs) {  // only if the lengths changed while this call runs
          sm.abort = 1;
          report(p.status, 2);
          return 0;
        }
        load_window(window + 32, stop);
        stop = __shfl_sync(0xffffffffu, w_end, 31);
      }
      stop = min(stop, tiles);
      const int32_t i = min(i0 + my_tile * n_step, stop - 1);
      int32_t k = 0;  // pairs of the window that end at or before tile i
#pragma unroll
      for (int d = 16; d > 0; d >>= 1)
        if (__shfl_sync(0xffffffffu, w_end, k + d - 1) <= i) k += d;
      const int32_t n = __shfl_sync(0xffffffffu, w.g.n, k), end_k = __shfl_sync(0xffffffffu, w_end, k);
      DecodeGeom g;
      g.L = __shfl_sync(0xffffffffu, w.g.L, k);
      g.a1 = __shfl_sync(0xffffffffu, w.g.a1, k);
      g.lo = __shfl_sync(0xffffffffu, w.g.lo, k);
      const int32_t off = __shfl_sync(0xffffffffu, w.off, k), sink = __shfl_sync(0xffffffffu, w.n_sink, k);
      const int32_t w0 = __shfl_sync(0xffffffffu, w.w0, k);
      const int32_t tile = i - (end_k - n);
      const DecodeSpan sp = decode_span(g, tile, p.log2_page);
      const int32_t t0 = sp.t0, lo = sp.lo, hi = sp.hi;
      const bool mine = i0 + my_tile * n_step < stop;
      nxt.h = header(i, tile, n, window + k, end_k, sp, mine && my_row == 0);
      nxt.h.b = __shfl_sync(0xffffffffu, w.b, k);
      nxt.h.h0 = __shfl_sync(0xffffffffu, w.h0, k);
      const int64_t tok = (int64_t)t0 + my_row;
      nxt.need = mine && my_tile < batch_tiles && tok + box > lo && tok < hi;
      nxt.row = (int32_t)(tok & (page - 1));
      nxt.id = 0;
      if (nxt.need) {  // nothing waits for the load before its batch is issued
        const int32_t lp = (int32_t)(tok >> p.log2_page);
        nxt.id = p.table[off + (lp < sink ? lp : lp - w0 + sink)];
      }
      return min(batch_tiles, (stop - i0 + n_step - 1) >> log2_step);
    };
    // Fills stage s with the run's tile i, whose boxes the lanes box_tile * boxes .. have in `c`.
    auto issue = [&](int s, int32_t i, const Box& c, int32_t box_tile) {
      uint8_t* stage = ring + s * C::STAGE_BYTES;
      uint8_t* extra = extras + s * C::EXTRA_BYTES;
      const bool load = my_tile == box_tile && c.need;
      const uint32_t have = __ballot_sync(0xffffffffu, load);
      const int leader = box_tile * boxes;
      const bool with_q = __shfl_sync(0xffffffffu, c.h.flags, leader) & 1;
      if (lane == leader) {
        sm.hdr[s] = c.h;
        sm.last[s] = i;
        ptx::mbar_arrive_expect_tx(&sm.full[s], __popc(have) * 2 * box * D * C::EB + (with_q ? heads * D * 2 : 0));
      }
      __syncwarp();
      if (load) issue_box<C>(stage, tk, tv, my_row, c.row, c.id, &sm.full[s]);
      if (with_q) {
        const int64_t row = (int64_t)__shfl_sync(0xffffffffu, c.h.b, leader) * Hq + __shfl_sync(0xffffffffu, c.h.h0, leader);
        if (lane < heads)
          bulk_load(extra + C::SCALE_BYTES + lane * C::Q_ROW, p.q + (row + lane) * D, D * 2, &sm.full[s]);
      }
      if (!BF) {
        // The tile's exponent bytes, [page][K, V][row], 16 of them a lane: a bulk copy per page would be as many
        // copies again as the codes take where pages are small.
        const int32_t at = lane * 16, from = leader + ((at >> (p.log2_page + 1)) << p.log2_page >> log2_box);
        // of a page of two boxes, either may be the only one that is loaded
        const int32_t box_at = (p.log2_page == log2_box || (have >> (from & 31) & 1) ? from : from + 1) & 31;
        const int32_t id = __shfl_sync(0xffffffffu, c.id, box_at);
        if (lane < C::SCALE_BYTES / 16 && (have >> box_at & 1))
          cp_async16(extra + at, p.kv_scale + ((int64_t)id << (p.log2_page + 1)) + (at & (2 * page - 1)));
        cp_async_arrive(&sm.full[s]);
      }
      __syncwarp();
    };
    auto check_id = [&](Box& c) {
      if (c.need && (uint32_t)c.id >= (uint32_t)p.num_pages) {
        report(p.status, 1);
        c.id = 0;
      }
    };
    // Joins the warps' results of the chunk in mail `k`: each helper those of its quarter's warps (w, w + 4, w + 8), then
    // all four together, a quarter of the columns each.
    uint32_t meets = 0;
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sm.sync);
      const uint32_t parity = meets++ & 1;
#pragma unroll 1
      for (int spin = 0; spin < 256; ++spin)
        if (__all_sync(0xffffffffu, ptx::mbar_test_wait(&sm.sync, parity))) return true;
      return warp_wait(&sm.sync, parity, &sm.abort, p.status);
    };
    constexpr int KS = D / 16, OC = D / 4;
    const int g = lane >> 2, t = lane & 3, quarter = warp & 3;
    auto join = [&](int k, uint32_t chunk) {
      const auto& mail = sm.mail[k];
      ptx::tc_fence_after();
      const int32_t b = mail.b, h0 = mail.h0, slot = mail.slot;
      // The largest unit of the warps' O. It is applied to the finished quotients: as part of a weight it would take
      // values near the smallest floats below them.
      int32_t vtop = 0;
      if (!BF) {
        const int32_t v = lane < C::WARPS ? mail.vref[lane] : 255 << 8;
        vtop = __reduce_max_sync(0xffffffffu, v & 255);
        if (vtop - __reduce_min_sync(0xffffffffu, v >> 8) > kDecodeSpread && warp == C::WARPS && lane == 0)
          sm.redo |= 1u << min(chunk, 31u);
      }
      const float unit = BF ? 1.f : row_scale(vtop);
#pragma unroll 1
      for (int nb = 0; nb < NB; ++nb) {
        const bool live = nb * 8 + 2 * t < heads;  // this lane's columns are heads of the group
        // the largest m of this lane's two heads and the sum of all l to it: lane (g, t) looks at warps g and g + 8
        float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
        float2 mx[2], lx[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          mx[x] = make_float2(-INFINITY, -INFINITY);
          lx[x] = make_float2(0.f, 0.f);
          if (8 * x + g < C::WARPS) {
            mx[x] = *reinterpret_cast<const float2*>(&mail.m[(8 * x + g) * 8 * NB + nb * 8 + 2 * t]);
            lx[x] = *reinterpret_cast<const float2*>(&mail.l[(8 * x + g) * 8 * NB + nb * 8 + 2 * t]);
          }
          top[0] = fmaxf(top[0], mx[x].x);
          top[1] = fmaxf(top[1], mx[x].y);
        }
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          top[0] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], d));
          top[1] = fmaxf(top[1], __shfl_xor_sync(0xffffffffu, top[1], d));
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          sum[0] += (mx[x].x == -INFINITY ? 0.f : ptx::ex2(mx[x].x - top[0])) * lx[x].x;
          sum[1] += (mx[x].y == -INFINITY ? 0.f : ptx::ex2(mx[x].y - top[1])) * lx[x].y;
        }
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], d);
          sum[1] += __shfl_xor_sync(0xffffffffu, sum[1], d);
        }
        float acc[OC];
#pragma unroll
        for (int c = 0; c < OC; ++c) acc[c] = 0.f;
#pragma unroll 1
        for (int x = 0; x < C::WARPS / 4; ++x) {
          uint32_t r[OC];
          tmem_get<OC>(tmem + k * C::MAIL_COLS + x * C::OCOLS + nb * OC, r);
          const int from = quarter + 4 * x;  // consumer warp w is on the quarter w mod 4
          const float2 mw = *reinterpret_cast<const float2*>(&mail.m[from * 8 * NB + nb * 8 + 2 * t]);
          const float rel = BF ? 1.f : exp2_int((mail.vref[from] & 255) - vtop - 14);
          const float w0 = mw.x == -INFINITY ? 0.f : ptx::ex2(mw.x - top[0]) * rel;
          const float w1 = mw.y == -INFINITY ? 0.f : ptx::ex2(mw.y - top[1]) * rel;
          ptx::tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < OC; ++c) acc[c] += __uint_as_float(r[c]) * (c & 1 ? w1 : w0);
        }
        float4* mine = merge + quarter * KS * 32 + lane;
#pragma unroll
        for (int mt = 0; mt < KS; ++mt)
          mine[mt * 32] = make_float4(acc[4 * mt], acc[4 * mt + 1], acc[4 * mt + 2], acc[4 * mt + 3]);
        if (!meet()) return false;
        if (live) {
          const float inv[2] = {__fdividef(1.f, sum[0]), __fdividef(1.f, sum[1])};
#pragma unroll
          for (int y = 0; y < KS / 4; ++y) {
            const int mt = quarter * (KS / 4) + y;
            float4 v[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) v[x] = merge[(x * KS + mt) * 32 + lane];
            const float out[2][2] = {{(v[0].x + v[1].x) + (v[2].x + v[3].x), (v[0].z + v[1].z) + (v[2].z + v[3].z)},
                                     {(v[0].y + v[1].y) + (v[2].y + v[3].y), (v[0].w + v[1].w) + (v[2].w + v[3].w)}};
            const int d0 = 16 * mt + (BF ? g : 2 * g), d1 = d0 + (BF ? 8 : 1);
#pragma unroll
            for (int j = 0; j < 2; ++j) {  // out[head][dim]
              const int head = nb * 8 + 2 * t + j;
              if (head >= heads) continue;
              if (slot < 0) {
                __nv_bfloat16* to = p.o + ((int64_t)b * Hq + h0 + head) * D;
                to[d0] = __float2bfloat16_rn(out[j][0] * inv[j] * unit);
                to[d1] = __float2bfloat16_rn(out[j][1] * inv[j] * unit);
              } else {
                float* to = p.part_o + ((int64_t)slot * kDecodeGroup + head) * D;
                to[d0] = out[j][0] * inv[j] * unit;
                to[d1] = out[j][1] * inv[j] * unit;
              }
            }
          }
          if (quarter == 0 && g == 0)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int head = nb * 8 + 2 * t + j;
              if (head >= heads) continue;
              if (slot < 0) p.lse[(int64_t)(h0 + head) * p.B + b] = 0.6931471805599453f * (top[j] + log2f(sum[j]));
              else p.part_sum[(int64_t)slot * kDecodeGroup + head] = make_float2(top[j], sum[j]);
            }
        }
        if (!meet()) return false;  // `merge` is free again
      }
      ptx::tc_fence_before();
      return true;
    };

    // Both jobs in turn: a copy as soon as its stage is free, a join as soon as a chunk is in the mail.
    int32_t i = warp - C::WARPS, left = 0, at_box = 0, ahead = -1;
    bool producing = tiles > 0 && i < n_step, done = tiles == 0;
    uint32_t mails = 0;
    int32_t idle = 0;
    cur.need = nxt.need = false;
    if (per == 1 && warp == C::WARPS && tiles > 0 && sm.window[0].g.n > sm.tile0) {
      // Tile 0 straight from its pair's geometry, 0.7 us before the first batch is planned.
      const DecodePair& w0 = sm.window[0];
      const int32_t tile = sm.tile0;
      const DecodeSpan sp = decode_span(w0.g, tile, p.log2_page);
      const int64_t tok = (int64_t)sp.t0 + my_row;
      cur.need = my_tile == 0 && tok + box > sp.lo && tok < sp.hi;
      cur.row = (int32_t)(tok & (page - 1));
      cur.id = 0;
      if (cur.need) {
        const int32_t lp = (int32_t)(tok >> p.log2_page);
        cur.id = p.table[w0.off + (lp < w0.n_sink ? lp : lp - w0.w0 + w0.n_sink)];
      }
      cur.h = header(0, tile, w0.g.n, sm.pair0, w0.g.n - tile, sp, lane == 0);
      cur.h.b = w0.b;
      cur.h.h0 = w0.h0;
      check_id(cur);
      issue(0, 0, cur, 0);
      i = n_step;
      cur.need = false;
    }
#pragma unroll 1
    while (producing || !done) {
      if (producing && left == 0) {  // the batch that was planned last becomes the current one
        if (ahead == 0) {
          producing = false;
          continue;
        }
        cur = nxt;
        left = max(ahead, 0);
        at_box = 0;
        ahead = plan(i + left * n_step);
        check_id(cur);
        continue;
      }
      if (producing) {
        const int s = i % C::STAGES;
        if (i < C::STAGES || __all_sync(0xffffffffu, ptx::mbar_try_wait(&sm.empty[s], ((i / C::STAGES) - 1) & 1))) {
          idle = 0;
          issue(s, i, cur, at_box);
          --left;
          ++at_box;
          i += n_step;
        }
      }
      if (!done) {
        const int k = mails % kDecodeMails;
        const uint32_t parity = mails / kDecodeMails & 1;
        if (__all_sync(0xffffffffu, producing ? ptx::mbar_test_wait(&sm.mail_full[k], parity)
                                              : ptx::mbar_try_wait(&sm.mail_full[k], parity))) {
          idle = 0;
          done = sm.mail[k].final != 0;
          if (!join(k, mails)) break;
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&sm.mail_empty[k]);
          ++mails;
        }
      }
      if ((++idle & (SEGPAGED_DECODE_IDLE_CHECK - 1)) == 0) {  // a bounded wait, as ptx::mbar_wait
        if (idle > SEGPAGED_DECODE_IDLE_TRIES) {
          sm.abort = 1;
          report(p.status, kDecodeStatusTimeout);
        }
        if (__any_sync(0xffffffffu, *(volatile int32_t*)&sm.abort != 0)) break;
      }
    }
  } else {
    // ----------------------------------------------------------------------------------- consumers
    constexpr int KS = D / 16;  // k16 steps of a logit, and m16 tiles of O^T
    const int g = lane >> 2, t = lane & 3;
    constexpr int MB = C::MB;
    const int turn = warp / C::TILE_WARPS;  // which tiles, counted modulo TURNS, this warp takes part in
    const int row0 = (warp % C::TILE_WARPS) * 16 * MB;
    // ldmatrix row of this lane in a block of 16 tokens, and its 16-byte chunk (0 or 1 of a pair). The swizzle XORs a
    // few row bits into the chunk bits of the address, so chunk c of the row is at (address of chunk 0) ^ (c << 4).
    const int lrow = row0 + (lane & 15), lchunk = lane >> 4;                                   // K, and 8-bit V
    const int trow = row0 + (lane & 7) + (lane >> 4) * 8, tchunk = (lane >> 3) & 1;            // bf16 V
    auto lane_base = [](int row, int chunk) {
      return C::ROWB == 128 ? row * 128 + ((chunk ^ (row & 7)) << 4) : row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
    };
    const uint32_t k_lane = lane_base(lrow, lchunk);
    const uint32_t v_lane = C::TILE_BYTES + (BF ? lane_base(trow, tchunk) : k_lane);
    // chunk c (even) of block mb
    auto chunk_addr = [](uint32_t base, int c, int mb) {
      return (base ^ ((c & 7) << 4)) + (c >> 3) * C::BLOCK_BYTES + mb * 16 * C::ROWB;
    };
    uint32_t qf[NB][KS][2];
    // Logits y are kept in log2 units, rounded to fp32 once, and a probability is 2^(y - m): at most 1, and 1 at the
    // maximum, whatever the size of y. (A product with the scale and the subtraction as one fma would be off by the
    // rounding of the scaled maximum, a factor of 2 or more from logits of 2^25 on: past the range of fp16, then of fp32.)
    float head_scale[NB][2];                     // of heads 2t, 2t + 1: what takes q' . k' to y but for the K row's exponent
    float m[NB][2], l[NB][2], o[NB][KS][4];
    int32_t vref = 0;                            // r + 127: the largest y of the chunk so far
    int32_t vlow = 255;                          // the smallest that this lane saw
    uint32_t mails = 0;
    int tick = 0, s = -1;
    uint32_t phase = 1;
    for (int32_t i = 0; i < tiles; ++i) {
      s = s + 1 == C::STAGES ? 0 : s + 1;
      phase ^= s == 0;
      if (!warp_wait(&sm.full[s], phase, &sm.abort, p.status)) break;
      const DecodeTileHeader h = sm.hdr[s];
      const int32_t v0 = h.rows & 0xffff, v1 = h.rows >> 16;
      const uint32_t kbase = ptx::smem_addr(ring + s * C::STAGE_BYTES) + k_lane;
      const uint32_t vbase = ptx::smem_addr(ring + s * C::STAGE_BYTES) + v_lane;
      const uint8_t* extra = extras + s * C::EXTRA_BYTES;
      if (h.flags & 1) {
        // ---- a chunk begins: query fragments, running values
        const uint8_t* qs = extra + C::SCALE_BYTES;
        vref = 0;
        vlow = 255;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const int head = nb * 8 + g;
          uint32_t top = 0;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              // fp16: the contraction runs in the order the code bytes lie in, 4t .. 4t+3 of each 16
              const int d = 16 * ks + (BF ? 2 * t + 8 * j : 4 * t + 2 * j);
              qf[nb][ks][j] = head < heads ? *reinterpret_cast<const uint32_t*>(qs + head * C::Q_ROW + 2 * d) : 0u;
              top = absmax2(top, qf[nb][ks][j]);
            }
          }
          if (BF) {
            head_scale[nb][0] = head_scale[nb][1] = p.scale_log2;
          } else {
            top = max2(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max2(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int32_t biased = (int32_t)(max(top & 0xffffu, top >> 16) >> 7);
            const int32_t e = biased == 255 ? 0 : 15 - max(biased - 127, -100);  // not finite: as it is
            const float up = exp2_int(e);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                qf[nb][ks][j] = pack_f16x2(bf16_lo(qf[nb][ks][j]) * up, bf16_hi(qf[nb][ks][j]) * up);
            const float back = p.scale_log2 * exp2_int(-e);
            head_scale[nb][0] = __shfl_sync(0xffffffffu, back, 8 * t);
            head_scale[nb][1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            m[nb][j] = -INFINITY;
            l[nb][j] = 0.f;
          }
#pragma unroll
          for (int mt = 0; mt < KS; ++mt) o[nb][mt][0] = o[nb][mt][1] = o[nb][mt][2] = o[nb][mt][3] = 0.f;
        }
      }
      const bool my_turn = C::TURNS == 1 || tick == turn;
      tick = tick + 1 == C::TURNS ? 0 : tick + 1;
      auto process = [&](auto edge_tile) {
        constexpr bool edge = decltype(edge_tile)::value;  // some of the warp's tokens are hidden
        // ---- logits: rows = tokens g, g + 8 of each block; columns = heads 2t, 2t + 1
        float sc[MB][NB][4];
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) sc[mb][nb][0] = sc[mb][nb][1] = sc[mb][nb][2] = sc[mb][nb][3] = 0.f;
        if (BF) {
#pragma unroll
          for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) {
              uint32_t a[4];
              ldsm4(chunk_addr(kbase, 2 * ks, mb), a);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
                mma16816<true>(sc[mb][nb], a[0], a[1], a[2], a[3], qf[nb][ks][0], qf[nb][ks][1]);
            }
        } else {
#pragma unroll
          for (int ks = 0; ks < KS; ks += 2)
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) {
              uint32_t a[4];
              ldsm4(chunk_addr(kbase, ks, mb), a);
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                uint32_t a0, a1, a2, a3;
                codes_to_half2x2<FMT, false>(a[2 * j], a0, a2);
                codes_to_half2x2<FMT, false>(a[2 * j + 1], a1, a3);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
                  mma16816<false>(sc[mb][nb], a0, a1, a2, a3, qf[nb][ks + j][0], qf[nb][ks + j][1]);
              }
            }
        }
        bool in[MB][2];
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          const int r = row0 + 16 * mb + g;
          in[mb][0] = !edge || (r >= v0 && r < v1);
          in[mb][1] = !edge || (r + 8 >= v0 && r + 8 < v1);
        }
        // Exponents: lane x works out token x's (of the warp's 16 MB), the lanes that hold its logits fetch them.
        float kscale[MB][2], vscale[MB][2], vshift = 1.f;
        if (!BF) {
          const int r = row0 + (lane & (16 * MB - 1));
          const uint8_t* at = extra + r + (r >> p.log2_page << p.log2_page);  // [page of the tile][K, V][row]
          const float k_mine = row_scale(at[0]);
          const int32_t y = at[1 << p.log2_page];
          const bool seen = !edge || (r >= v0 && r < v1);
          const int32_t top = max(vref, __reduce_max_sync(0xffffffffu, seen && y != kRowNaN ? y : 0));
          vlow = min(vlow, seen ? y : 255);
          // a hidden token's byte may be anything: its weight is zero whatever that says
          const float v_mine = !seen ? 0.f : y == kRowNaN ? __uint_as_float(0x7fffffffu) : exp2_int(y - top + 14);
          vshift = exp2_int(vref - top);
          vref = top;
#pragma unroll
          for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              kscale[mb][j] = __shfl_sync(0xffffffffu, k_mine, 16 * mb + 8 * j + g);
              vscale[mb][j] = __shfl_sync(0xffffffffu, v_mine, 16 * mb + 8 * j + g);
            }
        }
        uint32_t pf[MB][NB][2], pl[MB][NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const float f0 = head_scale[nb][0], f1 = head_scale[nb][1];
          float n0 = -INFINITY, n1 = -INFINITY;
#pragma unroll
          for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float& x0 = sc[mb][nb][2 * j];
              float& x1 = sc[mb][nb][2 * j + 1];
              x0 *= f0;  // before the K row's exponent: a scale that makes up for large keys does so in time
              x1 *= f1;
              if (!BF) {
                x0 *= kscale[mb][j];
                x1 *= kscale[mb][j];
              }
              if (edge) {
                x0 = in[mb][j] ? x0 : -INFINITY;
                x1 = in[mb][j] ? x1 : -INFINITY;
              }
              n0 = fmaxf(n0, x0);
              n1 = fmaxf(n1, x1);
            }
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) {
            n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, d));
            n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, d));
          }
          n0 = fmaxf(n0, m[nb][0]);
          n1 = fmaxf(n1, m[nb][1]);
          // a larger maximum (or V exponent) rescales what was summed so far
          if (__any_sync(0xffffffffu, n0 != m[nb][0] || n1 != m[nb][1] || vshift != 1.f)) {
            const float c0 = m[nb][0] == -INFINITY ? 0.f : ptx::ex2(m[nb][0] - n0);
            const float c1 = m[nb][1] == -INFINITY ? 0.f : ptx::ex2(m[nb][1] - n1);
            // NaN sums stay NaN: 0 * NaN
            l[nb][0] *= c0;
            l[nb][1] *= c1;
            const float w0 = c0 * vshift, w1 = c1 * vshift;
#pragma unroll
            for (int mt = 0; mt < KS; ++mt) {
              o[nb][mt][0] *= w0;
              o[nb][mt][1] *= w1;
              o[nb][mt][2] *= w0;
              o[nb][mt][3] *= w1;
            }
            m[nb][0] = n0;
            m[nb][1] = n1;
          }
          const float b0 = n0 == -INFINITY ? 0.f : n0, b1 = n1 == -INFINITY ? 0.f : n1;
#pragma unroll
          for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float p0 = ptx::ex2(sc[mb][nb][2 * j] - b0), p1 = ptx::ex2(sc[mb][nb][2 * j + 1] - b1);
              l[nb][0] += p0;
              l[nb][1] += p1;
              if (BF) {
                const uint32_t hi = ptx::pack_bf16x2(p0, p1);
                pf[mb][nb][j] = transpose8x8(hi);
                pl[mb][nb][j] = transpose8x8(ptx::pack_bf16x2(p0 - bf16_lo(hi), p1 - bf16_hi(hi)));
              } else {
                pf[mb][nb][j] = transpose8x8(pack_f16x2(p0 * vscale[mb][j], p1 * vscale[mb][j]));
              }
            }
        }
        // ---- O^T += V^T P^T. Rows outside [v0, v1) may hold NaN: their bits are cleared (tokens 2t, 2t+1 | +8)
        uint32_t keep[MB][2];
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int j = 0; edge && j < 2; ++j) {
            const int r = row0 + 16 * mb + 8 * j + 2 * t;
            keep[mb][j] = (r >= v0 && r < v1 ? 0xffffu : 0u) | (r + 1 >= v0 && r + 1 < v1 ? 0xffff0000u : 0u);
          }
        if (BF) {
#pragma unroll
          for (int mt = 0; mt < KS; ++mt)
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) {
              uint32_t a[4];
              ldsm4_t(chunk_addr(vbase, 2 * mt, mb), a);
              if (edge) {
                a[0] &= keep[mb][0];
                a[1] &= keep[mb][0];
                a[2] &= keep[mb][1];
                a[3] &= keep[mb][1];
              }
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                mma16816<true>(o[nb][mt], a[0], a[1], a[2], a[3], pf[mb][nb][0], pf[mb][nb][1]);
                mma16816<true>(o[nb][mt], a[0], a[1], a[2], a[3], pl[mb][nb][0], pl[mb][nb][1]);
              }
            }
        } else {
#pragma unroll
          for (int mt = 0; mt < KS; mt += 2)
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) {
              uint32_t a[4];
              ldsm4_t(chunk_addr(vbase, mt, mb), a);
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                // bytes of a register: token 2t's codes of dims 2g, 2g+1, then token 2t+1's
                uint32_t a0, a1, a2, a3;
                codes_to_half2x2<FMT, true>(a[2 * j], a0, a1);
                codes_to_half2x2<FMT, true>(a[2 * j + 1], a2, a3);
                if (edge) {
                  a0 &= keep[mb][0];
                  a1 &= keep[mb][0];
                  a2 &= keep[mb][1];
                  a3 &= keep[mb][1];
                }
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
                  mma16816<false>(o[nb][mt + j], a0, a1, a2, a3, pf[mb][nb][0], pf[mb][nb][1]);
              }
            }
        }
      };
      if (my_turn && row0 + 16 * MB > v0 && row0 < v1) {
        if (row0 < v0 || row0 + 16 * MB > v1) process(Flag<true>{});
        else process(Flag<false>{});
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sm.empty[s]);  // this warp has read its rows
      if (!(h.flags & 2)) continue;

      // ---- a chunk ends: this warp's result goes into the mail, and it goes on to the next chunk
      const int k = mails % kDecodeMails;
      if (mails >= kDecodeMails && !warp_wait(&sm.mail_empty[k], (mails / kDecodeMails - 1) & 1, &sm.abort, p.status)) break;
      ++mails;
      ptx::tc_fence_after();
      auto& mail = sm.mail[k];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) l[nb][j] += __shfl_xor_sync(0xffffffffu, l[nb][j], d);
          if (g == 0) {
            mail.m[(warp * NB + nb) * 8 + 2 * t + j] = m[nb][j];
            mail.l[(warp * NB + nb) * 8 + 2 * t + j] = l[nb][j];
          }
        }
        tmem_put<D / 4>(tmem + k * C::MAIL_COLS + (warp >> 2) * C::OCOLS + nb * (D / 4),
                        reinterpret_cast<const uint32_t*>(&o[nb][0][0]));
      }
      if (!BF) vlow = __reduce_min_sync(0xffffffffu, vlow);
      if (lane == 0) {
        mail.vref[warp] = vref | vlow << 8;
        if (warp == 0) {
          mail.b = h.b;
          mail.h0 = h.h0;
          mail.slot = (h.flags >> 2) - 1;
          mail.final = i + 1 == tiles;
        }
      }
      ptx::tmem_st_wait();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sm.mail_full[k]);
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == C::WARPS) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(sm.tmem, C::TMEM_COLS);
    // After a timeout: the copies in flight land before the block's memory is given up. Nobody issues any more, so that the
    // last tile of a stage is the one its barrier's phase is at. (For its tile before that a parity could be one of two.)
    if (sm.abort) {
#pragma unroll 1
      for (int s = 0; s < C::STAGES; ++s)
        if (sm.last[s] >= 0)
          ptx::mbar_wait(&sm.full[s], (sm.last[s] / C::STAGES) & 1, nullptr, p.status, kDecodeStatusTimeout);
    }
  }
  if constexpr (!BF) {
    static_assert(4 * redo_scratch<D>(C::WARPS + kDecodeHelpers) <= C::STAGES * C::STAGE_BYTES, "decode_redo's scratch");
    if (sm.redo != 0 && !sm.abort)
      decode_redo<D, FMT>(p, reinterpret_cast<float*>(ring), sm.pair0, sm.tile0, sm.end_rank - sm.first_rank, sm.redo,
                          C::WARPS + kDecodeHelpers);
  }
}

// Joins the chunks of the pairs that several CTAs shared: with w_c = 2^(m_c - m) l_c, m the largest m_c, O is the mean of the
// O_c weighted by w_c and LSE = ln 2 (m + log2 sum_c w_c). (A chunk's m + log2 l as one float would lose its l to rounding
// where m is large.)
// CTA c's last pair, if it goes on behind it, has n chunks: CTA c's second slot and the first slots of the n - 1 CTAs
// after it. Block (c, head) joins them: each of its eight warps takes every eighth chunk, a lane D/32 columns, and the
// warps' sums are added in order. The loads of five chunks a warp are in flight together with those of all the log
// sums, so a pair of up to 40 chunks waits for memory twice (which pair, then its chunks), one of 148 five times.
constexpr int kDecodeCombineWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kDecodeCombineWarps, 5) decode_combine_kernel(const DecodeParams p) {
  constexpr int E = D / 32, NW = kDecodeCombineWarps, U = 5;
  __shared__ float s_m[kDecodeMaxCtas], s_l[kDecodeMaxCtas], s_sum[NW], s_top[NW], s_o[NW][D];
  const int32_t cta = blockIdx.x, head = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  early_start();  // the partial results of the launch before this one
  const int2 meta = *reinterpret_cast<const int2*>(p.part_meta + 2 * cta);
  const int32_t pair = meta.x, n = min(meta.y, kDecodeMaxCtas);
  if (n <= 1) return;
  auto slot = [&](int32_t c) { return (c == 0 ? 2 * cta + 1 : 2 * (cta + c)) * kDecodeGroup + head; };
  float v[U][E];
  auto load = [&](int32_t c0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int32_t c = c0 + u * NW;
      if (c >= n) continue;
      const float* from = p.part_o + (int64_t)slot(c) * D + lane * E;
      if (E == 4) *reinterpret_cast<float4*>(v[u]) = *reinterpret_cast<const float4*>(from);
      else *reinterpret_cast<float2*>(v[u]) = *reinterpret_cast<const float2*>(from);
    }
  };
  load(warp);  // on its way while the weights are worked out
  float top = -INFINITY;
  for (int32_t c = threadIdx.x; c < n; c += 32 * NW) {
    const float2 x = p.part_sum[slot(c)];
    s_m[c] = x.x;
    s_l[c] = x.y;
    top = fmaxf(top, x.x);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  if (lane == 0) s_top[warp] = top;
  __syncthreads();
#pragma unroll
  for (int x = 0; x < NW; ++x) top = fmaxf(top, s_top[x]);
  float sum = 0.f, o[E] = {};
  for (int32_t c0 = warp; c0 < n; c0 += U * NW) {
    if (c0 != warp) load(c0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int32_t c = c0 + u * NW;
      if (c >= n) continue;
      const float w = (s_m[c] == -INFINITY ? 0.f : ptx::ex2(s_m[c] - top)) * s_l[c];
      sum += w;
#pragma unroll
      for (int k = 0; k < E; ++k) o[k] += w == 0.f ? 0.f : w * v[u][k];
    }
  }
#pragma unroll
  for (int k = 0; k < E; ++k) s_o[warp][lane * E + k] = o[k];
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  const int d = threadIdx.x;
  if (d >= D) return;
  float acc = 0.f;
  sum = 0.f;
#pragma unroll
  for (int x = 0; x < NW; ++x) {
    acc += s_o[x][d];
    sum += s_sum[x];
  }
  const int32_t bk = pair >> p.log2_hg, b = bk / p.Hkv;
  const int32_t h = (bk - b * p.Hkv) * p.G + (pair - (bk << p.log2_hg)) * kDecodeGroup + head;
  p.o[((int64_t)b * p.Hkv * p.G + h) * D + d] = __float2bfloat16_rn(__fdividef(acc, sum));
  if (d == 0) p.lse[(int64_t)h * p.B + b] = 0.6931471805599453f * (top + log2f(sum));
}

}  // namespace segpaged
