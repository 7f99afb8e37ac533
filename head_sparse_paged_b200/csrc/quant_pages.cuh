// quant_pages.cuh -- the kernels that write 8-bit pages, append new rows to a pool, and read 8-bit pages back.
//
// All three move each byte once and are bound by HBM: 2 bytes read and 1 written per element (the write), or the
// reverse (the read back). A warp takes 8 rows of a page and issues all their loads before it uses the first: 4 KB (2 KB
// for the read back) in flight a warp, in slices small enough to spread evenly over the GPU. On a batch of four 16-32K
// contexts (126 MB) that takes 23.2 us for the write and 22.8 us for the read back, 5.4 and 5.5 TB/s, where a plain copy of
// as many bytes takes 23.4 us. (Without the early start of the launches 25.1 and 25.0 us, against 26.8 and 25.0 us with
// slices of 16 rows, and 30.7 us both ways with a whole page per block, found by a binary search: 2.5 us of dependent loads
// before each page's data, and blocks with three pages beside blocks with two.)
// In the kernels that quantise, lane c of a row holds its elements 8c .. 8c+7 and D/2 + 8c .. D/2 + 8c+7, the pairs that
// the RoPE re-alignment rotates, so that the row's largest magnitude is taken of the rotated bf16 values: a pool written
// here holds the quantised form of exactly the rows that build_scatter_kernel would store.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "build_kernel.cuh"
#include "plan.h"
#include "quant_rows.cuh"
#include "rope.cuh"

namespace segpaged {

constexpr int kLog2SliceRows = 3, kSliceRows = 1 << kLog2SliceRows;  // rows of a page that one warp takes
constexpr int kSliceWarps = 4;  // warps of a block

// Pages of one (sequence, KV head) as storage_split gives them, with shifts for its divisions, from arrays that no host
// check has seen: a negative length or sink counts as 0, a window below 1 as 1, fewer than min_q query rows as that.
struct HeadPages {
  int32_t L, sink, window, n_sink, w0, total;
  bool global;
  // logical page of table index t, and the table index of a logical page (-1: not kept)
  __device__ __forceinline__ int32_t logical(int32_t t) const { return t < n_sink ? t : w0 + (t - n_sink); }
  __device__ __forceinline__ int32_t index(int32_t lp) const { return lp < n_sink ? lp : lp < w0 ? -1 : lp - w0 + n_sink; }
};

__device__ __forceinline__ HeadPages head_pages(int32_t L, int32_t lq, const int32_t* cls, int32_t bk, int32_t log2_page) {
  HeadPages r;
  const int32_t last = (1 << log2_page) - 1;
  r.L = max(L, 0);
  r.global = cls[3 * bk] != 0;
  r.sink = min(max(cls[3 * bk + 1], 0), r.L);
  r.window = max(cls[3 * bk + 2], 1);
  const int32_t n_all = (int32_t)(((uint32_t)r.L + last) >> log2_page);
  r.n_sink = (int32_t)(((uint32_t)r.sink + last) >> log2_page);
  r.w0 = (int32_t)(max((int64_t)r.L - lq - r.window + 1, (int64_t)0) >> log2_page);
  if (r.global || r.w0 <= r.n_sink) r.n_sink = r.w0 = n_all;  // sink and window pages meet: everything is kept
  r.total = r.n_sink + n_all - r.w0;
  return r;
}
__device__ __forceinline__ HeadPages head_pages(const int32_t* ctx_len, const int32_t* q_len, const int32_t* cls, int32_t b,
                                                int32_t bk, int32_t log2_page, int32_t min_q) {
  return head_pages(ctx_len[b], max(q_len ? q_len[b] : 1, min_q), cls, bk, log2_page);
}

// Largest index i in [0, n) with start[i] <= x (0 if there is none), for ascending starts: 32 of them a round. Whatever
// the array holds, the result is in [0, n).
__device__ __forceinline__ int32_t warp_find(const int32_t* start, int32_t n, int64_t x) {
  int32_t lo = 0;
  while (n > 1) {
    const int32_t step = (n + 31) >> 5, i = (threadIdx.x & 31) * step;
    const bool le = i < n && start[lo + i] <= x;
    const int32_t k = max(__popc(__ballot_sync(0xffffffffu, le)) - 1, 0) * step;
    lo += k;
    n = min(step, n - k);
  }
  return lo;
}

// One row's piece: elements 8c .. 8c+7 (lo) and D/2 + 8c .. (hi) of lane c.
struct RowPiece {
  uint4 lo, hi;
};

// The row's exponent byte, from the pieces of its LANES lanes (a power of two, aligned within the warp).
template <int FMT, int LANES>
__device__ __forceinline__ int32_t row_byte(const RowPiece& r) {
  uint32_t m = absmax2(absmax2(absmax2(absmax2(0u, r.lo.x), r.lo.y), r.lo.z), r.lo.w);
  m = absmax2(absmax2(absmax2(absmax2(m, r.hi.x), r.hi.y), r.hi.z), r.hi.w);
#pragma unroll
  for (int d = LANES / 2; d > 0; d >>= 1) m = max2(m, __shfl_xor_sync(0xffffffffu, m, d));
  return row_exponent_byte<FMT>(max(m & 0xffffu, m >> 16));
}

template <int FMT>
__device__ __forceinline__ void store_codes(uint8_t* row, int c, int half, const RowPiece& r, int32_t y) {
  uint2 lo = make_uint2(0, 0), hi = lo;
  if (y != kRowNaN) {
    const float inv = row_inverse_scale(y);
    lo = make_uint2(quantise4<FMT>(r.lo.x, r.lo.y, inv), quantise4<FMT>(r.lo.z, r.lo.w, inv));
    hi = make_uint2(quantise4<FMT>(r.hi.x, r.hi.y, inv), quantise4<FMT>(r.hi.z, r.hi.w, inv));
  }
  *reinterpret_cast<uint2*>(row + 8 * c) = lo;
  *reinterpret_cast<uint2*>(row + half + 8 * c) = hi;
}

// For kernels that may be launched while the work before them still runs: waits for its end, before anything is read or
// written, and lets the launch after this one get ready meanwhile. What that work wrote is read with ordinary loads:
// __ldg takes memory that nobody writes while the kernel runs, its wait included, and may be moved above the wait.
__device__ __forceinline__ void early_start() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

struct BuildQuantParams {
  BuildParams b;       // k_pool, v_pool unused
  uint8_t* k_pool;     // [num_pages][P][D] codes
  uint8_t* v_pool;
  uint8_t* kv_scale;   // [num_pages][2][P] exponent bytes, K then V
  int64_t table_len;
  int32_t log2_page;
};

template <int D, int FMT, bool ROPE>
__global__ void __launch_bounds__(32 * kSliceWarps) build_quant_kernel(BuildQuantParams q) {
  const BuildParams& p = q.b;
  constexpr int LANES = D / 16, ROWS = 32 / LANES, N = kSliceRows / ROWS;  // lanes of a row, rows a pass, passes
  const int lane = threadIdx.x & 31, c = lane % LANES;
  early_start();
  const int nheads = p.B * p.Hkv, log2_slices = q.log2_page - kLog2SliceRows;
  const int64_t slices = q.table_len << log2_slices, begin = p.offs[0], entries = p.offs[nheads];
  if (blockIdx.x == 0 && threadIdx.x == 0 && entries > q.table_len) report(p.status, 2);
  const int64_t warps = (int64_t)gridDim.x * kSliceWarps;
  for (int64_t x = (int64_t)blockIdx.x * kSliceWarps + (threadIdx.x >> 5); x < slices; x += warps) {
    const int64_t e = x >> log2_slices;
    const int32_t row0 = (int32_t)(x & ((1 << log2_slices) - 1)) * kSliceRows;
    const int32_t pid = p.table[e];
    if (e < begin) continue;  // spare room before the first table
    if (e >= entries) break;  // and behind the last
    const int bk = warp_find(p.offs, nheads, e), b = bk / p.Hkv, kh = bk - b * p.Hkv;
    const int32_t t = (int32_t)(e - p.offs[bk]);
    const int64_t src0 = p.cu_k[b];
    const HeadPages hp = head_pages((int32_t)(p.cu_k[b + 1] - src0), max(p.q_len[b], 0), p.cls, bk, q.log2_page);
    if (p.offs[bk + 1] - p.offs[bk] != hp.total) {
      if (lane == 0) report(p.status, 2);
      if (t < 0 || t >= hp.total) continue;
    }
    if (pid < 0 || pid >= p.num_pages) {
      if (lane == 0) report(p.status, 1);
      continue;
    }
    const int64_t tok0 = ((int64_t)hp.logical(t) << q.log2_page) + row0;
    RowPiece k[N], v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      k[i].lo = k[i].hi = v[i].lo = v[i].hi = make_uint4(0, 0, 0, 0);  // rows past the context end
      const int64_t tok = tok0 + i * ROWS + lane / LANES;
      if (tok >= hp.L) continue;
      const int64_t src = ((src0 + tok) * p.Hkv + kh) * D + 8 * c;
      k[i].lo = *reinterpret_cast<const uint4*>(p.k_dense + src);
      k[i].hi = *reinterpret_cast<const uint4*>(p.k_dense + src + D / 2);
      v[i].lo = *reinterpret_cast<const uint4*>(p.v_dense + src);
      v[i].hi = *reinterpret_cast<const uint4*>(p.v_dense + src + D / 2);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (ROPE) {  // (rows of zeros stay rows of zeros)
        const float4* t4 = reinterpret_cast<const float4*>(p.cos_sin + (int64_t)b * D + 16 * c);
        const float4 q0 = t4[0], q1 = t4[1], q2 = t4[2], q3 = t4[3];
        RowPiece r;
        r.lo.x = rot_pair(k[i].lo.x, k[i].hi.x, q0.x, q0.y, q0.z, q0.w, &r.hi.x);
        r.lo.y = rot_pair(k[i].lo.y, k[i].hi.y, q1.x, q1.y, q1.z, q1.w, &r.hi.y);
        r.lo.z = rot_pair(k[i].lo.z, k[i].hi.z, q2.x, q2.y, q2.z, q2.w, &r.hi.z);
        r.lo.w = rot_pair(k[i].lo.w, k[i].hi.w, q3.x, q3.y, q3.z, q3.w, &r.hi.w);
        k[i] = r;
      }
      const int32_t ky = row_byte<FMT, LANES>(k[i]), vy = row_byte<FMT, LANES>(v[i]);
      const int32_t row = row0 + i * ROWS + lane / LANES;
      const int64_t at = (((int64_t)pid << q.log2_page) + row) * D;
      store_codes<FMT>(q.k_pool + at, c, D / 2, k[i], ky);
      store_codes<FMT>(q.v_pool + at, c, D / 2, v[i], vy);
      if (c == 0) {
        uint8_t* sc = q.kv_scale + ((int64_t)pid << (q.log2_page + 1)) + row;
        sc[0] = (uint8_t)ky;
        sc[1 << q.log2_page] = (uint8_t)vy;
      }
    }
  }
}

struct AppendParams {
  const __nv_bfloat16* k_new;  // [total_new][Hkv][D]
  const __nv_bfloat16* v_new;
  const int32_t* cu_new;       // [B+1]
  const int32_t* ctx_len;      // [B]
  const int32_t* q_len;        // [B] or null
  const int32_t* cls;          // [B*Hkv][3]
  const int32_t* table;
  const int32_t* offs;         // [B*Hkv+1]
  uint8_t* k_pool;
  uint8_t* v_pool;
  uint8_t* kv_scale;           // null for bf16 pools
  int32_t* status;
  int64_t table_len;
  int32_t total_new, B, Hkv, log2_page, num_pages;
};

// A warp per 32 / (D/16) KV heads of one new row, both its K and its V: the search for the row's sequence is the warp's.
template <int D, int FMT>
__global__ void __launch_bounds__(32) append_kernel(AppendParams p) {
  constexpr int LANES = D / 16, HEADS = 32 / LANES;
  const int32_t r = (int32_t)blockIdx.x, lane = threadIdx.x, c = lane % LANES;
  const int32_t kh = (int32_t)blockIdx.y * HEADS + lane / LANES;
  bool ok = kh < p.Hkv;
  early_start();
  RowPiece k, v;
  k.lo = k.hi = v.lo = v.hi = make_uint4(0, 0, 0, 0);
  if (ok) {  // issued before the page look-up, whose loads depend on one another
    const int64_t src = ((int64_t)r * p.Hkv + kh) * D + 8 * c;
    k.lo = *reinterpret_cast<const uint4*>(p.k_new + src);
    k.hi = *reinterpret_cast<const uint4*>(p.k_new + src + D / 2);
    v.lo = *reinterpret_cast<const uint4*>(p.v_new + src);
    v.hi = *reinterpret_cast<const uint4*>(p.v_new + src + D / 2);
  }
  const int32_t first = p.cu_new[0], end = p.cu_new[p.B];
  if (r < first || r >= end) return;  // rows outside every sequence are left alone (the whole warp's row)
  const int32_t b = warp_find(p.cu_new, p.B, r);
  int64_t at = 0, sat = 0;
  if (ok) {
    const int32_t bk = b * p.Hkv + kh;
    const int64_t off = p.offs[bk], n = (int64_t)p.offs[bk + 1] - off;
    const HeadPages hp = head_pages(p.ctx_len, p.q_len, p.cls, b, bk, p.log2_page, 0);
    const int64_t pos = (int64_t)hp.L - p.cu_new[b + 1] + r;
    const int32_t row = (int32_t)(pos & ((1 << p.log2_page) - 1)), t = hp.index((int32_t)(pos >> p.log2_page));
    bool fits = pos >= 0 && n == hp.total;
    ok = pos >= 0 && t >= 0;  // t < 0: a page this head does not keep
    if (ok && (t >= n || off < 0 || off + t >= p.table_len)) ok = fits = false;
    if (!fits && c == 0) report(p.status, 2);
    if (ok) {
      const int32_t pid = p.table[off + t];
      if (pid < 0 || pid >= p.num_pages) {
        if (c == 0) report(p.status, 1);
        ok = false;
      }
      at = (((int64_t)pid << p.log2_page) + row) * D;
      sat = ((int64_t)pid << (p.log2_page + 1)) + row;
    }
  }
  if (FMT == kFmtBf16) {
    if (!ok) return;
    uint4* kd = reinterpret_cast<uint4*>(p.k_pool + 2 * at) + c;
    uint4* vd = reinterpret_cast<uint4*>(p.v_pool + 2 * at) + c;
    kd[0] = k.lo;
    kd[D / 16] = k.hi;
    vd[0] = v.lo;
    vd[D / 16] = v.hi;
    return;
  }
  const int32_t ky = row_byte<FMT, LANES>(k), vy = row_byte<FMT, LANES>(v);  // every lane of the warp takes part
  if (!ok) return;
  store_codes<FMT>(p.k_pool + at, c, D / 2, k, ky);
  store_codes<FMT>(p.v_pool + at, c, D / 2, v, vy);
  if (c == 0) {
    p.kv_scale[sat] = (uint8_t)ky;
    p.kv_scale[sat + (1 << p.log2_page)] = (uint8_t)vy;
  }
}

struct DequantParams {
  const int32_t* ctx_len;
  const int32_t* q_len;
  const int32_t* cls;
  const int32_t* table;
  const int32_t* offs;
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  const uint8_t* kv_scale;
  __nv_bfloat16* k_out;
  __nv_bfloat16* v_out;
  int32_t* status;
  int64_t table_len;
  int32_t B, Hkv, log2_page, num_pages;
};

// Eight codes as bf16: code * 2^(y - 127) rounded to nearest even. e4m3 has 4 and int8 7 significant bits, so only
// results below the bf16 normal range round at all.
template <int FMT>
__device__ __forceinline__ uint4 dequant8(uint2 w, float scale) {
  const uint32_t in[2] = {w.x, w.y};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h[2];
    codes_to_half2x2<FMT, false>(in[i], h[0], h[1]);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
      const __nv_bfloat162 r = __floats2bfloat162_rn(f.x * scale, f.y * scale);
      o[2 * i + j] = *reinterpret_cast<const uint32_t*>(&r);
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// D/8 lanes a row: 8-byte loads and 16-byte stores, both contiguous over the lanes.
template <int D, int FMT>
__global__ void __launch_bounds__(32 * kSliceWarps) dequant_pages_kernel(DequantParams p) {
  constexpr int LANES = D / 8, ROWS = 32 / LANES, N = kSliceRows / ROWS;
  const int lane = threadIdx.x & 31, c = lane % LANES;
  early_start();
  const int nheads = p.B * p.Hkv, log2_slices = p.log2_page - kLog2SliceRows;
  const int64_t slices = p.table_len << log2_slices, begin = p.offs[0], entries = p.offs[nheads];
  const int64_t warps = (int64_t)gridDim.x * kSliceWarps;
  if (blockIdx.x == 0 && threadIdx.x == 0 && entries > p.table_len) report(p.status, 2);
  for (int64_t x = (int64_t)blockIdx.x * kSliceWarps + (threadIdx.x >> 5); x < slices; x += warps) {
    const int64_t e = x >> log2_slices;
    const int32_t row0 = (int32_t)(x & ((1 << log2_slices) - 1)) * kSliceRows;
    const int32_t pid = p.table[e];
    if (e < begin) continue;  // spare room before the first table
    if (e >= entries) break;  // and behind the last
    if (pid < 0 || pid >= p.num_pages) {
      if (lane == 0) report(p.status, 1);
      continue;
    }
    // the codes are on their way while the head they belong to, and with it the context's end, is looked up
    const int64_t at = (((int64_t)pid << p.log2_page) + row0 + lane / LANES) * D + 8 * c;
    const uint8_t* sc = p.kv_scale + ((int64_t)pid << (p.log2_page + 1)) + row0 + lane / LANES;
    uint2 k[N], v[N];
    int32_t ky[N], vy[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      k[i] = *reinterpret_cast<const uint2*>(p.k_pool + at + i * ROWS * D);
      v[i] = *reinterpret_cast<const uint2*>(p.v_pool + at + i * ROWS * D);
      ky[i] = sc[i * ROWS];
      vy[i] = sc[i * ROWS + (1 << p.log2_page)];
    }
    const int bk = warp_find(p.offs, nheads, e), b = bk / p.Hkv;
    const int32_t t = (int32_t)(e - p.offs[bk]);
    const HeadPages hp = head_pages(p.ctx_len, p.q_len, p.cls, b, bk, p.log2_page, 0);
    if (p.offs[bk + 1] - p.offs[bk] != hp.total) {
      if (lane == 0) report(p.status, 2);
      if (t < 0 || t >= hp.total) continue;
    }
    const int64_t tok0 = ((int64_t)hp.logical(t) << p.log2_page) + row0 + lane / LANES;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool in = tok0 + i * ROWS < hp.L;  // rows past the context end are written as zero
      const uint4 zero = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(p.k_out + at + i * ROWS * D) = in ? dequant8<FMT>(k[i], row_scale(ky[i])) : zero;
      *reinterpret_cast<uint4*>(p.v_out + at + i * ROWS * D) = in ? dequant8<FMT>(v[i], row_scale(vy[i])) : zero;
    }
  }
}

}  // namespace segpaged
