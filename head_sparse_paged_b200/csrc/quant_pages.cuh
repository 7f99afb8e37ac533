// quant_pages.cuh -- the kernels that write 8-bit pages, append new rows to a pool, and read 8-bit pages back.
//
// All three move each byte once and are bound by HBM: 2 bytes read and 1 written per element (the write), or the
// reverse (the read back). D/16 lanes share a row. In the two that quantise, lane c of a row holds its elements
// 8c .. 8c+7 and D/2 + 8c .. D/2 + 8c+7, the pairs that the RoPE re-alignment rotates, so that the row's largest
// magnitude is taken of the rotated bf16 values: a pool written here holds the quantised form of exactly the rows
// that build_scatter_kernel would store.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "build_kernel.cuh"
#include "plan.h"
#include "quant_rows.cuh"
#include "rope.cuh"

namespace segpaged {

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
  for (int d = LANES / 2; d > 0; d >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, d));
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

struct BuildQuantParams {
  BuildParams b;       // k_pool, v_pool unused
  uint8_t* k_pool;     // [num_pages][P][D] codes
  uint8_t* v_pool;
  uint8_t* kv_scale;   // [num_pages][2][P] exponent bytes, K then V
};

template <int D, int FMT, bool ROPE>
__global__ void __launch_bounds__(256) build_quant_kernel(BuildQuantParams q) {
  const BuildParams& p = q.b;
  constexpr int LANES = D / 16;
  constexpr int kPass = 256 / LANES;  // rows a pass of the block takes
  const int nheads = p.B * p.Hkv;
  const int64_t E = p.offs[nheads];
  const int c = threadIdx.x % LANES;
  for (int64_t e = blockIdx.x; e < E; e += gridDim.x) {
    int lo = 0, hi = nheads;  // largest head with offs[head] <= e
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.offs[mid] <= e) lo = mid; else hi = mid;
    }
    const int bk = lo, b = bk / p.Hkv, kh = bk % p.Hkv;
    const int32_t t = (int32_t)(e - p.offs[bk]);
    const int32_t L = p.cu_k[b + 1] - p.cu_k[b];
    const Split sp = storage_split(L, p.q_len[b], p.cls[3 * bk], p.cls[3 * bk + 1], p.cls[3 * bk + 2], p.P);
    if (p.offs[bk + 1] - p.offs[bk] != sp.total) {
      if (t == 0 && threadIdx.x == 0) report(p.status, 2);
      if (t >= sp.total) continue;
    }
    const int32_t lp = t < sp.n_sink ? t : sp.w0 + (t - sp.n_sink);
    const int32_t pid = p.table[e];
    if (pid < 0 || pid >= p.num_pages) {
      if (threadIdx.x == 0) report(p.status, 1);
      continue;
    }
    for (int row0 = 0; row0 < p.P; row0 += kPass) {
      const int row = row0 + threadIdx.x / LANES;
      const int64_t tok = (int64_t)lp * p.P + row;
      RowPiece k, v;
      k.lo = k.hi = v.lo = v.hi = make_uint4(0, 0, 0, 0);  // rows past the context end
      if (row < p.P && tok < L) {
        const int64_t src = ((p.cu_k[b] + tok) * p.Hkv + kh) * D + 8 * c;
        k.lo = __ldg(reinterpret_cast<const uint4*>(p.k_dense + src));
        k.hi = __ldg(reinterpret_cast<const uint4*>(p.k_dense + src + D / 2));
        v.lo = __ldg(reinterpret_cast<const uint4*>(p.v_dense + src));
        v.hi = __ldg(reinterpret_cast<const uint4*>(p.v_dense + src + D / 2));
        if (ROPE) {
          const float4* t4 = reinterpret_cast<const float4*>(p.cos_sin + (int64_t)b * D + 16 * c);
          const float4 q0 = t4[0], q1 = t4[1], q2 = t4[2], q3 = t4[3];
          RowPiece r;
          r.lo.x = rot_pair(k.lo.x, k.hi.x, q0.x, q0.y, q0.z, q0.w, &r.hi.x);
          r.lo.y = rot_pair(k.lo.y, k.hi.y, q1.x, q1.y, q1.z, q1.w, &r.hi.y);
          r.lo.z = rot_pair(k.lo.z, k.hi.z, q2.x, q2.y, q2.z, q2.w, &r.hi.z);
          r.lo.w = rot_pair(k.lo.w, k.hi.w, q3.x, q3.y, q3.z, q3.w, &r.hi.w);
          k = r;
        }
      }
      const int32_t ky = row_byte<FMT, LANES>(k), vy = row_byte<FMT, LANES>(v);
      if (row >= p.P) continue;  // whole warps: kPass and P are multiples of a warp's rows or kPass > P >= 16
      const int64_t at = ((int64_t)pid * p.P + row) * D;
      store_codes<FMT>(q.k_pool + at, c, D / 2, k, ky);
      store_codes<FMT>(q.v_pool + at, c, D / 2, v, vy);
      if (c == 0) {
        uint8_t* sc = q.kv_scale + (int64_t)pid * 2 * p.P + row;
        sc[0] = (uint8_t)ky;
        sc[p.P] = (uint8_t)vy;
      }
    }
  }
}

// A sequence's geometry as the decode-side kernels read it from device memory: nothing there was checked on the
// host, so lengths and classes are brought into range first.
__device__ __forceinline__ Split device_split(const int32_t* ctx_len, const int32_t* q_len, const int32_t* cls, int b, int bk,
                                              int32_t P, int32_t min_q, int32_t* L_out) {
  const int32_t L = max(ctx_len[b], 0);
  const int32_t lq = max(q_len ? q_len[b] : 1, min_q);
  *L_out = L;
  return storage_split(L, lq, cls[3 * bk], max(cls[3 * bk + 1], 0), max(cls[3 * bk + 2], 1), P);
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
  int32_t total_new, B, Hkv, P, num_pages;
};

// One group of D/16 lanes per (new row, KV head), both its K and its V.
template <int D, int FMT>
__global__ void __launch_bounds__(128) append_kernel(AppendParams p) {
  constexpr int LANES = D / 16;
  const int64_t item = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / LANES;
  const int c = threadIdx.x % LANES;
  bool ok = item < (int64_t)p.total_new * p.Hkv;
  const int32_t r = ok ? (int32_t)(item / p.Hkv) : 0;
  const int kh = ok ? (int)(item % p.Hkv) : 0;
  RowPiece k, v;
  k.lo = k.hi = v.lo = v.hi = make_uint4(0, 0, 0, 0);
  if (ok) {  // issued before the page look-up, whose loads depend on one another
    const int64_t src = item * D + 8 * c;
    k.lo = __ldg(reinterpret_cast<const uint4*>(p.k_new + src));
    k.hi = __ldg(reinterpret_cast<const uint4*>(p.k_new + src + D / 2));
    v.lo = __ldg(reinterpret_cast<const uint4*>(p.v_new + src));
    v.hi = __ldg(reinterpret_cast<const uint4*>(p.v_new + src + D / 2));
  }
  ok = ok && r >= p.cu_new[0] && r < p.cu_new[p.B];  // rows outside every sequence are left alone
  int64_t at = 0, sat = 0;
  if (ok) {
    int lo = 0, hi = p.B;  // last sequence that starts at or before r
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.cu_new[mid] <= r) lo = mid; else hi = mid;
    }
    const int b = lo, bk = b * p.Hkv + kh;
    int32_t L;
    const Split sp = device_split(p.ctx_len, p.q_len, p.cls, b, bk, p.P, 0, &L);
    const int64_t pos = (int64_t)L - p.cu_new[b + 1] + r;
    const int64_t off = p.offs[bk], n = (int64_t)p.offs[bk + 1] - off;
    const int32_t lp = (int32_t)(pos / p.P), row = (int32_t)(pos % p.P);
    const int32_t t = lp < sp.n_sink ? lp : lp < sp.w0 ? -1 : lp - sp.w0 + sp.n_sink;
    bool fits = pos >= 0 && n == sp.total;
    ok = pos >= 0 && t >= 0;  // t < 0: a page this head does not keep
    if (ok && (t >= n || off < 0 || off + t >= p.table_len)) ok = fits = false;
    if (!fits && c == 0) report(p.status, 2);
    if (ok) {
      const int32_t pid = p.table[off + t];
      if (pid < 0 || pid >= p.num_pages) {
        if (c == 0) report(p.status, 1);
        ok = false;
      }
      at = ((int64_t)pid * p.P + row) * D;
      sat = (int64_t)pid * 2 * p.P + row;
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
    p.kv_scale[sat + p.P] = (uint8_t)vy;
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
  int32_t B, Hkv, P, num_pages;
};

// Sixteen codes (one 16-byte load) as bf16: code * 2^(y - 127) rounded to nearest even. e4m3 has 4 and int8 7
// significant bits, so only results below the bf16 normal range round at all.
template <int FMT>
__device__ __forceinline__ void dequant16(uint4 w, float scale, uint32_t (&o)[8]) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h[2];
    codes_to_half2x2<FMT, false>(in[i], h[0], h[1]);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
      const __nv_bfloat162 r = __floats2bfloat162_rn(f.x * scale, f.y * scale);
      o[2 * i + j] = *reinterpret_cast<const uint32_t*>(&r);
    }
  }
}

template <int D, int FMT>
__global__ void __launch_bounds__(256) dequant_pages_kernel(DequantParams p) {
  constexpr int LANES = D / 16;
  const int nheads = p.B * p.Hkv;
  const int64_t E = min((int64_t)p.offs[nheads], p.table_len);
  const int c = threadIdx.x % LANES;
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.offs[nheads] > p.table_len) report(p.status, 2);
  for (int64_t e = blockIdx.x; e < E; e += gridDim.x) {
    int lo = 0, hi = nheads;  // largest head with offs[head] <= e
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.offs[mid] <= e) lo = mid; else hi = mid;
    }
    const int bk = lo;
    const int32_t t = (int32_t)(e - p.offs[bk]);
    int32_t L;
    const Split sp = device_split(p.ctx_len, p.q_len, p.cls, bk / p.Hkv, bk, p.P, 0, &L);
    if (p.offs[bk + 1] - p.offs[bk] != sp.total) {
      if (t == 0 && threadIdx.x == 0) report(p.status, 2);
      if (t >= sp.total) continue;
    }
    const int32_t lp = t < sp.n_sink ? t : sp.w0 + (t - sp.n_sink);
    const int32_t pid = p.table[e];
    if (pid < 0 || pid >= p.num_pages) {
      if (threadIdx.x == 0) report(p.status, 1);
      continue;
    }
    for (int row = threadIdx.x / LANES; row < p.P; row += 256 / LANES) {
      const int64_t at = ((int64_t)pid * p.P + row) * D + 16 * c;
      uint32_t k[8] = {}, v[8] = {};
      if ((int64_t)lp * p.P + row < L) {
        const uint8_t* sc = p.kv_scale + (int64_t)pid * 2 * p.P + row;
        const uint4 kw = __ldg(reinterpret_cast<const uint4*>(p.k_pool + at));
        const uint4 vw = __ldg(reinterpret_cast<const uint4*>(p.v_pool + at));
        dequant16<FMT>(kw, row_scale(__ldg(sc)), k);
        dequant16<FMT>(vw, row_scale(__ldg(sc + p.P)), v);
      }
      uint4* ko = reinterpret_cast<uint4*>(p.k_out + at);
      uint4* vo = reinterpret_cast<uint4*>(p.v_out + at);
      ko[0] = make_uint4(k[0], k[1], k[2], k[3]);
      ko[1] = make_uint4(k[4], k[5], k[6], k[7]);
      vo[0] = make_uint4(v[0], v[1], v[2], v[3]);
      vo[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
  }
}

}  // namespace segpaged
