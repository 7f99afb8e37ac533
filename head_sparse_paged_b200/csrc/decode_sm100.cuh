// decode_sm100.cuh -- attention of one new token per sequence over its own stored pages.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "plan.h"
#include "quant_pages.cuh"
#include "sm100_ptx.cuh"

namespace segpaged {

struct DecodeParams {
  const __nv_bfloat16* q;      // [B][Hq][D]
  const uint8_t* k_pool;       // [num_pages][P][D], bf16 or codes
  const uint8_t* v_pool;
  const uint8_t* kv_scale;     // [num_pages][2][P], null for bf16
  const int32_t* table;
  const int32_t* offs;         // [B*Hkv+1]
  const int32_t* ctx_len;      // [B]
  const int32_t* q_len;        // [B] or null
  const int32_t* cls;          // [B*Hkv][3]
  __nv_bfloat16* o;            // [B][Hq][D]
  float* lse;                  // [Hq][B]
  int32_t* status;             // nullable
  int64_t table_len;
  int32_t B, Hkv, G, P, num_pages;
  float scale_log2;
};

// One warp per (sequence, query head): lanes split the row, tokens one after the other.
template <int D, int FMT>
__global__ void __launch_bounds__(128) decode_kernel(DecodeParams p) {
  constexpr int E = D / 32;  // elements of a lane
  const int lane = threadIdx.x & 31;
  const int Hq = p.Hkv * p.G;
  const int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (w >= (int64_t)p.B * Hq) return;
  const int b = (int)(w / Hq), h = (int)(w % Hq), bk = b * p.Hkv + h / p.G;
  int32_t L;
  const Split sp = device_split(p.ctx_len, p.q_len, p.cls, b, bk, p.P, 1, &L);
  const int32_t sink = p.cls[3 * bk] ? L : max(p.cls[3 * bk + 1], 0), lo = L - max(p.cls[3 * bk + 2], 1);
  const int64_t off = p.offs[bk], n = (int64_t)p.offs[bk + 1] - off;
  if (n != sp.total && lane == 0) report(p.status, 2);
  float q[E], o[E], m = -INFINITY, l = 0.f;
  for (int i = 0; i < E; ++i) {
    q[i] = __bfloat162float(p.q[w * D + lane * E + i]) * p.scale_log2;
    o[i] = 0.f;
  }
  for (int32_t t = 0; t < sp.total; ++t) {
    const int32_t lp = t < sp.n_sink ? t : sp.w0 + (t - sp.n_sink);
    int32_t pid = 0;
    if (t < n && off >= 0 && off + t < p.table_len) pid = p.table[off + t];
    else if (lane == 0) report(p.status, 2);
    if (pid < 0 || pid >= p.num_pages) {
      if (lane == 0) report(p.status, 1);
      pid = 0;
    }
    for (int32_t r = 0; r < p.P; ++r) {
      const int32_t tok = lp * p.P + r;
      if (tok >= L || (tok >= sink && tok < lo)) continue;
      const int64_t at = ((int64_t)pid * p.P + r) * D + lane * E;
      float s = 0.f, v[E], ks = 1.f, vs = 1.f;
      if (FMT != kFmtBf16) {
        ks = row_scale(p.kv_scale[(int64_t)pid * 2 * p.P + r]);
        vs = row_scale(p.kv_scale[(int64_t)pid * 2 * p.P + p.P + r]);
      }
      for (int i = 0; i < E; ++i) {
        float k;
        if (FMT == kFmtBf16) {
          k = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.k_pool)[at + i]);
          v[i] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.v_pool)[at + i]);
        } else {
          k = __low2float(codes_to_half2<FMT>(p.k_pool[at + i]));
          v[i] = __low2float(codes_to_half2<FMT>(p.v_pool[at + i])) * vs;
        }
        s += q[i] * k;
      }
      for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      s *= ks;
      const float mn = fmaxf(m, s), a = m == -INFINITY ? 0.f : exp2f(m - mn), pr = exp2f(s - mn);
      l = l * a + pr;
      for (int i = 0; i < E; ++i) o[i] = o[i] * a + pr * v[i];
      m = mn;
    }
  }
  for (int i = 0; i < E; ++i) p.o[w * D + lane * E + i] = __float2bfloat16_rn(L > 0 ? o[i] / l : 0.f);
  if (lane == 0) p.lse[(int64_t)h * p.B + b] = L > 0 ? 0.6931471805599453f * (m + log2f(l)) : -INFINITY;
}

}  // namespace segpaged
