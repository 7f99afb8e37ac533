// quant_rows.cuh -- the 8-bit form of a K or V row, shared by the kernels that write and read 8-bit pools.
//
// A row is the D values of one (token, KV head). Its 8-bit form is D codes c and one exponent byte y, and stands
// for c * 2^(y - 127). With a the largest magnitude of the row and M the largest code (448 for e4m3, 127 for int8),
// e = y - 127 is the smallest whole number >= -126 with a <= M * 2^e, and c = x * 2^-e rounded to nearest even.
// A power of two instead of a / M: x * 2^-e is then exact in fp32, so every code is the correctly rounded one (a
// quotient rounded first can move a code by one at a tie), e4m3 loses no precision by it (its relative step does not
// depend on the scale), the byte takes a quarter of a float's traffic, and kernels can apply it in an exponent.
// A row that holds an infinity or a NaN gets y = 255 and codes 0, and reads back as NaN throughout.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

namespace segpaged {

// SEGPAGED_KV_* of the C ABI
constexpr int kFmtBf16 = 0, kFmtE4m3 = 1, kFmtInt8 = 2;
constexpr int kRowNaN = 255;  // exponent byte of a row with an infinity or a NaN

// Larger of two bf16 pairs, each half by itself; a NaN (0x7fff) wins. (As an integer maximum of the bit patterns, which
// magnitudes order like, it is several instructions: 1390 instead of 1160 cycles for the queries of a chunk.)
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Largest magnitude of two packed bf16 pairs: 0x7f80 and above for infinities and NaNs.
__device__ __forceinline__ uint32_t absmax2(uint32_t m, uint32_t w) { return max2(m, w & 0x7fff7fffu); }

// Exponent byte of a row whose largest magnitude has the bf16 bits `top`.
template <int FMT>
__device__ __forceinline__ int32_t row_exponent_byte(uint32_t top) {
  if (top >= 0x7f80u) return kRowNaN;
  const int32_t exp = (int32_t)(top >> 7) - 127;  // -127 for zero and subnormals: below the clamp either way
  const int32_t man = (int32_t)(top & 0x7f);
  // 448 = 1.75 * 2^8, 127 = 1.984375 * 2^6: the bf16 mantissa up to which 2^exp * 1.man still fits
  const int32_t e = FMT == kFmtE4m3 ? exp - 8 + (man > 0x60) : exp - 6 + (man > 0x7e);
  return max(e, -126) + 127;
}

// 2^-(y - 127): a normal float for every byte row_exponent_byte gives but kRowNaN (1 .. 249).
__device__ __forceinline__ float row_inverse_scale(int32_t y) { return __uint_as_float((uint32_t)(254 - y) << 23); }

// 2^(y - 127), with 2^-127 (a subnormal) for y = 0 and NaN for y = 255.
__device__ __forceinline__ float row_scale(int32_t y) {
  const uint32_t bits = max((uint32_t)y << 23, 0x00400000u);
  return __uint_as_float(y == kRowNaN ? 0x7fffffffu : bits);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Codes of four values (two packed bf16 pairs), lowest byte first.
template <int FMT>
__device__ __forceinline__ uint32_t quantise4(uint32_t w0, uint32_t w1, float inv) {
  const float a = bf16_lo(w0) * inv, b = bf16_hi(w0) * inv, c = bf16_lo(w1) * inv, d = bf16_hi(w1) * inv;
  if (FMT == kFmtE4m3) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
  }
  const uint32_t lo = (__float2int_rn(a) & 0xff) | ((__float2int_rn(b) & 0xff) << 8);
  const uint32_t hi = (__float2int_rn(c) & 0xff) | ((__float2int_rn(d) & 0xff) << 8);
  return lo | (hi << 16);
}

// The four codes in w as two pairs of fp16 (both kinds of code are exact in fp16): a = bytes (0, 1) and b = bytes (2, 3),
// or with CROSS a = bytes (0, 2) and b = bytes (1, 3).
template <int FMT, bool CROSS>
__device__ __forceinline__ void codes_to_half2x2(uint32_t w, uint32_t& a, uint32_t& b) {
  if (FMT == kFmtE4m3) {
    if (CROSS) w = __byte_perm(w, 0, 0x3120);
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "mov.b32 {lo, hi}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(a), "=r"(b)
        : "r"(w));
  } else {
    // 0x6400 | u is 1024 + u in fp16; with u = code + 128, taking 1152 off leaves the code, exactly
    w ^= 0x80808080u;
    a = __byte_perm(w, 0x64646464u, CROSS ? 0x4240 : 0x4140);
    b = __byte_perm(w, 0x64646464u, CROSS ? 0x4341 : 0x4342);
    const uint32_t off = 0x64806480u;
    const __half2 ha = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&off));
    const __half2 hb = __hsub2(*reinterpret_cast<const __half2*>(&b), *reinterpret_cast<const __half2*>(&off));
    a = *reinterpret_cast<const uint32_t*>(&ha);
    b = *reinterpret_cast<const uint32_t*>(&hb);
  }
}

}  // namespace segpaged
