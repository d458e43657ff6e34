// E4M3 and E2M1 conversions shared by the kernels that write and read K/V pools.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

namespace dcpmla {

// 8 bf16 -> 8 E4M3 codes of x / scale (IEEE fp32 division, RNE, saturated).
__device__ __forceinline__ uint2 quantize8(uint4 x, float scale) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t out[2] = {0u, 0u};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float lo = __uint_as_float(w[e] << 16) / scale;
    const float hi = __uint_as_float(w[e] & 0xFFFF0000u) / scale;
    const __nv_fp8x2_storage_t c = __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
    out[e >> 1] |= (uint32_t)c << (16 * (e & 1));
  }
  return make_uint2(out[0], out[1]);
}

// Four E4M3 codes -> two f16x2 (codes 0 and 1, codes 2 and 3), exact.
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}

__device__ __forceinline__ uint64_t pair_f32(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
// 16 bf16 -> 16 E2M1 codes and their E4M3 block scale: block = E4M3(max |x| / (6 scale)), codes of
// x / (scale * block) (IEEE fp32 products and divisions, RNE, saturated; codes 0 for block 0). A block
// with an infinity or NaN, which have no code, gets the scale NaN: its values read as NaN.
__device__ __forceinline__ uint2 quantize16(uint4 lo, uint4 hi, float scale, uint8_t& block) {
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  uint32_t top = 0;  // the largest magnitude, by its bits: NaN lie above infinity, that above the rest
#pragma unroll
  for (int e = 0; e < 8; ++e)
    asm("max.u16x2 %0, %0, %1;" : "+r"(top) : "r"(w[e] & 0x7fff7fffu));
  top = max(top & 0xffffu, top >> 16);
  if (top >= 0x7f80u) {
    block = 0x7f;  // NaN
    return make_uint2(0u, 0u);
  }
  const float most = __uint_as_float(top << 16);
  block = (uint8_t)__nv_cvt_float_to_fp8(most / (6.0f * scale), __NV_SATFINITE, __NV_E4M3);
  const __half_raw b = __nv_cvt_fp8_to_halfraw(block, __NV_E4M3);
  const float step = scale * __half2float(*reinterpret_cast<const __half*>(&b));
  if (!(step > 0.f)) return make_uint2(0u, 0u);
  // Quotients by Markstein's method ("Computation of elementary functions on the IBM RISC
  // System/6000 processor", 1990): with r the reciprocal rounded to nearest and q within a unit of
  // x / step, q + (x - q step) r rounds to the quotient rounded to nearest, where x - q step is
  // exact (one FMA) and nothing leaves the range. The first correction brings q that near. Two at a
  // time; 2.5 operations a value, where a division takes four times as many (34 us for 20000 rows
  // of 2 x 1024 values).
  const float r = __frcp_rn(step);
  const bool plain = !(step > 1e-30f && step < 1e30f && most * r < 1e20f);
  const uint64_t r2 = pair_f32(r, r), s2 = pair_f32(-step, -step);
  uint32_t out[2] = {0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float lo_x = __uint_as_float(w[e] << 16), hi_x = __uint_as_float(w[e] & 0xFFFF0000u);
    uint64_t q, d;
    const uint64_t x2 = pair_f32(lo_x, hi_x);
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q) : "l"(x2), "l"(r2));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(q), "l"(s2), "l"(x2));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(q) : "l"(d), "l"(r2), "l"(q));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(q), "l"(s2), "l"(x2));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(q) : "l"(d), "l"(r2), "l"(q));
    // the sign is x's, also of a zero
    uint32_t a = ((uint32_t)q & 0x7fffffffu) | (w[e] << 16 & 0x80000000u);
    uint32_t b = ((uint32_t)(q >> 32) & 0x7fffffffu) | (w[e] & 0x80000000u);
    if (plain) a = __float_as_uint(lo_x / step), b = __float_as_uint(hi_x / step);
    uint32_t c;  // the second value in the upper half
    asm("{\n\t.reg .b8 c;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %1, %2;\n\t"
        "cvt.u32.u8 %0, c;\n\t}"
        : "=r"(c)
        : "f"(__uint_as_float(b)), "f"(__uint_as_float(a)));
    out[e >> 2] |= c << (8 * (e & 3));
  }
  return make_uint2(out[0], out[1]);
}

// Eight E2M1 codes -> four f16x2 (codes 2i and 2i + 1), exact.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t x, uint32_t (&y)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3])
      : "r"(x));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace dcpmla
