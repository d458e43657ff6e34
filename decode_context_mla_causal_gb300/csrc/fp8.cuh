// E4M3 conversions shared by the kernels that write and read K/V pools.
#pragma once

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

}  // namespace dcpmla
