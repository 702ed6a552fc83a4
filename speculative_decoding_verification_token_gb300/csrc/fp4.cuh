// fp4.cuh -- what quantisation to 4-bit blocks (fp4_quant.cu) and the product of such blocks
// (fp4_project.cu) share: the scale tiles' geometry and the 4- and 8-bit conversions.
//
// Packed rows: element i of a row in nibble i % 2 (0: low) of byte i / 2, rows padded with zeros
// to 32 elements.  Scales: one byte per block, in tiles of 128 rows by 4 consecutive blocks (a
// group) of 512 bytes, tile (r / 128, k / 4) row-major, row r's scale of block k at byte
// (r % 32) * 16 + (r / 32 % 4) * 4 + k % 4 -- the order in which tcgen05.cp spreads 512 bytes over
// 32 TMEM lanes of four columns, so a tile goes from memory to TMEM without a transposition.  A
// row's groups are padded to 256 elements (one k-block of the product), with scales of zero.
#pragma once

#include <cuda_fp16.h>

#include "sv_device.cuh"

namespace sv {

// Scale groups per row: 4 blocks each, whole k-blocks of 256 elements.
inline int32_t fp4_groups(int64_t H, int32_t format) {
  return static_cast<int32_t>((H + 255) / 256 * (format == SV_FP4_E8M0_32 ? 2 : 4));
}

// Eight values to e2m1 codes, nearest, ties to even, saturating at 6; element j in nibble j.
__device__ __forceinline__ uint32_t fp4x8(const float* t) {
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "f"(t[0]), "f"(t[1]), "f"(t[2]), "f"(t[3]), "f"(t[4]), "f"(t[5]), "f"(t[6]), "f"(t[7]));
  return w;
}

// The values of eight codes (exact).
__device__ __forceinline__ void fp4x8_values(uint32_t w, float* f) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
    f[2 * j] = v.x;
    f[2 * j + 1] = v.y;
  }
}

// The nearest finite e4m3 code of t >= 0 (ties to even, saturating at 448), and a code's value.
__device__ __forceinline__ uint32_t e4m3_of(float t) {
  uint16_t h;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(0.f), "f"(t));
  return h & 0xFFu;
}

__device__ __forceinline__ float e4m3_value(uint32_t code) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(code)));
  return __half2float(__ushort_as_half(static_cast<uint16_t>(h)));
}

}  // namespace sv
