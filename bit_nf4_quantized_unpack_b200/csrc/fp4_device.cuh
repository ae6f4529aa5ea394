// fp4_device.cuh -- storage of microscaled 4-bit floating-point matrices (MXFP4, NVFP4):
// block sizes, the tiled scale layout, and the conversions of codes and scales.
#pragma once

#include <cstdint>
#include <cstring>

#include <cuda_fp16.h>

#include "internal.h"
#include "sm100.cuh"

namespace qlora {

enum class Fp4 { kMx = QLORA_FP4_MX, kNv = QLORA_FP4_NV };

// Values per block scale.
template <Fp4 F>
constexpr int kFp4Block = F == Fp4::kMx ? 32 : 16;
// Columns that one 512-byte scale tile (128 rows x 4 blocks) covers.
template <Fp4 F>
constexpr int kFp4TileCols = 4 * kFp4Block<F>;

// Largest magnitude of an NVFP4 value in units of gscale: E2M1 6 times E4M3 448.
constexpr float kNvTop = 2688.f;

// Byte of (row, block) in the tiled scale array, ktiles = scale tiles along a row. The
// 512-byte tile is the order in which tcgen05.cp.32x128b.warpx4 spreads 128 rows over the
// 32 lanes x 4 columns of tensor memory that a block-scaled MMA reads.
__host__ __device__ __forceinline__ int64_t fp4_scale_offset(int64_t row, int64_t block,
                                                             int64_t ktiles) {
  return ((row >> 7) * ktiles + (block >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 +
         (block & 3);
}

// Eight fp32 values -> eight E2M1 codes (nearest, ties to the even code, 6 at most), value i
// in bits 4i..4i+3.
__device__ __forceinline__ uint32_t fp4_pack8(const float (&v)[8]) {
  uint32_t d;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(d)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return d;
}

// The two E2M1 codes of a byte (bits 0-7 of w) as fp32 values.
__device__ __forceinline__ float2 e2m1_pair(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t}"
      : "=r"(h)
      : "r"(w));
  __half2 v;
  memcpy(&v, &h, 4);
  return __half22float2(v);
}

// What the bf16 pair hi leaves of (a, b), as a bf16 pair: 0 where hi is infinite (or NaN).
__device__ __forceinline__ uint32_t bf16x2_rest_rn(float a, float b, uint32_t hi) {
  const float ra = (hi & 0x7F80u) == 0x7F80u ? 0.f : a - __uint_as_float(hi << 16);
  const float rb = (hi & 0x7F800000u) == 0x7F800000u ? 0.f : b - __uint_as_float(hi & 0xFFFF0000u);
  return pack_bf16x2_rn(ra, rb);
}

// fp32 -> E4M3 bits (nearest, ties to even, 448 at most).
__device__ __forceinline__ uint32_t e4m3_bits(float x) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(0.f), "f"(x));
  return d & 0xFFu;
}

// Value of a scale byte.
template <Fp4 F>
__device__ __forceinline__ float fp4_scale_value(uint32_t b) {
  if (F == Fp4::kMx)  // 2^(b - 127); 2^-127 is a subnormal, 255 is NaN
    return __uint_as_float(b == 0u ? 0x00400000u : b == 255u ? 0x7FFFFFFFu : b << 23);
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(b)));
  __half2 v;
  memcpy(&v, &h, 4);
  return __low2float(v);
}

// Scale byte of a block that holds a NaN or an infinity.
template <Fp4 F>
constexpr uint32_t kFp4NanScale = F == Fp4::kMx ? 0xFFu : 0x7Fu;

// Exponent e of the NVFP4 gscale 2^e of a set of values whose largest magnitude is `top`
// (fp32 bits): the smallest e >= -126 with top <= 2688 * 2^e; 0 for top = 0.
// 2688 = 1.3125 * 2^11, and 1.3125 has the mantissa field 0x280000.
__device__ __forceinline__ int nv_gscale_exp(uint32_t top) {
  if (top == 0u) return 0;
  const int e = static_cast<int>(top >> 23) - 127 - 11 + ((top & 0x7FFFFFu) > 0x280000u ? 1 : 0);
  return max(e, -126);  // subnormal tops have the exponent field 0 and end here too
}
// 2^e for -127 <= e <= 127.
__device__ __forceinline__ float pow2_f32(int e) {
  return __uint_as_float(e == -127 ? 0x00400000u : static_cast<uint32_t>(e + 127) << 23);
}

}  // namespace qlora
