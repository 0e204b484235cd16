// The FP8 cache row's quantisation and its inverse (the row and its rule are described
// in mla_fp8.cu), shared by the kernels that write and read such rows.
#pragma once

#include <cuda_fp8.h>
#include <stdint.h>

namespace mla {
namespace {

constexpr int kFp8RowBytes = 656;

// Magnitude of the non-negative E4M3 code c (0 .. 0x7E): exact in fp32.
__device__ __forceinline__ float e4m3_magnitude(uint32_t c) {
  const uint32_t e = c >> 3, m = c & 7u;
  // subnormal: m * 2^-9; normal: (8 + m) * 2^(e - 10)
  const float p2 = __uint_as_float((uint32_t)(127 + (e ? (int)e - 10 : -9)) << 23);
  return (float)(e ? 8u + m : m) * p2;
}

// E4M3 byte nearest to the exact quotient x / scale (scale > 0, finite), ties to
// the even mantissa, saturating at +-448.
__device__ __forceinline__ uint32_t e4m3_nearest(float x, float scale) {
  const __nv_fp8_storage_t c0 = __nv_cvt_float_to_fp8(__fdiv_rn(x, scale), __NV_SATFINITE, __NV_E4M3);
  const uint32_t sign = (uint32_t)c0 & 0x80u;
  uint32_t c = (uint32_t)c0 & 0x7Fu;
  const float a = fabsf(x);
  const float y = e4m3_magnitude(c);
  if (c < 0x7Eu) {
    const float mid = 0.5f * (y + e4m3_magnitude(c + 1));
    const float r = fmaf(mid, scale, -a);           // > 0: below the midpoint; 0: on it
    if (r < 0.f || (r == 0.f && (c & 1u))) c += 1;
  }
  if (c > 0u && c == ((uint32_t)c0 & 0x7Fu)) {
    const float mid = 0.5f * (e4m3_magnitude(c - 1) + y);
    const float r = fmaf(mid, scale, -a);
    if (r > 0.f || (r == 0.f && (c & 1u))) c -= 1;
  }
  return sign | c;
}

// Four E4M3 codes (the lowest byte first) times the tile's scale, as two bf16
// pairs: each code is widened exactly (to f16 by the E4M3 conversion, two codes
// per instruction, to fp32 by a mixed-precision multiply-add with 1), each pair
// multiplied by the fp32 scale in one packed multiply (each lane rounded to
// nearest, as two scalar multiplies), and the products rounded to bf16
// (measured faster than building the fp32 bits with integer operations).
// scale2: the scale in both halves.
__device__ __forceinline__ uint2 dequant4(uint32_t four, uint64_t scale2) {
  uint2 r;
  asm("{\n\t.reg .b16 c0, c1, l0, u0, l1, u1, one;\n\t.reg .b32 h0, h1;\n\t.reg .f32 a0, b0, a1, b1;\n\t"
      ".reg .b64 p0, p1;\n\t"
      "mov.b16 one, 0x3C00;\n\t"
      "mov.b32 {c0, c1}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 h0, c0;\n\t"
      "cvt.rn.f16x2.e4m3x2 h1, c1;\n\t"
      "mov.b32 {l0, u0}, h0;\n\t"
      "mov.b32 {l1, u1}, h1;\n\t"
      "fma.rn.f32.f16 a0, l0, one, 0f00000000;\n\t"
      "fma.rn.f32.f16 b0, u0, one, 0f00000000;\n\t"
      "fma.rn.f32.f16 a1, l1, one, 0f00000000;\n\t"
      "fma.rn.f32.f16 b1, u1, one, 0f00000000;\n\t"
      "mov.b64 p0, {a0, b0};\n\t"
      "mov.b64 p1, {a1, b1};\n\t"
      "mul.rn.f32x2 p0, p0, %3;\n\t"
      "mul.rn.f32x2 p1, p1, %3;\n\t"
      "mov.b64 {a0, b0}, p0;\n\t"
      "mov.b64 {a1, b1}, p1;\n\t"
      "cvt.rn.bf16x2.f32 %0, b0, a0;\n\t"
      "cvt.rn.bf16x2.f32 %1, b1, a1;\n\t}"
      : "=r"(r.x), "=r"(r.y)
      : "r"(four), "l"(scale2));
  return r;
}

// A warp's 512 latent values as E4M3 codes: lane l holds values [16 l, 16 l + 16)
// (tile l / 8, whose largest magnitude is reduced over its eight lanes); returns the
// lane's 16 codes and its tile's scale.  Every lane of the warp takes part.
__device__ __forceinline__ uint4 fp8_quantise16(const float (&x)[16], float* scale_out) {
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < 16; ++k) amax = fmaxf(amax, fabsf(x[k]));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float scale = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
  uint32_t packed[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t v = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v |= e4m3_nearest(x[4 * k + e], scale) << (8 * e);
    }
    packed[k] = v;
  }
  *scale_out = scale;
  return make_uint4(packed[0], packed[1], packed[2], packed[3]);
}

}  // namespace
}  // namespace mla
