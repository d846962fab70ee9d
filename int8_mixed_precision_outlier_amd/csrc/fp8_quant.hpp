// Device pieces of the operators that end in rows of numbers: a block's
// quantizer and the SiLU-gated product.
#pragma once

#include "fp8.hpp"

namespace i8mm {

// Maximum over the 16 lanes of a group, in every lane.
__device__ __forceinline__ float max16(float v) {
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) v = fmaxf(v, __shfl_xor(v, o, kWave));
  return v;
}

// Quantizes a lane's eight values of a 128-column block (the other lanes of
// its group of 16 hold the block's other values, zeros past the row's end):
// the packed e4m3 numbers, and the block's scale.
__device__ __forceinline__ uint2 quant8(const float (&y)[8], float& scale) {
  float a = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) a = fmaxf(a, fabsf(y[e]));
  a = fmaxf(max16(a), kScaleFloor);
  scale = a / kE4m3Max;
  const float inv = kE4m3Max / a;
  return make_uint2(pack_e4m3x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                    pack_e4m3x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
}

// silu(g) * u = g / (1 + exp(-g)) * u in fp32.  exp(-g) is 2^t times a
// correction for what t = -g log2(e) loses in its rounding (and log2(e) in
// its own), and the quotient is a product with the reciprocal instruction's
// result, at a third of the instructions of expf and the IEEE division, which
// bound k_fp8_blocks (2048x20480 with two blocks per group: 38.2 us; with expf
// and four: 50.8).  Within 8 half steps of 2^-24: the exponential and the
// reciprocal instruction 2 each, the correction (second-order terms and the
// rest of log2(e) add 2^-34), its fma to 1 + exp(-g) and the last two products
// 1 each.  The reciprocal is taken of (1 + exp(-g)) / 256 and the gate divided
// by 256, both exact: below g = -87.33 that of 1 + exp(-g) would leave the
// normal numbers, where the instruction gives 0, and so would y though a bf16
// u can be 3e38.  The gate's scaling costs 2 to 4 % (2048x20480 fp16 36.7 ->
// 38.2 us, 4096x12288 bf16 43.6 -> 44.6, calls in a graph); taken back per block
// behind a branch for products past 2^120 it cost as much.
// From g = -88.73 on exp(-g) is infinite and y a signed zero.
// The exponent's argument stops at 200, where exp is infinite or nothing
// beside 1 already, so that no product with log2(e) leaves the range: t and r
// would be infinities of both signs for the largest bf16 gates, and their
// result NaN.
__device__ __forceinline__ float silu_mul(float g, float u) {
  constexpr float kLog2e = 0x1.715476p+0f, kLog2eLow = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;
  constexpr float kScale = 0x1p-8f;
  const float c = __builtin_amdgcn_fmed3f(g, -200.0f, 200.0f);
  const float t = -c * kLog2e;
  const float r = fmaf(-c, kLog2eLow, fmaf(-c, kLog2e, -t));
  const float d = fmaf(__builtin_amdgcn_exp2f(t), fmaf(r, kLn2 * kScale, kScale), kScale);
  return g * kScale * __builtin_amdgcn_rcpf(d) * u;
}

}  // namespace i8mm
