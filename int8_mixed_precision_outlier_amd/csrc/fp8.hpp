// Block-scaled 8-bit floating point (e4m3): device helpers and internal
// launchers shared by the quantizers (fp8_rows.hip) and the products
// (fp8_gemm.hip, fp8_decode.hip).
//
// A row of numbers is held as e4m3 numbers (4 exponent bits, 3 mantissa
// bits, no infinities, largest 448) with one fp32 scale per block of 128
// columns, so that an outlier column costs precision only within its own
// block:
//   a = max(max |x| over the block, 2^-100),  s = a / 448,
//   q = e4m3_rne(RN32(x * RN32(448 / a))),    x ~ q * s.
// The floor of 2^-100 keeps 448 / a finite for an all-zero block and for
// blocks of subnormal bf16 values.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"

namespace i8mm {

typedef int v8i __attribute__((ext_vector_type(8)));

constexpr int kFp8Block = 128;        // columns (and features) per scale
constexpr float kE4m3Max = 448.0f;    // largest e4m3 magnitude
constexpr float kScaleFloor = 0x1p-100f;
// A buffer offset past every operand (they hold at most 2^31 bytes).
constexpr uint32_t kOutOfRange = 0xffffff00u;

// The 16-bit types: kF16 / kBf16 name them in template arguments.
constexpr int kF16 = 0, kBf16 = 1;

// One 16-bit value -> fp32 (exact).
template <int T>
__device__ __forceinline__ float to_f32(uint16_t b) {
  if constexpr (T == kF16) return h2f(b);
  return __builtin_bit_cast(float, (uint32_t)b << 16);
}

// Two fp32 values as a packed pair of 16-bit ones, round to nearest even.
template <int T>
__device__ __forceinline__ uint32_t pack16x2(float a, float b) {
  if constexpr (T == kF16) {
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    const h2 h = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, h);
  } else {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    const b2 h = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, h);
  }
}

// Eight 16-bit values (16 bytes) -> fp32.
template <int T>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = to_f32<T>((uint16_t)(d[e >> 1] >> (16 * (e & 1))));
}

// Four fp32 values as four e4m3 numbers, round to nearest even (NaN stays
// NaN).  The quantizers' products stay below 448 (1 + 2^-22), which rounds
// to 448, so the conversion never meets a value out of range.
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
  return (uint32_t)r;
}

// 16x16x128 e4m3 MFMA into a fresh fp32 block: P[16][16] = A[16 rows][128 k]
// . B[16 cols][128 k]^T.  Lane l supplies row/col l % 16 and 32 k-bytes of
// quarter l / 16; A and B use the same (lane, byte) -> k assignment, so any
// consistent permutation of k gives the same sum.  Register i of lane l
// holds P[row = 4*(l/16) + i][col = l%16].
// Precision: the instruction adds the exact products of a lane's 8
// consecutive bytes after cutting each off below 2^-13 of 2^E, E the largest
// sum of the two factors' exponents among the 8, and the sums of 8 in fp32
// (found with single products; the 16x16x32 form does the same at half the
// rate).  Against e4m3's own rounding, 2^-4, and the 16-bit result's that is
// small (a random product of 5136 columns stays at the fp16 result's
// rounding, 2.1e-4), so the products stay on it instead of on fp16 matrix
// instructions at half the rate.
__device__ __forceinline__ v4f mfma16_e4m3(v8i a, v8i b) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, v4f{}, 0, 0, 0, 0, 0, 0);
}

// 16x16x32 matrix instruction on fp16 or bf16 operands with fp32 accumulation
// (lane convention as mfma16_f16).
template <int T>
__device__ __forceinline__ v4f mfma32(v4i a, v4i b, v4f c) {
  if constexpr (T == kF16) {
    return mfma16_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c);
  } else {
    typedef __bf16 v8b __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, a),
                                                   __builtin_bit_cast(v8b, b), c, 0, 0, 0);
  }
}

// ---- packed layout of an e4m3 weight: 16-row x 128-column blocks of 2 KB,
// row-block major, columns zero-padded to a multiple of 128.  Inside a block
// the eight 16-byte column chunks are stored chunk-major, so each half block
// is one contiguous 64-lane x 16-byte load (lane l: row l % 16, chunks l/16
// and 4 + l/16) and the whole block one MFMA operand.
__host__ __device__ __forceinline__ int64_t fp8_kpad(int64_t K) { return (K + 127) / 128 * 128; }
__host__ __device__ __forceinline__ int64_t fp8_pack_offset(int64_t row, int64_t k, int64_t KB) {
  return ((row >> 4) * KB + (k >> 7)) * 2048 + (((k >> 4) & 7) * 16 + (row & 15)) * 16 + (k & 15);
}

hipError_t launch_fp8_quantize(const void* X, int type, int M, int K, void* Xq, float* xs,
                               hipStream_t st);
hipError_t launch_fp8_silu_mul(const void* GU, int type, int M, int I, void* Aq, float* as,
                               hipStream_t st);
hipError_t launch_fp8_rms_norm(const void* X, const void* R, const void* g, int type, int M, int K,
                               float eps, void* H, void* Xq, float* xs, hipStream_t st);
// One call of the norms on both sides of a residual's addition; pointers as in
// include/int8mm.h (gate null: none; Y null: quantized into Xq, xs).
struct SandwichCall {
  const uint16_t *X, *R, *post, *pre, *gate;
  uint16_t *H, *Y;
  uint8_t* Xq;
  float* xs;
  int M, K, tokens_per_gate, type;
  float alpha, eps;
};
hipError_t launch_sandwich_norm(const SandwichCall& c, hipStream_t st);
hipError_t launch_fp8_quantize_weight(const void* W, int type, int K, int N, void* Wq, float* ws,
                                      hipStream_t st);
hipError_t launch_fp8_pack_weight(const void* src, int N, int K, void* dst, hipStream_t st);

// One block-scaled product.  bias and Y are of `type`; the operands as in
// include/int8mm.h.
struct Fp8Call {
  const uint8_t* X;
  const float* xs;
  const uint8_t* W;
  const float* ws;
  const uint16_t* bias;
  uint16_t* Y;
  int M, N, K, type;
};

// The kernels of an M x N product.  Tiles: features [0, n1) in tiles `first`,
// [n1, N) (if any) in tiles `second`; kDecode: the weight-streaming kernel
// with R feature and T token blocks of 16.
enum { kDecode = -1, kTile256 = 0, kTile256x128 = 1, kTile128 = 2, kTile128Deep = 3, kTile64x128 = 4 };
struct Fp8Plan {
  int first, n1, second;
};
Fp8Plan fp8_plan(int M, int N);
constexpr int kFp8DecodeMaxM = 128;
struct Fp8DecodePlan {
  int R, T;
  int64_t cost;  // rounds of workgroups * (R + T)
};
Fp8DecodePlan fp8_decode_plan(int M, int N);  // M <= kFp8DecodeMaxM
hipError_t launch_fp8_decode(const Fp8Call& c, hipStream_t st);
hipError_t launch_fp8_matmul(const Fp8Call& c, hipStream_t st);

}  // namespace i8mm
