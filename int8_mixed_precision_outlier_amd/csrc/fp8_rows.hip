// Quantizers of the block-scaled e4m3 path (gfx950), with the formulas of
// fp8.hpp: rows alone, rows after a root-mean-square norm (with the
// residual's addition), rows of a SiLU-gated product, and weights (offline).
// All of them are bound by HBM traffic at many rows and by latency at few:
// every 16-bit input is read once, 16 bytes per lane, and a block's 128
// columns are one 16-lane group's eight values each, so its maximum is four
// shuffle steps and no LDS.
//
// The scales leave k-major, xs[kb][m]: the product reads one block's scales
// of a tile's tokens as contiguous words.
#include "fp8.hpp"
#include "launch.hpp"

namespace i8mm {

namespace {

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
// bound this kernel (2048x20480 with two blocks per group: 38.2 us; with expf
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

}  // namespace

// Rows alone (GATED: the SiLU-gated product of a row's two halves).  A group
// of 16 lanes takes one block of one row, so a wavefront covers four rows
// and stores their four scales of a block as 16 contiguous bytes; the
// workgroup's four wavefronts cover 16 rows of U consecutive blocks.
template <int T, bool GATED, int U>
__global__ __launch_bounds__(256) void k_fp8_blocks(const uint16_t* __restrict__ X, int m0, int M,
                                                    int K, int strips, uint8_t* __restrict__ Xq,
                                                    float* __restrict__ xs) {
  const int t = threadIdx.x, lane16 = t & 15;
  const int strip = blockIdx.x % strips;
  const int m = m0 + blockIdx.x / strips * 16 + (t >> 4);
  if (m >= M) return;  // whole groups of 16 lanes
  const int KB = (K + kFp8Block - 1) / kFp8Block;
  const uint16_t* row = X + (size_t)m * (GATED ? 2 * (size_t)K : (size_t)K);
  uint4 a[U], b[GATED ? U : 1];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int k = (strip * U + u) * kFp8Block + lane16 * 8;
    a[u] = make_uint4(0, 0, 0, 0);
    if constexpr (GATED) b[u] = make_uint4(0, 0, 0, 0);
    if (k < K) {
      a[u] = *reinterpret_cast<const uint4*>(row + k);
      if constexpr (GATED) b[u] = *reinterpret_cast<const uint4*>(row + K + k);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int kb = strip * U + u;
    const int k = kb * kFp8Block + lane16 * 8;
    if (kb >= KB) break;  // the same for the whole workgroup
    float y[8];
    unpack8<T>(a[u], y);
    if constexpr (GATED) {
      float up[8];
      unpack8<T>(b[u], up);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = silu_mul(y[e], up[e]);
    }
    float s;
    const uint2 q = quant8(y, s);
    if (k < K) *reinterpret_cast<uint2*>(Xq + (size_t)m * K + k) = q;
    if (lane16 == 0) xs[(size_t)kb * M + m] = s;
  }
}

// Root-mean-square norm of one row per workgroup, the row in registers (C
// chunks of 8 columns per thread), so X (and the residual) is read once:
//   h = RN16(x + r)  (or x),  y = h * rsqrt(mean(h^2) + eps) * g,
// the statistics and y in fp32, y quantized unrounded.  H and R (or X) may
// be the same buffer: a thread reads its columns before it writes them.
template <int T, bool RES, int NT, int C>
__global__ __launch_bounds__(NT) void k_fp8_rms_norm(const uint16_t* X, const uint16_t* R,
                                                     const uint16_t* __restrict__ g, int m0, int M,
                                                     int K, float eps, uint16_t* H,
                                                     uint8_t* __restrict__ Xq,
                                                     float* __restrict__ xs) {
  constexpr int NW = NT / 64;
  __shared__ float part[NW];
  const int t = threadIdx.x;
  // consecutive rows on one XCD: their scales share cache lines
  const int m = m0 + xcd_remap(blockIdx.x, gridDim.x);
  const size_t base = (size_t)m * K;
  uint4 h[C], w[C];
  float ss = 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int k = (c * NT + t) * 8;
    h[c] = w[c] = make_uint4(0, 0, 0, 0);
    if (k < K) {
      h[c] = *reinterpret_cast<const uint4*>(X + base + k);
      if constexpr (RES) {
        float x[8], r[8];
        unpack8<T>(h[c], x);
        unpack8<T>(*reinterpret_cast<const uint4*>(R + base + k), r);
        h[c] = make_uint4(pack16x2<T>(x[0] + r[0], x[1] + r[1]), pack16x2<T>(x[2] + r[2], x[3] + r[3]),
                          pack16x2<T>(x[4] + r[4], x[5] + r[5]), pack16x2<T>(x[6] + r[6], x[7] + r[7]));
      }
      w[c] = *reinterpret_cast<const uint4*>(g + k);
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int k = (c * NT + t) * 8;
    if constexpr (RES) {
      if (k < K) *reinterpret_cast<uint4*>(H + base + k) = h[c];
    }
    float x[8];
    unpack8<T>(h[c], x);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) ss += __shfl_xor(ss, o, kWave);
  if constexpr (NW > 1) {
    if ((t & 63) == 0) part[t >> 6] = ss;
    __syncthreads();
    ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NW; ++i) ss += part[i];
  }
  const float rs = 1.0f / sqrtf(ss / (float)K + eps);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int k = (c * NT + t) * 8;
    if ((k & ~(kFp8Block - 1)) >= K) break;  // whole groups of 16 lanes
    float x[8], gw[8], y[8];
    unpack8<T>(h[c], x);
    unpack8<T>(w[c], gw);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = x[e] * rs * gw[e];
    float s;
    const uint2 q = quant8(y, s);
    if (k < K) *reinterpret_cast<uint2*>(Xq + base + k) = q;
    if ((t & 15) == 0) xs[(size_t)(k / kFp8Block) * M + m] = s;
  }
}

// Weight quantizer (offline): one workgroup per 128 (k) x 128 (n) block of
// W[K][N], read coalesced along n into LDS, its maximum taken on the way,
// and written transposed in the packed layout (padding columns zero).
template <int T>
__global__ __launch_bounds__(256) void k_fp8_weight(const uint16_t* __restrict__ W, int K, int N,
                                                    int KB, uint8_t* __restrict__ Wq,
                                                    float* __restrict__ ws) {
  constexpr int LD = 128 + 2;  // a stride of an odd number of words
  __shared__ uint16_t tile[128][LD];
  __shared__ float part[4];
  const int t = threadIdx.x;
  const int kb = blockIdx.x % KB, nb = blockIdx.x / KB;
  float a = 0.0f;
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int r = p * 16 + (t >> 4), c = (t & 15) * 8;
    const int k = kb * 128 + r, n = nb * 128 + c;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (k < K && n < N) v = *reinterpret_cast<const uint4*>(W + (size_t)k * N + n);
    float f[8];
    unpack8<T>(v, f);
    const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      a = fmaxf(a, fabsf(f[e]));
      tile[r][c + e] = (uint16_t)(d[e >> 1] >> (16 * (e & 1)));
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor(a, o, kWave));
  if ((t & 63) == 0) part[t >> 6] = a;
  __syncthreads();
  a = fmaxf(fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3])), kScaleFloor);
  const float inv = kE4m3Max / a;
  if (t == 0) ws[(size_t)nb * KB + kb] = a / kE4m3Max;
  // 1024 chunks of 16 k-bytes: chunk q = ((row block * 8 + chunk) * 16 + row)
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int q = p * 256 + t;
    const int rb = q >> 7, c = (q >> 4) & 7, r = q & 15;
    const int n = nb * 128 + rb * 16 + r;
    if (n < N) {
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          f[i] = to_f32<T>(tile[c * 16 + e * 4 + i][rb * 16 + r]) * inv;
        o[e] = pack_e4m3x4(f[0], f[1], f[2], f[3]);
      }
      *reinterpret_cast<uint4*>(Wq + fp8_pack_offset(n, kb * 128 + c * 16, KB)) =
          make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// Packs a row-major e4m3 matrix [N][K], zero-filling the k padding.  One
// thread per 16-byte chunk of the destination.
__global__ __launch_bounds__(256) void k_fp8_pack(const uint8_t* __restrict__ src, int K,
                                                  uint8_t* __restrict__ dst, int KB,
                                                  int64_t nchunks) {
  const int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (q >= nchunks) return;
  const int r = (int)(q & 15), c = (int)((q >> 4) & 7);
  const int64_t blk = q >> 7;
  const int64_t row = blk / KB * 16 + r;
  const int k = (int)(blk % KB) * 128 + c * 16;
  uint4 v = make_uint4(0, 0, 0, 0);
  if (k < K) v = *reinterpret_cast<const uint4*>(src + row * K + k);
  *reinterpret_cast<uint4*>(dst + q * 16) = v;
}

// Rows per launch: a launch holds fewer than 2^32 threads, and a matrix of
// 16 columns may have 2^27 rows.
constexpr int kRowsPerLaunch = 1 << 20;

template <int T, bool GATED, int U>
static hipError_t run_strips(const void* X, int M, int K, void* Xq, float* xs, hipStream_t st) {
  const int KB = (K + kFp8Block - 1) / kFp8Block, strips = (KB + U - 1) / U;
  for (int64_t m0 = 0; m0 < M; m0 += kRowsPerLaunch) {
    const int rows = (int)(M - m0 < kRowsPerLaunch ? M - m0 : kRowsPerLaunch);
    k_fp8_blocks<T, GATED, U><<<strips * ((rows + 15) / 16), 256, 0, st>>>(
        static_cast<const uint16_t*>(X), (int)m0, M, K, strips, static_cast<uint8_t*>(Xq), xs);
  }
  return hipGetLastError();
}

// One block per 16 lanes while that keeps the workgroups within one round of
// the chip (8 per CU): the calls are then bound by latency (1x20480 gated, U =
// 1, 2, 4: 2.5, 3.1, 4.0 us; 300x5120: 2.5, 2.8, 3.4).  Two for more: 4096x12288,
// U = 1, 2, 4, 8: 27.4, 24.9, 25.1, 27.1 us (6.1 TB/s); 2048x20480 gated: 38.8,
// 38.2, 38.8, 41.7 (5.5 TB/s).
template <int T, bool GATED>
static hipError_t run_blocks(const void* X, int M, int K, void* Xq, float* xs, hipStream_t st) {
  const int64_t groups = ((int64_t)M + 15) / 16 * ((K + kFp8Block - 1) / kFp8Block);
  return groups <= 8 * device_cu_count() ? run_strips<T, GATED, 1>(X, M, K, Xq, xs, st)
                                         : run_strips<T, GATED, 2>(X, M, K, Xq, xs, st);
}

hipError_t launch_fp8_quantize(const void* X, int type, int M, int K, void* Xq, float* xs,
                               hipStream_t st) {
  return type == kF16 ? run_blocks<kF16, false>(X, M, K, Xq, xs, st)
                      : run_blocks<kBf16, false>(X, M, K, Xq, xs, st);
}

hipError_t launch_fp8_silu_mul(const void* GU, int type, int M, int I, void* Aq, float* as,
                               hipStream_t st) {
  return type == kF16 ? run_blocks<kF16, true>(GU, M, I, Aq, as, st)
                      : run_blocks<kBf16, true>(GU, M, I, Aq, as, st);
}

struct NormCall {
  const uint16_t *X, *R, *g;
  int M, K;
  float eps;
  uint16_t* H;
  uint8_t* Xq;
  float* xs;
};

template <int T, int NT, int C>
static hipError_t run_norm(const NormCall& c, hipStream_t st) {
  auto kern = c.R ? k_fp8_rms_norm<T, true, NT, C> : k_fp8_rms_norm<T, false, NT, C>;
  for (int64_t m0 = 0; m0 < c.M; m0 += kRowsPerLaunch) {
    const int rows = (int)(c.M - m0 < kRowsPerLaunch ? c.M - m0 : kRowsPerLaunch);
    kern<<<rows, NT, 0, st>>>(c.X, c.R, c.g, (int)m0, c.M, c.K, c.eps, c.H, c.Xq, c.xs);
  }
  return hipGetLastError();
}

// Threads and chunks per thread that hold a row of K <= 65536 columns: about
// as many threads as chunks for few rows, which wait for one row's latency
// (1x4096, 512 x 1 against 256 x 2: 2.8 and 3.1 us; 333x4112, 512 x 2 against
// 256 x 3: 3.6 and 3.9), fewer threads for many, which need workgroups to
// overlap (2048x5120, 256 x 3 against 512 x 2: 12.9 and 13.6 us; 4096x12288,
// 768 x 2, 512 x 3, 256 x 6: 67.9, 68.8, 74.8 us = 5.2 TB/s; 4000x272, 64 x 1
// against 256 x 1: 4.1 and 4.7).
template <int T>
static hipError_t norm_shape(const NormCall& c, hipStream_t st) {
  const int chunks = (c.K + 7) / 8;
  const bool few = c.M <= 2 * device_cu_count();
  if (chunks <= 64) return run_norm<T, 64, 1>(c, st);
  if (chunks <= 128) return run_norm<T, 128, 1>(c, st);
  if (chunks <= 256) return run_norm<T, 256, 1>(c, st);
  if (chunks <= 512) return few ? run_norm<T, 512, 1>(c, st) : run_norm<T, 256, 2>(c, st);
  if (chunks <= 768 && !few) return run_norm<T, 256, 3>(c, st);
  if (chunks <= 1024) return run_norm<T, 512, 2>(c, st);
  if (chunks <= 1536) return run_norm<T, 768, 2>(c, st);
  if (chunks <= 2048) return run_norm<T, 1024, 2>(c, st);
  if (chunks <= 4096) return run_norm<T, 1024, 4>(c, st);
  return run_norm<T, 1024, 8>(c, st);
}

hipError_t launch_fp8_rms_norm(const void* X, const void* R, const void* g, int type, int M, int K,
                               float eps, void* H, void* Xq, float* xs, hipStream_t st) {
  const NormCall c{static_cast<const uint16_t*>(X), static_cast<const uint16_t*>(R),
                   static_cast<const uint16_t*>(g), M, K, eps, static_cast<uint16_t*>(H),
                   static_cast<uint8_t*>(Xq), xs};
  return type == kF16 ? norm_shape<kF16>(c, st) : norm_shape<kBf16>(c, st);
}

hipError_t launch_fp8_quantize_weight(const void* W, int type, int K, int N, void* Wq, float* ws,
                                      hipStream_t st) {
  const int KB = (K + 127) / 128, grid = KB * ((N + 127) / 128);
  const uint16_t* w = static_cast<const uint16_t*>(W);
  uint8_t* q = static_cast<uint8_t*>(Wq);
  if (type == kF16)
    k_fp8_weight<kF16><<<grid, 256, 0, st>>>(w, K, N, KB, q, ws);
  else
    k_fp8_weight<kBf16><<<grid, 256, 0, st>>>(w, K, N, KB, q, ws);
  return hipGetLastError();
}

hipError_t launch_fp8_pack_weight(const void* src, int N, int K, void* dst, hipStream_t st) {
  const int KB = (int)(fp8_kpad(K) / 128);
  const int64_t nchunks = (int64_t)N * KB * 8;
  k_fp8_pack<<<(unsigned)((nchunks + 255) / 256), 256, 0, st>>>(
      static_cast<const uint8_t*>(src), K, static_cast<uint8_t*>(dst), KB, nchunks);
  return hipGetLastError();
}

}  // namespace i8mm
