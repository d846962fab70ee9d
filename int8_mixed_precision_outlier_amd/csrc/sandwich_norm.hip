// The norms on both sides of a residual's addition (gfx950):
//   z = x * rsqrt(mean(x^2) + eps) * post        the norm after a block
//   h = alpha * r + gate * z                     the residual, scaled, and the gated block
//   y = h * rsqrt(mean(h^2) + eps) * pre         the norm before the next block
// One row per workgroup, in registers from the first sum to the last store, so
// that every input is read once: without the fusion h alone would be written
// and read again.  All of it in fp32; h is rounded to its type on its way out
// only, and y is made from the unrounded h (a rounding step between the two
// norms would turn the last bits of the first one's sum into whole steps of y).
#include "fp8.hpp"
#include "fp8_quant.hpp"
#include "launch.hpp"

namespace i8mm {

namespace {

// The sum of v over the workgroup's NT threads, in every thread, in one order.
template <int NT>
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
  if constexpr (NT > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) v += part[i];
  }
  return v;
}

// 16 bytes; STREAM: nontemporally.
template <bool STREAM>
__device__ __forceinline__ uint4 load16(const uint16_t* p) {
  const v4i* from = reinterpret_cast<const v4i*>(p);
  return __builtin_bit_cast(uint4, STREAM ? __builtin_nontemporal_load(from) : *from);
}

template <int T, bool QUANT, bool STREAM, int NT, int C>
__global__ __launch_bounds__(NT) void k_sandwich_norm(SandwichCall c, int m0) {
  __shared__ float part[2][NT / 64];
  const int t = threadIdx.x;
  // consecutive rows on one XCD: their scales share cache lines
  const int m = m0 + xcd_remap(blockIdx.x, gridDim.x);
  const int K = c.K;
  const size_t base = (size_t)m * K;
  const uint16_t* gate = c.gate ? c.gate + (size_t)(m / c.tokens_per_gate) * K : nullptr;
  float h[C][8];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int k = (i * NT + t) * 8;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (k < K) v = load16<STREAM>(c.X + base + k);
    unpack8<T>(v, h[i]);
  }
  // the other operands' loads do not wait for the sum where registers hold them
  constexpr bool EARLY = C <= 2;
  uint4 r[EARLY ? C : 1], wp[EARLY ? C : 1], wg[EARLY ? C : 1], wn[EARLY ? C : 1];
  const uint32_t one = T == kF16 ? 0x3c003c00u : 0x3f803f80u;
  auto load = [&](int i, uint4& rr, uint4& p, uint4& g) {
    const int k = (i * NT + t) * 8;
    rr = p = make_uint4(0, 0, 0, 0);
    g = make_uint4(one, one, one, one);
    if (k < K) {
      rr = load16<STREAM>(c.R + base + k);
      p = *reinterpret_cast<const uint4*>(c.post + k);
      if (gate) g = *reinterpret_cast<const uint4*>(gate + k);
    }
  };
  auto load_pre = [&](int i, uint4& n) {
    const int k = (i * NT + t) * 8;
    n = make_uint4(0, 0, 0, 0);
    if (k < K) n = *reinterpret_cast<const uint4*>(c.pre + k);
  };
  if constexpr (EARLY) {
#pragma unroll
    for (int i = 0; i < C; ++i) load(i, r[i], wp[i], wg[i]), load_pre(i, wn[i]);
  }
#pragma unroll
  for (int i = 0; i < C; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(h[i][e], h[i][e], ss);
  ss = row_sum<NT>(ss, part[0]);
  const float rs = 1.0f / sqrtf(ss / (float)K + c.eps);
  ss = 0.0f;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int k = (i * NT + t) * 8;
    constexpr int L = EARLY ? 1 : 0;
    if constexpr (!EARLY) load(i, r[0], wp[0], wg[0]);
    float res[8], p[8], g[8];
    unpack8<T>(r[i * L], res);
    unpack8<T>(wp[i * L], p);
    unpack8<T>(wg[i * L], g);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      h[i][e] = fmaf(g[e], h[i][e] * rs * p[e], c.alpha * res[e]);
      ss = fmaf(h[i][e], h[i][e], ss);
    }
    if (k < K)
      *reinterpret_cast<uint4*>(c.H + base + k) =
          make_uint4(pack16x2<T>(h[i][0], h[i][1]), pack16x2<T>(h[i][2], h[i][3]),
                     pack16x2<T>(h[i][4], h[i][5]), pack16x2<T>(h[i][6], h[i][7]));
  }
  ss = row_sum<NT>(ss, part[1]);
  const float hs = 1.0f / sqrtf(ss / (float)K + c.eps);
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int k = (i * NT + t) * 8;
    if ((k & ~(kFp8Block - 1)) >= K) break;  // whole groups of 16 lanes
    constexpr int L = EARLY ? 1 : 0;
    if constexpr (!EARLY) load_pre(i, wn[0]);
    float n[8], y[8];
    unpack8<T>(wn[i * L], n);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = h[i][e] * hs * n[e];
    if constexpr (QUANT) {
      float s;
      const uint2 q = quant8(y, s);
      if (k < K) *reinterpret_cast<uint2*>(c.Xq + base + k) = q;
      if ((t & 15) == 0) c.xs[(size_t)(k / kFp8Block) * c.M + m] = s;
    } else if (k < K) {
      *reinterpret_cast<uint4*>(c.Y + base + k) =
          make_uint4(pack16x2<T>(y[0], y[1]), pack16x2<T>(y[2], y[3]), pack16x2<T>(y[4], y[5]),
                     pack16x2<T>(y[6], y[7]));
    }
  }
}

// Rows per launch: a launch holds fewer than 2^32 threads.
constexpr int kRowsPerLaunch = 1 << 20;

// Rows that the last-level cache (256 MB) cannot hold with what is written are
// read past it (4096x12288 quantized 79.5 -> 70.9 us = 5.0 TB/s, 16 bits 86.0 ->
// 73.7); smaller ones may be there still from their making (calls in turn on
// 220 MB, 2048x5120: 16.9 us, past it 20.1).
template <int T, int NT, int C>
hipError_t run(const SandwichCall& c, hipStream_t st) {
  const bool stream = (int64_t)c.M * c.K * 6 > (256ll << 20);
  auto kern = c.Y ? (stream ? k_sandwich_norm<T, false, true, NT, C>
                            : k_sandwich_norm<T, false, false, NT, C>)
                  : (stream ? k_sandwich_norm<T, true, true, NT, C>
                            : k_sandwich_norm<T, true, false, NT, C>);
  for (int64_t m0 = 0; m0 < c.M; m0 += kRowsPerLaunch)
    kern<<<(int)(c.M - m0 < kRowsPerLaunch ? c.M - m0 : kRowsPerLaunch), NT, 0, st>>>(c, (int)m0);
  return hipGetLastError();
}

// Threads and chunks of 8 columns per thread that hold a row of K <= 65536.  Two
// or three chunks per thread let more rows share a CU than one (us, calls in a
// graph, bf16: 4096x4096, 512 x 1 and 256 x 2: 23.3 and 22.1; 2048x5120, 640 x 1,
// 512 x 2, 384 x 2, 256 x 3: 20.4, 18.7, 18.1, 16.8; 4096x12288 through the cache,
// 768 x 2, 512 x 3, 384 x 4, 256 x 6: 81.2, 77.4, 83.4, 82.7); a few rows wait for
// one row's latency (1x5120, 384 x 2 and 256 x 3: 6.0 and 6.6).
template <int T>
hipError_t shape(const SandwichCall& c, hipStream_t st) {
  const int chunks = (c.K + 7) / 8;
  if (chunks <= 64) return run<T, 64, 1>(c, st);
  if (chunks <= 128) return run<T, 128, 1>(c, st);
  if (chunks <= 256) return run<T, 256, 1>(c, st);
  if (chunks <= 512) return run<T, 256, 2>(c, st);
  if (chunks <= 768)
    return c.M <= 2 * device_cu_count() ? run<T, 384, 2>(c, st) : run<T, 256, 3>(c, st);
  if (chunks <= 1536) return run<T, 512, 3>(c, st);
  if (chunks <= 2048) return run<T, 1024, 2>(c, st);
  if (chunks <= 4096) return run<T, 1024, 4>(c, st);
  return run<T, 1024, 8>(c, st);
}

}  // namespace

hipError_t launch_sandwich_norm(const SandwichCall& c, hipStream_t st) {
  return c.type == kF16 ? shape<kF16>(c, st) : shape<kBf16>(c, st);
}

}  // namespace i8mm
