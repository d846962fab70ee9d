// Block-scaled e4m3 product for few tokens, at most 128 (gfx950): the packed weight is
// streamed from HBM exactly once, every byte feeding a 16x16x128 e4m3 MFMA
// whose 16 columns are tokens.
//
// A workgroup owns R blocks of 16 features over all of K, so nothing is
// combined across workgroups; its KS wavefronts take the K blocks in turn and
// add their partial sums through LDS at the end in a fixed
// order.  A wavefront's K block of 16 features is 2 KB of contiguous W, two
// 16-byte loads per lane in exactly the MFMA's operand layout (nontemporal:
// the stream is never read again).  The tokens' bytes and scales reach a part
// of LDS that is the wavefront's own, by DMA, so no barrier is needed: an
// instruction moves 8 rows x 128 bytes, whole cache lines, with the chunks of
// a row swapped as in fp8_gemm.hip, where 16 rows x 64 bytes straight into
// registers fetched each line twice (a CU then took in 38 GB/s, too little
// for HBM's rate at more than 16 tokens: 32x20480x5120 33.6 us).  The next K
// block is on its way under the MFMAs and scaling fmas of the current one.
//
// Bound by HBM for a few tokens (1x12288x49152: 86 us = 7.0 TB/s, 32x12288x36864:
// 71 us = 6.4 TB/s).  Towards 128 tokens no unit is the bound: on 77x5136x20464
// (29 us, 3.6 TB/s of weight, 28 GB/s of both operands per CU) the one wavefront
// per SIMD issues 35 % of its time, waits for memory 36 % and for its turn or
// the matrix unit 29 %, and the matrix unit is busy 14 % of it (counters).
#include "common.hpp"
#include "fp8.hpp"
#include "launch.hpp"

#include <atomic>

namespace i8mm {

// LDS: two stages of a K block per wavefront, each T x 16 rows of 128 bytes
// and their scales (64 tokens per DMA); at the end the partial sums.
template <int R, int T, int KS>
struct DecodeLds {
  static constexpr int SDMA = (T + 3) / 4;  // DMAs of 64 token scales
  static constexpr int BLOCK = T * 2048 + SDMA * 256;
  static constexpr int WAVE = 2 * BLOCK;
  static constexpr int SUMS = KS * R * T * 1024;
  static constexpr int SIZE = KS * WAVE > SUMS ? KS * WAVE : SUMS;
  static_assert(SIZE <= 160 * 1024, "LDS budget");
};

template <int TY, int R, int T, int KS>
__global__ __launch_bounds__(KS * 64) void k_fp8_decode(
    const uint8_t* __restrict__ X, const float* __restrict__ xs, const uint8_t* __restrict__ W,
    const float* __restrict__ ws, const uint16_t* __restrict__ bias, uint16_t* __restrict__ Y,
    int M, int N, int K, int KB) {
  using L = DecodeLds<R, T, KS>;
  extern __shared__ __align__(16) int8_t smem[];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q4 = lane >> 4, r16 = lane & 15;
  const int nrb = N >> 4;
  const int rb0 = blockIdx.x * R;
  int8_t* mine = smem + w * L::WAVE;

  // rows past M and features past N repeat the last one: they only feed
  // outputs that are never stored
  const int xrow = lane >> 3;
  const uint32_t chunk = (lane & 7) ^ xrow;
  uint32_t xsrc[2 * T];
#pragma unroll
  for (int t = 0; t < 2 * T; ++t)
    xsrc[t] = (uint32_t)min(t * 8 + xrow, M - 1) * (uint32_t)K + chunk * 16u;
  uint32_t wsrc[R];
  // the weight scales through the constant address space: scalar loads
  typedef const __attribute__((address_space(4))) float* scalar_ptr;
  scalar_ptr wsrow[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int rb = min(rb0 + r, nrb - 1);
    wsrc[r] = (uint32_t)rb * (uint32_t)KB * 2048u;
    wsrow[r] = (scalar_ptr)(uintptr_t)(ws + (size_t)(rb / 8) * KB);
  }
  const uint32_t xbytes = (uint32_t)M * (uint32_t)K;
  const uint32_t wbytes = (uint32_t)nrb * (uint32_t)KB * 2048u;

  struct Weights {
    v4i w[R][2];
    float s[R];
  };
  // Loads of K block kb into registers and a stage of LDS.  A block at or past
  // KB gets empty descriptors and zero scales, and the columns at or past K of
  // a last block that K ends inside are read from an offset out of every
  // range: zeros.  So a load has no branch and always the same OPS vector
  // loads, which the wait in `step` counts.
  constexpr int OPS = 2 * T + L::SDMA + 2 * R;
  constexpr int kNonTemporal = 2;
  auto load = [&](int kb, int stage, Weights& o) {
    const bool live = kb < KB;
    const int k = live ? kb : 0;
    const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
        (void*)X, (short)0, live ? (int)xbytes : 0, 0x00020000);
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(xs + (size_t)k * M), (short)0, live ? M * 4 : 0, 0x00020000);
    const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
        (void*)W, (short)0, live ? (int)wbytes : 0, 0x00020000);
    const bool out = (uint32_t)k * 128u + chunk * 16u >= (uint32_t)K;
    int8_t* dst = mine + stage * L::BLOCK;
#pragma unroll
    for (int t = 0; t < 2 * T; ++t)
      dma16(rx, dst + t * 1024, (int)(out ? kOutOfRange : xsrc[t]), k * 128);
#pragma unroll
    for (int t = 0; t < L::SDMA; ++t) dma4(rs, dst + T * 2048 + t * 256, lane * 4 + t * 256, 0);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      o.s[r] = wsrow[r][k];  // block 0's past KB; `compute` takes zero there
#pragma unroll
      for (int h = 0; h < 2; ++h)
        o.w[r][h] = __builtin_bit_cast(
            v4i, __builtin_amdgcn_raw_buffer_load_b128(
                     rw, lane * 16, (int)(wsrc[r] + (uint32_t)k * 2048u + h * 1024u), kNonTemporal));
    }
  };

  v4f acc[R][T];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < T; ++t) acc[r][t] = v4f{};
  auto join = [](const v4i& lo, const v4i& hi) {
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  auto compute = [&](int kb, int stage, const Weights& o) {
    const bool live = kb < KB;
    const int8_t* src = mine + stage * L::BLOCK;
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const int8_t* row = src + (t * 16 + r16) * 128;
      const v8i x = join(*reinterpret_cast<const v4i*>(row + (q4 ^ (r16 & 7)) * 16),
                         *reinterpret_cast<const v4i*>(row + ((q4 + 4) ^ (r16 & 7)) * 16));
      const float sx = *reinterpret_cast<const float*>(src + T * 2048 + (t * 16 + r16) * 4);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float s = sx * (live ? o.s[r] : 0.0f);
        const v4f p = mfma16_e4m3(join(o.w[r][0], o.w[r][1]), x);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[r][t][e] = fmaf(p[e], s, acc[r][t][e]);
      }
    }
  };
  // a step: the next K block's loads, then the wait for the current one's
  auto step = [&](int kb, int stage, const Weights& cur, Weights& next) {
    load(kb + KS, stage ^ 1, next);
    wait_vm<OPS>();
    compute(kb, stage, cur);
    // the stage's reads are done before the next step's DMAs overwrite it
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  };

  Weights a, b;
  if (w < KB) {
    load(w, 0, a);
    for (int kb = w; kb < KB; kb += 2 * KS) {
      step(kb, 0, a, b);
      step(kb + KS, 1, b, a);
    }
  }
  wait_vm<0>();  // no DMA may still write LDS
  __syncthreads();  // the partial sums overwrite the stages
  v4f(*red)[R * T][64] = reinterpret_cast<v4f(*)[R * T][64]>(smem);
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < T; ++t) red[w][r * T + t][lane] = acc[r][t];
  __syncthreads();
  // the R * T blocks of 16 features x 16 tokens over the wavefronts: the
  // partial sums in wavefront order, the bias, one store of 4 features
  for (int o = w; o < R * T; o += KS) {
    v4f y = red[0][o][lane];
#pragma unroll
    for (int i = 1; i < KS; ++i) y += red[i][o][lane];
    const int n = (rb0 + o / T) * 16 + 4 * q4, m = o % T * 16 + r16;
    if (m < M && n < N) {
      if (bias) {
        const uint2 v = *reinterpret_cast<const uint2*>(bias + n);
        y[0] += to_f32<TY>((uint16_t)v.x);
        y[1] += to_f32<TY>((uint16_t)(v.x >> 16));
        y[2] += to_f32<TY>((uint16_t)v.y);
        y[3] += to_f32<TY>((uint16_t)(v.y >> 16));
      }
      *reinterpret_cast<uint2*>(Y + (size_t)m * N + n) =
          make_uint2(pack16x2<TY>(y[0], y[1]), pack16x2<TY>(y[2], y[3]));
    }
  }
}

template <int TY, int R, int T, int KS>
static hipError_t run_decode(const Fp8Call& c, hipStream_t st) {
  constexpr int SMEM = DecodeLds<R, T, KS>::SIZE;
  auto kern = k_fp8_decode<TY, R, T, KS>;
  // the dynamic-LDS limit is raised once per device the kernels run on
  static std::atomic<uint64_t> attr_set{0};
  int dev = 0;
  (void)hipGetDevice(&dev);
  const uint64_t bit = 1ull << (dev & 63);
  if (!(attr_set.load(std::memory_order_relaxed) & bit)) {
    const hipError_t e = hipFuncSetAttribute((const void*)kern,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != hipSuccess) return e;
    attr_set.fetch_or(bit, std::memory_order_relaxed);
  }
  const int KB = (c.K + kFp8Block - 1) / kFp8Block;
  kern<<<(c.N / 16 + R - 1) / R, KS * 64, SMEM, st>>>(c.X, c.xs, c.W, c.ws, c.bias, c.Y, c.M, c.N,
                                                      c.K, KB);
  return hipGetLastError();
}

// Feature blocks per workgroup.  The time goes about with the most loaded CU's
// rounds of workgroups times the blocks it reads per K block in each, R of the
// weight and T of the tokens; among the counts that are built, the choice that
// makes that least (ties: fewer) is the fastest or within 4 % of it at 28
// measured shapes of 9 to 128 tokens (32x5120x5120, R = 1, 2, 3, 4,
// 5: 12.0, 9.3, 11.2, 12.9, 13.6 us; 64x12288x36864, R = 1, 3, 5, 9: 155.6,
// 95.8, 86.9, 75.9; 128x5120x5120, R = 1, 2, 3: 26.6, 17.8, 21.1).  At most 8
// tokens bring little token traffic (the rows past M repeat the last one):
// with four or more blocks per CU one block per workgroup is best, the most
// loads in flight (1x12288x36864, R = 1, 3, 9: 65.4, 68.3, 69.9).  Above 64
// tokens the partial sums of more than 5 blocks would not fit LDS, and where 1
// to 4 blocks and the tokens' make more than 9, 64x128 tiles are faster
// (120x5120x16384, 4 blocks: 27.3 us against 23.6), above 112 tokens tiles
// also where 5 would be best.  7 and 8 are not built: they would gain where they
// just fill the CUs, near 28672 and 32768 features (weights that no cache
// holds, us as it is / with them: 16x8192x28672 40.2 / 38.7, 32x12288x28672 60.6 /
// 56.9, 48x4096x28672 25.3 / 23.8, 64x8192x28672 48.0 / 43.5, 32x5120x32000 30.0 /
// 29.5, 64x12288x32768 72.5 / 69.8).
constexpr int kDecodeR[] = {1, 2, 3, 4, 5, 6, 9};

Fp8DecodePlan fp8_decode_plan(int M, int N) {
  const int cus = device_cu_count(), nrb = N / 16, T = (M + 15) / 16;
  Fp8DecodePlan best{1, T, INT64_MAX};
  for (int R : kDecodeR) {
    if (T > 4 && R > 5) break;
    if (T > 4 && (R < 5 ? R + T > 9 : T > 7)) continue;
    const int64_t groups = (nrb + R - 1) / R, cost = (groups + cus - 1) / cus * (R + T);
    if (cost < best.cost) best = Fp8DecodePlan{R, T, cost};
    if (M <= 8 && nrb >= 4 * cus) break;
  }
  return best;
}

// Wavefronts that split K: eight for up to three feature and four token
// blocks, else four (registers for twice the accumulators and weights, LDS
// for twice the tokens).
template <int TY, int T>
static hipError_t decode_blocks(int R, const Fp8Call& c, hipStream_t st) {
  constexpr int KS = T <= 4 ? 8 : 4;
  if (R == 1) return run_decode<TY, 1, T, KS>(c, st);
  if constexpr (T <= 7) {
    if (R == 2) return run_decode<TY, 2, T, KS>(c, st);
    if (R == 5) return run_decode<TY, 5, T, 4>(c, st);
  }
  if constexpr (T <= 6)
    if (R == 3) return run_decode<TY, 3, T, KS>(c, st);
  if constexpr (T <= 5)
    if (R == 4) return run_decode<TY, 4, T, 4>(c, st);
  if constexpr (T <= 4)
    return R == 6 ? run_decode<TY, 6, T, 4>(c, st) : run_decode<TY, 9, T, 4>(c, st);
  return hipErrorInvalidValue;
}

template <int TY>
static hipError_t decode_tokens(const Fp8Call& c, hipStream_t st) {
  const Fp8DecodePlan p = fp8_decode_plan(c.M, c.N);
  switch (p.T) {
    case 1: return decode_blocks<TY, 1>(p.R, c, st);
    case 2: return decode_blocks<TY, 2>(p.R, c, st);
    case 3: return decode_blocks<TY, 3>(p.R, c, st);
    case 4: return decode_blocks<TY, 4>(p.R, c, st);
    case 5: return decode_blocks<TY, 5>(p.R, c, st);
    case 6: return decode_blocks<TY, 6>(p.R, c, st);
    case 7: return decode_blocks<TY, 7>(p.R, c, st);
    default: return decode_blocks<TY, 8>(p.R, c, st);
  }
}

hipError_t launch_fp8_decode(const Fp8Call& c, hipStream_t st) {
  return c.type == kF16 ? decode_tokens<kF16>(c, st) : decode_tokens<kBf16>(c, st);
}

}  // namespace i8mm
