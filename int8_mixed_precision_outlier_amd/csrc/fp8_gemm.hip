// Tiled block-scaled e4m3 product (gfx950):
//   Y[m][n] = sum_kb xs[kb][m] * ws[n/128][kb] * P_kb[m][n]  (+ bias[n]),
//   P_kb[m][n] = sum over the 128 columns of block kb of X[m][k] * W[n][k].
//
// One 16x16x128 e4m3 MFMA covers exactly one scale block, so its result is
// the unscaled P_kb of 16 features x 16 tokens, started from zero; the
// running sum takes it with one fp32 fma per element.  The weight is the
// MFMA's "A" operand (rows = features), the activations "B" (columns =
// tokens): register e of lane l holds feature 4*(l/16) + e of token l%16, so
// a lane's four products of one block share one token's scale, and the
// block of 128 features its weight scale: one product of scales per
// 16-token block and K block.
//
// Both operands reach LDS by direct DMA, one K block (128 bytes of every
// row) per stage.  W is packed (fp8.hpp): 1 KB contiguous per instruction.  X
// is row-major: an instruction moves 8 rows x 128 bytes, whole cache lines,
// and each lane fetches the 16-byte chunk (l % 8) ^ (row % 8) of its row, so
// that the 16 lanes of a fragment read (same chunk, rows 0-15) meet distinct
// LDS banks without any padding.  The tokens' scales come by DMA too, the
// weight's scales of the tile are staged once.
#include "common.hpp"
#include "fp8.hpp"

#include <atomic>

namespace i8mm {

namespace {

constexpr int kMaxKB = 65536 / kFp8Block;
// A buffer offset past every operand (they hold at most 2^31 bytes).
constexpr uint32_t kOutOfRange = 0xffffff00u;

// Four values of one token at features n .. n+3 (n % 4 == 0, N % 16 == 0).
template <int T>
__device__ __forceinline__ void store4(const v4f& y, int n, int m, int M, int N,
                                       uint16_t* __restrict__ Y) {
  if (m < M && n < N)
    *reinterpret_cast<uint2*>(Y + (size_t)m * N + n) =
        make_uint2(pack16x2<T>(y[0], y[1]), pack16x2<T>(y[2], y[3]));
}

}  // namespace

template <int T, int BM, int BN, int WM, int WN, int STAGES>
__global__ __launch_bounds__(WM* WN * 64, 2) void k_fp8_gemm(
    const uint8_t* __restrict__ X, const float* __restrict__ xs, const uint8_t* __restrict__ W,
    const float* __restrict__ ws, const uint16_t* __restrict__ bias, uint16_t* __restrict__ Y,
    int M, int N, int K, int KB, int tilesM, int tilesN, int groupM) {
  constexpr int NWAVE = WM * WN;
  constexpr int WTM = BM / WM, WTN = BN / WN;
  constexpr int FM = WTM / 16, FN = WTN / 16;
  constexpr int STAGE = (BM + BN) * 128;
  constexpr int WDMA = BN / 8, XDMA = BM / 8;  // 1 KB DMA instructions of a stage
  constexpr int DPW = (WDMA + XDMA) / NWAVE;
  constexpr int SDMA = WTM / 64;  // DMA instructions of a wavefront's token scales
  static_assert((WDMA + XDMA) % NWAVE == 0 && WTM % 64 == 0 && 128 % WTN == 0, "tiling");
  constexpr int OPS = DPW + SDMA;  // DMA instructions of a wavefront per stage
  constexpr int SX = STAGES * STAGE;                  // token scales: [stage][wavefront][WTM]
  constexpr int SW = SX + STAGES * NWAVE * WTM * 4;   // weight scales: [wn block][KB]
  constexpr int NBT = BN > 128 ? BN / 128 : 1;        // scale blocks across the tile
  extern __shared__ __align__(16) int8_t smem[];

  const int Tt = tilesM * tilesN;
  const int b = xcd_remap(blockIdx.x, Tt);
  const int per_group = groupM * tilesN;
  const int g = b / per_group;
  const int first_m = g * groupM;
  const int gsz = min(tilesM - first_m, groupM);
  const int tm = first_m + (b % per_group) % gsz;
  const int tn = (b % per_group) / gsz;
  const int m0 = tm * BM, n0 = tn * BN;

  const int t = threadIdx.x, lane = t & 63;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wn = w % WN, wm = w / WN;
  const int nrb = N >> 4;
  const int q4 = lane >> 4, r16 = lane & 15;

  // the tile's weight scales (rows past the last 128-feature block repeat it:
  // they only feed outputs that are never stored)
  float* sw = reinterpret_cast<float*>(smem + SW);
  const int nbs = (N + kFp8Block - 1) / kFp8Block;
  for (int i = t; i < NBT * KB; i += NWAVE * 64) {
    const int nb = min(n0 / kFp8Block + i / KB, nbs - 1);
    sw[i] = ws[(size_t)nb * KB + i % KB];
  }
  const float* my_sw = sw + (wn * WTN / 128) * KB;

  // this wavefront's DMA sources: 1 KB pieces J = w*DPW + j of a stage, the
  // weight's first.  Rows past N or M are clamped to the last valid one:
  // they only feed outputs that are never stored.
  uint32_t src[DPW];
  bool isw[DPW];
  const int xrow = lane >> 3;
  const uint32_t chunk = (lane & 7) ^ (xrow & 7);  // the column chunk of this lane's X pieces
#pragma unroll
  for (int j = 0; j < DPW; ++j) {
    const int J = w * DPW + j;
    isw[j] = J < WDMA;
    if (isw[j]) {
      const int rb = min(n0 / 16 + J / 2, nrb - 1);
      src[j] = (uint32_t)rb * (uint32_t)KB * 2048u + (J & 1) * 1024u + lane * 16u;
    } else {
      const int r = (J - WDMA) * 8 + xrow;
      const int row = min(m0 + r, M - 1);
      src[j] = (uint32_t)row * (uint32_t)K + chunk * 16u;
    }
  }
  const uint32_t wbytes = (uint32_t)nrb * (uint32_t)KB * 2048u;
  const uint32_t xbytes = (uint32_t)M * (uint32_t)K;

  // DMAs of K block kb into its stage.  Blocks at or past KB get empty
  // descriptors (zeros).  In a last block that K ends inside, chunks at or
  // past K read from an offset out of every range (zeros).
  auto dma = [&](int kb, int stage) {
    const bool live = kb < KB;
    const uint32_t k0 = live ? (uint32_t)kb : 0u;
    const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(W + (size_t)k0 * 2048), (short)0, live ? (int)(wbytes - k0 * 2048u) : 0, 0x00020000);
    const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(X + (size_t)k0 * 128), (short)0, live ? (int)(xbytes - k0 * 128u) : 0, 0x00020000);
    const bool out = k0 * 128u + chunk * 16u >= (uint32_t)K;
    int8_t* dst = smem + stage * STAGE + w * DPW * 1024;
#pragma unroll
    for (int j = 0; j < DPW; ++j) {
      dma16(isw[j] ? rw : rx, dst + j * 1024, (int)(out && !isw[j] ? kOutOfRange : src[j]), 0);
    }
    // scales of the wavefront's tokens (lanes past M read zeros)
    const int mw = min(m0 + wm * WTM, M - 1);
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(xs + (size_t)k0 * M + mw), (short)0, live ? min(M - mw, WTM) * 4 : 0, 0x00020000);
#pragma unroll
    for (int s = 0; s < SDMA; ++s)
      dma4(rs, smem + SX + ((stage * NWAVE + w) * WTM + s * 64) * 4, lane * 4 + s * 256, 0);
  };

  v4f acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[i][j] = v4f{};

#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) dma(s, s);
  __syncthreads();  // the weight scales (and, conservatively, the first DMAs)

  int stage = 0;
  for (int kb = 0; kb < KB; ++kb) {
    // K block kb landed in every wavefront, and every wavefront is done with
    // the stage of kb - 1, which the next DMA overwrites
    barrier_vm<(STAGES - 2) * OPS>();
    dma(kb + STAGES - 1, stage == 0 ? STAGES - 1 : stage - 1);
    const int8_t* wb = smem + stage * STAGE + (wn * WTN / 16) * 2048 + lane * 16;
    const int8_t* xb = smem + stage * STAGE + BN * 128 + wm * WTM * 128;
    const float* sb = reinterpret_cast<const float*>(smem + SX) + (stage * NWAVE + w) * WTM;
    const float s_w = my_sw[kb];
    v8i fx[FM];
    float s[FM];
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      const int8_t* p = xb + (j * 16 + r16) * 128;
      const v4i lo = *reinterpret_cast<const v4i*>(p + ((q4 ^ (r16 & 7)) * 16));
      const v4i hi = *reinterpret_cast<const v4i*>(p + (((q4 + 4) ^ (r16 & 7)) * 16));
      fx[j] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      s[j] = sb[j * 16 + r16] * s_w;
    }
#pragma unroll
    for (int i = 0; i < FN; ++i) {
      const v4i lo = *reinterpret_cast<const v4i*>(wb + i * 2048);
      const v4i hi = *reinterpret_cast<const v4i*>(wb + i * 2048 + 1024);
      const v8i fw = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
      for (int j = 0; j < FM; ++j) {
        const v4f p = mfma16_e4m3(fw, fx[j]);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(p[e], s[j], acc[i][j][e]);
      }
    }
    stage = stage + 1 == STAGES ? 0 : stage + 1;
  }
  __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));  // no DMA may still write LDS

#pragma unroll
  for (int i = 0; i < FN; ++i) {
    const int n = n0 + wn * WTN + i * 16 + 4 * q4;
    float bv[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (bias && n < N) {
      const uint2 v = *reinterpret_cast<const uint2*>(bias + n);
      bv[0] = to_f32<T>((uint16_t)v.x);
      bv[1] = to_f32<T>((uint16_t)(v.x >> 16));
      bv[2] = to_f32<T>((uint16_t)v.y);
      bv[3] = to_f32<T>((uint16_t)(v.y >> 16));
    }
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      v4f y = acc[i][j];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] += bv[e];
      store4<T>(y, n, m0 + wm * WTM + j * 16 + r16, M, N, Y);
    }
  }
}

template <int T, int BM, int BN, int WM, int WN, int STAGES>
static hipError_t run_gemm(const Fp8Call& c, hipStream_t st) {
  const int KB = (c.K + kFp8Block - 1) / kFp8Block;
  constexpr int NBT = BN > 128 ? BN / 128 : 1;
  constexpr int NWAVE = WM * WN;
  constexpr int SMEM = STAGES * (BM + BN) * 128 + STAGES * NWAVE * (BM / WM) * 4;
  static_assert(SMEM + NBT * kMaxKB * 4 <= 160 * 1024, "LDS budget");
  const int shm = SMEM + (NBT * KB * 4 + 255) / 256 * 256;
  const int tilesM = (c.M + BM - 1) / BM, tilesN = (c.N + BN - 1) / BN;
  auto kern = k_fp8_gemm<T, BM, BN, WM, WN, STAGES>;
  // the dynamic-LDS limit is raised once per device the kernels run on
  static std::atomic<uint64_t> attr_set{0};
  int dev = 0;
  (void)hipGetDevice(&dev);
  const uint64_t bit = 1ull << (dev & 63);
  if (!(attr_set.load(std::memory_order_relaxed) & bit)) {
    const hipError_t e =
        hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize,
                            SMEM + NBT * kMaxKB * 4);
    if (e != hipSuccess) return e;
    attr_set.fetch_or(bit, std::memory_order_relaxed);
  }
  kern<<<tilesM * tilesN, NWAVE * 64, shm, st>>>(c.X, c.xs, c.W, c.ws, c.bias, c.Y, c.M, c.N, c.K,
                                                 KB, tilesM, tilesN, tilesM < 4 ? tilesM : 4);
  return hipGetLastError();
}

template <int T>
static hipError_t run_matmul(const Fp8Call& c, hipStream_t st) {
  return run_gemm<T, 128, 128, 2, 2, 2>(c, st);
}

hipError_t launch_fp8_matmul(const Fp8Call& c, hipStream_t st) {
  return c.type == kF16 ? run_matmul<kF16>(c, st) : run_matmul<kBf16>(c, st);
}

}  // namespace i8mm
