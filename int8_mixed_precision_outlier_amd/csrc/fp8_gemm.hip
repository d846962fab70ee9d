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
#include "launch.hpp"

#include <atomic>
#include <utility>

namespace i8mm {

namespace {

constexpr int kMaxKB = 65536 / kFp8Block;

// LDS of a tile: S stages of one K block each (W's half blocks, then X's
// rows), the token scales [stage][wavefront][its tokens] (PW > 0: [stage][the
// tile's tokens]), the tile's weight scales [128-feature block][KB + S], and its bias in fp32.
template <int BM, int BN, int WM, int WN, int S, int PW>
struct GemmLds {
  static constexpr int STAGE = (BM + BN) * 128;
  static constexpr int SX = S * STAGE;
  static constexpr int SB = SX + S * (PW > 0 ? 1 : WN) * BM * 4;
  static constexpr int SW = SB + BN * 4;
  static constexpr int NBT = BN > 128 ? BN / 128 : 1;
  static constexpr int MAX = SW + NBT * (kMaxKB + S) * 4;
  static_assert(MAX <= 160 * 1024, "LDS budget");
};

// Order of one feature block's instructions: each of its MFMAs followed by
// four fmas, then LDS reads (R0 after the first, R1 after each of the others)
// and an even share of V DMAs.
constexpr int kSgMfma = 0x008, kSgValu = 0x002, kSgDsRead = 0x100, kSgVmemRead = 0x020;
template <int R0, int R1, int V, int... Js>
__device__ __forceinline__ void order_impl(std::integer_sequence<int, Js...>) {
  constexpr int FM = sizeof...(Js);
  ((__builtin_amdgcn_sched_group_barrier(kSgMfma, 1, 0),
    __builtin_amdgcn_sched_group_barrier(kSgValu, 4, 0),
    __builtin_amdgcn_sched_group_barrier(kSgDsRead, Js == 0 ? R0 : R1, 0),
    __builtin_amdgcn_sched_group_barrier(kSgVmemRead, (Js + 1) * V / FM - Js * V / FM, 0)),
   ...);
  __builtin_amdgcn_sched_barrier(0);
}
template <int FM, int R0, int R1, int V>
__device__ __forceinline__ void order() {
  order_impl<R0, R1, V>(std::make_integer_sequence<int, FM>{});
}

template <class F, int... Is>
__device__ __forceinline__ void unroll(F&& f, std::integer_sequence<int, Is...>) {
  (f(std::integral_constant<int, Is>{}), ...);
}

// Two 16x16 blocks of adjacent features (nb .. nb+15 in ya, nb+16 .. +31 in
// yb) of the same 16 tokens as one 16-byte store per lane: swapping rows 1
// and 3 of the first with rows 0 and 2 of the second leaves 8 consecutive
// features of a token in each lane.  N % 16 == 0, so they are all in range or
// all out.
template <int T>
__device__ __forceinline__ void store32(const v4f& ya, const v4f& yb, int nb, int mb, int M, int N,
                                        uint16_t* __restrict__ Y) {
  const int lane = threadIdx.x & 63, q = lane >> 4;
  const auto lo = __builtin_amdgcn_permlane16_swap(pack16x2<T>(ya[0], ya[1]),
                                                   pack16x2<T>(yb[0], yb[1]), false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap(pack16x2<T>(ya[2], ya[3]),
                                                   pack16x2<T>(yb[2], yb[3]), false, false);
  const int m = mb + (lane & 15), n = nb + 8 * (q >> 1) + 16 * (q & 1);
  if (m < M && n < N)
    *reinterpret_cast<uint4*>(Y + (size_t)m * N + n) = make_uint4(lo[0], hi[0], lo[1], hi[1]);
}

}  // namespace

template <int T, int BM, int BN, int WM, int WN, int S, int PW>
__global__ __launch_bounds__((WM * WN + PW) * 64, 2) void k_fp8_gemm(
    const uint8_t* __restrict__ X, const float* __restrict__ xs, const uint8_t* __restrict__ W,
    const float* __restrict__ ws, const uint16_t* __restrict__ bias, uint16_t* __restrict__ Y,
    int M, int N, int K, int KB, int tilesM, int tilesN, int groupM, int nbase) {
  using L = GemmLds<BM, BN, WM, WN, S, PW>;
  constexpr int NWAVE = WM * WN;
  constexpr int WTM = BM / WM, WTN = BN / WN;
  constexpr int FM = WTM / 16, FN = WTN / 16;
  // PW > 0: the last PW wavefronts only issue the DMAs, the others compute.  A
  // wavefront that issues waits for the address unit, 16 cycles per DMA; where
  // one wavefront per SIMD computes, nothing else would use that time
  // (256x5120x5120 on 64x128 tiles: 18.4 us with the DMAs in the computing
  // wavefronts, 15.8 with four more, both with three stages; 128x128 tiles, in
  // eight computing ones / in four more beside four, calls in a graph:
  // 1024x4096x4096 22.8 / 21.0, 512x5120x5120 23.3 / 21.4, 512x5120x8192 28.1 / 25.0).
  constexpr int DW = PW > 0 ? PW : NWAVE;  // wavefronts that share the DMAs
  // 1 KB DMAs of a wavefront per K block: of X, of either half of W, and of
  // its token scales
  constexpr int XDMA = BM / 8 / DW, HDMA = BN / 16 / DW, SDMA = PW > 0 ? 1 : WTM / 64;
  static_assert(BN / 16 % DW == 0 && BM / 8 % DW == 0 && WTM % 64 == 0, "DMA split");
  constexpr int SROW = PW > 0 ? BM : NWAVE * WTM;  // token scales of a stage
  static_assert(128 % WTN == 0 && FN % 2 == 0 && FM >= 4, "a wavefront's features share a scale block");
  extern __shared__ __align__(16) int8_t smem[];

  const int Tt = tilesM * tilesN;
  const int b = xcd_remap(blockIdx.x, Tt);
  const int per_group = groupM * tilesN;
  const int g = b / per_group;
  const int first_m = g * groupM;
  const int gsz = min(tilesM - first_m, groupM);
  const int tm = first_m + (b % per_group) % gsz;
  const int tn = (b % per_group) / gsz;
  // the launch covers the features from nbase on, tilesN tiles of BN
  const int m0 = tm * BM, n0 = nbase + tn * BN;

  const int t = threadIdx.x, lane = t & 63;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wn = w % WN, wm = w / WN;
  const int dw = PW > 0 ? max(w - NWAVE, 0) : w;
  const int nrb = N >> 4;
  const int q4 = lane >> 4, r16 = lane & 15;

  // the tile's weight scales (blocks past the last 128 features repeat it:
  // they only feed outputs that are never stored) and its bias; the loads of
  // the first round are in flight under the first DMAs
  float* sw = reinterpret_cast<float*>(smem + L::SW);
  float* sb = reinterpret_cast<float*>(smem + L::SB);
  const int nbs = (N + kFp8Block - 1) / kFp8Block;
  const int KS = KB + S;  // zeros behind each block's scales
  auto weight_scale = [&](int i) {
    const int nb = min(n0 / kFp8Block + i / KS, nbs - 1), kb = i % KS;
    return kb < KB ? ws[(size_t)nb * KB + kb] : 0.0f;
  };
  const float sw_first = t < L::NBT * KS ? weight_scale(t) : 0.0f;
  const uint16_t bias_first = bias && t < BN && n0 + t < N ? bias[n0 + t] : (uint16_t)0;
  static_assert(BN <= NWAVE * 64, "one bias value per thread");
  const float* my_sw = sw + (wn * WTN / 128) * KS;

  // DMA sources of this wavefront: XDMA pieces of 8 rows of X, and HDMA half
  // blocks of either half of W, the first and the second FN / 2 feature
  // blocks of every wavefront.  Rows past N or M are clamped to the last
  // valid one: they only feed outputs that are never stored.
  const int xrow = lane >> 3;
  const uint32_t chunk = (lane & 7) ^ xrow;  // the column chunk of this lane's X pieces
  uint32_t xsrc[XDMA], wsrc[2][HDMA];
  int wdst[2][HDMA];
#pragma unroll
  for (int j = 0; j < XDMA; ++j) {
    const int row = min(m0 + (dw * XDMA + j) * 8 + xrow, M - 1);
    xsrc[j] = (uint32_t)row * (uint32_t)K + chunk * 16u;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < HDMA; ++j) {
      const int q = dw * HDMA + j;  // half block q % 2 of the half's feature block q / 2
      const int a = q / 2, fb = a / (FN / 2) * FN + a % (FN / 2) + h * (FN / 2);
      const int rb = min(n0 / 16 + fb, nrb - 1);
      wsrc[h][j] = __builtin_amdgcn_readfirstlane((uint32_t)rb * (uint32_t)KB * 2048u + (q & 1) * 1024u);
      wdst[h][j] = __builtin_amdgcn_readfirstlane(fb * 2048 + (q & 1) * 1024);
    }
  // the tokens whose scales it loads, and their place in a stage: its own, or
  // 64 of the tile's (some twice, where PW * 64 exceeds them)
  constexpr int STOK = SDMA * 64;
  const int stok = PW > 0 ? dw % (BM / 64) * 64 : wm * WTM;
  const int sdst = PW > 0 ? stok : w * WTM;
  const int mw = min(m0 + stok, M - 1);
  const uint32_t wbytes = (uint32_t)nrb * (uint32_t)KB * 2048u;
  const uint32_t xbytes = (uint32_t)M * (uint32_t)K;

  // This wavefront's DMAs of K block kb: `a` takes X, the token scales and
  // the first half of W, `b` the second half.  Blocks at or past KB get
  // empty descriptors (zeros), so the loop needs no branch and every
  // wavefront counts the same number of DMAs.  In a last block that K ends
  // inside, chunks at or past K read from an offset out of every range
  // (zeros); tokens past M read zero scales.
  constexpr int OPA = XDMA + SDMA + HDMA, OPB = HDMA, OPS = OPA + OPB;
  constexpr int AHEAD = (S - 1) * OPS;  // DMAs that may be in flight at a barrier
  auto dma_w = [&](int kb, int stage, int h, int j) {
    const bool live = kb < KB;
    const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
        (void*)W, (short)0, live ? (int)wbytes : 0, 0x00020000);
    dma16(rw, smem + stage * L::STAGE + wdst[h][j], lane * 16,
          (int)(wsrc[h][j] + (uint32_t)(live ? kb : 0) * 2048u));
  };
  auto dma_b = [&](int kb, int stage, int d0, int d1) {
#pragma unroll
    for (int d = d0; d < d1; ++d) dma_w(kb, stage, 1, d);
  };
  auto dma_a = [&](int kb, int stage, int d0, int d1) {
    const bool live = kb < KB;
    const int k = live ? kb : 0;
    const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
        (void*)X, (short)0, live ? (int)xbytes : 0, 0x00020000);
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(xs + (size_t)k * M + mw), (short)0, live ? min(M - mw, STOK) * 4 : 0, 0x00020000);
    const bool out = (uint32_t)k * 128u + chunk * 16u >= (uint32_t)K;
#pragma unroll
    for (int d = d0; d < d1; ++d) {
      if (d < XDMA) {
        dma16(rx, smem + stage * L::STAGE + BN * 128 + (dw * XDMA + d) * 1024,
              (int)(out ? kOutOfRange : xsrc[d]), k * 128);
      } else if (d < XDMA + HDMA) {
        dma_w(kb, stage, 0, d - XDMA);
      } else {
        const int j = d - XDMA - HDMA;
        dma4(rs, smem + L::SX + (stage * SROW + sdst + j * 64) * 4, lane * 4 + j * 256, 0);
      }
    }
  };

  auto dma_one = [&](int kb, int stage, int d) {
    if (d < OPA) dma_a(kb, stage, d, d + 1);
    else dma_b(kb, stage, d - OPA, d - OPA + 1);
  };

  constexpr bool DB = S > 2;  // two K blocks' fragments in registers
  static_assert(DB ? FN <= 4 : FN % 4 == 0 && PW == 0, "registers; whole halves of W");
  v4f acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[i][j] = v4f{};

  // The last four partial products, each scaled in kLag MFMAs after its own.
  constexpr int kLag = 3;
  v4f p[4] = {};
  float s[FM] = {};
  auto scale_in = [&](int o) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      acc[o / FM][o % FM][e] = fmaf(p[o & 3][e], s[o % FM], acc[o / FM][o % FM][e]);
  };
  // MFMA number n of a K block, and the scaling of the one kLag before it;
  // sx, s_w: the K block's scales, which count from its product 0 on
  auto mma = [&](int n, const v8i& fw, const v8i& fx, const float(&sx)[FM], float s_w) {
    p[n & 3] = mfma16_e4m3(fw, fx);
    if (n == kLag) {  // the previous block's products are all in
#pragma unroll
      for (int q = 0; q < FM; ++q) s[q] = sx[q] * s_w;
    }
    scale_in((n + FN * FM - kLag) % (FN * FM));
  };
  // LDS offsets of the lane's fragments within a stage, and its reads
  const int wo = (wn * WTN / 16) * 2048 + lane * 16;
  const int xo = BN * 128 + (wm * WTM + r16) * 128;
  const int xlo = xo + (q4 ^ (r16 & 7)) * 16, xhi = xo + ((q4 + 4) ^ (r16 & 7)) * 16;
  auto join = [](const v4i& lo, const v4i& hi) {
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  auto read_w = [&](int at, int i) {
    const int8_t* q = smem + at + i * 2048;
    return join(*reinterpret_cast<const v4i*>(q), *reinterpret_cast<const v4i*>(q + 1024));
  };
  auto read_x = [&](int lo, int hi, int j) {
    return join(*reinterpret_cast<const v4i*>(smem + lo + j * 2048),
                *reinterpret_cast<const v4i*>(smem + hi + j * 2048));
  };
  const float* sbase =
      reinterpret_cast<const float*>(smem + L::SX) + (PW > 0 ? wm : w) * WTM + r16;
  auto read_s = [&](int stage, int kb, float(&sx)[FM], float& s_w) {
#pragma unroll
    for (int j = 0; j < FM; ++j) sx[j] = sbase[stage * SROW + j * 16];
    s_w = my_sw[kb];
  };

  const bool issues = PW == 0 || w >= NWAVE;
  if (KB > 0 && issues) {
#pragma unroll
    for (int k = 0; k < S; ++k) {
      dma_a(k, k, 0, OPA);
      if (DB || k < S - 1) dma_b(k, k, 0, OPB);
    }
  }
  if (t < BN) sb[t] = to_f32<T>(bias_first);
  if (KB > 0)
    for (int i = t; i < L::NBT * KS; i += (NWAVE + PW) * 64) sw[i] = i == t ? sw_first : weight_scale(i);

  if constexpr (DB) {
    // 256x128 and four-stage 128x128 tiles (64 tokens x 64 features per
    // wavefront) and 64x128 tiles (64 x 32): the registers hold all fragments
    // of two K blocks.  The next block's are read under the current one's
    // MFMAs, which so never wait for LDS, and a K block needs one barrier: its
    // stage is free as soon as the fragments are in registers.  Its DMAs run
    // S - 1 blocks ahead.
    v8i fw[2][FN], fx[2][FM];
    float sx[2][FM], s_w[2];
    auto read = [&](int stage, int f, v8i(&gw)[FN], v8i(&gx)[FM]) {  // in the order of use
      const int base = stage * L::STAGE;
      if (f == 0) gw[0] = read_w(base + wo, 0);
      else if (f <= FM) gx[f - 1] = read_x(base + xlo, base + xhi, f - 1);
      else gw[f - FM] = read_w(base + wo, f - FM);
    };
    if (PW > 0 && w >= NWAVE) {
      // a wavefront that only issues: the same barriers as the others
      if (KB > 0) {
        barrier_vm<(S - 1) * OPS>();
        barrier_vm<(S - 2) * OPS>();
        int st = 0;
        for (int kb = 0; kb < (KB + 1) / 2 * 2; ++kb) {
          dma_a(kb + S, st, 0, OPA);
          dma_b(kb + S, st, 0, OPB);
          barrier_vm<(S - 2) * OPS>();
          st = st + 1 == S ? 0 : st + 1;
        }
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));  // no DMA may still write LDS
      } else {
        __syncthreads();  // the bias
      }
      return;
    }
    if (KB > 0) {
      barrier_vm<(S - 1) * OPS>();  // the weight scales, and K block 0
#pragma unroll
      for (int f = 0; f < FM + FN; ++f) read(0, f, fw[0], fx[0]);
      read_s(0, 0, sx[0], s_w[0]);
      barrier_vm<(S - 2) * OPS>();  // stage 0 is free, K block 1 has landed
    }
    int st = 0;
    auto step = [&](auto P, int kb) {
      constexpr int c = decltype(P)::value;  // the parity of kb
      const int sn = st + 1 == S ? 0 : st + 1;
      auto block = [&](auto I) {
        constexpr int i = decltype(I)::value;
        constexpr int d0 = i * OPS / FN, d1 = (i + 1) * OPS / FN;
        constexpr int R = (FM + FN) / FN;  // fragments read under a feature block
#pragma unroll
        for (int j = 0; j < FM; ++j) {
          mma(i * FM + j, fw[c][i], fx[c][j], sx[c], s_w[c]);
          if (j < R) read(sn, i * R + j, fw[c ^ 1], fx[c ^ 1]);
        }
        if constexpr (i == FN - 1) read_s(sn, kb + 1, sx[c ^ 1], s_w[c ^ 1]);
        if constexpr (PW == 0) {
#pragma unroll
          for (int d = d0; d < d1; ++d) dma_one(kb + S, st, d);
        }
        order<FM, 2, (R > 2 ? 2 : 1), (PW == 0 ? d1 - d0 : 0)>();
      };
      unroll(block, std::make_integer_sequence<int, FN>{});
      // every wavefront holds K block kb + 1, whose stage may be overwritten,
      // and its DMAs of kb + 2 have landed (since then issued: those of the
      // S - 2 blocks kb + 3 .. kb + S)
      barrier_vm<(S - 2) * OPS>();
      __builtin_amdgcn_sched_barrier(0);
      st = sn;
    };
    for (int kb = 0; kb < KB; kb += 2) {  // behind an odd KB a block of zeros
      step(std::integral_constant<int, 0>{}, kb);
      step(std::integral_constant<int, 1>{}, kb + 1);
    }
  } else {
    // The two tiles with two stages, 256x256 (64 tokens x 128 features per
    // wavefront) and 128x128 above one per CU (64 x 64; two workgroups share a
    // CU): the registers hold two weight fragments (the next feature block's
    // loaded under the current one's MFMAs) and the tokens' FM fragments.  X and the two halves of W leave their stages separately,
    // at two barriers per K block, so that their DMAs run S - 0.5 blocks ahead
    // in S stages (one barrier and S - 1.15 blocks: 4096x12288x49152 2066 us
    // against 1967).
    v8i fw[2], fx[FM];
    float sx[FM], s_w = 0.0f;
    // the stages' offsets; the empty asm hides that one is another plus a
    // constant: as immediate offsets of the reads the constants do not fit,
    // and would be added anew in front of each
    int wst[S], lst[S], hst[S];
#pragma unroll
    for (int st = 0; st < S; ++st) {
      wst[st] = st * L::STAGE + wo;
      lst[st] = st * L::STAGE + xlo;
      hst[st] = st * L::STAGE + xhi;
      asm volatile("" : "+v"(wst[st]), "+v"(lst[st]), "+v"(hst[st]));
    }
    if (KB > 0) {
      barrier_vm<AHEAD>();  // the weight scales, and the first DMAs of block 0
      read_s(0, 0, sx, s_w);
#pragma unroll
      for (int j = 0; j < FM; ++j) fx[j] = read_x(lst[0], hst[0], j);
      fw[0] = read_w(wst[0], 0);
    }
    auto step = [&](auto ST, int kb) {
      constexpr int st = decltype(ST)::value, sn = (st + 1) % S;
      auto upto = [&](auto I) {
        constexpr int i = decltype(I)::value;
        constexpr int A = FN / 2 - 1;  // first feature block after the first barrier
        // the DMAs a barrier has made room for, spread over the feature blocks
        // up to the other barrier: a burst fills the address unit's queue and
        // holds up the MFMAs behind it
        constexpr int a0 = i < A ? 0 : (i - A) * OPA / (FN - 1 - A);
        constexpr int a1 = i < A ? 0 : (i + 1 - A) * OPA / (FN - 1 - A);
        constexpr int b0 = i < A ? i * OPB / A : 0, b1 = i < A ? (i + 1) * OPB / A : 0;
        static_assert(A > 0, "");
#pragma unroll
        for (int j = 0; j < FM; ++j) {
          mma(i * FM + j, fw[i & 1], fx[j], sx, s_w);
          if (j == 0) fw[(i + 1) & 1] = read_w(wst[st], i + 1);
        }
        dma_a(kb + S, st, a0, a1);
        dma_b(kb + S - 1, (st + S - 1) % S, b0, b1);
        order<FM, 2, 0, a1 - a0 + b1 - b0>();
        if constexpr (i == A - 1) {
          // every wavefront has read X and the first half of W of this K block,
          // and its DMAs of the second half have landed (issued S - 0.5 K blocks
          // ago; since then the A and B parts of kb + 1 .. kb + S - 1)
          barrier_vm<AHEAD>();
          __builtin_amdgcn_sched_barrier(0);
        }
      };
      unroll(upto, std::make_integer_sequence<int, FN - 1>{});
      // every wavefront has read the second half of W, and its DMAs of the next
      // K block's X and first half of W have landed (since then issued: the B
      // parts of kb + 1 .. kb + S - 1 and the A parts of kb + 2 .. kb + S)
      barrier_vm<AHEAD>();
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < FM; ++j) {
        mma((FN - 1) * FM + j, fw[(FN - 1) & 1], fx[j], sx, s_w);
        if (j == 0) fw[0] = read_w(wst[sn], 0);
        fx[j] = read_x(lst[sn], hst[sn], j);
      }
      read_s(sn, kb + 1, sx, s_w);
      order<FM, 4, 3, 0>();
    };
    // S K blocks per iteration, so that the stage is a constant in each; behind
    // the last come blocks of zero operands and zero scales
    for (int kb = 0; kb < KB; kb += S)
      unroll([&](auto ST) { step(ST, kb + decltype(ST)::value); },
             std::make_integer_sequence<int, S>{});
  }
  __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));  // no DMA may still write LDS
  if (KB == 0) __syncthreads();              // the bias
#pragma unroll
  for (int o = FN * FM - kLag; o < FN * FM; ++o) scale_in(o);

  // two feature blocks at a time: each token's 64 bytes leave in one store
#pragma unroll
  for (int i = 0; i < FN; i += 2) {
    const int nl = wn * WTN + i * 16;
    const v4f ba = *reinterpret_cast<const v4f*>(sb + nl + 4 * q4);
    const v4f bb = *reinterpret_cast<const v4f*>(sb + nl + 16 + 4 * q4);
#pragma unroll
    for (int j = 0; j < FM; ++j)
      store32<T>(acc[i][j] + ba, acc[i + 1][j] + bb, n0 + nl, m0 + wm * WTM + j * 16, M, N, Y);
  }
}

// One launch over the features [nbase, nend); nend is N, or a multiple of BN
// above nbase.
template <int T, int BM, int BN, int WM, int WN, int S, int PW = 0>
static hipError_t run_gemm(const Fp8Call& c, int nbase, int nend, hipStream_t st) {
  using L = GemmLds<BM, BN, WM, WN, S, PW>;
  const int KB = (c.K + kFp8Block - 1) / kFp8Block;
  const int shm = L::SW + L::NBT * (KB + S) * 4;
  const int tilesM = (c.M + BM - 1) / BM, tilesN = (nend - nbase + BN - 1) / BN;
  auto kern = k_fp8_gemm<T, BM, BN, WM, WN, S, PW>;
  // the dynamic-LDS limit is raised once per device the kernels run on
  static std::atomic<uint64_t> attr_set{0};
  int dev = 0;
  (void)hipGetDevice(&dev);
  const uint64_t bit = 1ull << (dev & 63);
  if (!(attr_set.load(std::memory_order_relaxed) & bit)) {
    const hipError_t e = hipFuncSetAttribute((const void*)kern,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, L::MAX);
    if (e != hipSuccess) return e;
    attr_set.fetch_or(bit, std::memory_order_relaxed);
  }
  // groups of 4 token tiles: the 32 tiles an XCD runs at once share 4 token
  // and 8 feature panels in its L2 (4096x12288x49152: 1963 us; 2 tiles 2035,
  // 8 tiles 1975, 16 tiles 2040)
  kern<<<tilesM * tilesN, (WM * WN + PW) * 64, shm, st>>>(
      c.X, c.xs, c.W, c.ws, c.bias, c.Y, c.M, c.N, c.K, KB, tilesM, tilesN,
      tilesM < 4 ? tilesM : 4, nbase);
  return hipGetLastError();
}

template <int T>
static hipError_t run_tiles(int cfg, const Fp8Call& c, int nbase, int nend, hipStream_t st) {
  switch (cfg) {
    case kTile64x128: return run_gemm<T, 64, 128, 1, 4, 4, 4>(c, nbase, nend, st);
    case kTile128Deep: return run_gemm<T, 128, 128, 2, 2, 4, 4>(c, nbase, nend, st);
    case kTile128: return run_gemm<T, 128, 128, 2, 2, 2>(c, nbase, nend, st);
    case kTile256x128: return run_gemm<T, 256, 128, 4, 2, 3>(c, nbase, nend, st);
    default: return run_gemm<T, 256, 256, 4, 2, 2>(c, nbase, nend, st);
  }
}

// Kernel and tile configuration.  The cost of a launch is counted in rounds
// of workgroups over the chip, in units of a round of 256x256 tiles (8
// wavefronts of 64 tokens x 128 features, one workgroup per CU: 57-66 us at K
// = 5120), fitted at K = 4096 and 5120 (us; 256x256 / 256x128 / 128x128):
//   256x128  0.70 per round (one workgroup per CU; 2048x4096x4096: 46.4 /
//            35.9 / 37.2);
//   128x128  0.74 per round of two workgroups per CU (512x5120x20480: 62.0 /
//            80.1 / 74.4); a last round of at most one per CU takes 0.40, in
//            the form with four stages (512x5120x5120: 52.9 / 34.5 / 20.7, with
//            two stages 26.2; 256x12288x12288: 134.9 / 91.4 / 64.3);
//   64x128   0.28 on at most 5/8 of the CUs (256x5120x5120: 14.7 us against
//            20.3 of 128x128; 15.8 with three stages), 0.305 on more
//            (192x5120x10240: 16.0 against 22.2; 256x12288x8192: 46.7 against
//            59.6), with two per CU it loses (512x5120x5120: 28.8 against 21.5);
//   decode   0.031 per block of 16 features or tokens that the most loaded CU
//            reads per K block (77x5136x20464: 30.7 us against 33.2 on 128x128
//            tiles; with weights that no cache holds, decode / 64x128 tiles:
//            104x5120x8192 17.8 / 19.4, 120x5120x5120 22.1 / 20.4, 96x5120x12288
//            20.1 / 20.7, 120x5120x16384 27.3 / 23.6, but 120x12288x12288 45.2 /
//            48.9; with weights in the last-level cache 104x5120x12288 22.9 /
//            15.1; 128x12288x49152: 161 against 144 on 128x128 tiles).
// Up to 64 tokens the decode kernel runs whatever the costs.  Fitted above
// that, they would put tiles in its place where one per CU just fills the chip
// (64x128 tiles near 32768 features, 128x128 near 65536).  With weights that no
// cache holds (decode / tiles, us) that loses up to 32 tokens: 1x12288x28672
// 52.8 / 61.4, 8x5120x20480 19.1 / 20.9, 16x8192x28672 40.0 / 42.4, 32x12288x32768
// 65.7 / 71.5, 4x5120x51200 42.8 / 52.5 (32x5120x25600 25.9 / 25.3); towards 64
// it would gain at most of these sizes: 64x5120x26000 32.0 / 27.9, 56x5120x28672
// 32.4 / 28.7, 64x12288x28672 68.4 / 67.3, 64x4096x32768 29.3 / 27.7, 64x5120x51200
// 64.3 / 57.1, 64x12288x57344 143.2 / 136.9, but 64x5120x24576 26.3 / 27.4,
// 40x5120x51200 53.2 / 54.9.
// When 256x256 tiles would leave the last round partly empty, the features
// can be split: [0, n1) in whole rounds of 256x256 tiles, [n1, N) in a second
// launch of smaller tiles (kGap for its fill and drain, taken when it saves
// more than kMargin).
constexpr double kF128 = 0.74, kF128Deep = 0.40, kF64 = 0.28, kF64More = 0.305,
                 kF256x128 = 0.70, kFDecode = 0.031, kGap = 0.04, kMargin = 0.05;

// The cheapest single launch over n features; ties keep the larger tile.
static int cheapest_tile(long M, long n, long cus, double* cost) {
  const long tm = (M + 255) / 256, t128 = (M + 127) / 128 * ((n + 127) / 128);
  int best = kTile256;
  *cost = (double)((tm * ((n + 255) / 256) + cus - 1) / cus);
  const double c1 = kF256x128 * (double)((tm * ((n + 127) / 128) + cus - 1) / cus);
  if (c1 < *cost) {
    best = kTile256x128;
    *cost = c1;
  }
  const long last = t128 % (2 * cus);
  const double c2 = kF128 * (double)(t128 / (2 * cus)) +
                    (last == 0 ? 0.0 : last <= cus ? kF128Deep : kF128);
  if (c2 < *cost) {
    best = t128 <= cus ? kTile128Deep : kTile128;
    *cost = c2;
  }
  const long t64 = (M + 63) / 64 * ((n + 127) / 128);
  const double c3 = 8 * t64 <= 5 * cus ? kF64 : kF64More;
  if (t64 <= cus && c3 < *cost) {
    best = kTile64x128;
    *cost = c3;
  }
  return best;
}

Fp8Plan fp8_plan(int M, int N) {
  const long cus = device_cu_count();
  double cbest;
  Fp8Plan best{cheapest_tile(M, N, cus, &cbest), N, 0};
  if (M <= kFp8DecodeMaxM && (M <= 64 || kFDecode * (double)fp8_decode_plan(M, N).cost < cbest))
    return Fp8Plan{kDecode, N, 0};
  const long tm = (M + 255) / 256, t256 = tm * ((N + 255) / 256);
  for (long R = 1; R * cus < t256; ++R) {
    const long n1 = R * cus / tm * 256;
    if (n1 <= 0 || n1 >= N) continue;
    double rest;
    const int second = cheapest_tile(M, N - n1, cus, &rest);
    const double c = (double)((tm * (n1 / 256) + cus - 1) / cus) + kGap + rest;
    if (second != kTile256 && c < cbest - kMargin) {
      best = Fp8Plan{kTile256, (int)n1, second};
      cbest = c;
    }
  }
  return best;
}

template <int T>
static hipError_t run_matmul(const Fp8Call& c, hipStream_t st) {
  const Fp8Plan p = fp8_plan(c.M, c.N);
  if (p.first == kDecode) return launch_fp8_decode(c, st);
  const hipError_t e = run_tiles<T>(p.first, c, 0, p.n1, st);
  if (e != hipSuccess || p.n1 >= c.N) return e;
  return run_tiles<T>(p.second, c, p.n1, c.N, st);
}

hipError_t launch_fp8_matmul(const Fp8Call& c, hipStream_t st) {
  return c.type == kF16 ? run_matmul<kF16>(c, st) : run_matmul<kBf16>(c, st);
}

}  // namespace i8mm
