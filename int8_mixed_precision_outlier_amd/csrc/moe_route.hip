// The router of a mixture of experts (gfx950): logits = X . W^T, a softmax over
// the experts, and the top_k largest of each token.
//
// Which expert comes first is a comparison of numbers that may lie as close as
// they like, so it is decided on sums of 64 bits.  For few tokens all sums are:
// the products of two 16-bit numbers are exact in fp32 already.  For more, the
// matrix instructions add 32 products each in fp32, these sums are added in 64
// bits, and a bound of what the fp32 additions may have lost comes with every
// logit; only a token whose chosen experts, or the first one left out, lie closer
// than that has its candidates summed again in 64 bits.  Equal logits (the same
// row of W twice) are summed in the same order and go to the lower index.
#include "fp8.hpp"
#include "launch.hpp"
#include "moe.hpp"

#include <atomic>

namespace i8mm {

namespace {

// ---- few tokens: one wavefront per token and expert, its lanes share the columns

// The sum of x * w in 64 bits over 8 columns from `first` on and again after each
// `step`, in every lane: the lanes' columns in turn, then 6 steps of pairwise
// sums, the same order for every row.
template <int TY>
__device__ __forceinline__ double dot64(const uint16_t* x, const uint16_t* w, int K, int first,
                                        int step) {
  double acc = 0.0;
#pragma unroll 4
  for (int k = first; k < K; k += step) {
    float a[8], b[8];
    unpack8<TY>(*reinterpret_cast<const uint4*>(x + k), a);
    unpack8<TY>(*reinterpret_cast<const uint4*>(w + k), b);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc = fma((double)a[e], (double)b[e], acc);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) acc += __shfl_xor(acc, o, kWave);
  return acc;
}

template <int TY>
__global__ __launch_bounds__(256) void k_moe_logits(const uint16_t* __restrict__ X,
                                                    const uint16_t* __restrict__ W, int64_t first,
                                                    int64_t dots, int K, int E,
                                                    double* __restrict__ L) {
  const int64_t i = first + (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (i >= dots) return;
  const int lane = threadIdx.x & 63;
  const double v = dot64<TY>(X + i / E * K, W + i % E * K, K, lane * 8, 512);
  if (lane == 0) L[i] = v;
}

// ---- more tokens: matrix instructions ---------------------------------------
//
// A workgroup makes 16 tokens x 32 EW experts with KS wavefronts along the columns
// for each 32 experts.  A wavefront takes steps of 64 columns in turn; the rows
// come by DMA into a part of LDS of its own, STAGES steps ahead, so that no
// barrier is needed (a DMA moves 8 rows of 128 bytes, whole cache lines, the
// 16-byte chunks swapped by the row's low bits against bank conflicts).  The
// sums are added at the end, in the wavefronts' order.  Every instruction starts
// from zero, so that its sum of 32 products is rounded only inside it; a second
// one on the operands' magnitudes gives the bound.
// What a sum of 32 products may be off, relative to the sum of their magnitudes:
// each of its additions within 2^-23 of what it has by then, and a quarter more
// for the bound's own rounding (at most K / 32 additions of 2^-23).  Measured against
// 64 bits, a sum of 32 is off by at most 4 * 2^-23 in both types (one large product
// in any place and 31 that the alignment to it cuts short; 1.1 * 2^-23 for random
// and cancelling ones): the tenfold room costs a few more sums made again.
constexpr float kLost = 40.0f * 0x1p-23f;
// Logits closer than this are always compared in 64 bits: the bound does not hold
// for sums below fp32's normal numbers.
constexpr float kTiny = 0x1p-100f;

template <int EW, int KS>
struct Tile {
  static constexpr int WAVES = EW * KS, STAGES = 3;
  static constexpr int STEP = 6 * 1024;  // 16 + 32 rows of 128 bytes
  static constexpr int LDS = WAVES * STAGES * STEP;
};

template <int TY, int EW, int KS>
__global__ __launch_bounds__(EW * KS * 64) void k_moe_logits_tile(
    const uint16_t* __restrict__ X, const uint16_t* __restrict__ W, int M, int K, int E,
    int eblocks, double* __restrict__ L, float* __restrict__ bound) {
  using T = Tile<EW, KS>;
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 63, q4 = lane >> 4, r16 = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m0 = blockIdx.x / eblocks * 16;
  const int e0 = (blockIdx.x % eblocks * EW + w / KS) * 32, kw = w % KS;
  uint8_t* mine = smem + w * T::STAGES * T::STEP;
  const int xrows = min(16, M - m0), wrows = max(0, min(32, E - e0));
  const void* xbase = X + (size_t)m0 * K;
  const void* wbase = W + (size_t)min(e0, E - 1) * K;
  const int drow = lane >> 3;
  const uint32_t chunk = (lane & 7) ^ drow;
  uint32_t src[4];  // rows past the end of either operand are out of its range: zeros
#pragma unroll
  for (int i = 0; i < 4; ++i) src[i] = (uint32_t)(i * 8 + drow) * (uint32_t)K * 2u + chunk * 16u;
  const int steps = (K + 63) / 64;
  constexpr int OPS = 6;
  auto load = [&](int s, int stage) {
    const bool live = s < steps;
    const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
        (void*)xbase, (short)0, live ? (int)((uint32_t)xrows * (uint32_t)K * 2u) : 0, 0x00020000);
    const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
        (void*)wbase, (short)0, live ? (int)((uint32_t)wrows * (uint32_t)K * 2u) : 0, 0x00020000);
    const bool out = s * 64 + (int)chunk * 8 >= K;
    uint8_t* dst = mine + stage * T::STEP;
    const int at = live ? s * 128 : 0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      dma16(rx, dst + i * 1024, (int)(out ? kOutOfRange : src[i] + at), 0);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      dma16(rw, dst + 2048 + i * 1024, (int)(out ? kOutOfRange : src[i] + at), 0);
  };
  double acc[2][4];
  v4f mag[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    mag[j] = v4f{};
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[j][e] = 0.0;
  }
  auto compute = [&](int stage) {
    const uint8_t* from = mine + stage * T::STEP + r16 * 128;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = ((h * 4 + q4) ^ (r16 & 7)) * 16;
      const v4i x = *reinterpret_cast<const v4i*>(from + c);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const v4i v = *reinterpret_cast<const v4i*>(from + 2048 + j * 2048 + c);
        const v4f sum = mfma32<TY>(x, v, v4f{});
        mag[j] = mfma32<TY>(x & 0x7fff7fff, v & 0x7fff7fff, mag[j]);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] += (double)sum[e];
      }
    }
    // read before a DMA overwrites it
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < T::STAGES - 1; ++i) load(kw + i * KS, i);
  for (int s = kw; s < steps; s += T::STAGES * KS)
#pragma unroll
    for (int i = 0; i < T::STAGES; ++i) {  // steps past the end add zeros
      load(s + (i + T::STAGES - 1) * KS, (i + T::STAGES - 1) % T::STAGES);
      wait_vm<OPS*(T::STAGES - 1)>();
      compute(i);
    }
  wait_vm<0>();
  __syncthreads();
  double(*red)[2][4][64] = reinterpret_cast<double(*)[2][4][64]>(smem);
  float(*red_b)[2][4][64] = reinterpret_cast<float(*)[2][4][64]>(smem + sizeof(double) * T::WAVES * 512);
  static_assert(T::WAVES * 512 * 12 <= T::LDS, "the sums fit where the stages were");
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) red[w][j][e][lane] = acc[j][e], red_b[w][j][e][lane] = mag[j][e];
  __syncthreads();
  // the 8 registers of each 32 experts' sums over its KS wavefronts
  for (int o = kw; o < 8; o += KS) {
    const int j = o >> 2, i = o & 3, first = w / KS * KS;
    double v = 0.0;
    float g = 0.0f;
#pragma unroll
    for (int u = 0; u < KS; ++u) v += red[first + u][j][i][lane], g += red_b[first + u][j][i][lane];
    const int m = m0 + q4 * 4 + i, e = e0 + j * 16 + r16;
    if (m < M && e < E) {
      L[(size_t)m * E + e] = v;
      bound[(size_t)m * E + e] = fmaf(g, kLost, kTiny);
    }
  }
}

// ---- softmax and choice -----------------------------------------------------

// The largest of the lanes' numbers, uniform: each row of 16 lanes, then the rows
// behind each other (lane 63 has met all).
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#define I8MM_STEP(ctrl, rows)                                                            \
  {                                                                                      \
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, rows, 0xf, false); \
    v = v > o ? v : o;                                                                   \
  }
  I8MM_STEP(0x111, 0xf)  // row_shr 1, 2, 4, 8
  I8MM_STEP(0x112, 0xf)
  I8MM_STEP(0x114, 0xf)
  I8MM_STEP(0x118, 0xf)
  I8MM_STEP(0x142, 0xa)  // row_bcast 15 into rows 1 and 3
  I8MM_STEP(0x143, 0xc)  // row_bcast 31 into rows 2 and 3
#undef I8MM_STEP
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
  return v;
}

// A number as an integer that orders as it does; a NaN as -inf.  0 is below all.
__device__ __forceinline__ uint64_t order_key(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v == v ? v : -__builtin_inf());
  return b >> 63 ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ double key_value(uint64_t k) {
  return __builtin_bit_cast(double, k >> 63 ? k & ~(1ull << 63) : ~k);
}

// The `count` largest keys of the wavefront in descending order, ties to the lower
// expert (EPL per lane, expert i * 64 + lane): lane j gets the j-th and its expert.
template <int EPL>
__device__ __forceinline__ void choose(const uint64_t (&key)[EPL], int count, int lane,
                                       uint64_t& mine, int& chosen) {
  uint64_t left[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) left[i] = key[i];
  for (int j = 0; j < count; ++j) {
    uint64_t best = left[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) best = left[i] > best ? left[i] : best;
    const uint32_t hi = wave_max((uint32_t)(best >> 32));
    const uint32_t lo = wave_max((uint32_t)(best >> 32) == hi ? (uint32_t)best : 0u);
    const uint64_t top = (uint64_t)hi << 32 | lo;
    int at = -1;
#pragma unroll
    for (int i = EPL - 1; i >= 0; --i) {
      const uint64_t has = __ballot(left[i] == top);
      if (has) at = i * 64 + __builtin_ctzll(has);
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (at == i * 64 + lane) left[i] = 0;
    if (lane == j) mine = top, chosen = at;
  }
}

// One wavefront per token.  With a bound, the workgroup's wavefronts then share
// the columns of what is summed again for those of its four tokens whose order
// the bound leaves open.
template <int TY, int EPL>
__global__ __launch_bounds__(256) void k_moe_topk(RouteCall c) {
  __shared__ uint64_t open[4][EPL];      // a token's experts to sum again, a bit each
  __shared__ double again[4][EPL * 64];  // their sums over each wavefront's columns
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int m = blockIdx.x * 4 + w;
  const int E = c.E;
  const bool live = m < c.M;
  double v[EPL];
  uint64_t key[EPL];
  uint64_t mine = 0;
  int chosen = 0;
  uint32_t worst = 0;  // the largest bound's bits (a NaN's are above every number's)
  if (live) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = i * 64 + lane;
      if (c.bound && e < E) {
        const uint32_t b = __builtin_bit_cast(uint32_t, c.bound[(size_t)m * E + e]);
        worst = b > worst ? b : worst;
      }
      v[i] = e < E ? c.logits[(size_t)m * E + e] : 0.0;
      key[i] = e < E ? order_key(v[i]) : 0;  // below every number's
    }
  }
  if (c.bound) {
    bool close = false;
    if (lane < EPL) open[w][lane] = 0;
    if (live) {
      // one more than are chosen: the first one left out
      const int count = min(c.top_k + 1, E);
      choose(key, count, lane, mine, chosen);
      const double off = 2.0 * (double)__builtin_bit_cast(float, wave_max(worst));
      const double value = key_value(mine);
      const double next = __shfl_down(value, 1, kWave);
      // neighbours whose order is open; not (value - next > off): also where one
      // of them is no number.  A single expert has none, but its sum may have
      // passed fp32's range and would make its weight NaN.
      const bool alone = count == 1 && lane == 0 && !(off < __builtin_inf());
      const uint64_t gaps = __ballot((lane + 1 < count && !(value - next > off)) || alone);
      close = gaps != 0;
      // who has such a neighbour is summed again; the others stay further than
      // `off` from them and from each other
      if ((gaps | gaps << 1) >> lane & 1)
        atomicOr(reinterpret_cast<unsigned long long*>(&open[w][chosen >> 6]), 1ull << (chosen & 63));
      if (gaps >> (c.top_k - 1) & 1) {  // the last place is open: also to those not listed
        const double last = __shfl(value, c.top_k - 1, kWave);
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          const uint64_t set = __ballot(i * 64 + lane < E && !(fabs(v[i] - last) > off));
          if (lane == 0) atomicOr(reinterpret_cast<unsigned long long*>(&open[w][i]), set);
        }
      }
    }
    __syncthreads();
    for (int t = 0; t < 4; ++t) {
      uint64_t any = 0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) any |= open[t][i];
      if (any == 0) continue;  // the same for the whole workgroup
      const uint16_t* row = c.X + (size_t)(blockIdx.x * 4 + t) * c.K;
      for (int i = 0; i < EPL; ++i)
        for (uint64_t set = open[t][i]; set; set &= set - 1) {
          const int e = i * 64 + __builtin_ctzll(set);
          const double d =
              dot64<TY>(row, c.W + (size_t)e * c.K, c.K, (int)threadIdx.x * 8, 256 * 8);
          if (lane == 0) again[w][e] = d;
        }
      __syncthreads();
      if (w == t) {
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (open[t][i] >> lane & 1) {
            const int e = i * 64 + lane;
            v[i] = again[0][e] + again[1][e] + again[2][e] + again[3][e];
            key[i] = order_key(v[i]);
          }
      }
      __syncthreads();
    }
    if (live && close) choose(key, c.top_k, lane, mine, chosen);
  } else if (live) {
    choose(key, c.top_k, lane, mine, chosen);
  }
  if (!live) return;
  // the softmax's differences in 64 bits, its exponentials and sum in fp32
  const double top = __shfl(key_value(mine), 0, kWave);
  float total = 0.0f;
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    if (i * 64 + lane < E) total += expf((float)(v[i] - top));
  total = wave_sum(total);
  float p = 0.0f;
  if (lane < c.top_k) p = expf((float)(key_value(mine) - top)) / total;
  const float sum = wave_sum(p);
  if (lane < c.top_k) {
    c.experts[(size_t)m * c.top_k + lane] = chosen;
    c.weights[(size_t)m * c.top_k + lane] = c.normalize ? p / sum : p;
  }
}

template <int TY>
hipError_t route(const RouteCall& call, hipStream_t st) {
  RouteCall c = call;
  const int64_t dots = (int64_t)c.M * c.E;
  if (!route_by_tiles(c.M, c.K, c.E)) {
    c.bound = nullptr;
    // a launch holds fewer than 2^32 threads; rows without columns can be 2^28 sums
    constexpr int64_t kPerLaunch = 1 << 24;
    for (int64_t i = 0; i < dots; i += kPerLaunch) {
      const int64_t n = dots - i < kPerLaunch ? dots - i : kPerLaunch;
      k_moe_logits<TY><<<(unsigned)((n + 3) / 4), 256, 0, st>>>(c.X, c.W, i, dots, c.K, c.E,
                                                                c.logits);
    }
  } else {
    auto go = [&](auto kern, int ew, size_t lds, std::atomic<uint64_t>& asked) {
      int dev = 0;
      (void)hipGetDevice(&dev);
      const uint64_t bit = 1ull << (dev & 63);
      if (!(asked.load(std::memory_order_relaxed) & bit)) {
        const hipError_t r = hipFuncSetAttribute(
            (const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (r != hipSuccess) return r;
        asked.fetch_or(bit, std::memory_order_relaxed);
      }
      const int eblocks = (c.E + 32 * ew - 1) / (32 * ew);
      kern<<<(c.M + 15) / 16 * eblocks, 512, lds, st>>>(c.X, c.W, c.M, c.K, c.E, eblocks, c.logits,
                                                        c.bound);
      return hipGetLastError();
    };
    static std::atomic<uint64_t> asked[2];
    // 32 experts a workgroup while that is at most two rounds of the chip (one
    // fits a CU), else 128, which share the tokens' rows in L1 (us, calls in a
    // graph with the choice, 32 and 128 at a time: 128x4096 of 128 17.8 and 27.9,
    // 2048x4096 of 128 31.5 and 33.4, 4096x4096 of 96 40.4 and 35.6, 4096x5120 of
    // 128 58.8 and 46.3)
    const int64_t tiles = (int64_t)((c.M + 15) / 16) * ((c.E + 31) / 32);
    const hipError_t e = tiles <= 2 * device_cu_count()
                             ? go(k_moe_logits_tile<TY, 1, 8>, 1, Tile<1, 8>::LDS, asked[0])
                             : go(k_moe_logits_tile<TY, 4, 2>, 4, Tile<4, 2>::LDS, asked[1]);
    if (e != hipSuccess) return e;
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int epl = (c.E + 63) / 64;
  auto kern = epl <= 1   ? k_moe_topk<TY, 1>
              : epl <= 2 ? k_moe_topk<TY, 2>
              : epl <= 4 ? k_moe_topk<TY, 4>
                         : k_moe_topk<TY, 16>;
  kern<<<(c.M + 3) / 4, 256, 0, st>>>(c);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_route(const RouteCall& c, hipStream_t st) {
  return c.type == kF16 ? route<kF16>(c, st) : route<kBf16>(c, st);
}

}  // namespace i8mm
