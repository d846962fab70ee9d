// A mixture of experts' gated feed-forward for few tokens (gfx950), from
// block-scaled e4m3 weights and 16-bit activations:
//   a[p]  = silu(x . G_e^T) * (x . U_e^T)     for each pair p of a token and its expert e
//   y[m]  = sum over the token's pairs of weight[p] * (a[p] . D_e^T)
//
// Few tokens are bound by the stream of the chosen experts' weights, so each
// chosen expert is read once for all its tokens, and the activations stay in 16
// bits: quantizing them would not shorten the stream.  The e4m3 numbers become
// fp16 or bf16 in registers (exactly) and meet the tokens in 16x16x32 matrix
// instructions; the sum of a 128-column block is scaled once in fp32 (see
// split_scale).  The gated product between the two kernels keeps 16 bits of mantissa as a sum of
// two bf16 numbers, which feed two matrix instructions each: one bf16 number
// would add as much error as the result's own rounding, and an fp16 one could
// overflow.
#include "fp8.hpp"
#include "fp8_quant.hpp"
#include "launch.hpp"
#include "moe.hpp"

#include <atomic>
#include <type_traits>

namespace i8mm {

namespace {

// A row offset past every operand (at most 2^31 bytes), with room below 2^32
// for the offsets inside a block.
constexpr uint32_t kNoRow = 0xfffff000u;

// A block's scale s = power * rest, exactly, the same for the whole wavefront.
// Left operands of fp32's range times numbers of up to 448, 128 times, can pass it
// where s brings the sum back, so the conversions of the block's numbers take its
// power of two with them (they read no more than the exponent), and what multiplies
// the sum is 1 to 2 in magnitude: the sum passes the range only where its scaled
// value nearly does.  The power stays within 2^-100 .. 2^100, so that the numbers
// times it are normal bf16 ones; a scale further out (or zero, subnormal, infinite,
// NaN) leaves the rest to `rest`.  fp16 operands' sums cannot pass fp32's range,
// and fp16 could not hold the scaled numbers.
struct Scale {
  float power, rest;
};
template <int TY>
__device__ __forceinline__ Scale split_scale(float s) {
  if constexpr (TY == kF16) return {1.0f, s};
  // scalar instructions: the median of three is a vector one, and takes registers
  const int low = max((int)(__builtin_bit_cast(uint32_t, s) >> 23 & 255), 27);
  const int e = min(__builtin_amdgcn_readfirstlane(low), 227);
  const float rest = s * __builtin_bit_cast(float, (254 - e) << 23);
  return {__builtin_bit_cast(float, e << 23),
          __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, rest)))};
}

// Two e4m3 numbers (the low or high half of a dword) as fp16, or times a power of
// two as bf16, exactly.
template <int TY, bool HIGH>
__device__ __forceinline__ int widen2(int w, float power) {
  if constexpr (TY == kF16)
    return __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HIGH));
  else
    return __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, power, HIGH));
}

// A lane's 16 e4m3 numbers of a half block as two matrix operands.
template <int TY>
__device__ __forceinline__ void widen16(const v4i& w, float power, v4i (&o)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    o[i] = v4i{widen2<TY, false>(w[2 * i], power), widen2<TY, true>(w[2 * i], power),
               widen2<TY, false>(w[2 * i + 1], power), widen2<TY, true>(w[2 * i + 1], power)};
}

// The expert of slot s: the experts in turn, or, where there are fewer pairs
// than experts, that of pair s if s is the expert's first pair.  -1: none.
// Writes the expert's pairs to `list` in ascending order and their number to n.
template <int NT>
__device__ __forceinline__ int expert_of_slot(const MoeCall& c, int s, uint16_t* list, int* counts,
                                              int& n) {
  const int P = c.M * c.top_k;
  int e = P < c.E ? c.experts[s] : s;
  e = __builtin_amdgcn_readfirstlane(e);
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  constexpr int NW = NT / 64;
  // each wavefront counts its part of the pairs, then writes it behind the others'
  const int seg = ((P + NW - 1) / NW + 63) & ~63;
  const int lo = w * seg, hi = min(P, lo + seg);
  int mine = 0;
  for (int p = lo + lane; p - lane < hi; p += 64)
    mine += __builtin_popcountll(__ballot(p < hi && c.experts[p] == e));
  if (lane == 0) counts[w] = mine;
  __syncthreads();
  int at = 0;
  n = 0;
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    if (i < w) at += counts[i];
    n += counts[i];
  }
  for (int p = lo + lane; p - lane < hi; p += 64) {
    const bool is = p < hi && c.experts[p] == e;
    const uint64_t b = __ballot(is);
    if (is) list[at + __builtin_popcountll(b & ((1ull << lane) - 1))] = (uint16_t)p;
    at += __builtin_popcountll(b);
  }
  __syncthreads();
  n = __builtin_amdgcn_readfirstlane(n);
  if ((unsigned)e >= (unsigned)c.E || n == 0 || (P < c.E && list[0] != s)) return -1;
  return e;
}

// ---- the columns split over a workgroup's wavefronts -------------------------
//
// One product of NB blocks of 16 weight rows (at bytes w_at[b] of the expert's
// packed matrix, with scales s_at[b]) with T blocks of 16 tokens (rows[t]: byte
// offset of the lane's token in the operand, or kNoRow) over the wavefront's
// 128-column blocks w, w + KS, ...  Weights and tokens come straight to registers,
// a block ahead.  The operand holds `PLANES` numbers per column that are added: 16 columns are
// 32 bytes of the first, then 32 of the second.
template <int TY, int NB, int T, int PLANES, int KS>
struct Product {
  struct Stage {
    v4i w[NB][2];
    v4i x[T][2][PLANES][2];
    float s[NB];
  };
  typedef const __attribute__((address_space(4))) float* scalar_ptr;
  const uint8_t* W;
  uint32_t w_bytes;
  uint32_t w_at[NB];
  scalar_ptr s_at[NB];
  const void* X;
  uint32_t x_bytes;
  uint32_t rows[T];
  int K, KB, lane, q4;

  __device__ __forceinline__ void load_w(int kb, Stage& o) const {
    constexpr int kNonTemporal = 2;
    const bool live = kb < KB;
    const int k = live ? kb : 0;
    const __amdgpu_buffer_rsrc_t rw =
        __builtin_amdgcn_make_buffer_rsrc((void*)W, (short)0, live ? (int)w_bytes : 0, 0x00020000);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      o.s[b] = s_at[b][k];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        o.w[b][h] = __builtin_bit_cast(
            v4i, __builtin_amdgcn_raw_buffer_load_b128(
                     rw, lane * 16, (int)(w_at[b] + (uint32_t)k * 2048u + h * 1024u), kNonTemporal));
    }
  }

  __device__ __forceinline__ void load_x(int kb, Stage& o) const {
    const bool live = kb < KB;
    const int k = live ? kb : 0;
    const __amdgpu_buffer_rsrc_t rx =
        __builtin_amdgcn_make_buffer_rsrc((void*)X, (short)0, live ? (int)x_bytes : 0, 0x00020000);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool out = k * 128 + h * 64 + q4 * 16 >= K;
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const uint32_t at = (out ? kNoRow : rows[t]) + h * 128 * PLANES;
#pragma unroll
        for (int p = 0; p < PLANES; ++p)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            o.x[t][h][p][i] = __builtin_bit_cast(
                v4i, __builtin_amdgcn_raw_buffer_load_b128(
                         rx, (int)(at + p * 32 + i * 16), k * (256 * PLANES), 0));
      }
    }
  }

  __device__ __forceinline__ void compute(const Stage& s, v4f (&acc)[NB][T]) const {
    v4f sum[NB][T];
    Scale sc[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      sc[b] = split_scale<TY>(s.s[b]);
#pragma unroll
      for (int t = 0; t < T; ++t) sum[b][t] = v4f{};
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        v4i w[2];
        widen16<TY>(s.w[b][h], sc[b].power, w);
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
          for (int p = 0; p < PLANES; ++p)
#pragma unroll
            for (int i = 0; i < 2; ++i) sum[b][t] = mfma32<TY>(w[i], s.x[t][h][p][i], sum[b][t]);
      }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[b][t][e] = fmaf(sum[b][t][e], sc[b].rest, acc[b][t][e]);
  }

  __device__ __forceinline__ void run(int w, v4f (&acc)[NB][T]) const {
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int t = 0; t < T; ++t) acc[b][t] = v4f{};
    if (w >= KB) return;
    Stage a, b;
    load_x(w, a);
    load_w(w, a);
    for (int kb = w; kb < KB; kb += 2 * KS) {
      load_x(kb + KS, b);
      load_w(kb + KS, b);
      compute(a, acc);
      if (kb + KS >= KB) break;
      load_x(kb + 2 * KS, a);
      load_w(kb + 2 * KS, a);
      compute(b, acc);
    }
  }
};

// The wavefronts' sums through LDS, [KS][NB * T][64]: any wavefront can then add
// those of tile o = b * T + t, in wavefront order.
template <int NB, int T, int KS>
__device__ __forceinline__ void spread_partials(const v4f (&acc)[NB][T], int w, int lane, v4f* red) {
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int t = 0; t < T; ++t) red[(w * NB * T + b * T + t) * 64 + lane] = acc[b][t];
  __syncthreads();
}
template <int NB, int T, int KS>
__device__ __forceinline__ v4f joined(const v4f* red, int o, int lane) {
  v4f y = red[o * 64 + lane];
#pragma unroll
  for (int i = 1; i < KS; ++i) y += red[(i * NB * T + o) * 64 + lane];
  return y;
}

// The gated product of a lane's four features of one pair, as two bf16 numbers.
__device__ __forceinline__ void store_gated(const v4f& g, const v4f& u, uint8_t* at) {
  float hi[4], lo[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = silu_mul(g[i], u[i]);
    // a finite one past the largest bf16 number is that number and a rest; an
    // infinity leaves none (its difference would be NaN)
    constexpr float kLargest = 3.4028235e38f, kLargestBf16 = 0x1.fep127f;
    hi[i] = (float)(__bf16)a;
    if (fabsf(a) > kLargestBf16 && fabsf(a) <= kLargest) hi[i] = copysignf(kLargestBf16, a);
    lo[i] = fabsf(hi[i]) <= kLargest ? a - hi[i] : 0.0f;
  }
  *reinterpret_cast<uint2*>(at) =
      make_uint2(pack16x2<kBf16>(hi[0], hi[1]), pack16x2<kBf16>(hi[2], hi[3]));
  *reinterpret_cast<uint2*>(at + 32) =
      make_uint2(pack16x2<kBf16>(lo[0], lo[1]), pack16x2<kBf16>(lo[2], lo[3]));
}

// First product: workgroup (f, s) makes 16 features of the gated product, gate
// and up rows side by side, for all tokens of slot s's expert.
template <int TY, int T, int KS>
__device__ __forceinline__ void up_tokens(const MoeCall& c, int e, int j0, int n,
                                          const uint16_t* list, v4f* red) {
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q4 = lane >> 4, r16 = lane & 15;
  const int f = blockIdx.x;
  using P = Product<TY, 2, T, 1, KS>;
  P p;
  p.K = c.K;
  p.KB = (c.K + kFp8Block - 1) / kFp8Block;
  p.lane = lane;
  p.q4 = q4;
  p.w_bytes = (uint32_t)(2 * c.I) * (uint32_t)(p.KB * kFp8Block);
  p.W = c.up + (size_t)e * p.w_bytes;
  const float* scales = c.up_scale + (size_t)e * ((2 * c.I + 127) / 128) * p.KB;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int rb = b * (c.I / 16) + f;
    p.w_at[b] = (uint32_t)rb * (uint32_t)p.KB * 2048u;
    p.s_at[b] = (typename P::scalar_ptr)(uintptr_t)(scales + (size_t)(rb / 8) * p.KB);
  }
  p.X = c.X;
  p.x_bytes = (uint32_t)c.M * (uint32_t)c.K * 2u;
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const int j = j0 + t * 16 + r16;
    p.rows[t] = j < n ? (uint32_t)(list[j] / c.top_k) * (uint32_t)c.K * 2u + q4 * 32u : kNoRow;
  }
  v4f acc[2][T];
  p.run(w, acc);
  spread_partials<2, T, KS>(acc, w, lane, red);
  for (int t = w; t < T; t += KS) {
    const v4f g = joined<2, T, KS>(red, t, lane), u = joined<2, T, KS>(red, T + t, lane);
    const int j = j0 + t * 16 + r16;
    if (j < n) store_gated(g, u, c.act + ((size_t)list[j] * c.I + f * 16) * 4 + q4 * 8);
  }
  __syncthreads();  // `red` is free
}

// Second product: workgroup (f, s) makes 16 * NB features of slot s's expert's
// output for all its tokens, times their weights.
template <int NB, int T, int KS>
__device__ __forceinline__ void down_tokens(const MoeCall& c, int e, int j0, int n,
                                            const uint16_t* list, v4f* red) {
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q4 = lane >> 4, r16 = lane & 15;
  const int rb0 = blockIdx.x * NB, nrb = c.K / 16;
  using P = Product<kBf16, NB, T, 2, KS>;
  P p;
  p.K = c.I;
  p.KB = (c.I + kFp8Block - 1) / kFp8Block;
  p.lane = lane;
  p.q4 = q4;
  p.w_bytes = (uint32_t)c.K * (uint32_t)(p.KB * kFp8Block);
  p.W = c.down + (size_t)e * p.w_bytes;
  const float* scales = c.down_scale + (size_t)e * ((c.K + 127) / 128) * p.KB;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int rb = min(rb0 + b, nrb - 1);  // past the end: the last one, never stored
    p.w_at[b] = (uint32_t)rb * (uint32_t)p.KB * 2048u;
    p.s_at[b] = (typename P::scalar_ptr)(uintptr_t)(scales + (size_t)(rb / 8) * p.KB);
  }
  p.X = c.act;
  p.x_bytes = (uint32_t)c.M * (uint32_t)c.top_k * (uint32_t)c.I * 4u;
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const int j = j0 + t * 16 + r16;
    p.rows[t] = j < n ? (uint32_t)list[j] * (uint32_t)c.I * 4u + q4 * 64u : kNoRow;
  }
  v4f acc[NB][T];
  p.run(w, acc);
  spread_partials<NB, T, KS>(acc, w, lane, red);
  for (int o = w; o < NB * T; o += KS) {
    const v4f y = joined<NB, T, KS>(red, o, lane);
    const int j = j0 + o % T * 16 + r16, rb = rb0 + o / T;
    if (j < n && rb < nrb) {
      const float s = c.weights[list[j]];
      *reinterpret_cast<v4f*>(c.part + (size_t)list[j] * c.K + rb * 16 + q4 * 4) = y * s;
    }
  }
  __syncthreads();
}

template <int TY, int TMAX, int KS>
__global__ __launch_bounds__(KS * 64) void k_moe_up(MoeCall c) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int counts[KS];
  v4f* red = reinterpret_cast<v4f*>(smem);
  uint16_t* list = reinterpret_cast<uint16_t*>(smem + KS * 2 * TMAX * 1024);
  int n;
  const int e = expert_of_slot<KS * 64>(c, blockIdx.y, list, counts, n);
  if (e < 0) return;
  for (int j0 = 0; j0 < n; j0 += 16 * TMAX) {
    if (TMAX >= 4 && n - j0 > 32)
      up_tokens<TY, TMAX, KS>(c, e, j0, n, list, red);
    else if (TMAX >= 2 && n - j0 > 16)
      up_tokens<TY, TMAX < 2 ? 1 : 2, KS>(c, e, j0, n, list, red);
    else
      up_tokens<TY, 1, KS>(c, e, j0, n, list, red);
  }
}

template <int NB, int TMAX, int KS>
__global__ __launch_bounds__(KS * 64) void k_moe_down(MoeCall c) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int counts[KS];
  v4f* red = reinterpret_cast<v4f*>(smem);
  uint16_t* list = reinterpret_cast<uint16_t*>(smem + KS * NB * TMAX * 1024);
  int n;
  const int e = expert_of_slot<KS * 64>(c, blockIdx.y, list, counts, n);
  if (e < 0) return;
  for (int j0 = 0; j0 < n; j0 += 16 * TMAX) {
    if (TMAX >= 4 && n - j0 > 32)
      down_tokens<NB, TMAX, KS>(c, e, j0, n, list, red);
    else if (TMAX >= 2 && n - j0 > 16)
      down_tokens<NB, TMAX < 2 ? 1 : 2, KS>(c, e, j0, n, list, red);
    else
      down_tokens<NB, 1, KS>(c, e, j0, n, list, red);
  }
}

// ---- many workgroups: no split of the columns --------------------------------
//
// A workgroup's eight wavefronts take two blocks of 16 weight rows each, over all
// columns, and share the tokens' tile of a 128-column block in LDS, which comes by
// DMA a block ahead (two blocks ahead it took as long: 512x4096 of 128 experts
// 541 and 546 us).  The weights go straight to the wavefront that uses them,
// requested two blocks ahead.  The loop goes by two blocks and may end after the
// first, so the compiled first step waits for all but 0 to 5 of the loads on their
// way, the next block's weights and tile among them, in front of its products; only
// the second step's run under the stream.  The figures here are with those waits.
// A tile row is 256 bytes per number of an operand column, its 16-byte chunks
// swapped by the row's low four bits: a read of 16 bytes serves 16 lanes at once,
// eight of one chunk and eight of the next one, and they meet all 64 banks (by
// three bits, half of the reads' cycles were conflicts).
template <int TY, int T, int PLANES>
struct Wide {
  static constexpr int WAVES = 8, NB = 2, NT = WAVES * 64;
  static constexpr int ROW = 256 * PLANES, CHUNKS = ROW / 16;
  static constexpr int STAGE = T * 16 * ROW;
  static constexpr int LOADS = (T * 16 * CHUNKS + NT - 1) / NT;  // DMAs of a wavefront
  typedef const __attribute__((address_space(4))) float* scalar_ptr;
  struct Weights {
    v4i w[NB][2];
    float s[NB];
  };
  const uint8_t* W;
  uint32_t w_bytes;
  uint32_t w_at[NB];
  scalar_ptr s_at[NB];
  const void* X;
  uint32_t x_bytes;
  int K, KB;

  // list[j0 .. j0 + 16 T) of n pairs are the tile's rows; a row's operand starts
  // at byte (pair / per) * stride.
  __device__ __forceinline__ void run(const uint16_t* list, int j0, int n, int per, uint32_t stride,
                                      uint8_t* smem, v4f (&acc)[NB][T]) const {
    const int tid = threadIdx.x, lane = tid & 63, q4 = lane >> 4, r16 = lane & 15;
    const __amdgpu_buffer_rsrc_t rw =
        __builtin_amdgcn_make_buffer_rsrc((void*)W, (short)0, (int)w_bytes, 0x00020000);
    const __amdgpu_buffer_rsrc_t rx =
        __builtin_amdgcn_make_buffer_rsrc((void*)X, (short)0, (int)x_bytes, 0x00020000);
    // The tile's chunk number i * NT + thread of LDS holds the swapped chunk of its row.
    uint32_t src[LOADS];
    const int slot = tid % CHUNKS, row0 = tid / CHUNKS;
    const int c = slot ^ (row0 & 15);  // NT / CHUNKS rows further the low bits are the same
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int j = j0 + row0 + i * (NT / CHUNKS);
      src[i] = j < n ? (uint32_t)(list[j] / per) * stride + c * 16u : kNoRow;
    }
    // columns of a chunk: 8 of one number, or 16 of two numbers in four chunks
    const int col = PLANES == 1 ? c * 8 : (c >> 2) * 16;
    const int first = __builtin_amdgcn_readfirstlane(tid & ~63);
    auto load_x = [&](int kb, int stage) {
      const bool out = kb * 128 + col >= K;
      uint8_t* dst = smem + stage * STAGE + first * 16;
#pragma unroll
      for (int i = 0; i < LOADS; ++i)
        if (i * NT + first < T * 16 * CHUNKS)  // whole wavefronts
          dma16(rx, dst + i * NT * 16, (int)(out ? kNoRow : src[i]), kb * ROW);
    };
    auto load_w = [&](int kb, Weights& o) {
      constexpr int kNonTemporal = 2;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        o.s[b] = s_at[b][kb];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          o.w[b][h] = __builtin_bit_cast(
              v4i, __builtin_amdgcn_raw_buffer_load_b128(
                       rw, lane * 16, (int)(w_at[b] + (uint32_t)kb * 2048u + h * 1024u),
                       kNonTemporal));
      }
    };
    auto compute = [&](const Weights& o, int stage) {
      v4i w[2][NB][2];
      Scale sc[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) sc[b] = split_scale<TY>(o.s[b]);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int b = 0; b < NB; ++b) widen16<TY>(o.w[b][h], sc[b].power, w[h][b]);
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const uint8_t* row = smem + stage * STAGE + (t * 16 + r16) * ROW;
        v4f sum[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) sum[b] = v4f{};
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int p = 0; p < PLANES; ++p)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int c = (h * 4 + q4) * 2 * PLANES + p * 2 + i;
              const v4i f = *reinterpret_cast<const v4i*>(row + (c ^ r16) * 16);
#pragma unroll
              for (int b = 0; b < NB; ++b) sum[b] = mfma32<TY>(w[h][b][i], f, sum[b]);
            }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[b][t][e] = fmaf(sum[b][e], sc[b].rest, acc[b][t][e]);
        // one block of tokens' reads at a time: more would not fit the registers
        __builtin_amdgcn_sched_barrier(0);
      }
    };
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int t = 0; t < T; ++t) acc[b][t] = v4f{};
    if (KB == 0) return;
    Weights a, b;
    constexpr int WOPS = 2 * NB;  // vector loads of a block's weights
    load_x(0, 0);
    // the waits count the loads behind the tile's, so none may be moved in front of it
    __builtin_amdgcn_sched_barrier(0);
    load_w(0, a);
    load_w(min(1, KB - 1), b);
    barrier_vm<2 * WOPS>();  // the first tile is there
    auto step = [&](int kb, Weights& cur) {
      const int stage = kb & 1;
      load_x(min(kb + 1, KB - 1), stage ^ 1);
      __builtin_amdgcn_sched_barrier(0);
      compute(cur, stage);
      load_w(min(kb + 2, KB - 1), cur);
      barrier_vm<WOPS>();  // the next tile is there, and this one free
    };
    for (int kb = 0; kb < KB; kb += 2) {
      step(kb, a);
      if (kb + 1 < KB) step(kb + 1, b);
    }
    barrier_vm<0>();  // no DMA may still write LDS
  }
};

template <int TY, int T>
__device__ __forceinline__ void up_wide(const MoeCall& c, int group, int e, int j0, int n,
                                        const uint16_t* list, uint8_t* smem) {
  const int lane = threadIdx.x & 63, q4 = lane >> 4, r16 = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  using P = Wide<TY, T, 1>;
  const int f = group * P::WAVES + w, nf = c.I / 16, fc = min(f, nf - 1);
  P p;
  p.K = c.K;
  p.KB = (c.K + kFp8Block - 1) / kFp8Block;
  p.w_bytes = (uint32_t)(2 * c.I) * (uint32_t)(p.KB * kFp8Block);
  p.W = c.up + (size_t)e * p.w_bytes;
  const float* scales = c.up_scale + (size_t)e * ((2 * c.I + 127) / 128) * p.KB;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int rb = b * nf + fc;
    p.w_at[b] = (uint32_t)rb * (uint32_t)p.KB * 2048u;
    p.s_at[b] = (typename P::scalar_ptr)(uintptr_t)(scales + (size_t)(rb / 8) * p.KB);
  }
  p.X = c.X;
  p.x_bytes = (uint32_t)c.M * (uint32_t)c.K * 2u;
  v4f acc[2][T];
  p.run(list, j0, n, c.top_k, (uint32_t)c.K * 2u, smem, acc);
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const int j = j0 + t * 16 + r16;
    if (j < n && f < nf)
      store_gated(acc[0][t], acc[1][t], c.act + ((size_t)list[j] * c.I + f * 16) * 4 + q4 * 8);
  }
}

template <int T>
__device__ __forceinline__ void down_wide(const MoeCall& c, int group, int e, int j0, int n,
                                          const uint16_t* list, uint8_t* smem) {
  const int lane = threadIdx.x & 63, q4 = lane >> 4, r16 = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  using P = Wide<kBf16, T, 2>;
  const int rb0 = (group * P::WAVES + w) * 2, nrb = c.K / 16;
  P p;
  p.K = c.I;
  p.KB = (c.I + kFp8Block - 1) / kFp8Block;
  p.w_bytes = (uint32_t)c.K * (uint32_t)(p.KB * kFp8Block);
  p.W = c.down + (size_t)e * p.w_bytes;
  const float* scales = c.down_scale + (size_t)e * ((c.K + 127) / 128) * p.KB;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int rb = min(rb0 + b, nrb - 1);
    p.w_at[b] = (uint32_t)rb * (uint32_t)p.KB * 2048u;
    p.s_at[b] = (typename P::scalar_ptr)(uintptr_t)(scales + (size_t)(rb / 8) * p.KB);
  }
  p.X = c.act;
  p.x_bytes = (uint32_t)c.M * (uint32_t)c.top_k * (uint32_t)c.I * 4u;
  v4f acc[2][T];
  p.run(list, j0, n, 1, (uint32_t)c.I * 4u, smem, acc);
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const int j = j0 + t * 16 + r16;
    if (j < n) {
      const float s = c.weights[list[j]];
#pragma unroll
      for (int b = 0; b < 2; ++b)
        if (rb0 + b < nrb)
          *reinterpret_cast<v4f*>(c.part + (size_t)list[j] * c.K + (rb0 + b) * 16 + q4 * 4) =
              acc[b][t] * s;
    }
  }
}

// Bytes of LDS for the two tiles of the most tokens.
template <int PLANES>
constexpr int kWideLds = 2 * Wide<kF16, 4, PLANES>::STAGE;

// UP: the first product, else the second.  Up to 64 of an expert's tokens per
// pass over its weights.  `groups` workgroups make an expert's features; they run
// on one XCD, whose L2 then holds the expert's tokens for all of them.
template <int TY, bool UP>
__global__ __launch_bounds__(512, 4) void k_moe_wide(MoeCall c, int groups) {
  extern __shared__ __align__(16) uint8_t smem[];
  // The counts lie where the tiles will be: the tiles and a list of the most pairs
  // are 80 KB, two workgroups fill a CU's LDS to the byte (with 32 bytes more one
  // fits: the second product of 1024x4096, 128 experts, 8 places took 394 us, not 306).
  int* counts = reinterpret_cast<int*>(smem);
  uint16_t* list = reinterpret_cast<uint16_t*>(smem + kWideLds<UP ? 1 : 2>);
  const int at = xcd_remap(blockIdx.x, gridDim.x), group = at % groups;
  int n;
  const int e = expert_of_slot<512>(c, at / groups, list, counts, n);
  if (e < 0) return;
  auto pass = [&](auto t, int j0) {
    if constexpr (UP)
      up_wide<TY, t()>(c, group, e, j0, n, list, smem);
    else
      down_wide<t()>(c, group, e, j0, n, list, smem);
  };
  for (int j0 = 0; j0 < n; j0 += 64) {
    const int blocks = (n - j0 + 15) / 16;
    if (blocks >= 4)
      pass(std::integral_constant<int, 4>{}, j0);
    else if (blocks == 3)
      pass(std::integral_constant<int, 3>{}, j0);
    else if (blocks == 2)
      pass(std::integral_constant<int, 2>{}, j0);
    else
      pass(std::integral_constant<int, 1>{}, j0);
  }
}

// ---- a few pairs: vector products -------------------------------------------
//
// With far fewer pairs than experts an expert has hardly ever two tokens, so each
// pair goes alone, without matrix instructions: a lane multiplies its 16 numbers
// of a row, times their scale's power of two, by the pair's activations (fp32, in
// LDS, read by 16 lanes at once).
// That needs one accumulator a row block and no operand registers, so that many
// wavefronts fit a CU with CB blocks of weights on their way each, refilled as
// they are used; these calls wait for latency (1x4096 of 128 experts, 8 places of
// 1408: 30 us in a graph, 18 + 10.5 in the two kernels = 5.1 TB/s; CB = 4 and 6,
// without the order of the reads below, 32).  The compiler orders the first CB
// blocks' loads as it likes and has a round's first use wait for all that are on
// their way; the figures are with that wait.

// The sums over columns [kb0, kb1) * 128 of NB row blocks; lane l has that of row
// l % 16 in every of its four quarters.  x.load(kb) starts the loads of the
// activations of CB blocks (zeros past the end) and x.store(at) leaves them as
// fp32 in LDS of the wavefront's own.  Those of kb0 are on their way already:
// they do not wait for what the weights' address waits for.
template <int NB, int CB, typename Activations>
__device__ __forceinline__ void vector_product(const uint8_t* W, uint32_t w_bytes,
                                               const uint32_t (&w_at)[NB],
                                               const float* const (&s_at)[NB], int kb0, int kb1,
                                               float* at, Activations& x, float (&acc)[NB]) {
  constexpr int kNonTemporal = 2;
  const int lane = threadIdx.x & 63, q4 = lane >> 4;
  v4i w[CB][NB][2];
  float s[NB];
  // a block at or past kb1 gets an empty descriptor: zeros, and nothing is read
  auto load_w = [&](int kb, v4i (&o)[NB][2]) {
    const bool live = kb < kb1;
    const __amdgpu_buffer_rsrc_t rw =
        __builtin_amdgcn_make_buffer_rsrc((void*)W, (short)0, live ? (int)w_bytes : 0, 0x00020000);
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        o[b][h] = __builtin_bit_cast(
            v4i, __builtin_amdgcn_raw_buffer_load_b128(
                     rw, lane * 16 + h * 1024, live ? (int)(w_at[b] + (uint32_t)kb * 2048u) : 0,
                     kNonTemporal));
  };
  // the blocks' scales, one a lane: scalar loads would be waited for with the
  // first read of LDS
  auto load_scales = [&](int kb) {
#pragma unroll
    for (int b = 0; b < NB; ++b) s[b] = s_at[b][min(kb + lane, kb1 - 1)];
  };
#pragma unroll
  for (int b = 0; b < NB; ++b) acc[b] = 0.0f;
  if (kb0 >= kb1) return;
  load_scales(kb0);
#pragma unroll
  for (int c = 0; c < CB; ++c) load_w(kb0 + c, w[c]);
  for (int kb = kb0; kb < kb1; kb += CB) {
    x.store(at);
    float now[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) now[b] = s[b];
    if (kb + CB < kb1) {
      x.load(kb + CB);
      load_scales(kb + CB);
    }
#pragma unroll
    for (int c = 0; c < CB; ++c) {
      float sum[NB][2] = {};
      Scale sc[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b)
        sc[b] = split_scale<kBf16>(__builtin_bit_cast(
            float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, now[b]), c)));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const v4f* from = reinterpret_cast<const v4f*>(at + c * 128 + h * 64 + q4 * 16);
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const v4f v = from[d];
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            typedef float v2f __attribute__((ext_vector_type(2)));
            const float p = sc[b].power;
            const v2f lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[c][b][h][d], p, false);
            const v2f hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[c][b][h][d], p, true);
            sum[b][0] = fmaf(lo[0], v[0], sum[b][0]);
            sum[b][1] = fmaf(lo[1], v[1], sum[b][1]);
            sum[b][0] = fmaf(hi[0], v[2], sum[b][0]);
            sum[b][1] = fmaf(hi[1], v[3], sum[b][1]);
          }
          // else the reads and conversions of all blocks are brought forward, and
          // their registers cost more than they hide
          if (d & 1) __builtin_amdgcn_sched_barrier(0);
        }
      }
      load_w(kb + CB + c, w[c]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[b] = fmaf(sum[b][0] + sum[b][1], sc[b].rest, acc[b]);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read before it is written again
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    acc[b] += __shfl_xor(acc[b], 16, kWave);
    acc[b] += __shfl_xor(acc[b], 32, kWave);
  }
}

// First product: workgroup (f, p) makes 16 features of pair p's gated product
// (fp32), the columns split over its wavefronts.
constexpr int kFewUpWaves = 8, kFewUpBlocks = 2;
template <int TY>
struct FewTokens {
  const uint16_t* row;
  int K, lane;
  uint2 v;
  __device__ __forceinline__ void load(int kb) {  // 4 columns a lane
    static_assert(kFewUpBlocks * 128 == 64 * 4, "one load per lane");
    const int k = kb * 128 + lane * 4;
    v = k < K ? *reinterpret_cast<const uint2*>(row + k) : make_uint2(0, 0);
  }
  __device__ __forceinline__ void store(float* at) const {
    *reinterpret_cast<v4f*>(at + lane * 4) =
        v4f{to_f32<TY>((uint16_t)v.x), to_f32<TY>((uint16_t)(v.x >> 16)),
            to_f32<TY>((uint16_t)v.y), to_f32<TY>((uint16_t)(v.y >> 16))};
  }
};
template <int TY>
__global__ __launch_bounds__(kFewUpWaves * 64) void k_moe_up_few(MoeCall c) {
  __shared__ __align__(16) float x[kFewUpWaves][kFewUpBlocks * 128];
  __shared__ float red[kFewUpWaves][2][16];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int f = blockIdx.x, pair = blockIdx.y;
  const int KB = (c.K + kFp8Block - 1) / kFp8Block;
  const int kb0 = KB * w / kFewUpWaves, kb1 = KB * (w + 1) / kFewUpWaves;
  // columns past the wavefront's own meet weights of zero, and are none themselves
  FewTokens<TY> tokens{c.X + (size_t)(pair / c.top_k) * c.K, min(c.K, kb1 * 128), lane, {}};
  tokens.load(kb0);
  const int e = __builtin_amdgcn_readfirstlane(c.experts[pair]);
  if ((unsigned)e >= (unsigned)c.E) return;
  const uint32_t w_bytes = (uint32_t)(2 * c.I) * (uint32_t)(KB * kFp8Block);
  uint32_t w_at[2];
  const float* s_at[2];
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int rb = b * (c.I / 16) + f;
    w_at[b] = (uint32_t)rb * (uint32_t)KB * 2048u;
    s_at[b] = c.up_scale + ((size_t)e * ((2 * c.I + 127) / 128) + rb / 8) * KB;
  }
  float acc[2];
  vector_product<2, kFewUpBlocks>(c.up + (size_t)e * w_bytes, w_bytes, w_at, s_at, kb0, kb1, x[w],
                                  tokens, acc);
  if (lane < 16) red[w][0][lane] = acc[0], red[w][1][lane] = acc[1];
  __syncthreads();
  if (threadIdx.x < 16) {
    float g = 0.0f, u = 0.0f;
#pragma unroll
    for (int i = 0; i < kFewUpWaves; ++i) g += red[i][0][lane], u += red[i][1][lane];
    reinterpret_cast<float*>(c.act)[(size_t)pair * c.I + f * 16 + lane] = silu_mul(g, u);
  }
}

// Second product and the sum over the pairs: a workgroup owns 16 features of all
// pairs, so nothing is joined in another launch; its wavefronts take the pairs in turn, or, where there are fewer pairs,
// one of `parts` shares of a pair's columns.
constexpr int kFewDownWaves = 16, kFewDownBlocks = 2;
constexpr int kFewPairs = 64;
struct FewGated {
  const float* row;
  int I, lane;
  v4f v[kFewDownBlocks / 2];
  __device__ __forceinline__ void load(int kb) {  // 4 columns a lane and load
#pragma unroll
    for (int i = 0; i < kFewDownBlocks / 2; ++i) {
      const int k = kb * 128 + i * 256 + lane * 4;
      v[i] = k < I ? *reinterpret_cast<const v4f*>(row + k) : v4f{};
    }
  }
  __device__ __forceinline__ void store(float* at) const {
#pragma unroll
    for (int i = 0; i < kFewDownBlocks / 2; ++i)
      *reinterpret_cast<v4f*>(at + i * 256 + lane * 4) = v[i];
  }
};
template <int TY>
__global__ __launch_bounds__(kFewDownWaves * 64) void k_moe_down_few(MoeCall c, int parts) {
  __shared__ __align__(16) float x[kFewDownWaves][kFewDownBlocks * 128];
  __shared__ float sums[kFewPairs][16];  // parts * pairs <= kFewPairs
  __shared__ float shares[kFewPairs];    // the pairs' weights
  const int P = c.M * c.top_k;
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rb = blockIdx.x, KB = (c.I + kFp8Block - 1) / kFp8Block;
  const uint32_t w_bytes = (uint32_t)c.K * (uint32_t)(KB * kFp8Block);
  const uint32_t w_at[1] = {(uint32_t)rb * (uint32_t)KB * 2048u};
  // a pair without an expert: zeros, whatever its weight
  float share = 0.0f;
  if (tid < P && (unsigned)c.experts[tid] < (unsigned)c.E) share = c.weights[tid];
  for (int item = w; item < P * parts; item += kFewDownWaves) {
    const int pair = item / parts, q = item % parts;
    const int kb0 = KB * q / parts, kb1 = KB * (q + 1) / parts;
    FewGated gated{reinterpret_cast<const float*>(c.act) + (size_t)pair * c.I,
                   min(c.I, kb1 * 128), lane, {}};
    gated.load(kb0);
    const int e = __builtin_amdgcn_readfirstlane(c.experts[pair]);
    if ((unsigned)e >= (unsigned)c.E) {
      if (lane < 16) sums[item][lane] = 0.0f;
      continue;
    }
    const float* const s_at[1] = {c.down_scale + ((size_t)e * ((c.K + 127) / 128) + rb / 8) * KB};
    float acc[1];
    vector_product<1, kFewDownBlocks>(c.down + (size_t)e * w_bytes, w_bytes, w_at, s_at, kb0, kb1,
                                      x[w], gated, acc);
    if (lane < 16) sums[item][lane] = acc[0];
  }
  if (tid < P) shares[tid] = share;
  __syncthreads();
  for (int o = tid; o < c.M * 16; o += kFewDownWaves * 64) {
    const int m = o >> 4, f = o & 15;
    float y = 0.0f;
    for (int j = 0; j < c.top_k; ++j) {
      const int pair = m * c.top_k + j;
      float v = 0.0f;
      for (int q = 0; q < parts; ++q) v += sums[pair * parts + q][f];
      y = fmaf(v, shares[pair], y);
    }
    c.Y[(size_t)m * c.K + rb * 16 + f] = (uint16_t)pack16x2<TY>(y, 0.0f);
  }
}

// y[m] = the sum of the token's pairs in their order, rounded once; a thread
// per 8 columns.  Eight pairs' loads at a time, also those of pairs whose sums
// were not made (their places are read and dropped): with a branch around each
// load one token of 8 experts took 4.8 us instead of 2.
template <int TY>
__global__ __launch_bounds__(256) void k_moe_join(MoeCall c) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int chunks = c.K / 8;
  if (i >= (int64_t)c.M * chunks) return;
  const int m = (int)(i / chunks), k = (int)(i % chunks) * 8;
  v4f a = {}, b = {};
  for (int j0 = 0; j0 < c.top_k; j0 += 8) {
    v4f u[8], v[8];
    bool made[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int p = m * c.top_k + min(j0 + j, c.top_k - 1);
      made[j] = j0 + j < c.top_k && (unsigned)c.experts[p] < (unsigned)c.E && c.I > 0;
      const v4f* from = reinterpret_cast<const v4f*>(c.part + (size_t)p * c.K + k);
      u[j] = from[0];
      v[j] = from[1];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[e] += made[j] ? u[j][e] : 0.0f;
        b[e] += made[j] ? v[j][e] : 0.0f;
      }
  }
  *reinterpret_cast<uint4*>(c.Y + (size_t)m * c.K + k) =
      make_uint4(pack16x2<TY>(a[0], a[1]), pack16x2<TY>(a[2], a[3]), pack16x2<TY>(b[0], b[1]),
                 pack16x2<TY>(b[2], b[3]));
}

// Launches with more than the 64 KB of dynamic LDS that need no leave: asked
// for once per device the kernels run on.
template <typename Kernel>
hipError_t launch_wide(Kernel kern, std::atomic<uint64_t>& asked, int groups, int slots, size_t lds,
                       const MoeCall& c, hipStream_t st) {
  int dev = 0;
  (void)hipGetDevice(&dev);
  const uint64_t bit = 1ull << (dev & 63);
  if (!(asked.load(std::memory_order_relaxed) & bit)) {
    const hipError_t e = hipFuncSetAttribute(
        (const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, 96 * 1024);
    if (e != hipSuccess) return e;
    asked.fetch_or(bit, std::memory_order_relaxed);
  }
  kern<<<groups * slots, 512, lds + (size_t)c.M * c.top_k * 2, st>>>(c, groups);
  return hipGetLastError();
}

template <int TY, int TMAX>
hipError_t split_up(const MoeCall& c, int slots, hipStream_t st) {
  constexpr int KS = TMAX == 1 ? 8 : 4;
  k_moe_up<TY, TMAX, KS><<<dim3(c.I / 16, slots), KS * 64,
                           KS * 2 * TMAX * 1024 + (size_t)c.M * c.top_k * 2, st>>>(c);
  return hipGetLastError();
}

template <int TMAX>
hipError_t split_down(const MoeCall& c, int slots, hipStream_t st) {
  constexpr int KS = 4, NB = 2;
  k_moe_down<NB, TMAX, KS><<<dim3((c.K / 16 + NB - 1) / NB, slots), KS * 64,
                             KS * NB * TMAX * 1024 + (size_t)c.M * c.top_k * 2, st>>>(c);
  return hipGetLastError();
}

template <int TY>
hipError_t wide_up(const MoeCall& c, int slots, hipStream_t st) {
  static std::atomic<uint64_t> asked;
  return launch_wide(k_moe_wide<TY, true>, asked, (c.I / 16 + 7) / 8, slots, kWideLds<1>, c, st);
}

inline hipError_t wide_down(const MoeCall& c, int slots, hipStream_t st) {
  static std::atomic<uint64_t> asked;
  return launch_wide(k_moe_wide<kBf16, false>, asked, (c.K / 16 + 15) / 16, slots, kWideLds<2>, c,
                     st);
}

// Whether each pair goes alone: one token, or so few pairs that they seldom
// share an expert, whose weights are then read for each of them (us with and
// without, tokens x columns, expert's width, experts, places: 1x4096 1408 128 8
// 29.5 and 35.7; 2x4096 1408 128 8 53.0 and 61.7; 4x4096 1408 128 8 90.2 and 99.1;
// 8x4096 1408 128 8 168 and 149; 1x5120 8192 8 2 52.9 and 59.5; 2x5120 8192 8 2
// 86.8 and 87.1; 2x2048 768 128 8 22.7 and 27.4).
bool few_pairs(const MoeCall& c) {
  const int P = c.M * c.top_k;
  return P <= kFewPairs && (c.M == 1 || 4 * P <= c.E);
}

template <int TY>
hipError_t run_few(const MoeCall& c, hipStream_t st) {
  const int P = c.M * c.top_k;
  k_moe_up_few<TY><<<dim3(c.I / 16, P), kFewUpWaves * 64, 0, st>>>(c);
  const int parts = P < kFewDownWaves ? kFewDownWaves / P : 1;
  k_moe_down_few<TY><<<c.K / 16, kFewDownWaves * 64, 0, st>>>(c, parts);
  return hipGetLastError();
}

// First product, us of a call in a graph (tokens x columns, expert's width,
// experts, places):
//   up to 4 tokens an expert, or 16 in all: the columns split, 16 tokens at a time,
//     against shared tiles: 64x4096 1408 128 8: 358 and 373, 48x5120 1408 64 6: 231
//     and 253 (96x4096 1408 128 8, 6 tokens an expert: 425 and 401);
//   else shared tiles, where their workgroups are more than half of the CUs,
//     against the columns split and 64 tokens at a time: 364x720 1824 12 5: 137 and
//     157, 385x7008 608 114 4: 368 and 396 (128x4096 512 8 2, 32 workgroups: 66 and 41).
template <int TY>
hipError_t first_product(const MoeCall& c, int slots, hipStream_t st) {
  if (c.M <= 16 || c.M * c.top_k < 5 * c.E) return split_up<TY, 1>(c, slots, st);
  if (2 * (int64_t)slots * ((c.I + 127) / 128) > device_cu_count())
    return wide_up<TY>(c, slots, st);
  return split_up<TY, 4>(c, slots, st);
}

// Second product, the same way:
//   shared tiles, where their workgroups fill the chip once, against the columns
//     split and 16 tokens at a time: 385x7008 608 114 4: 368 and 510, 24x4096 1408
//     128 8: 268 and 279 (32x5120 8192 8 2, 160 workgroups: 201 and 199, 8x5120
//     8192 8 2: 177 and 156);
//   else the columns split: 64 tokens at a time for many tokens an expert, and
//     columns to split, against 16: 364x720 1824 12 5: 137 and 158, 200x256 2816 4
//     2: 70 and 76 (132x1904 144 9 7, two column blocks: 54 and 47).
hipError_t second_product(const MoeCall& c, int slots, hipStream_t st) {
  if ((int64_t)slots * ((c.K + 255) / 256) >= 2 * device_cu_count())
    return wide_down(c, slots, st);
  if (c.M * c.top_k > 64 * slots && c.I >= 8 * kFp8Block) return split_down<4>(c, slots, st);
  return split_down<1>(c, slots, st);
}

template <int TY>
hipError_t run(const MoeCall& c, hipStream_t st) {
  const int P = c.M * c.top_k, slots = P < c.E ? P : c.E;
  if (c.I > 0) {  // else nothing is made, and the sums over the pairs are zeros
    if (few_pairs(c)) return run_few<TY>(c, st);
    hipError_t e = first_product<TY>(c, slots, st);
    if (e == hipSuccess) e = second_product(c, slots, st);
    if (e != hipSuccess) return e;
  }
  k_moe_join<TY><<<(unsigned)(((int64_t)c.M * (c.K / 8) + 255) / 256), 256, 0, st>>>(c);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_moe(const MoeCall& c, hipStream_t st) {
  return c.type == kF16 ? run<kF16>(c, st) : run<kBf16>(c, st);
}

}  // namespace i8mm
