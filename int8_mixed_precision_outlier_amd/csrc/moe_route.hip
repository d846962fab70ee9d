// The router of a mixture of experts (gfx950): logits = X . W^T, a softmax over
// the experts, and the top_k largest of each token.
//
// Which expert comes first is a comparison of numbers that may lie as close as
// they like, so the sums are held in 64 bits: the products of two 16-bit
// numbers are exact in fp32 already, and a choice then changes only where two
// logits agree to about 2^-50.  Equal logits (the same row of W twice) are
// summed in the same order and go to the lower index.
#include "fp8.hpp"
#include "launch.hpp"
#include "moe.hpp"

namespace i8mm {

namespace {

// One wavefront per MT tokens x ET experts; its lanes share the columns.
template <int TY, int MT, int ET>
__global__ __launch_bounds__(256) void k_moe_logits(const uint16_t* __restrict__ X,
                                                    const uint16_t* __restrict__ W, int M, int K,
                                                    int E, int eblocks, double* __restrict__ L) {
  const int lane = threadIdx.x & 63;
  const int64_t tile = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int m0 = (int)(tile / eblocks) * MT, e0 = (int)(tile % eblocks) * ET;
  if (m0 >= M) return;
  double acc[MT][ET];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < ET; ++j) acc[i][j] = 0.0;
  for (int k = lane * 8; k < K; k += 512) {
    float x[MT][8], w[ET][8];
#pragma unroll
    for (int i = 0; i < MT; ++i)  // rows past the end repeat the last one, unused
      unpack8<TY>(*reinterpret_cast<const uint4*>(X + (size_t)min(m0 + i, M - 1) * K + k), x[i]);
#pragma unroll
    for (int j = 0; j < ET; ++j)
      unpack8<TY>(*reinterpret_cast<const uint4*>(W + (size_t)min(e0 + j, E - 1) * K + k), w[j]);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < ET; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[i][j] = fma((double)x[i][e], (double)w[j][e], acc[i][j]);
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < ET; ++j) {
      double v = acc[i][j];
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
      if (lane == 0 && m0 + i < M && e0 + j < E) L[(size_t)(m0 + i) * E + e0 + j] = v;
    }
}

// One wavefront per token, EPL experts per lane (expert i * 64 + lane).
template <int EPL>
__global__ __launch_bounds__(256) void k_moe_topk(const double* __restrict__ L, int M, int E,
                                                  int top_k, int normalize,
                                                  int32_t* __restrict__ experts,
                                                  float* __restrict__ weights) {
  const int lane = threadIdx.x & 63;
  const int m = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (m >= M) return;
  const double* row = L + (size_t)m * E;
  // a NaN ranks with -inf; the weights of its row are all NaN
  double v[EPL], key[EPL];
  double top = -__builtin_inf();
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = i * 64 + lane;
    v[i] = e < E ? row[e] : -__builtin_inf();
    key[i] = v[i] == v[i] ? v[i] : -__builtin_inf();
    top = fmax(top, key[i]);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = fmax(top, __shfl_xor(top, o, kWave));
  // the softmax's differences in 64 bits, its exponentials and sum in fp32
  float total = 0.0f;
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    if (i * 64 + lane < E) total += expf((float)(v[i] - top));
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) total += __shfl_xor(total, o, kWave);
  uint32_t taken = 0;  // bit i: expert i * 64 + lane
  float mine = 0.0f, sum = 0.0f;
  int chosen = 0;
  for (int j = 0; j < top_k; ++j) {
    double best = -__builtin_inf();
    int at = 0x7fffffff;  // no expert: any other precedes it
#pragma unroll
    for (int i = EPL - 1; i >= 0; --i) {
      const int e = i * 64 + lane;
      if (e < E && !(taken >> i & 1u) && (key[i] >= best)) best = key[i], at = e;
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      const double b = __shfl_xor(best, o, kWave);
      const int a = __shfl_xor(at, o, kWave);
      if (b > best || (b == best && a < at)) best = b, at = a;
    }
    if ((at & 63) == lane) taken |= 1u << (at >> 6);
    // the value itself (a NaN stays one) from the lane that holds it
    double raw = v[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i)
      if (i == at >> 6) raw = v[i];
    raw = __shfl(raw, at & 63, kWave);
    const float p = expf((float)(raw - top)) / total;
    sum += p;
    if (lane == j) mine = p, chosen = at;
  }
  if (lane < top_k) {
    experts[(size_t)m * top_k + lane] = chosen;
    weights[(size_t)m * top_k + lane] = normalize ? mine / sum : mine;
  }
}

template <int TY>
hipError_t logits(const RouteCall& c, hipStream_t st) {
  auto go = [&](auto kern, int mt, int et) {
    const int eblocks = (c.E + et - 1) / et;
    const int64_t tiles = (int64_t)((c.M + mt - 1) / mt) * eblocks;
    kern<<<(unsigned)((tiles + 3) / 4), 256, 0, st>>>(c.X, c.W, c.M, c.K, c.E, eblocks, c.logits);
    return hipGetLastError();
  };
  if ((int64_t)c.M * c.E <= 16 * 4 * device_cu_count()) return go(k_moe_logits<TY, 1, 1>, 1, 1);
  return go(k_moe_logits<TY, 4, 4>, 4, 4);
}

}  // namespace

hipError_t launch_moe_route(const RouteCall& c, hipStream_t st) {
  const hipError_t e = c.type == kF16 ? logits<kF16>(c, st) : logits<kBf16>(c, st);
  if (e != hipSuccess) return e;
  const int epl = (c.E + 63) / 64;
  auto kern = epl <= 1   ? k_moe_topk<1>
              : epl <= 2 ? k_moe_topk<2>
              : epl <= 4 ? k_moe_topk<4>
                         : k_moe_topk<16>;
  kern<<<(c.M + 3) / 4, 256, 0, st>>>(c.logits, c.M, c.E, c.top_k, c.normalize, c.experts,
                                      c.weights);
  return hipGetLastError();
}

}  // namespace i8mm
