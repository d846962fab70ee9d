// Mixture-of-experts operators: the router (moe_route.hip) and the experts'
// gated feed-forward for few tokens (moe_experts.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace i8mm {

// Workspace fields start at multiples of this.
constexpr size_t kMoeAlign = 256;
constexpr size_t moe_align(size_t n) { return (n + kMoeAlign - 1) / kMoeAlign * kMoeAlign; }

struct RouteCall {
  const uint16_t *X, *W;
  int32_t* experts;
  float* weights;
  double* logits;  // workspace: [M][E]
  float* bound;    // workspace: [M][E], what a logit may be off
  int M, K, E, top_k, type;
  bool normalize;
};
// Whether the logits come from matrix instructions: above 2^25 products (us,
// calls in a graph, each sum in 64 bits and by matrix instructions: 77x5136 of 61
// experts 13.0 and 15.1, 64x4096 of 128 14.0 and 17.7, 128x4096 of 128 20.5 and
// 17.8, 512x4096 of 128 56.2 and 20.5).
inline bool route_by_tiles(int64_t M, int64_t K, int64_t E) { return M * E * K > (1 << 25); }
inline size_t route_logits_bytes(int64_t M, int64_t E) { return (size_t)M * E * sizeof(double); }
inline size_t route_bound_bytes(int64_t M, int64_t K, int64_t E) {
  return route_by_tiles(M, K, E) ? (size_t)M * E * sizeof(float) : 0;
}
hipError_t launch_moe_route(const RouteCall& c, hipStream_t st);

// A (token, place) pair p = m * top_k + j has the expert experts[p]; a pair
// whose expert is not one of 0 .. E-1 contributes nothing.
struct MoeCall {
  const uint16_t* X;
  const int32_t* experts;
  const float* weights;
  const uint8_t *up, *down;  // packed, expert after expert
  const float *up_scale, *down_scale;
  uint16_t* Y;
  uint8_t* act;  // workspace: [pairs][I] of the gated product, two bf16 each
  float* part;   // workspace: [pairs][K] of the second product
  int M, K, I, E, top_k, type;
};
inline size_t moe_act_bytes(int64_t pairs, int64_t I) { return (size_t)pairs * I * 4; }
inline size_t moe_part_bytes(int64_t pairs, int64_t K) { return (size_t)pairs * K * 4; }
hipError_t launch_fp8_moe(const MoeCall& c, hipStream_t st);

}  // namespace i8mm
