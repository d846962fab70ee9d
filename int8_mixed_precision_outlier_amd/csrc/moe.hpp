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
  int M, K, E, top_k, type;
  bool normalize;
};
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
