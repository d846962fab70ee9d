// C-ABI layer of the mixture-of-experts operators: argument checks and kernel
// dispatch.  Host code only; it never allocates, frees or synchronizes.  The
// operations are described in include/int8mm.h.
#include "../../include/int8mm.h"
#include "api_internal.hpp"
#include "fp8.hpp"
#include "moe.hpp"

using namespace i8mm;

namespace {

inline bool aligned_to(const void* p, uintptr_t n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

int check_choice(int64_t E, int64_t top_k) {
  if (E < 1 || E > INT8MM_MAX_EXPERTS) return INT8MM_EINVAL;
  return top_k < 1 || top_k > INT8MM_MAX_TOP_K ? INT8MM_EINVAL : INT8MM_OK;
}

int check_route(int64_t M, int64_t K, int64_t E, int64_t top_k) {
  int st = check_rows(INT8MM_F16, M, K, K);
  if (st != INT8MM_OK) return st;
  st = check_choice(E, top_k);
  if (st != INT8MM_OK) return st;
  return top_k > E || M > INT8MM_ROUTE_MAX_TOKENS ? INT8MM_EINVAL : INT8MM_OK;
}

int check_moe(int64_t M, int64_t K, int64_t I, int64_t E, int64_t top_k) {
  int st = check_choice(E, top_k);
  if (st != INT8MM_OK) return st;
  if (M < 0 || M > INT8MM_MOE_MAX_PAIRS || M * top_k > INT8MM_MOE_MAX_PAIRS) return INT8MM_EINVAL;
  if (I < 0 || I > INT8MM_MAX_K) return INT8MM_EINVAL;
  st = check_weight(K, 2 * I);
  return st != INT8MM_OK ? st : check_weight(I, K);
}

}  // namespace

extern "C" {

size_t moe_route_workspace_size(int64_t M, int64_t K, int64_t E, int64_t top_k) {
  if (check_route(M, K, E, top_k) != INT8MM_OK) return 0;
  return moe_align(route_logits_bytes(M, E)) + moe_align(route_bound_bytes(M, K, E));
}

int moe_route(const void* X, const void* W, int type, int64_t M, int64_t K, int64_t E,
              int64_t top_k, int normalize, int32_t* experts, float* weights, void* workspace,
              size_t workspace_bytes, hipStream_t stream) {
  if (type != INT8MM_F16 && type != INT8MM_BF16) return INT8MM_EINVAL;
  const int st = check_route(M, K, E, top_k);
  if (st != INT8MM_OK) return st;
  if (M == 0) return INT8MM_OK;
  if (!experts || !weights || !workspace || (K > 0 && (!X || !W))) return INT8MM_EINVAL;
  if (!aligned16(X) || !aligned16(W) || !aligned_to(experts, 4) || !aligned_to(weights, 4) ||
      !aligned_to(workspace, kMoeAlign))
    return INT8MM_EALIGN;
  if (workspace_bytes < moe_route_workspace_size(M, K, E, top_k)) return INT8MM_EWORKSPACE;
  const RouteCall c{static_cast<const uint16_t*>(X), static_cast<const uint16_t*>(W), experts,
                    weights, static_cast<double*>(workspace),
                    reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) +
                                             moe_align(route_logits_bytes(M, E))),
                    (int)M, (int)K, (int)E, (int)top_k, type, normalize != 0};
  return hip_error_status(launch_moe_route(c, stream));
}

size_t fp8_moe_workspace_size(int64_t M, int64_t K, int64_t I, int64_t E, int64_t top_k) {
  if (check_moe(M, K, I, E, top_k) != INT8MM_OK) return 0;
  return moe_align(moe_act_bytes(M * top_k, I)) + moe_align(moe_part_bytes(M * top_k, K));
}

int fp8_moe(const void* X, int type, int64_t M, int64_t K, const int32_t* experts,
            const float* weights, int64_t top_k, const void* gate_up_f8,
            const float* gate_up_scale, const void* down_f8, const float* down_scale, int64_t I,
            int64_t E, void* Y, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (type != INT8MM_F16 && type != INT8MM_BF16) return INT8MM_EINVAL;
  const int st = check_moe(M, K, I, E, top_k);
  if (st != INT8MM_OK) return st;
  if (M == 0 || K == 0) return INT8MM_OK;
  if (!X || !experts || !weights || !Y || !workspace) return INT8MM_EINVAL;
  if (I > 0 && (!gate_up_f8 || !gate_up_scale || !down_f8 || !down_scale)) return INT8MM_EINVAL;
  if (!aligned16(X) || !aligned_to(experts, 4) || !aligned_to(weights, 4) ||
      !aligned16(gate_up_f8) || !aligned16(gate_up_scale) || !aligned16(down_f8) ||
      !aligned16(down_scale) || !aligned16(Y) || !aligned_to(workspace, kMoeAlign))
    return INT8MM_EALIGN;
  if (workspace_bytes < fp8_moe_workspace_size(M, K, I, E, top_k)) return INT8MM_EWORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const MoeCall c{static_cast<const uint16_t*>(X), experts, weights,
                  static_cast<const uint8_t*>(gate_up_f8), static_cast<const uint8_t*>(down_f8),
                  gate_up_scale, down_scale, static_cast<uint16_t*>(Y), ws,
                  reinterpret_cast<float*>(ws + moe_align(moe_act_bytes(M * top_k, I))),
                  (int)M, (int)K, (int)I, (int)E, (int)top_k, type};
  return hip_error_status(launch_fp8_moe(c, stream));
}

}  // extern "C"
