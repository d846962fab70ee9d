// C-ABI layer of the block-scaled e4m3 operators: argument checks and kernel
// dispatch.  Host code only; it never allocates, frees or synchronizes.  The
// operations are described in include/int8mm.h.
#include "../../include/int8mm.h"
#include "api_internal.hpp"
#include "fp8.hpp"

#include <math.h>

using namespace i8mm;

namespace i8mm {

int check_rows(int type, int64_t rows, int64_t K, int64_t width) {
  if (type != INT8MM_F16 && type != INT8MM_BF16) return INT8MM_EINVAL;
  if (rows < 0 || K < 0 || K > INT8MM_MAX_K || rows > INT8MM_MAX_MN) return INT8MM_EINVAL;
  if (rows * width > INT8MM_MAX_MN) return INT8MM_EINVAL;
  return K % 16 != 0 ? INT8MM_EALIGN : INT8MM_OK;
}

// N * 128 <= INT8MM_MAX_MN follows from the product's bound where K > 0; it
// keeps N within the kernels' integers and grids where K == 0.
int check_weight(int64_t K, int64_t N) {
  if (K < 0 || K > INT8MM_MAX_K || N < 0 || N > INT8MM_MAX_MN / kFp8Block) return INT8MM_EINVAL;
  if (N * fp8_kpad(K) > INT8MM_MAX_MN) return INT8MM_EINVAL;
  return K % 16 != 0 || N % 16 != 0 ? INT8MM_EALIGN : INT8MM_OK;
}

}  // namespace i8mm

extern "C" {

int64_t fp8_packed_size(int64_t N, int64_t K) {
  return check_weight(K, N) == INT8MM_OK ? N * fp8_kpad(K) : -1;
}

int fp8_quantize_weight(const void* W, int type, int64_t K, int64_t N, void* W_f8, float* w_scale,
                        hipStream_t stream) {
  if (type != INT8MM_F16 && type != INT8MM_BF16) return INT8MM_EINVAL;
  const int st = check_weight(K, N);
  if (st != INT8MM_OK) return st;
  if (K == 0 || N == 0) return INT8MM_OK;
  if (!W || !W_f8 || !w_scale) return INT8MM_EINVAL;
  if (!aligned16(W) || !aligned16(W_f8) || !aligned16(w_scale)) return INT8MM_EALIGN;
  return hip_error_status(
      launch_fp8_quantize_weight(W, type, (int)K, (int)N, W_f8, w_scale, stream));
}

int fp8_pack_weight(const void* src, int64_t N, int64_t K, void* W_f8, hipStream_t stream) {
  const int st = check_weight(K, N);
  if (st != INT8MM_OK) return st;
  if (K == 0 || N == 0) return INT8MM_OK;
  if (!src || !W_f8) return INT8MM_EINVAL;
  if (!aligned16(src) || !aligned16(W_f8)) return INT8MM_EALIGN;
  return hip_error_status(launch_fp8_pack_weight(src, (int)N, (int)K, W_f8, stream));
}

int fp8_quantize(const void* X, int type, int64_t M, int64_t K, void* X_f8, float* x_scale,
                 hipStream_t stream) {
  const int st = check_rows(type, M, K, K);
  if (st != INT8MM_OK) return st;
  if (M == 0 || K == 0) return INT8MM_OK;
  if (!X || !X_f8 || !x_scale) return INT8MM_EINVAL;
  if (!aligned16(X) || !aligned16(X_f8) || !aligned16(x_scale)) return INT8MM_EALIGN;
  return hip_error_status(launch_fp8_quantize(X, type, (int)M, (int)K, X_f8, x_scale, stream));
}

int fp8_rms_norm(const void* X, const void* residual, const void* weight, int type, int64_t M,
                 int64_t K, float eps, void* H, void* X_f8, float* x_scale, hipStream_t stream) {
  const int st = check_rows(type, M, K, K);
  if (st != INT8MM_OK) return st;
  if (!(eps > 0.0f) || isinf(eps)) return INT8MM_EINVAL;
  if (M == 0 || K == 0) return INT8MM_OK;
  if (!X || !weight || !X_f8 || !x_scale || !residual != !H) return INT8MM_EINVAL;
  if (!aligned16(X) || !aligned16(weight) || !aligned16(X_f8) || !aligned16(x_scale) ||
      !aligned16(residual) || !aligned16(H))
    return INT8MM_EALIGN;
  return hip_error_status(launch_fp8_rms_norm(X, residual, weight, type, (int)M, (int)K, eps, H,
                                              X_f8, x_scale, stream));
}

int fp8_sandwich_norm(const void* X, const void* residual, const void* post_weight,
                      const void* pre_weight, const void* gate, int64_t gate_rows,
                      float residual_scale, int type, int64_t M, int64_t K, float eps, void* H,
                      void* Y, void* X_f8, float* x_scale, hipStream_t stream) {
  const int st = check_rows(type, M, K, K);
  if (st != INT8MM_OK) return st;
  if (!(eps > 0.0f) || isinf(eps) || !isfinite(residual_scale)) return INT8MM_EINVAL;
  if (gate_rows < 0 || !gate != !gate_rows) return INT8MM_EINVAL;
  if (gate_rows > 0 && M % gate_rows != 0) return INT8MM_EINVAL;
  if (M == 0 || K == 0) return INT8MM_OK;
  if (!X || !residual || !post_weight || !pre_weight || !H) return INT8MM_EINVAL;
  if (!X_f8 != !x_scale || !Y == !X_f8) return INT8MM_EINVAL;
  if (!aligned16(X) || !aligned16(residual) || !aligned16(post_weight) || !aligned16(pre_weight) ||
      !aligned16(gate) || !aligned16(H) || !aligned16(Y) || !aligned16(X_f8) ||
      !aligned16(x_scale))
    return INT8MM_EALIGN;
  const auto in = [](const void* p) { return static_cast<const uint16_t*>(p); };
  const SandwichCall c{in(X), in(residual), in(post_weight), in(pre_weight), in(gate),
                       static_cast<uint16_t*>(H), static_cast<uint16_t*>(Y),
                       static_cast<uint8_t*>(X_f8), x_scale, (int)M, (int)K,
                       (int)(gate ? M / gate_rows : 1), type, residual_scale, eps};
  return hip_error_status(launch_sandwich_norm(c, stream));
}

int fp8_silu_mul(const void* gate_up, int type, int64_t M, int64_t K, void* A_f8, float* a_scale,
                 hipStream_t stream) {
  const int st = check_rows(type, M, K, 2 * K);
  if (st != INT8MM_OK) return st;
  if (M == 0 || K == 0) return INT8MM_OK;
  if (!gate_up || !A_f8 || !a_scale) return INT8MM_EINVAL;
  if (!aligned16(gate_up) || !aligned16(A_f8) || !aligned16(a_scale)) return INT8MM_EALIGN;
  return hip_error_status(
      launch_fp8_silu_mul(gate_up, type, (int)M, (int)K, A_f8, a_scale, stream));
}

int fp8_matmul(const void* X_f8, const float* x_scale, int64_t M, int64_t K, const void* W_f8,
               const float* w_scale, int64_t N, const void* bias, int type, void* Y,
               hipStream_t stream) {
  int st = check_rows(type, M, K, K);
  if (st != INT8MM_OK) return st;
  st = check_weight(K, N);
  if (st != INT8MM_OK) return st;
  if (M * N > INT8MM_MAX_MN) return INT8MM_EINVAL;
  if (M == 0 || N == 0) return INT8MM_OK;
  if (!Y || (K > 0 && (!X_f8 || !x_scale || !W_f8 || !w_scale))) return INT8MM_EINVAL;
  if (!aligned16(Y) || !aligned16(bias) ||
      (K > 0 && (!aligned16(X_f8) || !aligned16(x_scale) || !aligned16(W_f8) || !aligned16(w_scale))))
    return INT8MM_EALIGN;
  const Fp8Call c{static_cast<const uint8_t*>(X_f8), x_scale,
                  static_cast<const uint8_t*>(W_f8), w_scale,
                  static_cast<const uint16_t*>(bias), static_cast<uint16_t*>(Y),
                  (int)M, (int)N, (int)K, type};
  return hip_error_status(launch_fp8_matmul(c, stream));
}

int fp8_matmul_config(int64_t M, int64_t N, int64_t K, int32_t* cfg) {
  int st = check_rows(INT8MM_F16, M, K, K);
  if (st != INT8MM_OK) return st;
  st = check_weight(K, N);
  if (st != INT8MM_OK) return st;
  if (!cfg || M == 0 || N == 0 || M * N > INT8MM_MAX_MN) return INT8MM_EINVAL;
  struct Tile {
    int32_t bm, bn, stages;
  };
  static constexpr Tile kTiles[] = {{256, 256, 2}, {256, 128, 3}, {128, 128, 2}, {128, 128, 4},
                                    {64, 128, 4}};
  const Fp8Plan p = fp8_plan((int)M, (int)N);
  if (p.first == kDecode) {
    const Fp8DecodePlan d = fp8_decode_plan((int)M, (int)N);
    cfg[0] = 0, cfg[1] = d.R, cfg[2] = d.T, cfg[3] = 0;
  } else if (p.n1 >= N) {
    const Tile t = kTiles[p.first];
    cfg[0] = 1, cfg[1] = t.bm, cfg[2] = t.bn, cfg[3] = t.stages;
  } else {
    const Tile t = kTiles[p.second];
    cfg[0] = 2, cfg[1] = p.n1, cfg[2] = t.bm, cfg[3] = t.stages;
  }
  return INT8MM_OK;
}

}  // extern "C"
