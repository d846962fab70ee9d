// Host-side pieces of the C-ABI layer shared between its source files.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace i8mm {

// The whole decomposed matmul on a caller-given workspace: argument checks,
// then detection, quantization + gather and the GEMM (or decode) kernel,
// all enqueued on `stream`.  Exactly one of W_f16 and cache is non-null
// (unless the call is a no-op).  Returns an int8mm_status.
int run_mixed(const void* X_f16, int64_t M, int64_t K, const int8_t* W_i8,
              const float* w_absmax, const void* W_f16, const void* cache, int64_t N,
              float alpha, const void* bias_f16, void* Y_f16, void* workspace,
              size_t workspace_bytes, int64_t n_cap, hipStream_t stream);

// INT8MM_OK for hipSuccess; otherwise records the error for
// int8mm_last_hip_error and returns INT8MM_EHIP.
int hip_error_status(hipError_t e);

// Argument checks shared by the e4m3 and the mixture-of-experts functions.
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// Type, sizes and alignment of a rows x K matrix (`width` columns are stored
// per row of the input: K, or 2K for a gated pair).
int check_rows(int type, int64_t rows, int64_t K, int64_t width);
// Sizes of an N x K e4m3 weight.
int check_weight(int64_t K, int64_t N);

}  // namespace i8mm
