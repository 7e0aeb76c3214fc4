// Internal interface between the host code of the feed-forward operators (lce_ffn_api.cu) and
// their kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "lce.h"

namespace lce {

// The epilogues of a feed-forward product.  Z = A B^T with A [M x K] and B [Ncols x K].
enum FfnMode : int {
  FFN_LINEAR = 0,     // C = act(Z + bias) + R
  FFN_GATED = 1,      // C = act(Z) * Z2, Z2 = A B2^T
  FFN_LINEAR_DZ = 2,  // C = D * act'(Z + bias)
  FFN_GATED_DGU = 3,  // C = D * Z2 * act'(Z), C2 = D * act(Z)
  FFN_GRADS = 4,      // C = Z, or Z + A2 B2^T (two pairs of operands into one sum)
};

// One product.  Strides in elements; an operand is row-major [rows x K], or with *_t set stored
// as [K x rows] (the contracted index is its row).
struct FfnGemm {
  int mode;
  lce_dtype_t dtype;
  lce_activation_t act;
  int64_t M, Ncols, K;
  const void* A; int64_t lda; bool a_t;
  const void* B; int64_t ldb; bool b_t;
  const void* A2; const void* B2;  // gated: B2 only; FFN_GRADS: the second pair, or null
  const void* bias;                // [Ncols] or null
  const void* R; int64_t ldr;      // FFN_LINEAR: residual, or null
  const void* D; int64_t ldd;      // outgoing gradient [M x Ncols]
  void* C; int64_t ldc;
  void* C2;                        // FFN_GATED_DGU (row stride ldc)
};

// CUDA cores, any mode, type and layout: lce_ffn_simt.cu
cudaError_t launch_ffn_simt(const FfnGemm& g, cudaStream_t stream);
// out[c] = sum over the N rows of x[., c], row stride ld: lce_ffn_simt.cu
cudaError_t launch_column_sum(const void* x, int64_t ld, int64_t N, int64_t cols, lce_dtype_t dtype,
                              void* out, cudaStream_t stream);

}  // namespace lce
