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

// A forward product of a few tokens (FFN_LINEAR or FFN_GATED): A is X [M x K], B (and B2) the weights
// [Ncols x K], all row-major with strides in elements.
struct FfnGemm {
  int mode;
  lce_activation_t act;
  int64_t M, Ncols, K;
  const void* A; int64_t lda;
  const void* B; const void* B2; int64_t ldb;
  const void* bias;                // [Ncols] or null
  const void* R; int64_t ldr;      // residual, or null
  void* C; int64_t ldc;
};

// An operand of the tensor-core kernel as it is stored: bf16 rows of stored_cols elements, ld
// elements apart; for fp32 three such arrays (the bf16 parts), part_stride elements apart.
struct FfnOperand {
  const void* ptr;
  int64_t stored_rows, stored_cols, ld;
  int64_t parts, part_stride;
};

// One product for the tensor-core kernel.  a_mn / b_mn: stored [K x rows]; A2, B2: the second weights
// (gated), or a second pair of operands summed into the same product (FFN_GRADS; ptr null: none).
// For LCE_F32 the pre-activation gradients C and C2 are written as bf16 parts (row stride ldc,
// part_stride apart), and C of the other modes as fp32.
struct FfnTc {
  int mode;
  lce_activation_t act;
  int64_t M, Ncols, K;
  FfnOperand A, B, A2, B2;
  bool a_mn, b_mn;
  const void* bias;
  const void* R; int64_t ldr;
  const void* D; int64_t ldd;
  void* C; int64_t ldc;
  void* C2;
  int64_t part_stride;
};

// What a call knows to be zero in the workspace header, updated by each launch.
struct CallState {
  bool flags = false;  // the error flags
  bool sched = false;  // the scheduler counters
};

// Tensor cores: lce_ffn_tc.cu.  Several jobs only for FFN_GRADS, where a job whose C is null is not
// computed but counted when the launch is planned; header: the workspace header.
cudaError_t launch_ffn_tc(const FfnTc* jobs, int njobs, lce_dtype_t dtype, unsigned* header,
                          CallState* state, int num_sms, cudaStream_t stream);
// Copies of x [rows x cols], row stride ld, for several arrays: fp32 into three bf16 parts (parts = 3)
// of row stride ld_out, part_stride apart, or bf16 into rows of stride ld_out (parts = 1).  Clears the
// workspace header: lce_ffn_simt.cu
struct PackArray {
  const void* x;
  int64_t ld, rows, cols;
  void* out;
  int64_t ld_out, part_stride;
};
constexpr int MAX_PACK_ARRAYS = 3;
cudaError_t launch_pack(const PackArray* arrays, int count, int parts, unsigned* header,
                        cudaStream_t stream);
// Few tokens, bf16 (at most FFN_FEW_TOKENS rows): lce_ffn_few.cu.  Clears the error flags.
constexpr int64_t FFN_FEW_TOKENS = 160;
cudaError_t launch_ffn_few(const FfnGemm& g, unsigned* err, int num_sms, cudaStream_t stream);
// Few tokens, fp32: lce_ffn_simt.cu.  Clears the error flags.
cudaError_t launch_ffn_few_f32(const FfnGemm& g, unsigned* err, cudaStream_t stream);
// out[c] = sum over the N rows of x[., c], row stride ld.  parts = 1: x and out bf16; parts = 3: x
// holds three bf16 parts, part_stride apart, and out is fp32: lce_ffn_simt.cu
cudaError_t launch_column_sum(const void* x, int64_t ld, int64_t N, int64_t cols, int parts,
                              int64_t part_stride, void* out, cudaStream_t stream);

}  // namespace lce
