// C ABI of the feed-forward operators (declared in include/lce.h): argument checks, workspace
// layout and the order of their launches.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "lce.h"
#include "lce_ffn.h"
#include "lce_internal.h"

namespace lce {
namespace {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t elem(lce_dtype_t dt) { return dt == LCE_BF16 ? 2 : 4; }

bool dtype_ok(lce_dtype_t dt) { return dt == LCE_BF16 || dt == LCE_F32; }
bool act_ok(lce_activation_t a) { return a >= LCE_ACT_NONE && a <= LCE_ACT_GELU_TANH; }
// A width (or row stride): whole 16-byte rows.
bool width_ok(int64_t w, lce_dtype_t dt) {
  const int64_t mult = (dt == LCE_BF16) ? 8 : 4;
  return w >= mult && w % mult == 0 && w <= kMaxDim;
}
bool rows_ok(int64_t N) { return N >= 0 && N <= kMaxDim; }

// Workspace: header (error flags), then the gradients of the pre-activations [N x width] each.
struct Layout {
  size_t off_z[2];
  size_t total;
};

Layout layout(int64_t N, int64_t width, int nz, lce_dtype_t dt) {
  Layout L{};
  size_t off = WS_HEADER_BYTES;
  for (int i = 0; i < nz; ++i) {
    L.off_z[i] = off;
    off += align256(static_cast<size_t>(N) * static_cast<size_t>(width) * elem(dt));
  }
  L.total = off;
  return L;
}

cudaError_t gemm(int kid, const FfnGemm& g, cudaStream_t stream) {
  if (g.M == 0) return cudaSuccess;
  return traced(kid, stream, [&] { return launch_ffn_simt(g, stream); });
}

cudaError_t zero(void* p, size_t bytes, cudaStream_t stream) {
  return (p && bytes) ? note(cudaMemsetAsync(p, 0, bytes, stream)) : cudaSuccess;
}

// dX = dZ W (+ dZ2 W2) and dW = dZ^T X (and dW2 = dZ2^T X) for dZ [N x width] with row stride ldz.
lce_status_t products(const void* X, int64_t ldx, const void* W, const void* W2, const void* dZ,
                      const void* dZ2, int64_t ldz, int64_t N, int64_t d, int64_t width,
                      lce_dtype_t dt, void* dX, void* dW, void* dW2, cudaStream_t stream) {
  FfnGemm g{};
  g.mode = FFN_GRADS;
  g.dtype = dt;
  g.act = LCE_ACT_NONE;
  for (int i = 0; i < (dW2 ? 2 : 1); ++i) {
    if (!dW) break;
    g.M = width; g.Ncols = d; g.K = N;
    g.A = i ? dZ2 : dZ; g.lda = ldz; g.a_t = true;
    g.B = X; g.ldb = ldx; g.b_t = true;
    g.C = i ? dW2 : dW; g.ldc = d;
    if (gemm(K_FFN_GRADS, g, stream) != cudaSuccess) return LCE_ERR_CUDA;
  }
  if (dX) {
    g.M = N; g.Ncols = d; g.K = width;
    g.A = dZ; g.lda = ldz; g.a_t = false;
    g.B = W; g.ldb = d; g.b_t = true;
    g.A2 = dZ2; g.B2 = W2;
    g.C = dX; g.ldc = d;
    if (gemm(K_FFN_GRADS, g, stream) != cudaSuccess) return LCE_ERR_CUDA;
  }
  return LCE_OK;
}

}  // namespace
}  // namespace lce

using namespace lce;

extern "C" {

size_t lce_linear_workspace_size(int64_t N, int64_t d_in, int64_t d_out, lce_activation_t activation,
                                 int32_t backward, lce_dtype_t dtype) {
  if (!dtype_ok(dtype) || !act_ok(activation) || (backward != 0 && backward != 1)) return 0;
  if (!rows_ok(N) || !width_ok(d_in, dtype) || !width_ok(d_out, dtype)) return 0;
  return layout(N, d_out, (backward && activation != LCE_ACT_NONE) ? 1 : 0, dtype).total;
}

lce_status_t lce_linear_forward(const void* X, int64_t ldx, const void* W, const void* bias,
                                const void* residual, int64_t ldr, int64_t N, int64_t d_in,
                                int64_t d_out, lce_activation_t activation, lce_dtype_t dtype,
                                void* Y, int64_t ldy, void* workspace, size_t ws_bytes,
                                void* stream_) {
  if (!dtype_ok(dtype) || !act_ok(activation)) return LCE_ERR_INVALID_ARG;
  if (!W || !workspace || (N > 0 && (!X || !Y))) return LCE_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(W) || !aligned16(bias) || !aligned16(residual) || !aligned16(Y) ||
      !aligned16(workspace))
    return LCE_ERR_INVALID_ARG;
  const size_t need = lce_linear_workspace_size(N, d_in, d_out, activation, 0, dtype);
  if (need == 0 || !width_ok(ldx, dtype) || ldx < d_in || !width_ok(ldy, dtype) || ldy < d_out ||
      (residual && (!width_ok(ldr, dtype) || ldr < d_out)))
    return LCE_ERR_UNSUPPORTED_SHAPE;
  if (N > 0 && (Y == X || Y == W || (Y == residual && ldr != ldy))) return LCE_ERR_INVALID_ARG;
  if (ws_bytes < need) return LCE_ERR_WORKSPACE_TOO_SMALL;
  int num_sms = 0;
  lce_status_t st = check_device(&num_sms);
  if (st != LCE_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (zero(workspace, WS_HEADER_BYTES, stream) != cudaSuccess) return LCE_ERR_CUDA;
  FfnGemm g{};
  g.mode = FFN_LINEAR;
  g.dtype = dtype; g.act = activation;
  g.M = N; g.Ncols = d_out; g.K = d_in;
  g.A = X; g.lda = ldx; g.B = W; g.ldb = d_in;
  g.bias = bias; g.R = residual; g.ldr = ldr;
  g.C = Y; g.ldc = ldy;
  return gemm(K_LIN, g, stream) == cudaSuccess ? LCE_OK : LCE_ERR_CUDA;
}

lce_status_t lce_linear_backward(const void* X, int64_t ldx, const void* W, const void* bias,
                                 const void* dY, int64_t ldy, int64_t N, int64_t d_in,
                                 int64_t d_out, lce_activation_t activation, lce_dtype_t dtype,
                                 void* dX, void* dW, void* dbias, void* workspace,
                                 size_t ws_bytes, void* stream_) {
  if (!dtype_ok(dtype) || !act_ok(activation)) return LCE_ERR_INVALID_ARG;
  if (!W || !workspace || (N > 0 && (!X || !dY))) return LCE_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(W) || !aligned16(bias) || !aligned16(dY) || !aligned16(dX) ||
      !aligned16(dW) || !aligned16(dbias) || !aligned16(workspace))
    return LCE_ERR_INVALID_ARG;
  const size_t need = lce_linear_workspace_size(N, d_in, d_out, activation, 1, dtype);
  if (need == 0 || !width_ok(ldx, dtype) || ldx < d_in || !width_ok(ldy, dtype) || ldy < d_out)
    return LCE_ERR_UNSUPPORTED_SHAPE;
  if (ws_bytes < need) return LCE_ERR_WORKSPACE_TOO_SMALL;
  int num_sms = 0;
  lce_status_t st = check_device(&num_sms);
  if (st != LCE_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (zero(workspace, WS_HEADER_BYTES, stream) != cudaSuccess) return LCE_ERR_CUDA;
  if (N == 0) {
    const size_t e = elem(dtype);
    if (zero(dW, static_cast<size_t>(d_in) * d_out * e, stream) != cudaSuccess ||
        zero(dbias, static_cast<size_t>(d_out) * e, stream) != cudaSuccess)
      return LCE_ERR_CUDA;
    return LCE_OK;
  }
  const void* dZ = dY;
  int64_t ldz = ldy;
  if (activation != LCE_ACT_NONE) {
    const Layout L = layout(N, d_out, 1, dtype);
    void* z = static_cast<char*>(workspace) + L.off_z[0];
    FfnGemm g{};
    g.mode = FFN_LINEAR_DZ;
    g.dtype = dtype; g.act = activation;
    g.M = N; g.Ncols = d_out; g.K = d_in;
    g.A = X; g.lda = ldx; g.B = W; g.ldb = d_in;
    g.bias = bias; g.D = dY; g.ldd = ldy;
    g.C = z; g.ldc = d_out;
    if (gemm(K_LIN_DZ, g, stream) != cudaSuccess) return LCE_ERR_CUDA;
    dZ = z;
    ldz = d_out;
  }
  if (dbias && traced(K_COLSUM, stream, [&] {
        return launch_column_sum(dZ, ldz, N, d_out, dtype, dbias, stream);
      }) != cudaSuccess)
    return LCE_ERR_CUDA;
  return products(X, ldx, W, nullptr, dZ, nullptr, ldz, N, d_in, d_out, dtype, dX, dW, nullptr,
                  stream);
}

size_t lce_gated_workspace_size(int64_t N, int64_t d, int64_t F, int32_t backward,
                                lce_dtype_t dtype) {
  if (!dtype_ok(dtype) || (backward != 0 && backward != 1)) return 0;
  if (!rows_ok(N) || !width_ok(d, dtype) || !width_ok(F, dtype)) return 0;
  return layout(N, F, backward ? 2 : 0, dtype).total;
}

lce_status_t lce_gated_forward(const void* X, int64_t ldx, const void* Wg, const void* Wu, int64_t N,
                               int64_t d, int64_t F, lce_activation_t activation,
                               lce_dtype_t dtype, void* H, int64_t ldh, void* workspace,
                               size_t ws_bytes, void* stream_) {
  if (!dtype_ok(dtype) || !act_ok(activation)) return LCE_ERR_INVALID_ARG;
  if (!Wg || !Wu || !workspace || (N > 0 && (!X || !H))) return LCE_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(Wg) || !aligned16(Wu) || !aligned16(H) || !aligned16(workspace))
    return LCE_ERR_INVALID_ARG;
  const size_t need = lce_gated_workspace_size(N, d, F, 0, dtype);
  if (need == 0 || !width_ok(ldx, dtype) || ldx < d || !width_ok(ldh, dtype) || ldh < F)
    return LCE_ERR_UNSUPPORTED_SHAPE;
  if (N > 0 && (H == X || H == Wg || H == Wu)) return LCE_ERR_INVALID_ARG;
  if (ws_bytes < need) return LCE_ERR_WORKSPACE_TOO_SMALL;
  int num_sms = 0;
  lce_status_t st = check_device(&num_sms);
  if (st != LCE_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (zero(workspace, WS_HEADER_BYTES, stream) != cudaSuccess) return LCE_ERR_CUDA;
  FfnGemm g{};
  g.mode = FFN_GATED;
  g.dtype = dtype; g.act = activation;
  g.M = N; g.Ncols = F; g.K = d;
  g.A = X; g.lda = ldx; g.B = Wg; g.B2 = Wu; g.ldb = d;
  g.C = H; g.ldc = ldh;
  return gemm(K_GATED, g, stream) == cudaSuccess ? LCE_OK : LCE_ERR_CUDA;
}

lce_status_t lce_gated_backward(const void* X, int64_t ldx, const void* Wg, const void* Wu,
                                const void* dH, int64_t ldh, int64_t N, int64_t d, int64_t F,
                                lce_activation_t activation, lce_dtype_t dtype, void* dX, void* dWg,
                                void* dWu, void* workspace, size_t ws_bytes, void* stream_) {
  if (!dtype_ok(dtype) || !act_ok(activation)) return LCE_ERR_INVALID_ARG;
  if (!Wg || !Wu || !workspace || (N > 0 && (!X || !dH)) || (!dWg != !dWu))
    return LCE_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(Wg) || !aligned16(Wu) || !aligned16(dH) || !aligned16(dX) ||
      !aligned16(dWg) || !aligned16(dWu) || !aligned16(workspace))
    return LCE_ERR_INVALID_ARG;
  const size_t need = lce_gated_workspace_size(N, d, F, 1, dtype);
  if (need == 0 || !width_ok(ldx, dtype) || ldx < d || !width_ok(ldh, dtype) || ldh < F)
    return LCE_ERR_UNSUPPORTED_SHAPE;
  if (ws_bytes < need) return LCE_ERR_WORKSPACE_TOO_SMALL;
  int num_sms = 0;
  lce_status_t st = check_device(&num_sms);
  if (st != LCE_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (zero(workspace, WS_HEADER_BYTES, stream) != cudaSuccess) return LCE_ERR_CUDA;
  if (N == 0) {
    const size_t bytes = static_cast<size_t>(d) * F * elem(dtype);
    if (zero(dWg, bytes, stream) != cudaSuccess || zero(dWu, bytes, stream) != cudaSuccess)
      return LCE_ERR_CUDA;
    return LCE_OK;
  }
  const Layout L = layout(N, F, 2, dtype);
  char* ws = static_cast<char*>(workspace);
  FfnGemm g{};
  g.mode = FFN_GATED_DGU;
  g.dtype = dtype; g.act = activation;
  g.M = N; g.Ncols = F; g.K = d;
  g.A = X; g.lda = ldx; g.B = Wg; g.B2 = Wu; g.ldb = d;
  g.D = dH; g.ldd = ldh;
  g.C = ws + L.off_z[0]; g.C2 = ws + L.off_z[1]; g.ldc = F;
  if (gemm(K_GATED_DGU, g, stream) != cudaSuccess) return LCE_ERR_CUDA;
  return products(X, ldx, Wg, Wu, g.C, g.C2, F, N, d, F, dtype, dX, dWg, dWu, stream);
}

}  // extern "C"
