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

// Tiles are addressed with 32-bit coordinates, the last one a tile's width past the end at most; sizes
// of arrays stay far from 64 bits.
constexpr int64_t kMaxDim = (int64_t(1) << 31) - 512;
constexpr int64_t kMaxElements = int64_t(1) << 48;

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
bool sizes_ok(int64_t N, int64_t d, int64_t width, lce_dtype_t dt) {
  return rows_ok(N) && width_ok(d, dt) && width_ok(width, dt) && N * d <= kMaxElements &&
         N * width <= kMaxElements && d * width <= kMaxElements;
}

// Whether a forward product of N tokens runs as a weight stream (lce_ffn_few.cu; fp32:
// lce_ffn_simt.cu) rather than in tiles of 256 tokens (lce_ffn_tc.cu).  us inside a captured graph,
// stream / tiles:
//   linear 128 x 8192 -> 4096 18 / 24, 128 x 5224 -> 13384 45 / 39, 160 x 11008 -> 4096 24 / 30, 192: 28 / 31;
//     160 x 4096 -> 11008 26 / 25: the stream cuts long K loops into more pieces
//   gated 128 x 4096 x 11008 40 / 47, 160: 42 / 47, 192: 49 / 48 (a tile for each of more than half the
//     SMs, no joining); 48 x 4096 x 8192 27 / 27, 96: 32 / 27 (two sums to join per tile);
//     96 x 2048 x 1024 8.7 / 11.9, 128: 22 / 12 (its partial sums no longer fit)
//   fp32 linear 32 x 2048 -> 8192 50 / 65, 48: 64 / 65, 64: 83 / 65, 40 x 4096 -> 4096 69 / 80: up to 48
//     tokens, the crossing of weights that fit in L2.  The stream reads them once per eight tokens, so
//     that larger ones cross at about 34: 6144 -> 16384 with 32 tokens 293 / 322, 40: 390 / 322, 48:
//     471 / 322; 4096 -> 16384 32: 207 / 220, 48: 315 / 220; gated 32 x 6144 -> 16384 583 / 633.  Small products, for
//     which the tiles take about 12 us + 6 per 1000 of d: 64 x 512 -> 1024 4.5 / 14, 256: 14.9 / 14.5,
//     100 x 1024 -> 1024 12.6 / 16.5, 500 x 256 -> 512 10.0 / 12.2, 1000: 17.4 / 12.4, 100 x 6000 -> 512
//     31 / 48; a result costs about as much as 100 more of d (4096 x 128 -> 144 15.9 / 10.0)
bool few_tokens(int64_t N, int64_t d, int64_t width, int weights, lce_dtype_t dt) {
  if (dt == LCE_F32)
    return N <= 48 ||
           (N <= 4096 && static_cast<double>(N) * width * weights * (d + 100) <= 1e8 + 5.6e4 * d);
  if (N <= 32) return true;
  if (weights == 1) return N <= 128 || (N <= FFN_FEW_TOKENS && d >= 2 * width);
  const int64_t tiles = (width + 127) / 128;  // of the stream: feature rows of one CTA
  if (tiles > 76 && tiles <= 152) return N <= FFN_FEW_TOKENS;
  return N <= (tiles <= 16 ? 112 : 48);
}

// Rows of the workspace's arrays start on 128-byte lines.
int64_t round64(int64_t x) { return (x + 63) & ~int64_t(63); }

// Whether a bf16 operand with rows of `width` elements is copied into aligned rows before the products
// read it.  Rows that start between 32-byte sectors cost a K-major operand of the tensor-core kernel a
// third of its rate (10240 x 1672 x 3008: 96 us, 1664 wide 68 us); the copy costs a pass over the
// operands, which pays when every element enters enough products (4096 x 4104 x 4096 forward: 99 us
// with, 116 without; 1024 x 4104 x 4096: 36 with, 32 without).  MN-major operands lose 8% only, and
// rows whose stride is a multiple of 32 bytes but not of 128 lose 10%: they are left alone.
bool misaligned(int64_t width) { return width % 16 != 0; }
bool copy_pays(int64_t N, int64_t width) { return N * width >= 1200 * (N + width); }

// One array of the workspace: bf16, or for LCE_F32 three bf16 parts of it.
struct Slot {
  size_t off;
  int64_t ld, part_stride;
};

// Workspace: header (error flags, scheduler counters), then the copies of X and of the weights that
// the tensor-core kernel reads (LCE_F32: their parts; LCE_BF16: where copy_pays), then the gradients
// of the pre-activations.
struct Layout {
  bool copies;
  Slot x, w[2], z[2];
  size_t total;
};

// k_major: a product contracts X and the weights over d (the forward pass, or pre-activations that are
// recomputed).
Layout layout(int64_t N, int64_t d, int64_t width, int weights, int nz, bool backward, bool k_major,
              lce_dtype_t dt) {
  Layout L{};
  size_t off = WS_HEADER_BYTES;
  auto take = [&](Slot& s, int64_t rows, int64_t cols) {
    s.off = off;
    s.ld = round64(cols);
    s.part_stride = rows * s.ld;
    off += align256(static_cast<size_t>(s.part_stride) * 2 * (dt == LCE_BF16 ? 1 : 3));
  };
  L.copies = (backward || !few_tokens(N, d, width, weights, dt)) &&
             (dt == LCE_F32 || (k_major && misaligned(d) && copy_pays(N, width * weights)));
  if (L.copies) {
    take(L.x, N, d);
    for (int i = 0; i < weights; ++i) take(L.w[i], width, d);
  }
  for (int i = 0; i < nz; ++i) take(L.z[i], N, width);
  L.total = off;
  return L;
}

// Whether dZ has an array of its own in the workspace.  With no activation dZ is dY: read in place,
// or copied like the other operands.
bool own_dz(int64_t N, int64_t d_in, int64_t d_out, lce_activation_t act, lce_dtype_t dt) {
  return act != LCE_ACT_NONE || dt == LCE_F32 || (misaligned(d_out) && copy_pays(N, d_in));
}
Layout linear_layout(int64_t N, int64_t d_in, int64_t d_out, lce_activation_t act, bool backward,
                     lce_dtype_t dt) {
  const int nz = backward && own_dz(N, d_in, d_out, act, dt) ? 1 : 0;
  return layout(N, d_in, d_out, 1, nz, backward, !backward || act != LCE_ACT_NONE, dt);
}
Layout gated_layout(int64_t N, int64_t d, int64_t F, bool backward, lce_dtype_t dt) {
  return layout(N, d, F, 2, backward ? 2 : 0, backward, true, dt);
}

cudaError_t zero(void* p, size_t bytes, cudaStream_t stream) {
  return (p && bytes) ? note(cudaMemsetAsync(p, 0, bytes, stream)) : cudaSuccess;
}

// What the launches of one call share.
struct Call {
  lce_dtype_t dt;
  char* ws;
  int num_sms;
  cudaStream_t stream;
  CallState state{};
  PackArray pack[MAX_PACK_ARRAYS];
  int npack = 0;

  unsigned* flags() const { return reinterpret_cast<unsigned*>(ws); }
  cudaError_t few(int kid, const FfnGemm& g) {
    return traced(kid, stream, [&] {
      return dt == LCE_BF16 ? launch_ffn_few(g, flags(), num_sms, stream)
                            : launch_ffn_few_f32(g, flags(), stream);
    });
  }
  cudaError_t tc(int kid, const FfnTc* jobs, int n) {
    return traced(kid, stream,
                  [&] { return launch_ffn_tc(jobs, n, dt, flags(), &state, num_sms, stream); });
  }
  // x [rows x cols] as an operand of the tensor-core kernel: itself, or its copy in slot s (if there
  // is one), which the next pack_all() writes
  FfnOperand operand(const void* x, int64_t ld, int64_t rows, int64_t cols, const Slot* s) {
    if (dt == LCE_BF16 && (!s || !misaligned(ld))) return FfnOperand{x, rows, cols, ld, 1, 0};
    pack[npack++] = PackArray{x, ld, rows, cols, ws + s->off, s->ld, s->part_stride};
    return own(*s, rows, cols);
  }
  cudaError_t pack_all() {
    if (npack == 0) return cudaSuccess;
    state.flags = state.sched = true;  // the launch clears the header
    return traced(K_PACK, stream,
                  [&] { return launch_pack(pack, npack, dt == LCE_BF16 ? 1 : 3, flags(), stream); });
  }
  // an array of the workspace as an operand
  FfnOperand own(const Slot& s, int64_t rows, int64_t cols) const {
    return FfnOperand{ws + s.off, rows, cols, s.ld, dt == LCE_BF16 ? 1 : 3, s.part_stride};
  }
};

// dX = dZ W (+ dZ2 W2), dW = dZ^T X (and dW2 = dZ2^T X) in one launch, the longer sums first.
// nw = 1 or 2 weights; dX or the dW may be null.
cudaError_t products(Call& c, const FfnOperand& X, const FfnOperand* W, const FfnOperand* Z,
                     int nw, int64_t N, int64_t d, int64_t width, void* dX, void* const* dW) {
  if (!dX && !dW[0]) return cudaSuccess;
  FfnTc jobs[3];
  const bool dx_first = nw * width >= N;
  FfnTc& x = jobs[dx_first ? 0 : nw] = FfnTc{};
  x.M = N; x.Ncols = d; x.K = width;
  x.A = Z[0]; x.B = W[0]; x.b_mn = true;
  if (nw == 2) { x.A2 = Z[1]; x.B2 = W[1]; }
  x.C = dX; x.ldc = d;
  for (int i = 0; i < nw; ++i) {
    FfnTc& w = jobs[dx_first ? i + 1 : i] = FfnTc{};
    w.M = width; w.Ncols = d; w.K = N;
    w.A = Z[i]; w.B = X; w.a_mn = w.b_mn = true;
    w.C = dW[i]; w.ldc = d;
  }
  for (int i = 0; i <= nw; ++i) { jobs[i].mode = FFN_GRADS; jobs[i].act = LCE_ACT_NONE; }
  return c.tc(K_FFN_GRADS, jobs, nw + 1);
}

}  // namespace
}  // namespace lce

using namespace lce;

extern "C" {

size_t lce_linear_workspace_size(int64_t N, int64_t d_in, int64_t d_out, lce_activation_t activation,
                                 int32_t backward, lce_dtype_t dtype) {
  if (!dtype_ok(dtype) || !act_ok(activation) || (backward != 0 && backward != 1)) return 0;
  if (!sizes_ok(N, d_in, d_out, dtype)) return 0;
  return linear_layout(N, d_in, d_out, activation, backward != 0, dtype).total;
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
  if (N == 0)  // otherwise the first launch clears the error flags
    return zero(workspace, WS_HEADER_BYTES, stream) == cudaSuccess ? LCE_OK : LCE_ERR_CUDA;
  Call c{dtype, static_cast<char*>(workspace), num_sms, stream};
  if (few_tokens(N, d_in, d_out, 1, dtype)) {
    FfnGemm g{};
    g.mode = FFN_LINEAR;
    g.act = activation;
    g.M = N; g.Ncols = d_out; g.K = d_in;
    g.A = X; g.lda = ldx; g.B = W; g.ldb = d_in;
    g.bias = bias; g.R = residual; g.ldr = ldr;
    g.C = Y; g.ldc = ldy;
    return c.few(K_LIN, g) == cudaSuccess ? LCE_OK : LCE_ERR_CUDA;
  }
  const Layout L = linear_layout(N, d_in, d_out, activation, false, dtype);
  FfnTc g{};
  g.mode = FFN_LINEAR;
  g.act = activation;
  g.M = N; g.Ncols = d_out; g.K = d_in;
  g.bias = bias; g.R = residual; g.ldr = ldr;
  g.C = Y; g.ldc = ldy;
  g.A = c.operand(X, ldx, N, d_in, L.copies ? &L.x : nullptr);
  g.B = c.operand(W, d_in, d_out, d_in, L.copies ? &L.w[0] : nullptr);
  if (c.pack_all() != cudaSuccess || c.tc(K_LIN, &g, 1) != cudaSuccess) return LCE_ERR_CUDA;
  return LCE_OK;
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
  if (N == 0) {
    if (zero(workspace, WS_HEADER_BYTES, stream) != cudaSuccess) return LCE_ERR_CUDA;
    const size_t e = elem(dtype);
    if (zero(dW, static_cast<size_t>(d_in) * d_out * e, stream) != cudaSuccess ||
        zero(dbias, static_cast<size_t>(d_out) * e, stream) != cudaSuccess)
      return LCE_ERR_CUDA;
    return LCE_OK;
  }
  Call c{dtype, static_cast<char*>(workspace), num_sms, stream};
  const Layout L = linear_layout(N, d_in, d_out, activation, true, dtype);
  const FfnOperand x = c.operand(X, ldx, N, d_in, L.copies ? &L.x : nullptr);
  const FfnOperand w = c.operand(W, d_in, d_out, d_in, L.copies ? &L.w[0] : nullptr);
  const bool none = activation == LCE_ACT_NONE;
  const bool own_z = own_dz(N, d_in, d_out, activation, dtype);
  const FfnOperand z = none ? c.operand(dY, ldy, N, d_out, own_z ? &L.z[0] : nullptr)
                            : c.own(L.z[0], N, d_out);
  if (c.pack_all() != cudaSuccess) return LCE_ERR_CUDA;
  if (!none) {
    FfnTc g{};
    g.mode = FFN_LINEAR_DZ;
    g.act = activation;
    g.M = N; g.Ncols = d_out; g.K = d_in;
    g.A = x; g.B = w;
    g.bias = bias; g.D = dY; g.ldd = ldy;
    g.C = c.ws + L.z[0].off; g.ldc = L.z[0].ld; g.part_stride = L.z[0].part_stride;
    if (c.tc(K_LIN_DZ, &g, 1) != cudaSuccess) return LCE_ERR_CUDA;
  }
  if (dbias && traced(K_COLSUM, stream, [&] {
        return launch_column_sum(z.ptr, z.ld, N, d_out, static_cast<int>(z.parts), z.part_stride,
                                 dbias, stream);
      }) != cudaSuccess)
    return LCE_ERR_CUDA;
  if (products(c, x, &w, &z, 1, N, d_in, d_out, dX, &dW) != cudaSuccess) return LCE_ERR_CUDA;
  // no launch that clears the error flags (dbias alone, or nothing asked for)
  if (!c.state.flags && zero(workspace, WS_HEADER_BYTES, stream) != cudaSuccess) return LCE_ERR_CUDA;
  return LCE_OK;
}

size_t lce_gated_workspace_size(int64_t N, int64_t d, int64_t F, int32_t backward,
                                lce_dtype_t dtype) {
  if (!dtype_ok(dtype) || (backward != 0 && backward != 1)) return 0;
  if (!sizes_ok(N, d, F, dtype)) return 0;
  return gated_layout(N, d, F, backward != 0, dtype).total;
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
  if (N == 0)  // otherwise the first launch clears the error flags
    return zero(workspace, WS_HEADER_BYTES, stream) == cudaSuccess ? LCE_OK : LCE_ERR_CUDA;
  Call c{dtype, static_cast<char*>(workspace), num_sms, stream};
  if (few_tokens(N, d, F, 2, dtype)) {
    FfnGemm g{};
    g.mode = FFN_GATED;
    g.act = activation;
    g.M = N; g.Ncols = F; g.K = d;
    g.A = X; g.lda = ldx; g.B = Wg; g.B2 = Wu; g.ldb = d;
    g.C = H; g.ldc = ldh;
    return c.few(K_GATED, g) == cudaSuccess ? LCE_OK : LCE_ERR_CUDA;
  }
  const Layout L = gated_layout(N, d, F, false, dtype);
  FfnTc g{};
  g.mode = FFN_GATED;
  g.act = activation;
  g.M = N; g.Ncols = F; g.K = d;
  g.C = H; g.ldc = ldh;
  g.A = c.operand(X, ldx, N, d, L.copies ? &L.x : nullptr);
  g.B = c.operand(Wg, d, F, d, L.copies ? &L.w[0] : nullptr);
  g.B2 = c.operand(Wu, d, F, d, L.copies ? &L.w[1] : nullptr);
  if (c.pack_all() != cudaSuccess || c.tc(K_GATED, &g, 1) != cudaSuccess) return LCE_ERR_CUDA;
  return LCE_OK;
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
  if (N == 0) {
    if (zero(workspace, WS_HEADER_BYTES, stream) != cudaSuccess) return LCE_ERR_CUDA;
    const size_t bytes = static_cast<size_t>(d) * F * elem(dtype);
    if (zero(dWg, bytes, stream) != cudaSuccess || zero(dWu, bytes, stream) != cudaSuccess)
      return LCE_ERR_CUDA;
    return LCE_OK;
  }
  Call c{dtype, static_cast<char*>(workspace), num_sms, stream};
  const Layout L = gated_layout(N, d, F, true, dtype);
  const FfnOperand x = c.operand(X, ldx, N, d, L.copies ? &L.x : nullptr);
  const FfnOperand w[2] = {c.operand(Wg, d, F, d, L.copies ? &L.w[0] : nullptr),
                           c.operand(Wu, d, F, d, L.copies ? &L.w[1] : nullptr)};
  const FfnOperand z[2] = {c.own(L.z[0], N, F), c.own(L.z[1], N, F)};
  if (c.pack_all() != cudaSuccess) return LCE_ERR_CUDA;
  FfnTc g{};
  g.mode = FFN_GATED_DGU;
  g.act = activation;
  g.M = N; g.Ncols = F; g.K = d;
  g.A = x; g.B = w[0]; g.B2 = w[1];
  g.D = dH; g.ldd = ldh;
  g.C = c.ws + L.z[0].off; g.C2 = c.ws + L.z[1].off;
  g.ldc = L.z[0].ld; g.part_stride = L.z[0].part_stride;
  if (c.tc(K_GATED_DGU, &g, 1) != cudaSuccess) return LCE_ERR_CUDA;
  void* const dW[2] = {dWg, dWu};
  return products(c, x, w, z, 2, N, d, F, dX, dW) == cudaSuccess ? LCE_OK : LCE_ERR_CUDA;
}

}  // extern "C"
