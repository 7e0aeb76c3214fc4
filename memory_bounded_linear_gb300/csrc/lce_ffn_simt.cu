// CUDA-core kernels of the feed-forward operators: fp32 products of a few tokens, column sums
// (dbias), and the split of fp32 operands into bf16 parts.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "bf16_parts.cuh"
#include "lce_act.cuh"
#include "lce_ffn.h"
#include "lce_internal.h"

namespace lce {
namespace {

// ---------------------------------------------------------------- fp32 products of a few tokens
// Bound by reading the weights once (HBM).  A block computes ROWS features (of Wg and Wu both, when
// gated) for NT tokens; its eight warps take 512-byte pieces of K in turn, lanes four elements each,
// and each weight vector loaded serves NT tokens from registers (X comes from L1/L2).  The lanes'
// sums meet by shuffles, the warps' in shared memory, in a fixed order.
constexpr int WARPS = 8;
constexpr int ROWS = 4;

template <int NT, bool GATED>
__global__ void __launch_bounds__(WARPS * 32) few_f32_kernel(const FfnGemm g,
                                                             unsigned* err) {
  constexpr int R = GATED ? 2 * ROWS : ROWS;
  __shared__ float sh[WARPS][R * NT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *err = 0u;  // this kernel never waits
  const int64_t f0 = static_cast<int64_t>(blockIdx.x) * ROWS;
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * NT;
  const float* X = static_cast<const float*>(g.A);
  const float* w[R];
  const float* x[NT];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    // features and tokens past the end repeat the last one; their results are dropped
    const int64_t f = min(f0 + r % ROWS, g.Ncols - 1);
    w[r] = static_cast<const float*>(r < ROWS ? g.B : g.B2) + f * g.ldb;
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) x[t] = X + min(t0 + t, g.M - 1) * g.lda;
  float acc[R][NT] = {};
  for (int64_t k = (warp * 32 + lane) * 4; k < g.K; k += WARPS * 128) {
    float4 wv[R];
#pragma unroll
    for (int r = 0; r < R; ++r) wv[r] = __ldcs(reinterpret_cast<const float4*>(w[r] + k));
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float4 xv = __ldg(reinterpret_cast<const float4*>(x[t] + k));
#pragma unroll
      for (int r = 0; r < R; ++r)
        acc[r][t] = fmaf(wv[r].x, xv.x, fmaf(wv[r].y, xv.y, fmaf(wv[r].z, xv.z, fmaf(wv[r].w, xv.w, acc[r][t]))));
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float v = acc[r][t];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == 0) sh[warp][r * NT + t] = v;
    }
  __syncthreads();
  const int i = threadIdx.x;  // one result per thread
  if (i >= ROWS * NT) return;
  const int r = i % ROWS, t = i / ROWS;
  const int64_t f = f0 + r, m = t0 + t;
  if (f >= g.Ncols || m >= g.M) return;
  float z = 0.f, u = 0.f;
#pragma unroll
  for (int k = 0; k < WARPS; ++k) {
    z += sh[k][r * NT + t];
    if (GATED) u += sh[k][(ROWS + r) * NT + t];
  }
  float v;
  dispatch_act(g.act, [&](auto tag) {
    constexpr int ACT = decltype(tag)::value;
    if (GATED) {
      v = act<ACT, false>(z) * u;
    } else {
      if (g.bias) z += static_cast<const float*>(g.bias)[f];
      v = act<ACT, false>(z);
      if (g.R) v += static_cast<const float*>(g.R)[m * g.ldr + f];
    }
  });
  static_cast<float*>(g.C)[m * g.ldc + f] = v;
}

template <bool GATED>
cudaError_t few_f32(const FfnGemm& g, unsigned* err, cudaStream_t stream) {
  const unsigned bx = static_cast<unsigned>((g.Ncols + ROWS - 1) / ROWS);
  const auto by = [&](int nt) { return dim3(bx, static_cast<unsigned>((g.M + nt - 1) / nt)); };
  if (g.M == 1) few_f32_kernel<1, GATED><<<by(1), WARPS * 32, 0, stream>>>(g, err);
  else if (g.M == 2) few_f32_kernel<2, GATED><<<by(2), WARPS * 32, 0, stream>>>(g, err);
  else if (g.M <= 4) few_f32_kernel<4, GATED><<<by(4), WARPS * 32, 0, stream>>>(g, err);
  else few_f32_kernel<8, GATED><<<by(8), WARPS * 32, 0, stream>>>(g, err);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------- column sums
// One thread per column, rows in order.
template <typename E, int PARTS, typename O>
__global__ void column_sum_kernel(const E* x, int64_t ld, int64_t part_stride, int64_t N, int64_t cols,
                                  O* out) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (c >= cols) return;
  float s = 0.f;
  for (int64_t r = 0; r < N; ++r) {
    float v = 0.f;
#pragma unroll
    for (int k = PARTS - 1; k >= 0; --k) v += static_cast<float>(x[k * part_stride + r * ld + c]);
    s += v;
  }
  out[c] = static_cast<O>(s);
}

// fp32 rows into bf16 parts, four columns per thread.
__global__ void split_bf16_kernel(const float* x, int64_t ld, int64_t rows, int64_t cols,
                                  __nv_bfloat16* out, int64_t ld_out, int64_t part_stride) {
  const int64_t c4 = cols / 4;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < rows * c4;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t r = i / c4, c = (i - r * c4) * 4;
    const float4 v = *reinterpret_cast<const float4*>(x + r * ld + c);
    float p[4][3];
    split_bf16(v.x, p[0]);
    split_bf16(v.y, p[1]);
    split_bf16(v.z, p[2]);
    split_bf16(v.w, p[3]);
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      __nv_bfloat162 h[2] = {__floats2bfloat162_rn(p[0][k], p[1][k]),
                             __floats2bfloat162_rn(p[2][k], p[3][k])};
      *reinterpret_cast<uint2*>(out + k * part_stride + r * ld_out + c) =
          *reinterpret_cast<uint2*>(h);
    }
  }
}

}  // namespace

cudaError_t launch_ffn_few_f32(const FfnGemm& g, unsigned* err, cudaStream_t stream) {
  return g.mode == FFN_GATED ? few_f32<true>(g, err, stream) : few_f32<false>(g, err, stream);
}

cudaError_t launch_column_sum(const void* x, int64_t ld, int64_t N, int64_t cols, int parts,
                              int64_t part_stride, void* out, cudaStream_t stream) {
  const unsigned blocks = static_cast<unsigned>((cols + 127) / 128);
  const __nv_bfloat16* h = static_cast<const __nv_bfloat16*>(x);
  if (parts == 3)
    column_sum_kernel<__nv_bfloat16, 3><<<blocks, 128, 0, stream>>>(h, ld, part_stride, N, cols,
                                                                    static_cast<float*>(out));
  else
    column_sum_kernel<__nv_bfloat16, 1>
        <<<blocks, 128, 0, stream>>>(h, ld, 0, N, cols, static_cast<__nv_bfloat16*>(out));
  return cudaGetLastError();
}

cudaError_t launch_split_bf16(const float* x, int64_t ld, int64_t rows, int64_t cols, void* out,
                              int64_t ld_out, int64_t part_stride, cudaStream_t stream) {
  const int64_t need = (rows * (cols / 4) + 255) / 256;
  const unsigned blocks = static_cast<unsigned>(need < 152 * 16 ? need : 152 * 16);
  split_bf16_kernel<<<blocks, 256, 0, stream>>>(x, ld, rows, cols, static_cast<__nv_bfloat16*>(out),
                                                ld_out, part_stride);
  return cudaGetLastError();
}

}  // namespace lce
