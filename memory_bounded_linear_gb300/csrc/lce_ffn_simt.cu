// Feed-forward products on the CUDA cores: one kernel for every mode, type and operand layout.
// A block computes a 64 x 64 tile of Z (and of Z2) with 4 x 4 outputs per thread, k-blocks of 16
// through shared memory, fp32 FMA; the epilogue is elementwise on the accumulators.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "bf16_parts.cuh"
#include "lce_act.cuh"
#include "lce_ffn.h"
#include "lce_internal.h"

namespace lce {
namespace {

constexpr int T = 64, KB = 16;

template <typename E>
__device__ __forceinline__ float ld(const void* p, int64_t i) {
  return static_cast<float>(static_cast<const E*>(p)[i]);
}

template <typename E, int MODE>
__global__ void __launch_bounds__(256) ffn_simt_kernel(const FfnGemm g) {
  constexpr bool DUAL = MODE == FFN_GATED || MODE == FFN_GATED_DGU;
  constexpr bool FAST = sizeof(E) == 2;
  __shared__ float sa[KB][T + 4], sb[KB][T + 4], sb2[DUAL ? KB : 1][T + 4];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * T, n0 = static_cast<int64_t>(blockIdx.y) * T;
  float z[4][4] = {}, z2[4][4] = {};
  const int pairs = (MODE == FFN_GRADS && g.A2) ? 2 : 1;
  for (int pair = 0; pair < pairs; ++pair) {
    const void* A = pair ? g.A2 : g.A;
    const void* B = pair ? g.B2 : g.B;
    for (int64_t k0 = 0; k0 < g.K; k0 += KB) {
      for (int i = threadIdx.x; i < T * KB; i += 256) {
        // neighbouring threads walk the operand's contiguous index
        const int ka = g.a_t ? i / T : i % KB, ra = g.a_t ? i % T : i / KB;
        const int64_t m = m0 + ra, k = k0 + ka;
        sa[ka][ra] = (m < g.M && k < g.K) ? ld<E>(A, g.a_t ? k * g.lda + m : m * g.lda + k) : 0.f;
        const int kb = g.b_t ? i / T : i % KB, rb = g.b_t ? i % T : i / KB;
        const int64_t n = n0 + rb, kk = k0 + kb;
        const bool ok = n < g.Ncols && kk < g.K;
        const int64_t off = g.b_t ? kk * g.ldb + n : n * g.ldb + kk;
        sb[kb][rb] = ok ? ld<E>(B, off) : 0.f;
        if (DUAL) sb2[kb][rb] = ok ? ld<E>(g.B2, off) : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < KB; ++k) {
        float a[4], b[4], b2[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = sa[k][ty * 4 + i];
          b[i] = sb[k][tx * 4 + i];
          if (DUAL) b2[i] = sb2[k][tx * 4 + i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            z[i][j] = fmaf(a[i], b[j], z[i][j]);
            if (DUAL) z2[i][j] = fmaf(a[i], b2[j], z2[i][j]);
          }
      }
      __syncthreads();
    }
  }
  E* C = static_cast<E*>(g.C);
  dispatch_act(g.act, [&](auto tag) {
    constexpr int ACT = decltype(tag)::value;
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j) {
        const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
        if (m >= g.M || n >= g.Ncols) continue;
        const int64_t c = m * g.ldc + n;
        float v = z[i][j];
        if ((MODE == FFN_LINEAR || MODE == FFN_LINEAR_DZ) && g.bias) v += ld<E>(g.bias, n);
        if (MODE == FFN_LINEAR) {
          v = act<ACT, FAST>(v);
          if (g.R) v += ld<E>(g.R, m * g.ldr + n);
        } else if (MODE == FFN_GATED) {
          v = act<ACT, FAST>(v) * z2[i][j];
        } else if (MODE == FFN_LINEAR_DZ || MODE == FFN_GATED_DGU) {
          float a, d;
          act_grad<ACT, FAST>(v, a, d);
          const float o = ld<E>(g.D, m * g.ldd + n);
          if (DUAL) {
            static_cast<E*>(g.C2)[c] = static_cast<E>(o * a);
            v = o * z2[i][j] * d;
          } else {
            v = o * d;
          }
        }
        C[c] = static_cast<E>(v);
      }
  });
}

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

template <typename E>
cudaError_t simt(const FfnGemm& g, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((g.M + T - 1) / T), static_cast<unsigned>((g.Ncols + T - 1) / T));
  switch (g.mode) {
    case FFN_LINEAR: ffn_simt_kernel<E, FFN_LINEAR><<<grid, 256, 0, stream>>>(g); break;
    case FFN_GATED: ffn_simt_kernel<E, FFN_GATED><<<grid, 256, 0, stream>>>(g); break;
    case FFN_LINEAR_DZ: ffn_simt_kernel<E, FFN_LINEAR_DZ><<<grid, 256, 0, stream>>>(g); break;
    case FFN_GATED_DGU: ffn_simt_kernel<E, FFN_GATED_DGU><<<grid, 256, 0, stream>>>(g); break;
    default: ffn_simt_kernel<E, FFN_GRADS><<<grid, 256, 0, stream>>>(g);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_ffn_simt(const FfnGemm& g, cudaStream_t stream) {
  return g.dtype == LCE_BF16 ? simt<__nv_bfloat16>(g, stream) : simt<float>(g, stream);
}

cudaError_t launch_column_sum(const void* x, int64_t ld, int64_t N, int64_t cols, lce_dtype_t dtype,
                              int parts, int64_t part_stride, void* out, cudaStream_t stream) {
  const unsigned blocks = static_cast<unsigned>((cols + 127) / 128);
  const __nv_bfloat16* h = static_cast<const __nv_bfloat16*>(x);
  if (parts == 3)
    column_sum_kernel<__nv_bfloat16, 3><<<blocks, 128, 0, stream>>>(h, ld, part_stride, N, cols,
                                                                    static_cast<float*>(out));
  else if (dtype == LCE_BF16)
    column_sum_kernel<__nv_bfloat16, 1>
        <<<blocks, 128, 0, stream>>>(h, ld, 0, N, cols, static_cast<__nv_bfloat16*>(out));
  else
    column_sum_kernel<float, 1><<<blocks, 128, 0, stream>>>(static_cast<const float*>(x), ld, 0, N, cols,
                                                            static_cast<float*>(out));
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
