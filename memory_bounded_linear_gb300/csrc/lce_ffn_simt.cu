// CUDA-core kernels of the feed-forward operators: fp32 products of a few tokens, column sums
// (dbias), and copies of operands (fp32 into bf16 parts, bf16 into aligned rows).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "bf16_parts.cuh"
#include "lce_act.cuh"
#include "lce_ffn.h"
#include "lce_internal.h"
#include "ptx.cuh"

namespace lce {
namespace {

// ---------------------------------------------------------------- fp32 products of a few tokens
// Up to eight tokens bound by reading the weights once (HBM).  A warp computes ROWS features (4; gated 2
// of Wg and 2 of Wu) for NT tokens, at most eight, or WAYS warps of a block together: they take 512-byte
// pieces of K in turn, lanes four elements each, and each weight vector loaded serves NT tokens from
// registers (X comes from L1/L2).  The lanes' sums meet by shuffles, the warps' in shared memory, in a
// fixed order.  Every further tile of eight tokens reads all weights again, from L2 at best: the token
// tile is the slower grid index.  Inside a captured graph 1 x 2048 -> 8192 takes 12.3 us (5.5 TB/s), 8: 17,
// 16: 29, 32: 50, 48: 64; 6144 -> 16384 (403 MB) 8: 85, 16: 162, 32: 293, 48: 471; 2 x 2048 -> 2048 4.4
// (3.8 TB/s; most of it the launch and the latency of the first loads).
constexpr int WARPS = 8;

template <int NT, int WAYS, bool GATED>
__global__ void __launch_bounds__(WARPS * 32) few_f32_kernel(const FfnGemm g,
                                                             unsigned* err) {
  constexpr int ROWS = GATED ? 2 : 4, R = 4;
  __shared__ float sh[WARPS][R * NT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  ptx::wait_for_previous();  // no memory of the caller is touched before this
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *err = 0u;  // this kernel never waits
  // all warps together: the same features for the whole block, which keeps their addresses uniform
  const int way = WAYS == WARPS ? warp : warp % WAYS, group = WAYS == WARPS ? 0 : warp / WAYS;
  const int64_t f0 = (static_cast<int64_t>(blockIdx.x) * (WARPS / WAYS) + group) * ROWS;
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
  for (int64_t k = (way * 32 + lane) * 4; k < g.K; k += WAYS * 128) {
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
  ptx::launch_dependents();
  // The lanes' sums: at each step a lane keeps half of its values and adds the other lane's to them, so
  // that the last one ends with value lane / (32 / V), in 31 shuffles for 32 values instead of 160.
  constexpr int V = R * NT;
  float s[V];
#pragma unroll
  for (int i = 0; i < V; ++i) s[i] = acc[i / NT][i % NT];
#pragma unroll
  for (int o = 16, n = V / 2; o > 0; o >>= 1, n >>= 1) {
    if (n == 0) {
      s[0] += __shfl_xor_sync(0xffffffffu, s[0], o);
      continue;
    }
    const bool upper = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float other = __shfl_xor_sync(0xffffffffu, upper ? s[i] : s[i + n], o);
      s[i] = (upper ? s[i + n] : s[i]) + other;
    }
  }
  if (lane % (32 / V) == 0) sh[warp][lane / (32 / V)] = s[0];
  __syncthreads();
  if (way != 0 || lane >= ROWS * NT) return;  // one result per thread, of the first warp's lanes
  const int r = lane % ROWS, t = lane / ROWS;
  const int64_t f = f0 + r, m = t0 + t;
  if (f >= g.Ncols || m >= g.M) return;
  float z = 0.f, u = 0.f;
#pragma unroll
  for (int k = 0; k < WAYS; ++k) {
    z += sh[group * WAYS + k][r * NT + t];
    if (GATED) u += sh[group * WAYS + k][(ROWS + r) * NT + t];
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

template <int NT, bool GATED>
cudaError_t few_f32(const FfnGemm& g, unsigned* err, cudaStream_t stream) {
  constexpr int ROWS = GATED ? 2 : 4;
  const int64_t groups = (g.Ncols + ROWS - 1) / ROWS, token_tiles = (g.M + NT - 1) / NT;
  auto blocks = [&](int ways) { return (groups * ways + WARPS - 1) / WARPS; };
  auto launch = [&](auto kernel, int ways) {
    const dim3 grid(static_cast<unsigned>(blocks(ways)), static_cast<unsigned>(token_tiles));
    return launch_kernel(kernel, grid, WARPS * 32, stream, g, err);
  };
  // The cheapest by an estimate: waves of the blocks that fit on the SMs at once, each the steps of K
  // and about two more for the sums.  (us with 8, 4, 2, 1 warps: 8 x 2048 -> 8192 21.6, 20.0, 19.1, 17.1;
  // 12 x 1024 -> 2048 7.5, 5.8, 4.7, 7.1; 16 x 6000 -> 1500 19.9, 24.5, 25.5.)  One token always takes
  // eight: the loads in flight decide (1 x 4096 -> 4096 13.2, 17.6 with two).
  int ways = WARPS;
  if (NT > 1) {
    constexpr int PLACES = 152 * (NT == 2 ? 3 : 2);
    int64_t best = INT64_MAX;
    for (int w = WARPS; w >= 1; w /= 2) {
      const int64_t cost = ((blocks(w) * token_tiles + PLACES - 1) / PLACES) *
                           ((g.K + 128 * w - 1) / (128 * w) + 2);
      if (cost < best) { best = cost; ways = w; }
    }
  }
  if constexpr (NT > 1) {
    if (ways == 1) return launch(few_f32_kernel<NT, 1, GATED>, 1);
    if (ways == 2) return launch(few_f32_kernel<NT, 2, GATED>, 2);
    if (ways == 4) return launch(few_f32_kernel<NT, 4, GATED>, 4);
  }
  return launch(few_f32_kernel<NT, WARPS, GATED>, WARPS);
}
template <bool GATED>
cudaError_t few_f32(const FfnGemm& g, unsigned* err, cudaStream_t stream) {
  if (g.M == 1) return few_f32<1, GATED>(g, err, stream);
  if (g.M == 2) return few_f32<2, GATED>(g, err, stream);
  if (g.M <= 4) return few_f32<4, GATED>(g, err, stream);
  return few_f32<8, GATED>(g, err, stream);
}

// ---------------------------------------------------------------------------- column sums
// Bound by reading x once; with few columns by how many rows are in flight.  A cluster of eight blocks
// takes a strip of LANES x 4 columns; every LANES lanes of its 64 warps read rows of the strip, eight at a
// time: with LANES = 16 rows of 128 contiguous bytes and 1,024 of them in flight per strip; with 8,
// for up to NARROW columns, 2,048.  Lanes meet by shuffles, warps in shared memory, blocks through
// distributed shared memory, in a fixed order: one launch, no workspace, no atomics.  4095 x 8192 bf16
// takes 12 us (5.6 TB/s).
constexpr int64_t NARROW = 2048;
constexpr int SUM_SPLIT = 8;
constexpr int SUM_UNROLL = 8;

__device__ __forceinline__ void add4(float (&s)[4], const uint2& q) {
  s[0] += __uint_as_float(q.x << 16);
  s[1] += __uint_as_float(q.x & 0xffff0000u);
  s[2] += __uint_as_float(q.y << 16);
  s[3] += __uint_as_float(q.y & 0xffff0000u);
}

template <int PARTS, int LANES, typename O>
__global__ void __cluster_dims__(SUM_SPLIT, 1, 1) __launch_bounds__(WARPS * 32)
    column_sum_kernel(const __nv_bfloat16* __restrict__ x, int64_t ld, int64_t part_stride, int64_t N,
                      int64_t cols, O* __restrict__ out) {
  constexpr int SUM_COLS = LANES * 4, PER_WARP = 32 / LANES;  // columns; rows a warp reads at once
  ptx::wait_for_previous();
  __shared__ float sh[WARPS][SUM_COLS];
  __shared__ float total[SUM_COLS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(blockIdx.x) % SUM_SPLIT;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x / SUM_SPLIT) * SUM_COLS;
  const int64_t c = c0 + (lane & (LANES - 1)) * 4;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  if (c < cols) {
    constexpr int64_t STEP = SUM_SPLIT * WARPS * PER_WARP;
    const int64_t step = STEP * ld;
    int64_t r = (rank * WARPS + warp) * PER_WARP + lane / LANES;
    const __nv_bfloat16* p = x + r * ld + c;
    for (; r + (SUM_UNROLL - 1) * STEP < N; r += SUM_UNROLL * STEP, p += SUM_UNROLL * step) {
      uint2 q[SUM_UNROLL][PARTS];
#pragma unroll
      for (int u = 0; u < SUM_UNROLL; ++u)
#pragma unroll
        for (int k = 0; k < PARTS; ++k)
          q[u][k] = __ldg(reinterpret_cast<const uint2*>(p + u * step + k * part_stride));
#pragma unroll
      for (int u = 0; u < SUM_UNROLL; ++u) {
        float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = PARTS - 1; k >= 0; --k) add4(v, q[u][k]);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += v[i];
      }
    }
    for (; r < N; r += STEP, p += step) {
      float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = PARTS - 1; k >= 0; --k)
        add4(v, __ldg(reinterpret_cast<const uint2*>(p + k * part_stride)));
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] += v[i];
    }
  }
  ptx::launch_dependents();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int o = 16; o >= LANES; o >>= 1) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
    if (lane < LANES) sh[warp][lane * 4 + i] = s[i];
  }
  __syncthreads();
  if (threadIdx.x < SUM_COLS) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) v += sh[w][threadIdx.x];
    total[threadIdx.x] = v;
  }
  ptx::cluster_sync();
  if (rank == 0 && threadIdx.x < SUM_COLS && c0 + threadIdx.x < cols) {
    const uint32_t at = ptx::smem_addr(&total[threadIdx.x]);
    float v = 0.f;
#pragma unroll
    for (int r = 0; r < SUM_SPLIT; ++r) v += ptx::ld_shared_cluster(ptx::mapa_shared(at, r));
    out[c0 + threadIdx.x] = static_cast<O>(v);
  }
  ptx::cluster_sync();  // no block leaves while its sums are read
}

// ---------------------------------------------------------------------------- operand copies
// Up to MAX_PACK_ARRAYS arrays in one launch, bound by memory: fp32 into three bf16 parts (PARTS = 3,
// 4 bytes read and 6 written per element) or bf16 into rows of another stride (PARTS = 1).  A block
// takes PACK_VECS 16-byte groups of one array; block 0 also clears the workspace header, as the first
// launch of its call.
constexpr int PACK_UNROLL = 4;
constexpr int PACK_VECS = WARPS * 32 * PACK_UNROLL;

struct PackParams {
  PackArray a[MAX_PACK_ARRAYS];
  int64_t first[MAX_PACK_ARRAYS];  // first block of each array
  int count;
  unsigned* header;
};

template <int PARTS>
__global__ void __launch_bounds__(WARPS * 32) pack_kernel(const __grid_constant__ PackParams p) {
  constexpr int VEC = PARTS == 3 ? 4 : 8;  // elements per 16 bytes read
  ptx::wait_for_previous();  // no memory of the caller is touched before this
  if (blockIdx.x == 0 && threadIdx.x < WS_HEADER_BYTES / 4) p.header[threadIdx.x] = 0u;
  int k = 0;
  while (k + 1 < p.count && p.first[k + 1] <= blockIdx.x) ++k;
  const PackArray& a = p.a[k];
  const uint32_t groups = static_cast<uint32_t>(a.cols / VEC);  // per row
  const int64_t i0 = (blockIdx.x - p.first[k]) * static_cast<int64_t>(PACK_VECS);
  const int64_t r0 = i0 / groups;
  const uint32_t o0 = static_cast<uint32_t>(i0 - r0 * groups);  // group of the block's first
  uint4 v[PACK_UNROLL];
  int64_t row[PACK_UNROLL];
  uint32_t col[PACK_UNROLL];
#pragma unroll
  for (int u = 0; u < PACK_UNROLL; ++u) {
    const uint32_t o = o0 + threadIdx.x + u * WARPS * 32;
    row[u] = r0 + o / groups;
    col[u] = o % groups * VEC;
    if (row[u] < a.rows)
      v[u] = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.x) +
                                             (row[u] * a.ld + col[u]) * (16 / VEC));
  }
  ptx::launch_dependents();
#pragma unroll
  for (int u = 0; u < PACK_UNROLL; ++u) {
    if (row[u] >= a.rows) break;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + row[u] * a.ld_out + col[u];
    if constexpr (PARTS == 1) {
      *reinterpret_cast<uint4*>(out) = v[u];
    } else {
      float q[4][3];
      split_bf16(__uint_as_float(v[u].x), q[0]);
      split_bf16(__uint_as_float(v[u].y), q[1]);
      split_bf16(__uint_as_float(v[u].z), q[2]);
      split_bf16(__uint_as_float(v[u].w), q[3]);
#pragma unroll
      for (int s = 0; s < 3; ++s) {
        __nv_bfloat162 h[2] = {__floats2bfloat162_rn(q[0][s], q[1][s]),
                               __floats2bfloat162_rn(q[2][s], q[3][s])};
        *reinterpret_cast<uint2*>(out + s * a.part_stride) = *reinterpret_cast<uint2*>(h);
      }
    }
  }
}

}  // namespace

cudaError_t launch_ffn_few_f32(const FfnGemm& g, unsigned* err, cudaStream_t stream) {
  return g.mode == FFN_GATED ? few_f32<true>(g, err, stream) : few_f32<false>(g, err, stream);
}

cudaError_t launch_column_sum(const void* x, int64_t ld, int64_t N, int64_t cols, int parts,
                              int64_t part_stride, void* out, cudaStream_t stream) {
  const __nv_bfloat16* h = static_cast<const __nv_bfloat16*>(x);
  auto launch = [&](auto kernel, int strip, auto* result) {
    const dim3 grid(static_cast<unsigned>((cols + strip - 1) / strip * SUM_SPLIT));
    return launch_kernel(kernel, grid, WARPS * 32, stream, h, ld, part_stride, N, cols, result);
  };
  if (parts == 3) {
    float* o = static_cast<float*>(out);
    return cols <= NARROW ? launch(column_sum_kernel<3, 8, float>, 32, o)
                          : launch(column_sum_kernel<3, 16, float>, 64, o);
  }
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out);
  return cols <= NARROW ? launch(column_sum_kernel<1, 8, __nv_bfloat16>, 32, o)
                        : launch(column_sum_kernel<1, 16, __nv_bfloat16>, 64, o);
}

cudaError_t launch_pack(const PackArray* arrays, int count, int parts, unsigned* header,
                        cudaStream_t stream) {
  if (count < 1 || count > MAX_PACK_ARRAYS || (parts != 1 && parts != 3)) return cudaErrorInvalidValue;
  PackParams p{};
  p.count = count;
  p.header = header;
  int64_t blocks = 0;
  for (int i = 0; i < count; ++i) {
    p.a[i] = arrays[i];
    p.first[i] = blocks;
    blocks += (arrays[i].rows * (arrays[i].cols / (parts == 3 ? 4 : 8)) + PACK_VECS - 1) / PACK_VECS;
  }
  if (blocks > (int64_t(1) << 31) - 1) {
    set_error_detail("operand copy of %lld blocks: beyond a launch's grid", static_cast<long long>(blocks));
    return cudaErrorInvalidValue;
  }
  const dim3 grid(static_cast<unsigned>(blocks));
  return parts == 3 ? launch_kernel(pack_kernel<3>, grid, WARPS * 32, stream, p)
                    : launch_kernel(pack_kernel<1>, grid, WARPS * 32, stream, p);
}

}  // namespace lce
