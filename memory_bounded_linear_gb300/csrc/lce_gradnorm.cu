// Global gradient norm over many arrays, and clipping (declared in include/lce.h).
//
//   total = sqrt(sum over arrays of sum of g^2)   (or max |g|),   c = min(1, max_norm / (total + 1e-6))
//   out   = g c
//
// Two launches.  The first cuts the arrays into chunks of CHUNK elements and gives block b the chunks
// b, b + grid, ...; each block writes one partial.  The second reads all partials (every block for
// itself, in the same order), forms c and scales its chunks.  The table of the arrays is a kernel
// argument, so nothing is copied to the device and a captured graph holds its own table; lists
// longer than one table take several launches of each kind.
// Both passes are bound by memory: 2 x the arrays' bytes are read (the second time from L2 as far
// as they fit) and once written.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "lce.h"
#include "lce_internal.h"

namespace lce {
namespace {

constexpr int THREADS = 256;
constexpr int64_t CHUNK = 16384;       // elements: 64 per thread
constexpr int TABLE = 512;             // arrays per launch
constexpr int MAX_BLOCKS = 152 * 4;    // blocks of one norm launch

struct Table {
  const void* in[TABLE];
  void* out[TABLE];
  int64_t numel[TABLE];
  int64_t first[TABLE + 1];  // first chunk of each array
  unsigned char f32[TABLE];
  int count;
};

__device__ __forceinline__ int find(const Table& t, int64_t chunk) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// |x| as an integer: its order is that of the values, with inf above them and NaN above inf.
__device__ __forceinline__ unsigned mag(float x) { return __float_as_uint(x) & 0x7fffffffu; }

struct Acc {
  float s;     // sum of squares of at most CHUNK / THREADS values
  unsigned m;  // largest magnitude
  template <bool INF>
  __device__ __forceinline__ void add(float x) {
    if (INF) m = max(m, mag(x));
    else s = fmaf(x, x, s);
  }
};

template <typename E, bool INF>
__device__ __forceinline__ void visit(const E* p, int64_t n, Acc& a) {
  for (int64_t i = threadIdx.x; i < n; i += THREADS) a.add<INF>(static_cast<float>(p[i]));
}

template <bool INF>
__global__ void __launch_bounds__(THREADS) norm_kernel(const __grid_constant__ Table t, double* part) {
  double sum = 0.0;
  unsigned m = 0;
  for (int64_t c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
    const int k = find(t, c);
    const int64_t i0 = (c - t.first[k]) * CHUNK;
    const int64_t n = min(CHUNK, t.numel[k] - i0);
    Acc a{0.f, 0u};
    if (t.f32[k]) visit<float, INF>(static_cast<const float*>(t.in[k]) + i0, n, a);
    else visit<__nv_bfloat16, INF>(static_cast<const __nv_bfloat16*>(t.in[k]) + i0, n, a);
    sum += static_cast<double>(a.s);
    m = max(m, a.m);
  }
  __shared__ double sh[THREADS];
  sh[threadIdx.x] = INF ? static_cast<double>(m) : sum;
  __syncthreads();
  for (int w = THREADS / 2; w > 0; w >>= 1) {
    if (threadIdx.x < w) {
      const double o = sh[threadIdx.x + w];
      sh[threadIdx.x] = INF ? fmax(sh[threadIdx.x], o) : sh[threadIdx.x] + o;
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) part[blockIdx.x] = sh[0];
}

// The total from all partials: the same sum, in the same order, whichever block computes it.
template <bool INF>
__device__ float total_of(const double* part, int parts) {
  __shared__ double sh[THREADS];
  double v = 0.0;
  for (int i = threadIdx.x; i < parts; i += THREADS) v = INF ? fmax(v, part[i]) : v + part[i];
  sh[threadIdx.x] = v;
  __syncthreads();
  for (int w = THREADS / 2; w > 0; w >>= 1) {
    if (threadIdx.x < w) {
      const double o = sh[threadIdx.x + w];
      sh[threadIdx.x] = INF ? fmax(sh[threadIdx.x], o) : sh[threadIdx.x] + o;
    }
    __syncthreads();
  }
  return INF ? __uint_as_float(static_cast<unsigned>(sh[0])) : static_cast<float>(sqrt(sh[0]));
}

template <bool INF>
__global__ void __launch_bounds__(THREADS) total_kernel(const double* part, int parts, float* total) {
  const float v = total_of<INF>(part, parts);
  if (threadIdx.x == 0) *total = v;
}

template <typename E>
__device__ __forceinline__ void scale(const E* in, E* out, int64_t n, float c) {
  for (int64_t i = threadIdx.x; i < n; i += THREADS)
    out[i] = static_cast<E>(static_cast<float>(in[i]) * c);
}

template <bool INF>
__global__ void __launch_bounds__(THREADS)
    scale_kernel(const __grid_constant__ Table t, const double* part, int parts, float max_norm,
                 float* total) {
  const float v = total_of<INF>(part, parts);
  if (blockIdx.x == 0 && threadIdx.x == 0) *total = v;
  const float q = max_norm / (v + 1e-6f);
  const float c = q > 1.f ? 1.f : q;  // NaN stays
  for (int64_t ch = blockIdx.x; ch < t.first[t.count]; ch += gridDim.x) {
    const int k = find(t, ch);
    if (c == 1.f && t.in[k] == t.out[k]) continue;
    const int64_t i0 = (ch - t.first[k]) * CHUNK;
    const int64_t n = min(CHUNK, t.numel[k] - i0);
    if (t.f32[k])
      scale(static_cast<const float*>(t.in[k]) + i0, static_cast<float*>(t.out[k]) + i0, n, c);
    else
      scale(static_cast<const __nv_bfloat16*>(t.in[k]) + i0,
            static_cast<__nv_bfloat16*>(t.out[k]) + i0, n, c);
  }
}

// Calls f(table) for the list cut into tables; empty arrays are left out.
template <typename F>
cudaError_t for_tables(const void* const* grads, void* const* out, const int64_t* numels,
                       const int32_t* dtypes, int64_t count, F&& f) {
  Table t;
  t.count = 0;
  t.first[0] = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (numels[i] > 0) {
      const int k = t.count++;
      t.in[k] = grads[i];
      t.out[k] = out ? out[i] : const_cast<void*>(grads[i]);
      t.numel[k] = numels[i];
      t.f32[k] = dtypes[i] == LCE_F32;
      t.first[k + 1] = t.first[k] + (numels[i] + CHUNK - 1) / CHUNK;
    }
    if (t.count == TABLE || (i + 1 == count && t.count > 0)) {
      cudaError_t e = f(t);
      if (e != cudaSuccess) return e;
      t.count = 0;
    }
  }
  return cudaSuccess;
}

int64_t tables_of(int64_t count) { return (count + TABLE - 1) / TABLE; }

lce_status_t checks(const void* const* grads, void* const* out, const int64_t* numels,
                    const int32_t* dtypes, int64_t count, lce_norm_t norm, const float* total,
                    const void* workspace, size_t ws_bytes) {
  if (norm != LCE_NORM_L2 && norm != LCE_NORM_INF) return LCE_ERR_INVALID_ARG;
  if (count < 0 || !total || !workspace || (count > 0 && (!grads || !numels || !dtypes)))
    return LCE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(workspace) & 15u) || (reinterpret_cast<uintptr_t>(total) & 3u))
    return LCE_ERR_INVALID_ARG;
  for (int64_t i = 0; i < count; ++i) {
    if (dtypes[i] != LCE_BF16 && dtypes[i] != LCE_F32) return LCE_ERR_INVALID_ARG;
    if (numels[i] < 0 || numels[i] > (int64_t(1) << 48)) return LCE_ERR_UNSUPPORTED_SHAPE;
    const uintptr_t mask = dtypes[i] == LCE_F32 ? 3u : 1u;
    if (numels[i] > 0) {
      if (!grads[i] || (reinterpret_cast<uintptr_t>(grads[i]) & mask)) return LCE_ERR_INVALID_ARG;
      if (out && (!out[i] || (reinterpret_cast<uintptr_t>(out[i]) & mask)))
        return LCE_ERR_INVALID_ARG;
    }
  }
  if (ws_bytes < lce_grad_norm_workspace_size(count)) return LCE_ERR_WORKSPACE_TOO_SMALL;
  return LCE_OK;
}

template <bool INF>
lce_status_t run(const void* const* grads, void* const* out, const int64_t* numels,
                 const int32_t* dtypes, int64_t count, bool clip, float max_norm, float* total,
                 void* workspace, cudaStream_t stream) {
  double* part = reinterpret_cast<double*>(static_cast<char*>(workspace) + WS_HEADER_BYTES);
  int parts = 0;
  cudaError_t e = for_tables(grads, out, numels, dtypes, count, [&](const Table& t) {
    const int blocks = static_cast<int>(std::min<int64_t>(t.first[t.count], MAX_BLOCKS));
    const cudaError_t r = traced(K_GRAD_NORM, stream, [&] {
      norm_kernel<INF><<<blocks, THREADS, 0, stream>>>(t, part + parts);
      return cudaGetLastError();
    });
    parts += blocks;
    return r;
  });
  if (e != cudaSuccess) return LCE_ERR_CUDA;
  if (!clip || parts == 0) {
    e = traced(K_GRAD_NORM, stream, [&] {
      total_kernel<INF><<<1, THREADS, 0, stream>>>(part, parts, total);
      return cudaGetLastError();
    });
    return e == cudaSuccess ? LCE_OK : LCE_ERR_CUDA;
  }
  e = for_tables(grads, out, numels, dtypes, count, [&](const Table& t) {
    const int blocks = static_cast<int>(std::min<int64_t>(t.first[t.count], MAX_BLOCKS));
    return traced(K_GRAD_SCALE, stream, [&] {
      scale_kernel<INF><<<blocks, THREADS, 0, stream>>>(t, part, parts, max_norm, total);
      return cudaGetLastError();
    });
  });
  return e == cudaSuccess ? LCE_OK : LCE_ERR_CUDA;
}

lce_status_t entry(const void* const* grads, void* const* out, const int64_t* numels,
                   const int32_t* dtypes, int64_t count, lce_norm_t norm, bool clip, float max_norm,
                   float* total, void* workspace, size_t ws_bytes, void* stream) {
  lce_status_t st =
      checks(grads, out, numels, dtypes, count, norm, total, workspace, ws_bytes);
  if (st != LCE_OK) return st;
  int num_sms = 0;
  if ((st = check_device(&num_sms)) != LCE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return norm == LCE_NORM_INF
             ? run<true>(grads, out, numels, dtypes, count, clip, max_norm, total, workspace, s)
             : run<false>(grads, out, numels, dtypes, count, clip, max_norm, total, workspace, s);
}

}  // namespace
}  // namespace lce

using namespace lce;

extern "C" {

size_t lce_grad_norm_workspace_size(int64_t count) {
  if (count < 0 || count > (int64_t(1) << 31)) return 0;
  const size_t tables = static_cast<size_t>(std::max<int64_t>(1, tables_of(count)));
  return WS_HEADER_BYTES + tables * MAX_BLOCKS * sizeof(double);
}

lce_status_t lce_grad_norm(const void* const* grads, const int64_t* numels, const int32_t* dtypes,
                           int64_t count, lce_norm_t norm, float* total_norm, void* workspace,
                           size_t ws_bytes, void* stream) {
  return entry(grads, nullptr, numels, dtypes, count, norm, false, 0.f, total_norm, workspace,
               ws_bytes, stream);
}

lce_status_t lce_clip_grad_norm(const void* const* grads, void* const* out, const int64_t* numels,
                                const int32_t* dtypes, int64_t count, lce_norm_t norm,
                                float max_norm, float* total_norm, void* workspace,
                                size_t ws_bytes, void* stream) {
  if (!(max_norm >= 0.f)) return LCE_ERR_INVALID_ARG;
  return entry(grads, out, numels, dtypes, count, norm, true, max_norm, total_norm, workspace,
               ws_bytes, stream);
}

}  // extern "C"
