// Global gradient norm over many arrays, and clipping (declared in include/lce.h).
//
//   total = sqrt(sum over arrays of sum of g^2)   (or max |g|),   c = min(1, max_norm / (total + 1e-6))
//   out   = g c
//
// Two launches.  The first cuts the arrays into chunks (up to 64 KB, smaller where that would leave
// SMs without one) and gives block b the chunks b, b + grid, ...; each block writes one partial.  The
// second reads all partials (every block for itself, in the same order), forms c and scales the
// chunks, last one first, so that what the first pass left in L2 is not read from memory again.  The
// table of the arrays is a kernel argument: nothing is copied to the device, and a captured graph
// holds its own table; lists longer than one table take several launches of each kind.
// Both passes are bound by memory: the arrays are read twice and written once.  Inside a captured graph
// 20 arrays of 137 MB take 63.1 us (0.97 of the copy rate for three passes), 1.25 GB 578 us (0.96), 0.6
// MB 6.2 us (latency).  (Loading each vector of the next chunk as one is consumed was 2% slower from 100
// MB on.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "lce.h"
#include "lce_internal.h"
#include "ptx.cuh"

namespace lce {
namespace {

constexpr int THREADS = 512;
constexpr int UNROLL = 8;              // 16-byte vectors a thread has in flight
constexpr int TABLE = 512;             // arrays per launch,
constexpr int SMALL_TABLE = 40;        // or, for a short list, a table of 1.3 KB instead of 17
constexpr int MAX_BLOCKS = 152 * 2;    // blocks of one launch: 1,024 threads per SM

template <int CAP>
struct Table {
  const void* in[CAP];
  void* out[CAP];
  int64_t numel[CAP];
  int64_t first[CAP + 1];  // first chunk of each array
  unsigned char f32[CAP];
  int count;
  int vectors;               // 16-byte vectors per chunk: THREADS x 1, 2, 4 or 8
};

template <int CAP>
__device__ __forceinline__ int find(const Table<CAP>& t, int64_t chunk) {
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
  float s;     // sum of squares of at most 64 values (and two at the unaligned ends)
  unsigned m;  // largest magnitude
  template <bool INF>
  __device__ __forceinline__ void add(float x) {
    if (INF) m = max(m, mag(x));
    else s = fmaf(x, x, s);
  }
};

template <typename E>
constexpr int PER_VEC = 16 / sizeof(E);

template <typename E>
__device__ __forceinline__ void unpack(const uint4& q, float (&v)[PER_VEC<E>]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(E) == 2) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      v[i] = __uint_as_float(w[i]);
    }
  }
}

// The block's sum (or maximum) of v in a fixed order, in thread 0.
template <bool INF>
__device__ __forceinline__ double reduce(double v) {
  __shared__ double sh[THREADS / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double w = __shfl_xor_sync(0xffffffffu, v, o);
    v = INF ? fmax(v, w) : v + w;
  }
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 1; i < THREADS / 32; ++i) v = INF ? fmax(v, sh[i]) : v + sh[i];
  }
  return v;
}

// A chunk of the table: its elements, and where the whole 16-byte vectors among them begin.
struct Chunk {
  const char* in;
  char* out;
  int n, head, nvec;  // elements; those before the vectors; vectors
  bool f32;
};
template <int CAP>
__device__ __forceinline__ Chunk chunk_of(const Table<CAP>& t, int64_t c) {
  const int k = find(t, c);
  Chunk r;
  r.f32 = t.f32[k];
  const int bytes = r.f32 ? 4 : 2, per_vec = 16 / bytes;
  const int64_t size = static_cast<int64_t>(t.vectors) * per_vec, i0 = (c - t.first[k]) * size;
  r.n = static_cast<int>(min(size, t.numel[k] - i0));
  r.in = static_cast<const char*>(t.in[k]) + i0 * bytes;
  r.out = static_cast<char*>(t.out[k]) + i0 * bytes;
  r.head = min(static_cast<int>((16 - (reinterpret_cast<uintptr_t>(r.in) & 15)) & 15) / bytes, r.n);
  r.nvec = (r.n - r.head) / per_vec;
  return r;
}
// This thread's vectors of a chunk.  LAST: the last use of these values.
template <bool LAST>
__device__ __forceinline__ void load(const Chunk& c, uint4 (&q)[UNROLL]) {
  const uint4* v = reinterpret_cast<const uint4*>(c.in + c.head * (c.f32 ? 4 : 2));
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const int i = threadIdx.x + u * THREADS;
    q[u] = i >= c.nvec ? make_uint4(0, 0, 0, 0) : LAST ? __ldcs(v + i) : v[i];
  }
}

// Adds chunk c, whose vectors are in q.
template <typename E, bool INF>
__device__ __forceinline__ void visit(const Chunk& c, const uint4 (&q)[UNROLL], Acc& a) {
  const E* p = reinterpret_cast<const E*>(c.in);
  const int tail = c.n - c.head - c.nvec * PER_VEC<E>;
  if (threadIdx.x < c.head) a.add<INF>(static_cast<float>(p[threadIdx.x]));
  if (threadIdx.x < tail) a.add<INF>(static_cast<float>(p[c.n - tail + threadIdx.x]));
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    float f[PER_VEC<E>];
    unpack<E>(q[u], f);
#pragma unroll
    for (int i = 0; i < PER_VEC<E>; ++i) a.add<INF>(f[i]);
  }
}

template <bool INF, int CAP>
__global__ void __launch_bounds__(THREADS, 2)
    norm_kernel(const __grid_constant__ Table<CAP> t, double* part, unsigned* flags) {
  int64_t i = blockIdx.x;  // the grid is not larger than the number of chunks
  Chunk c = chunk_of(t, i);
  ptx::wait_for_previous();  // no memory of the caller is touched before this
  ptx::launch_dependents();  // its blocks take the places of this grid's as they end
  if (blockIdx.x == 0 && threadIdx.x == 0) *flags = 0u;  // nothing here can fail on the device
  double sum = 0.0;
  unsigned m = 0;
  while (true) {
    uint4 q[UNROLL];
    load<false>(c, q);
    Acc a{0.f, 0u};
    if (c.f32) visit<float, INF>(c, q, a);
    else visit<__nv_bfloat16, INF>(c, q, a);
    sum += static_cast<double>(a.s);
    m = max(m, a.m);
    i += gridDim.x;
    if (i >= t.first[t.count]) break;
    c = chunk_of(t, i);
  }
  const double r = reduce<INF>(INF ? static_cast<double>(m) : sum);
  if (threadIdx.x == 0) part[blockIdx.x] = r;
}

// The total from all partials: the same sum, in the same order, whichever block computes it.
template <bool INF>
__device__ __forceinline__ float total_of(const double* part, int parts) {
  __shared__ float total;
  double v = 0.0;
  for (int i = threadIdx.x; i < parts; i += THREADS) v = INF ? fmax(v, part[i]) : v + part[i];
  v = reduce<INF>(v);
  if (threadIdx.x == 0)
    total = INF ? __uint_as_float(static_cast<unsigned>(v)) : static_cast<float>(sqrt(v));
  __syncthreads();
  return total;
}

template <bool INF>
__global__ void __launch_bounds__(THREADS) total_kernel(const double* part, int parts, float* total,
                                                        unsigned* flags) {
  ptx::wait_for_previous();
  const float v = total_of<INF>(part, parts);
  if (threadIdx.x == 0) {
    *total = v;
    *flags = 0u;
  }
}

template <typename E>
__device__ __forceinline__ E scaled(E x, float c) {
  return static_cast<E>(static_cast<float>(x) * c);
}

// Writes chunk c, whose vectors are in q.
template <typename E>
__device__ __forceinline__ void scale(const Chunk& c, const uint4 (&q)[UNROLL], float f) {
  const E* in = reinterpret_cast<const E*>(c.in);
  E* out = reinterpret_cast<E*>(c.out);
  if ((reinterpret_cast<uintptr_t>(in) ^ reinterpret_cast<uintptr_t>(out)) & 15) {
    // the two are never 16-byte aligned together
    for (int i = threadIdx.x; i < c.n; i += THREADS) out[i] = scaled(in[i], f);
    return;
  }
  const int tail = c.n - c.head - c.nvec * PER_VEC<E>;
  uint4* o = reinterpret_cast<uint4*>(out + c.head);
  if (threadIdx.x < c.head) out[threadIdx.x] = scaled(in[threadIdx.x], f);
  if (threadIdx.x < tail)
    out[c.n - tail + threadIdx.x] = scaled(in[c.n - tail + threadIdx.x], f);
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    float v[PER_VEC<E>];
    unpack<E>(q[u], v);
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(E) == 2) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j] * f, v[2 * j + 1] * f);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        w[j] = __float_as_uint(v[j] * f);
      }
    }
    const int i = threadIdx.x + u * THREADS;
    if (i < c.nvec) __stcs(o + i, make_uint4(w[0], w[1], w[2], w[3]));
  }
}

template <bool INF, int CAP>
__global__ void __launch_bounds__(THREADS, 2)
    scale_kernel(const __grid_constant__ Table<CAP> t, const double* part, int parts, float max_norm,
                 float* total) {
  int64_t i = t.first[t.count] - 1 - blockIdx.x;  // the grid is not larger than the number of chunks
  Chunk c = chunk_of(t, i);
  // No memory of the caller is touched before this, the gradients neither: the kernel that wrote them
  // lies two launches back, and only a wait of its own makes those writes visible to this kernel.
  ptx::wait_for_previous();
  ptx::launch_dependents();
  uint4 q[UNROLL];
  load<true>(c, q);  // in flight while the partials are summed
  const float v = total_of<INF>(part, parts);
  if (blockIdx.x == 0 && threadIdx.x == 0) *total = v;
  const float r = isinf(v) ? 0.f : max_norm / (v + 1e-6f);  // also where max_norm is infinite
  const float f = r > 1.f ? 1.f : r;  // NaN stays
  while (true) {
    if (f != 1.f || c.in != c.out) {
      if (c.f32) scale<float>(c, q, f);
      else scale<__nv_bfloat16>(c, q, f);
    }
    i -= gridDim.x;
    if (i < 0) break;
    c = chunk_of(t, i);
    load<true>(c, q);
  }
}

// Calls f(table) for the list cut into tables; empty arrays are left out.
template <int CAP, typename F>
cudaError_t for_tables(const void* const* grads, void* const* out, const int64_t* numels,
                       const int32_t* dtypes, int64_t count, F&& f) {
  double bytes = 0.0;
  for (int64_t i = 0; i < count; ++i)
    bytes += static_cast<double>(numels[i]) * (dtypes[i] == LCE_F32 ? 4 : 2);
  Table<CAP> t;
  t.vectors = THREADS;
  // a chunk for every SM at most, while that is enough: a block of the second pass then fits beside one
  // of the first and begins with it (27 arrays of 2 MB 6.2 us, 8.7 with twice as many smaller chunks)
  while (t.vectors < THREADS * UNROLL && bytes / (16.0 * t.vectors) + count > MAX_BLOCKS / 2)
    t.vectors *= 2;
  t.count = 0;
  t.first[0] = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (numels[i] > 0) {
      const int k = t.count++;
      const int64_t size = static_cast<int64_t>(t.vectors) * (dtypes[i] == LCE_F32 ? 4 : 8);
      t.in[k] = grads[i];
      t.out[k] = out ? out[i] : const_cast<void*>(grads[i]);
      t.numel[k] = numels[i];
      t.f32[k] = dtypes[i] == LCE_F32;
      t.first[k + 1] = t.first[k] + (numels[i] + size - 1) / size;
    }
    if (t.count == CAP || (i + 1 == count && t.count > 0)) {
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

template <bool INF, int CAP>
lce_status_t run(const void* const* grads, void* const* out, const int64_t* numels,
                 const int32_t* dtypes, int64_t count, bool clip, float max_norm, float* total,
                 void* workspace, cudaStream_t stream) {
  double* part = reinterpret_cast<double*>(static_cast<char*>(workspace) + WS_HEADER_BYTES);
  unsigned* flags = static_cast<unsigned*>(workspace);
  int parts = 0;
  cudaError_t e = for_tables<CAP>(grads, out, numels, dtypes, count, [&](const Table<CAP>& t) {
    const int blocks = static_cast<int>(std::min<int64_t>(t.first[t.count], MAX_BLOCKS));
    const cudaError_t r = traced(K_GRAD_NORM, stream, [&] {
      return launch_kernel(norm_kernel<INF, CAP>, dim3(blocks), THREADS, stream, t, part + parts,
                           flags);
    });
    parts += blocks;
    return r;
  });
  if (e != cudaSuccess) return LCE_ERR_CUDA;
  if (!clip || parts == 0) {
    e = traced(K_GRAD_NORM, stream, [&] {
      return launch_kernel(total_kernel<INF>, dim3(1), THREADS, stream, part, parts, total, flags);
    });
    return e == cudaSuccess ? LCE_OK : LCE_ERR_CUDA;
  }
  e = for_tables<CAP>(grads, out, numels, dtypes, count, [&](const Table<CAP>& t) {
    const int blocks = static_cast<int>(std::min<int64_t>(t.first[t.count], MAX_BLOCKS));
    return traced(K_GRAD_SCALE, stream, [&] {
      return launch_kernel(scale_kernel<INF, CAP>, dim3(blocks), THREADS, stream, t, part, parts,
                           max_norm, total);
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
  auto go = [&](auto inf) {
    constexpr bool INF = decltype(inf)::value;
    return count <= SMALL_TABLE
               ? run<INF, SMALL_TABLE>(grads, out, numels, dtypes, count, clip, max_norm, total,
                                       workspace, s)
               : run<INF, TABLE>(grads, out, numels, dtypes, count, clip, max_norm, total, workspace,
                                 s);
  };
  return norm == LCE_NORM_INF ? go(std::true_type{}) : go(std::false_type{});
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
