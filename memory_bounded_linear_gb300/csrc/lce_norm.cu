// Layer normalisation and its gradients (declared in include/lce.h).
//
//   c = x - mean(x),  r = 1 / sqrt(mean(c^2) + eps),  x^ = c r,  y = x^ w + b
//   g = dy w,  dx = r (g - mean(g) - x^ mean(g x^)),  dw = sum over rows of dy x^,  db = sum of dy
//
// Bound by memory, closely followed by the instructions of a row: x is read once and y written once.  T threads
// share a row; the grid is as large as the SMs hold and walks over the rows, the next two on their way
// into shared memory (cp.async, each thread for itself) while one is summed.  What pays is few warps a
// row: reductions and the exchange between warps cost about 250 instructions a warp, as many as 16 vectors do, and with
// the next rows in registers instead of shared memory there were not enough left for it.  Arithmetic is packed in pairs.
// The backward pass recomputes both statistics from x, which it reads anyway: the forward pass keeps nothing.  Its
// blocks hold the columns' partial sums of dw and db in registers over all their rows and write them once; a
// second launch adds them in a fixed order (2 to 4 us).
// Inside a captured graph, bf16: forward 32768 x 6144 128 us (0.92 of the copy rate), 16384 x 4096 46 (0.86);
// backward 32768 x 6144 199 (0.89), 16384 x 4096 70 (0.85), 16384 x 2048 41 (0.73); forward of one row 2.0.  At
// 16384 x 4096 backward with 64 / 128 / 256 / 512 threads a row: 68 / 75 / 100 / 204 us; forward with 64 / 128 / 256:
// 55 / 45 / 62.  Rows that fill no class run masked: 16384 x 7168 92 and 149 us (0.75, 0.70).
// Farther from their floor: 16384 x 2046 bf16 by 4 bytes 37 and 60 us (0.53, 0.49), 16384 x 2047 by single elements 54 and
// 84 (0.36); rows that are read again, 2048 x 20000 70 and 137 (0.35, 0.26).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "lce.h"
#include "lce_internal.h"
#include "lce_vec.cuh"
#include "per_device.h"
#include "ptx.cuh"

namespace lce {
namespace {

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 512;
constexpr int64_t kMaxWidth = int64_t(1) << 30;  // columns are counted in 32 bits, a step past the end too
constexpr int64_t kMaxElements = int64_t(1) << 48;

// Partial sums of dw and db, blocks of the backward pass, at most: a bound for the workspace, whatever the device.
int64_t max_parts(int64_t N, int64_t d) {
  return std::min<int64_t>(std::max<int64_t>(N, 1), d > 1024 ? 152 * 4 : 152 * 8);
}

struct NormArgs {
  const void* x;
  const void* w;   // or null
  const void* b;   // or null
  const void* dy;  // backward
  void* y;         // forward: y; backward: dx or null
  int64_t ldx, ldy, ldo;  // of x, of dy, of y or dx
  int64_t N;
  int d;
  float eps;
  float* part;     // [2][parts][d]: dw, db; null: neither is wanted
  float4* stats;   // [N], wide rows
  unsigned* flags;
};

// Threads of a block: T of them share a row.
template <int T>
constexpr int kBlock = T < 128 ? 128 : T;

// Blocks of an SM that a kernel is compiled for, by the 16-byte vectors of a row that a thread holds.
// (narrow vectors: 4 bytes and less).
template <int T, int NV, bool NARROW>
constexpr int kForwardResident = ((NARROW ? 768 : NV > 2 ? 640 : 768) + kBlock<T> - 1) / kBlock<T>;
template <int T, int NV, bool NARROW>
constexpr int kGradResident = ((NARROW ? 512 : NV > 4 ? 256 : NV > 2 ? 384 : NV > 1 ? 512 : 768) + kBlock<T> - 1) / kBlock<T>;

// Statistics of the rows that T threads hold in registers, NV vectors of V elements each.  Each warp takes
// its own mean first and all sums of differences to that, so that one exchange between the warps
// is enough: with n_w elements, mean m_w and the sums S, Q of c = x - m_w and c^2 of warp w,
//   mean = sum of (n_w m_w + S) / d,   sum of (x - mean)^2 = sum of Q + 2 (m_w - mean) S + n_w (m_w - mean)^2
// and with g the same for the sums of g and g (x - mean).  S is 0 but for the rounding of m_w; with it rows far
// off centre lose no bits.
// FULL: the vectors fill the row exactly, so that none has to be asked for.
template <typename E, int V, int T, int NV, bool FULL>
struct RowOf {
  int t, d;
  int first;   // of this thread's columns; the others follow T V apart
  int n_warp;  // elements of this warp
  float inv_warp, inv_d;
  __device__ __forceinline__ RowOf(int d_) : t(threadIdx.x % T), d(d_), first((threadIdx.x % T) * V) {
    n_warp = 0;
    if (FULL) d = T * NV * V;
#pragma unroll
    for (int i = 0; i < NV; ++i) n_warp += max(0, min(32 * V, d - (i * T + (t & ~31)) * V));
    inv_warp = 1.f / static_cast<float>(max(n_warp, 1));
    inv_d = 1.f / static_cast<float>(d);
  }
  __device__ __forceinline__ int col(int i) const { return first + i * T * V; }
  __device__ __forceinline__ bool in(int i) const { return FULL || col(i) < d; }

  __device__ __forceinline__ static float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
  // Sums of K = 2 or 4 values over a warp: halves of the warp take half the values each, so that 4 values take
  // 6 shuffles instead of 20.  The sum of value k is left in the lanes whose number modulo K is k.
  template <int K>
  __device__ __forceinline__ static float warp_sums(const float (&q)[K]) {
    const int lane = threadIdx.x & 31;
    float v;
    if constexpr (K == 4) {
      const bool odd = lane & 1, high = lane & 2;
      const float a = (odd ? q[1] : q[0]) + __shfl_xor_sync(0xffffffffu, odd ? q[0] : q[1], 1);
      const float b = (odd ? q[3] : q[2]) + __shfl_xor_sync(0xffffffffu, odd ? q[2] : q[3], 1);
      v = (high ? b : a) + __shfl_xor_sync(0xffffffffu, high ? a : b, 2);
    } else {
      const bool odd = lane & 1;
      v = (odd ? q[1] : q[0]) + __shfl_xor_sync(0xffffffffu, odd ? q[0] : q[1], 1);
      v += __shfl_xor_sync(0xffffffffu, v, 2);
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
  // Barrier of the T threads of a row.
  __device__ __forceinline__ static void row_barrier() {
    if constexpr (T == kBlock<T>) __syncthreads();
    else asm volatile("bar.sync %0, %1;" ::"r"(static_cast<int>(threadIdx.x) / T + 1), "n"(T) : "memory");
  }

  // The warp's mean of a row whose vectors x(i) gives.
  template <typename X>
  __device__ __forceinline__ float mean_of(X&& x) const {
    Lane<V> s;
    spread(0.f, s);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!in(i)) continue;
      Lane<V> v[kLanes<V>];
      unpack2<E, V>(x(i), v);
#pragma unroll
      for (int j = 0; j < kLanes<V>; ++j) s = add2(s, v[j]);
    }
    return warp_sum(both(s)) * inv_warp;
  }
  // K sums of each warp (of c, c^2 and, for K = 4, g, g c), those of the whole row afterwards; *shift: what c + shift
  // is the difference to the row's mean.  sh: two rooms of K + 2 floats a warp, taken in turn, so that one barrier
  // is enough.
  static constexpr int ROOM = 8;
  template <int K>
  __device__ __forceinline__ void join(float m, float (&q)[K], float* sh, int& turn, float* shift) const {
    const float v = warp_sums<K>(q);
    if constexpr (T == 32) {
#pragma unroll
      for (int k = 0; k < K; ++k) q[k] = __shfl_sync(0xffffffffu, v, k);
      const float off = q[0] * inv_d;
      q[1] = fmaf(-off, q[0], q[1]);
      if constexpr (K == 4) q[3] = fmaf(-off, q[2], q[3]);
      *shift = -off;
    } else {
      float* room = sh + (turn * kBlock<T> / T + threadIdx.x / T) * (T / 32) * ROOM;
      turn ^= 1;
      const int lane = threadIdx.x & 31;
      float* mine = room + (t >> 5) * ROOM;
      if (lane < K) mine[lane] = v;
      else if (lane == K) mine[6] = m;
      else if (lane == K + 1) mine[7] = static_cast<float>(n_warp);
      row_barrier();
      // differences to warp 0's mean: small numbers, whose sums lose nothing
      const float m0 = room[6];
      float a = 0.f;
#pragma unroll 4
      for (int w = 0; w < T / 32; ++w) {
        const float* e = room + w * ROOM;
        a += fmaf(e[7], e[6] - m0, e[0]);
      }
      const float mean = a * inv_d;  // of the row, less m0
      float q1 = 0.f, q2 = 0.f, q3 = 0.f;
#pragma unroll 4
      for (int w = 0; w < T / 32; ++w) {
        const float* e = room + w * ROOM;
        const float off = (e[6] - m0) - mean;
        q1 += fmaf(off, fmaf(e[7], off, 2.f * e[0]), e[1]);
        if constexpr (K == 4) {
          q2 += e[2];
          q3 += fmaf(off, e[2], e[3]);
        }
      }
      q[1] = q1;
      if constexpr (K == 4) q[2] = q2, q[3] = q3;
      *shift = (m - m0) - mean;
    }
  }
};
// The next rows of ARRAYS arrays, on their way into shared memory while the current one is summed.  Each thread
// copies the vectors that it will read itself: no thread waits for another, and no register holds what is still to
// come.  Single bf16 (rows that are not even 4-byte aligned) are loaded where they are used.
template <typename E, int V, int T, int NV, int ARRAYS, bool FULL>
struct Ahead {
  static constexpr int BYTES_EACH = Raw<E, V>::BYTES;
  static constexpr bool COPIES = BYTES_EACH >= 4;
  static constexpr size_t STAGE = static_cast<size_t>(ARRAYS) * NV * kBlock<T> * BYTES_EACH;
  static constexpr int STAGES = !COPIES ? 0 : STAGE <= 16384 ? 3 : 2;
  static constexpr size_t BYTES = STAGES * STAGE;
  using Row = RowOf<E, V, T, NV, FULL>;
  const Row& p;
  const E* base[ARRAYS];
  int64_t ld[ARRAYS];
  int64_t N, step;
  uint32_t room;  // of the block, in shared memory
  int stage = 0;
  Raw<E, V> now[COPIES ? 1 : ARRAYS][COPIES ? 1 : NV];

  __device__ __forceinline__ uint32_t slot(int st, int array, int i) const {
    return room + (((st * ARRAYS + array) * NV + i) * kBlock<T> + threadIdx.x) * BYTES_EACH;
  }
  __device__ __forceinline__ void issue(int64_t row, int st) {
    if constexpr (COPIES) {
      if (row < N) {
#pragma unroll
        for (int k = 0; k < ARRAYS; ++k) {
#pragma unroll
          for (int i = 0; i < NV; ++i)
            if (p.in(i)) {
              const E* from = base[k] + row * ld[k] + p.col(i);
              if constexpr (BYTES_EACH == 16) ptx::copy16_async(slot(st, k, i), from, true);
              else ptx::copy4_async(slot(st, k, i), from);
            }
        }
      }
      ptx::copy_commit();
    }
  }
  // Before the first row.
  __device__ __forceinline__ void begin(int64_t row) {
#pragma unroll
    for (int st = 0; st + 1 < STAGES; ++st) issue(row + st * step, st);
  }
  // The row is there; the one STAGES - 1 steps on is sent for.
  __device__ __forceinline__ void next(int64_t row) {
    if constexpr (COPIES) {
      issue(row + (STAGES - 1) * step, stage == 0 ? STAGES - 1 : stage - 1);
      ptx::copy_wait<STAGES - 1>();
    } else {
#pragma unroll
      for (int k = 0; k < ARRAYS; ++k) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (p.in(i)) now[k][i] = load_raw_once<E, V>(base[k] + row * ld[k] + p.col(i));
      }
    }
  }
  __device__ __forceinline__ Raw<E, V> get(int array, int i) const {
    if constexpr (BYTES_EACH == 16) {
      return Raw<E, V>{ptx::ld_shared_v4(slot(stage, array, i))};
    } else if constexpr (COPIES) {
      return Raw<E, V>{ptx::ld_shared_u32(slot(stage, array, i))};
    } else {
      return now[array][i];
    }
  }
  __device__ __forceinline__ void done() {
    if constexpr (COPIES) stage = stage + 1 == STAGES ? 0 : stage + 1;
  }
};
// 1 / sqrt(var + eps) from the sum of squared differences; NaN where that is not finite (an inf or NaN in
// the row).
__device__ __forceinline__ float inverse_deviation(float squares, float inv_d, float eps) {
  if (!(squares < INFINITY)) return NAN;
  return rsqrtf(fmaf(fmaxf(squares, 0.f), inv_d, eps));
}

template <typename E, int V, int T, int NV, bool FULL>
__global__ void __launch_bounds__(kBlock<T>, kForwardResident<T, NV, V < kVec<E>>)
    layer_norm_kernel(const NormArgs a) {
  using Row = RowOf<E, V, T, NV, FULL>;
  __shared__ alignas(16) float sh[2 * kBlock<T> / 32 * Row::ROOM];
  constexpr int ROWS = kBlock<T> / T;
  const Row p(a.d);
  const int64_t step = static_cast<int64_t>(gridDim.x) * ROWS;
  int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / T;
  const E* w = static_cast<const E*>(a.w);
  const E* b = static_cast<const E*>(a.b);
  extern __shared__ uint4 rows_ahead[];
  int turn = 0;
  ptx::wait_for_previous();
  ptx::launch_dependents();
  Ahead<E, V, T, NV, 1, FULL> ahead{p, {static_cast<const E*>(a.x)}, {a.ldx}, a.N, step, ptx::smem_addr(rows_ahead)};
  ahead.begin(row);
  Raw<E, V> rw[NV], rb[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    rw[i] = w && p.in(i) ? load_raw<E, V>(w + p.col(i)) : zero_raw<E, V>();
    rb[i] = b && p.in(i) ? load_raw<E, V>(b + p.col(i)) : zero_raw<E, V>();
  }
  for (; row < a.N; row += step) {
    stay_packed(rw);
    stay_packed(rb);
    ahead.next(row);
    auto x = [&](int i) { return ahead.get(0, i); };
    const float m = p.mean_of(x);
    Lane<V> minus, s0, s1;
    spread(-m, minus);
    spread(0.f, s0);
    spread(0.f, s1);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!p.in(i)) continue;
      Lane<V> v[kLanes<V>];
      unpack2<E, V>(x(i), v);
#pragma unroll
      for (int j = 0; j < kLanes<V>; ++j) {
        const Lane<V> c = add2(v[j], minus);
        s0 = add2(s0, c);
        s1 = fma2(c, c, s1);
      }
    }
    float q[2] = {both(s0), both(s1)}, shift;
    p.template join<2>(m, q, sh, turn, &shift);
    Lane<V> r2, shift2;
    spread(inverse_deviation(q[1], p.inv_d, a.eps), r2);
    spread(shift, shift2);
    E* out = static_cast<E*>(a.y) + row * a.ldo;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!p.in(i)) continue;
      Lane<V> v[kLanes<V>], fw[kLanes<V>], fb[kLanes<V>];
      unpack2<E, V>(x(i), v);
      unpack2<E, V>(rw[i], fw);
      unpack2<E, V>(rb[i], fb);
#pragma unroll
      for (int j = 0; j < kLanes<V>; ++j) {
        Lane<V> o = mul2(add2(add2(v[j], minus), shift2), r2);
        if (w) o = b ? fma2(o, fw[j], fb[j]) : mul2(o, fw[j]);
        else if (b) o = add2(o, fb[j]);
        v[j] = o;
      }
      store_raw<E, V>(out + p.col(i), pack2<E, V>(v));
    }
    ahead.done();
  }
}

// PARTS = false: neither dw nor db is wanted.  Roundings are written out so that dX is the same in both.
template <typename E, int V, int T, int NV, bool FULL, bool PARTS>
__global__ void __launch_bounds__(kBlock<T>, kGradResident<T, NV, V < kVec<E>>)
    layer_norm_grad_kernel(const NormArgs a) {
  using Row = RowOf<E, V, T, NV, FULL>;
  __shared__ alignas(16) float sh[2 * kBlock<T> / 32 * Row::ROOM];
  constexpr int ROWS = kBlock<T> / T;
  const Row p(a.d);
  const int64_t step = static_cast<int64_t>(gridDim.x) * ROWS;
  int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / T;
  const E* w = static_cast<const E*>(a.w);
  extern __shared__ uint4 rows_ahead[];
  int turn = 0;
  ptx::wait_for_previous();
  ptx::launch_dependents();
  if (a.flags && blockIdx.x == 0 && threadIdx.x == 0) *a.flags = 0u;  // nothing here can fail on the device
  Ahead<E, V, T, NV, 2, FULL> ahead{p,     {static_cast<const E*>(a.x), static_cast<const E*>(a.dy)}, {a.ldx, a.ldy}, a.N, step,
                              ptx::smem_addr(rows_ahead)};
  ahead.begin(row);
  constexpr int L = kLanes<V>;
  Raw<E, V> rw[NV];
  Lane<V> sw[PARTS ? NV : 1][L], sb[PARTS ? NV : 1][L];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    rw[i] = w && p.in(i) ? load_raw<E, V>(w + p.col(i)) : zero_raw<E, V>();
    if (PARTS) {
#pragma unroll
      for (int j = 0; j < L; ++j) spread(0.f, sw[i][j]), spread(0.f, sb[i][j]);
    }
  }
  for (; row < a.N; row += step) {
    stay_packed(rw);
    ahead.next(row);
    auto x = [&](int i) { return ahead.get(0, i); };
    auto dy = [&](int i) { return ahead.get(1, i); };
    const float m = p.mean_of(x);
    Lane<V> minus, s0, s1, s2, s3;  // sums of c, c^2, g, g c
    spread(-m, minus);
    spread(0.f, s0);
    s1 = s2 = s3 = s0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!p.in(i)) continue;
      Lane<V> v[L], g[L], fw[L];
      unpack2<E, V>(x(i), v);
      unpack2<E, V>(dy(i), g);
      unpack2<E, V>(rw[i], fw);
#pragma unroll
      for (int j = 0; j < L; ++j) {
        const Lane<V> c = add2(v[j], minus);
        if (w) g[j] = mul2(g[j], fw[j]);
        s0 = add2(s0, c);
        s1 = fma2(c, c, s1);
        s2 = add2(s2, g[j]);
        s3 = fma2(g[j], c, s3);
      }
    }
    float q[4] = {both(s0), both(s1), both(s2), both(s3)}, shift;
    stay_packed(rw);
    p.template join<4>(m, q, sh, turn, &shift);
    const float r = inverse_deviation(q[1], p.inv_d, a.eps);
    Lane<V> r2, shift2, a1, a2;
    spread(r, r2);
    spread(shift, shift2);
    spread(-(q[2] * p.inv_d) * r, a1);      // -r mean(g)
    spread(-(q[3] * p.inv_d * r) * r, a2);  // -r mean(g x^)
    E* out = static_cast<E*>(a.y) + row * a.ldo;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!p.in(i)) continue;
      Lane<V> v[L], g[L], fw[L];
      unpack2<E, V>(x(i), v);
      unpack2<E, V>(dy(i), g);
      unpack2<E, V>(rw[i], fw);
#pragma unroll
      for (int j = 0; j < L; ++j) {
        const Lane<V> h = mul2(add2(add2(v[j], minus), shift2), r2);
        if (PARTS) {
          sw[i][j] = fma2(g[j], h, sw[i][j]);
          sb[i][j] = add2(sb[i][j], g[j]);
        }
        if (w) g[j] = mul2(g[j], fw[j]);
        g[j] = fma2(h, a2, fma2(g[j], r2, a1));
      }
      if (a.y) store_raw<E, V>(out + p.col(i), pack2<E, V>(g));
    }
    ahead.done();
  }
  if constexpr (PARTS) {
    // [2][d], where the block's rows meet one after the other
    float* acc = reinterpret_cast<float*>(rows_ahead);
#pragma unroll 1
    for (int k = 0; k < ROWS; ++k) {
      if (ROWS > 1) __syncthreads();
      if (static_cast<int>(threadIdx.x) / T != k) continue;
      float* out = k < ROWS - 1 ? acc : a.part + static_cast<int64_t>(blockIdx.x) * a.d;
      const int64_t apart = k < ROWS - 1 ? a.d : static_cast<int64_t>(gridDim.x) * a.d;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (!p.in(i)) continue;
#pragma unroll
        for (int j = 0; j < L; ++j) {
          const int c = p.col(i) + j * (V / L);
          Lane<V> u = sw[i][j], v = sb[i][j];
          if (k > 0) {
            u = add2(u, *reinterpret_cast<const Lane<V>*>(acc + c));
            v = add2(v, *reinterpret_cast<const Lane<V>*>(acc + a.d + c));
          }
          *reinterpret_cast<Lane<V>*>(out + c) = u;
          *reinterpret_cast<Lane<V>*>(out + apart + c) = v;
        }
      }
    }
  }
}

// ------------------------------------------------------------------- rows wider than the registers
// The same with rows re-read (from L2 as a rule): once for each sum and once for the result.
template <typename E, int V, bool STATS>
__global__ void __launch_bounds__(1024) layer_norm_wide_kernel(const NormArgs a) {
  __shared__ float sh1[2 * 32], sh[2 * 4 * 32];
  const E* w = static_cast<const E*>(a.w);
  const E* b = static_cast<const E*>(a.b);
  const float inv_d = 1.f / static_cast<float>(a.d);
  int turn = 0, turn4 = 0;
  ptx::wait_for_previous();
  ptx::launch_dependents();
  if (STATS && blockIdx.x == 0 && threadIdx.x == 0) *a.flags = 0u;
  for (int64_t row = blockIdx.x; row < a.N; row += gridDim.x) {
    const E* x = static_cast<const E*>(a.x) + row * a.ldx;
    const E* dy = static_cast<const E*>(a.dy) + row * a.ldy;  // STATS
    float s[1] = {0.f};
    for (int c = threadIdx.x * V; c < a.d; c += 1024 * V) {
      float v[V];
      unpack<E, V>(load_raw<E, V>(x + c), v);
#pragma unroll
      for (int j = 0; j < V; ++j) s[0] += v[j];
    }
    sum_over<1024, 1>(s, sh1, turn);
    const float mean = s[0] * inv_d;
    float q[4] = {0.f, 0.f, 0.f, 0.f};
    for (int c = threadIdx.x * V; c < a.d; c += 1024 * V) {
      float v[V], g[V], fw[V];
      unpack<E, V>(load_raw<E, V>(x + c), v);
      if (STATS) unpack<E, V>(load_raw<E, V>(dy + c), g);
      if (STATS && w) unpack<E, V>(load_raw<E, V>(w + c), fw);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        v[j] -= mean;
        q[0] += v[j];
        q[1] = fmaf(v[j], v[j], q[1]);
        if (STATS) {
          if (w) g[j] = __fmul_rn(g[j], fw[j]);
          q[2] += g[j];
          q[3] = fmaf(g[j], v[j], q[3]);
        }
      }
    }
    sum_over<1024, 4>(q, sh, turn4);
    const float off = q[0] * inv_d;
    float r = 1.f / sqrtf(fmaxf(fmaf(-off, off, q[1] * inv_d), 0.f) + a.eps);
    if (!(q[1] < INFINITY)) r = NAN;  // as inverse_deviation(): fmaxf above drops a NaN, and 1 / inf would be 0
    if constexpr (STATS) {
      // x^ = (x - mean - off) r keeps its bits only with both differences taken in turn
      if (threadIdx.x == 0) {
        a.stats[2 * row] = make_float4(mean, off, r, 0.f);
        a.stats[2 * row + 1] = make_float4(q[2] * inv_d, (q[3] - off * q[2]) * inv_d * r, 0.f, 0.f);
      }
    } else {
      E* out = static_cast<E*>(a.y) + row * a.ldo;
      for (int c = threadIdx.x * V; c < a.d; c += 1024 * V) {
        float v[V], fw[V], fb[V];
        unpack<E, V>(load_raw<E, V>(x + c), v);
        if (w) unpack<E, V>(load_raw<E, V>(w + c), fw);
        if (b) unpack<E, V>(load_raw<E, V>(b + c), fb);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          float o = ((v[j] - mean) - off) * r;
          if (w) o = b ? fmaf(o, fw[j], fb[j]) : o * fw[j];
          else if (b) o += fb[j];
          v[j] = o;
        }
        store_raw<E, V>(out + c, pack<E, V>(v));
      }
    }
  }
}

// Gradients of wide rows from their statistics: a block owns 256 x V columns and every gridDim.y-th row.
template <typename E, int V>
__global__ void __launch_bounds__(256) layer_norm_wide_grad_kernel(const NormArgs a) {
  ptx::wait_for_previous();
  ptx::launch_dependents();
  const int64_t c = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * V;
  if (c >= a.d) return;
  const E* w = static_cast<const E*>(a.w);
  float fw[V], sw[V], sb[V];
  if (w) unpack<E, V>(load_raw<E, V>(w + c), fw);
#pragma unroll
  for (int j = 0; j < V; ++j) sw[j] = sb[j] = 0.f;
  for (int64_t row = blockIdx.y; row < a.N; row += gridDim.y) {
    const float4 p = a.stats[2 * row], m = a.stats[2 * row + 1];
    float v[V], g[V];
    unpack<E, V>(load_raw<E, V>(static_cast<const E*>(a.x) + row * a.ldx + c), v);
    unpack<E, V>(load_raw<E, V>(static_cast<const E*>(a.dy) + row * a.ldy + c), g);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float h = __fmul_rn((v[j] - p.x) - p.y, p.z);
      sw[j] = fmaf(g[j], h, sw[j]);
      sb[j] += g[j];
      if (w) g[j] = __fmul_rn(g[j], fw[j]);
      g[j] = __fmul_rn(p.z, fmaf(-h, m.y, g[j] - m.x));
    }
    if (a.y) store_raw<E, V>(static_cast<E*>(a.y) + row * a.ldo + c, pack<E, V>(g));
  }
  if (a.part) {
    float* pw = a.part + static_cast<int64_t>(blockIdx.y) * a.d + c;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      pw[j] = sw[j];
      pw[static_cast<int64_t>(gridDim.y) * a.d + j] = sb[j];
    }
  }
}

// out[c] = sum over the parts, 32 columns a block and every 32nd part a warp; blockIdx.y: dw, db.
template <typename E>
__global__ void __launch_bounds__(1024, 2)
    layer_norm_sum_kernel(const float* part, int parts, int d, E* dw, E* db) {
  __shared__ float sh[32][33];
  ptx::wait_for_previous();
  ptx::launch_dependents();
  E* out = blockIdx.y == 0 ? dw : db;
  if (!out) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  const float* p = part + blockIdx.y * static_cast<int64_t>(parts) * d;
  float s = 0.f;
  if (c < d) {
#pragma unroll 8
    for (int k = warp; k < parts; k += 32) s += p[static_cast<int64_t>(k) * d + c];
  }
  sh[warp][lane] = s;
  __syncthreads();
  s = sh[lane][warp];  // column `warp` of the block, one part of its sum a lane
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int64_t mine = static_cast<int64_t>(blockIdx.x) * 32 + warp;
  if (lane == 0 && mine < d) out[mine] = static_cast<E>(s);
}

// ---------------------------------------------------------------------------------- host side
bool aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool dtype_ok(lce_dtype_t dt) { return dt == LCE_BF16 || dt == LCE_F32; }
size_t elem(lce_dtype_t dt) { return dt == LCE_BF16 ? 2 : 4; }
bool sizes_ok(int64_t N, int64_t d) {
  return N >= 0 && N <= kMaxRows && d >= 1 && d <= kMaxWidth && N * d <= kMaxElements;
}
bool stride_ok(int64_t ld, int64_t d, int64_t N) {
  return ld >= d && ld <= kMaxElements && (N <= 1 || ld <= (int64_t(1) << 62) / N);
}

// Widest row of the register kernels, in vectors of 16 bytes: 16,384 bf16 or 8,192 fp32.  Of narrow vectors: 8,192 bf16
// either way, and by words of 4 bytes 8,192 bf16 or 4,096 fp32 forward, twice that backward.
constexpr int kForwardVectors = 2048, kBackwardVectors = 2048;

// A dependent launch of one of the kernels above on as many blocks as the SMs hold at once; `resident` keeps how many
// an SM of a device holds, once the kernel may use its shared memory there.
template <typename K>
cudaError_t launch_rows(K kernel, int64_t blocks, int threads, size_t smem, PerDevice<kMaxDevices>& resident, int* grid,
                        int64_t most, int num_sms, cudaStream_t s, const NormArgs& a) {
  int dev = 0, n = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = resident.get(dev, [&](int* blocks_per_sm) {
    const cudaError_t set =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    return set != cudaSuccess ? set
                              : cudaOccupancyMaxActiveBlocksPerMultiprocessor(blocks_per_sm, kernel, threads, smem);
  }, &n);
  if (e != cudaSuccess) return e;
  *grid = static_cast<int>(std::min<int64_t>({blocks, int64_t(num_sms) * n, most}));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(*grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {dependent_launch()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}
template <typename E, int V, int T, int NV, bool FULL = false>
cudaError_t forward_rows(const NormArgs& a, int num_sms, cudaStream_t s) {
  if constexpr (V > 1 && !FULL) {
    if (a.d == T * NV * V) return forward_rows<E, V, T, NV, true>(a, num_sms, s);
  }
  static PerDevice<kMaxDevices> resident;
  constexpr int ROWS = kBlock<T> / T;
  int grid;
  return launch_rows(layer_norm_kernel<E, V, T, NV, FULL>, (a.N + ROWS - 1) / ROWS, kBlock<T>,
                     Ahead<E, V, T, NV, 1, FULL>::BYTES, resident, &grid, a.N, num_sms, s, a);
}
// Classes of rows by their vectors, each twice the one before: what a class does not fill is masked, and a row that fills
// it asks for nothing.  Between 512 and 1,024 there is one more, of 768 (no others were tried): us with it / without, bf16,
// forward of 32768 rows and backward of 16384: 4104 wide 136 / 149 and 120 / 127, 4608 136 / 151 and 111 / 118,
// 5120 142 / 155 and 115 / 121, 5632 152 / 162 and 126 / 132, 6144 129 / 168 and 107 / 135.
template <typename E, int V>
cudaError_t forward(const NormArgs& a, int num_sms, cudaStream_t s) {
  const int64_t nv = (a.d + V - 1) / V;
  if constexpr (V < kVec<E>) {  // narrow vectors, more of them a thread
    constexpr int NV = Raw<E, V>::BYTES == 4 ? 8 : 16;
    if (nv <= 32 * NV) return forward_rows<E, V, 32, NV>(a, num_sms, s);
    if (nv <= 64 * NV) return forward_rows<E, V, 64, NV>(a, num_sms, s);
    if (nv <= 128 * NV) return forward_rows<E, V, 128, NV>(a, num_sms, s);
    if (nv <= 256 * NV) return forward_rows<E, V, 256, NV>(a, num_sms, s);
    if (nv <= 512 * NV) return forward_rows<E, V, 512, NV>(a, num_sms, s);
  } else {
  if (nv <= 32) return forward_rows<E, V, 32, 1>(a, num_sms, s);
  if (nv <= 64) return forward_rows<E, V, 32, 2>(a, num_sms, s);
  if (nv <= 128) return forward_rows<E, V, 32, 4>(a, num_sms, s);
  if (nv <= 256) return forward_rows<E, V, 64, 4>(a, num_sms, s);
  if (nv <= 512) return forward_rows<E, V, 128, 4>(a, num_sms, s);
  if (nv <= 768) return forward_rows<E, V, 192, 4>(a, num_sms, s);
  if (nv <= 1024) return forward_rows<E, V, 256, 4>(a, num_sms, s);
  if (nv <= kForwardVectors) return forward_rows<E, V, 512, 4>(a, num_sms, s);
  }
  const int grid = static_cast<int>(std::min<int64_t>(a.N, 2 * num_sms));
  return launch_kernel(layer_norm_wide_kernel<E, V, false>, dim3(grid), 1024, s, a);
}

int64_t wide_chunks(int64_t N, int64_t d, int num_sms) {
  const int64_t tiles = (d + 2047) / 2048;
  return std::max<int64_t>(1, std::min<int64_t>({N, (int64_t(num_sms) * 8 + tiles - 1) / tiles, max_parts(N, d)}));
}

template <typename E, int V, int T, int NV, bool FULL = false>
cudaError_t backward_rows(const NormArgs& a, int* parts, int num_sms, cudaStream_t s) {
  if constexpr (V > 1 && !FULL) {
    if (a.d == T * NV * V) return backward_rows<E, V, T, NV, true>(a, parts, num_sms, s);
  }
  static PerDevice<kMaxDevices> resident[2];
  constexpr int ROWS = kBlock<T> / T;
  const int64_t blocks = (a.N + ROWS - 1) / ROWS;
  // two blocks an SM while a block has no more than four rows: partial sums are written and read once more
  const int64_t most = a.part ? std::min(max_parts(a.N, a.d), std::max<int64_t>(2 * num_sms, a.N / 4)) : a.N;
  // where a block has several rows, their sums meet in the same memory
  const size_t meet = ROWS > 1 ? 2 * sizeof(float) * NV * V * T : 0;
  const size_t bytes = std::max(Ahead<E, V, T, NV, 2, FULL>::BYTES, meet);
  if (a.part)
    return launch_rows(layer_norm_grad_kernel<E, V, T, NV, FULL, true>, blocks, kBlock<T>, bytes, resident[1], parts, most, num_sms, s, a);
  return launch_rows(layer_norm_grad_kernel<E, V, T, NV, FULL, false>, blocks, kBlock<T>, bytes, resident[0], parts, most, num_sms, s, a);
}
template <typename E, int V>
cudaError_t backward(const NormArgs& a, int* parts, int num_sms, cudaStream_t s) {
  const int64_t nv = (a.d + V - 1) / V;
  if constexpr (V < kVec<E>) {
    constexpr int NV = Raw<E, V>::BYTES == 4 ? 8 : 16;
    if (nv <= 32 * NV) return backward_rows<E, V, 32, NV>(a, parts, num_sms, s);
    if (nv <= 64 * NV) return backward_rows<E, V, 64, NV>(a, parts, num_sms, s);
    if (nv <= 128 * NV) return backward_rows<E, V, 128, NV>(a, parts, num_sms, s);
    if (nv <= 256 * NV) return backward_rows<E, V, 256, NV>(a, parts, num_sms, s);
    if (nv <= 512 * NV) return backward_rows<E, V, 512, NV>(a, parts, num_sms, s);
    if (NV < 16 && nv <= 512 * 16) return backward_rows<E, V, 512, 16>(a, parts, num_sms, s);
  } else {
  if (nv <= 32) return backward_rows<E, V, 32, 1>(a, parts, num_sms, s);
  if (nv <= 64) return backward_rows<E, V, 32, 2>(a, parts, num_sms, s);
  if (nv <= 128) return backward_rows<E, V, 32, 4>(a, parts, num_sms, s);
  if (nv <= 256) return backward_rows<E, V, 64, 4>(a, parts, num_sms, s);
  if (nv <= 512) return backward_rows<E, V, 64, 8>(a, parts, num_sms, s);
  if (nv <= 768) return backward_rows<E, V, 128, 6>(a, parts, num_sms, s);
  if (nv <= 1024) return backward_rows<E, V, 128, 8>(a, parts, num_sms, s);
  if (nv <= kBackwardVectors) return backward_rows<E, V, 256, 8>(a, parts, num_sms, s);
  }
  const int grid = static_cast<int>(std::min<int64_t>(a.N, 2 * num_sms));
  cudaError_t e = launch_kernel(layer_norm_wide_kernel<E, V, true>, dim3(grid), 1024, s, a);
  if (e != cudaSuccess) return e;
  ++g_extra_kernels;
  *parts = static_cast<int>(wide_chunks(a.N, a.d, num_sms));
  const unsigned tiles = static_cast<unsigned>((nv + 255) / 256);
  return launch_kernel(layer_norm_wide_grad_kernel<E, V>, dim3(tiles, *parts), 256, s, a);
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
// Whether rows of d elements may take the path of re-read rows (which depends on their alignment too).
bool may_be_wide(int64_t d) { return d > 8192; }

}  // namespace
}  // namespace lce

using namespace lce;

extern "C" {

size_t lce_layer_norm_workspace_size(int64_t N, int64_t d, lce_dtype_t dtype) {
  if (!dtype_ok(dtype) || !sizes_ok(N, d)) return 0;
  const size_t parts = static_cast<size_t>(max_parts(N, d));
  size_t total = WS_HEADER_BYTES + align256(2 * parts * static_cast<size_t>(d) * sizeof(float));
  if (may_be_wide(d)) total += static_cast<size_t>(N) * 2 * sizeof(float4);
  return total;
}

lce_status_t lce_layer_norm_forward(const void* X, int64_t ldx, const void* weight, const void* bias,
                                    int64_t N, int64_t d, float eps, lce_dtype_t dtype, void* Y,
                                    int64_t ldy, void* stream) {
  if (!dtype_ok(dtype) || !(eps > 0.f) || isinf(eps)) return LCE_ERR_INVALID_ARG;
  if (!sizes_ok(N, d) || !stride_ok(ldx, d, N) || !stride_ok(ldy, d, N)) return LCE_ERR_UNSUPPORTED_SHAPE;
  const size_t e = elem(dtype);
  if ((N > 0 && (!X || !Y)) || !aligned(X, e) || !aligned(Y, e) || !aligned(weight, e) || !aligned(bias, e))
    return LCE_ERR_INVALID_ARG;
  if (N > 0 && X == Y && ldx != ldy && N > 1) return LCE_ERR_INVALID_ARG;
  int num_sms = 0;
  const lce_status_t st = check_device(&num_sms);
  if (st != LCE_OK || N == 0) return st;
  NormArgs a{};
  a.x = X, a.w = weight, a.b = bias, a.y = Y, a.ldx = ldx, a.ldo = ldy, a.N = N;
  a.d = static_cast<int>(d), a.eps = eps;
  auto whole = [&](size_t n) {
    return aligned(X, n) && aligned(Y, n) && aligned(weight, n) && aligned(bias, n) && d * e % n == 0 &&
           (N <= 1 || (ldx * e % n == 0 && ldy * e % n == 0));
  };
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t err = traced(K_NORM, s, [&] {
    if (dtype == LCE_BF16)
      return whole(16)  ? forward<__nv_bfloat16, 8>(a, num_sms, s)
             : whole(4) ? forward<__nv_bfloat16, 2>(a, num_sms, s)
                        : forward<__nv_bfloat16, 1>(a, num_sms, s);
    return whole(16) ? forward<float, 4>(a, num_sms, s) : forward<float, 1>(a, num_sms, s);
  });
  return err == cudaSuccess ? LCE_OK : LCE_ERR_CUDA;
}

lce_status_t lce_layer_norm_backward(const void* X, int64_t ldx, const void* weight, const void* dY,
                                     int64_t ldy, int64_t N, int64_t d, float eps, lce_dtype_t dtype,
                                     void* dX, void* dweight, void* dbias, void* workspace,
                                     size_t ws_bytes, void* stream) {
  if (!dtype_ok(dtype) || !(eps > 0.f) || isinf(eps)) return LCE_ERR_INVALID_ARG;
  if (!sizes_ok(N, d) || !stride_ok(ldx, d, N) || !stride_ok(ldy, d, N)) return LCE_ERR_UNSUPPORTED_SHAPE;
  const size_t e = elem(dtype);
  if ((N > 0 && (!X || !dY)) || !workspace || !aligned(workspace, 16) || !aligned(X, e) ||
      !aligned(dY, e) || !aligned(weight, e) || !aligned(dX, e) || !aligned(dweight, e) ||
      !aligned(dbias, e))
    return LCE_ERR_INVALID_ARG;
  if (ws_bytes < lce_layer_norm_workspace_size(N, d, dtype)) return LCE_ERR_WORKSPACE_TOO_SMALL;
  int num_sms = 0;
  lce_status_t st = check_device(&num_sms);
  if (st != LCE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  NormArgs a{};
  a.x = X, a.w = weight, a.dy = dY, a.y = dX, a.ldx = ldx, a.ldy = ldy, a.ldo = d, a.N = N;
  a.d = static_cast<int>(d), a.eps = eps;
  a.flags = reinterpret_cast<unsigned*>(ws);
  float* part = reinterpret_cast<float*>(ws + WS_HEADER_BYTES);
  a.part = dweight || dbias ? part : nullptr;
  const size_t parts_max = static_cast<size_t>(max_parts(N, d));
  a.stats = reinterpret_cast<float4*>(ws + WS_HEADER_BYTES +
                                      align256(2 * parts_max * static_cast<size_t>(d) * sizeof(float)));
  int parts = 0;
  if (N > 0) {
    auto whole = [&](size_t n) {
      return aligned(X, n) && aligned(dY, n) && aligned(weight, n) && aligned(dX, n) && d * e % n == 0 &&
             (N <= 1 || (ldx * e % n == 0 && ldy * e % n == 0));
    };
    const cudaError_t err = traced(K_NORM_GRAD, s, [&] {
      if (dtype == LCE_BF16)
        return whole(16)  ? backward<__nv_bfloat16, 8>(a, &parts, num_sms, s)
               : whole(4) ? backward<__nv_bfloat16, 2>(a, &parts, num_sms, s)
                          : backward<__nv_bfloat16, 1>(a, &parts, num_sms, s);
      return whole(16) ? backward<float, 4>(a, &parts, num_sms, s) : backward<float, 1>(a, &parts, num_sms, s);
    });
    if (err != cudaSuccess) return LCE_ERR_CUDA;
  } else if (note(cudaMemsetAsync(workspace, 0, sizeof(unsigned), s)) != cudaSuccess) {
    return LCE_ERR_CUDA;
  }
  if (!a.part) return LCE_OK;
  const cudaError_t err = traced(K_NORM_SUM, s, [&] {
    const dim3 grid(static_cast<unsigned>((d + 31) / 32), 2);
    if (dtype == LCE_BF16)
      return launch_kernel(layer_norm_sum_kernel<__nv_bfloat16>, grid, 1024, s, part, parts, a.d,
                           static_cast<__nv_bfloat16*>(dweight), static_cast<__nv_bfloat16*>(dbias));
    return launch_kernel(layer_norm_sum_kernel<float>, grid, 1024, s, part, parts, a.d,
                         static_cast<float*>(dweight), static_cast<float*>(dbias));
  });
  return err == cudaSuccess ? LCE_OK : LCE_ERR_CUDA;
}

}  // extern "C"
