// Sampling from logits with temperature, top-k, top-p and min-p (declared in include/lce.h).
//
//   w_i = exp((z_i - max z) / temperature);  top-k, top-p and min-p keep a set that is a prefix of the
//   tokens ordered by (logit descending, index ascending);  the token is where the kept weights, summed
//   in the order of indices, pass u times their total
//
// One launch; a cluster of 1 to 8 CTAs holds a row in its shared memory (read in place where it does not fit), which
// is read from memory once.  Nothing is sorted but a few hundred candidates, in the cluster's first CTA:
//   - top-k up to 512: where k / ctas threads of each CTA have a largest logit above some bin's edge, no token behind
//     that bin is among the k largest.  What is left is ranked, cut by top-k, top-p and min-p, and drawn from there.
//   - top-p of all tokens: counts in 4096 bins of equal width between the largest and the smallest logit that has a
//     weight tell in which bin the border lies; one pass then adds all weights exactly and lists the tokens
//     around that bin (nucleus).  bf16 logits are counted by value, which gives the sums and the border at once
//     (nucleus_by_value).
//   - Otherwise (top-k of many, top-p of what top-k left, borders that the counts misplace) a search for the border, a
//     logit and an index: exact counts or weights in 2048 bins, the border's bin ranked if it holds at most 512
//     tokens, cut into 2048 bins again if more, decided by the indices if all its logits are equal (lower).
//   - A last pass adds the weights of the kept tokens by warp and CTA, and the one chunk in which the
//     target lies is added up token by token.
//
// Which token comes out depends on which side of a border a sum falls on, so the sums have to be right to
// many more bits than fp32 has, and must not depend on the order of additions.  Weights are integers of 2^-39:
// z log2(e) / temperature as a product with a constant of two floats, cut at an integer k of 256ths, whose difference
// to the product takes one rounding; a table of 2^(j/256) in two floats and a cubic for the rest, |rest| <= 1/2 of
// 256ths; relative error 2^-31.7 at most, 2^-34 as a rule, and up to a unit for the bits below it.  Sums of integers are
// exact in any order, also by atomics.
// Double precision exponentials would cost ten times as much here (two operations a cycle and SM); with errors of 2^-23
// about one row in some thousand would draw another token.
//
// Bound by latency: a row takes a dozen short steps, one after the other, which show as waits at barriers and as first
// executions of code, and where a row is not staged by reading L2 again in each.  Issue slots are 39 to 44% busy (25
// instructions for a weight, 6 for a bin; 125 a logit over all steps of top-p of fp32), so that instructions alone bound
// nothing.  Inside a captured graph over logits that are not in L2: 1 x 151,936 bf16 greedy 4.1 us, top-k 50 and top-p 0.95 12, all
// tokens 11, top-p 0.9 24; 64 x 151,936 fp32 greedy 17, all 37, top-p 0.9 78; 128 x 200,000 bf16 min-p 0.05 36 to 40, top-p
// 0.9 106 (by bins and lists 208).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <float.h>
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

constexpr int THREADS = 512, WARPS = THREADS / 32;
constexpr int MAX_CLUSTER = 8;
constexpr int BINS = 2048;
constexpr int LIST = 512;
constexpr int WEIGHT_BITS = 39;
constexpr float T_MAX = 40.f;  // weights of 2^-40 and less are 0
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 512;
constexpr int64_t kMaxVocabulary = int64_t(1) << 22;  // sums of weights stay below 2^62

// ------------------------------------------------------------------------------------ weights
// 2^39 2^((255 - j) / 256), j = 0 .. 255, as a float and the rest, from the exponential series.
struct Powers {
  float hi[256], lo[256];
  constexpr Powers() : hi(), lo() {
    for (int j = 0; j < 256; ++j) {
      const double y = (255 - j) * (0.693147180559945309417 / 256);
      double term = 1.0, sum = 1.0;
      for (int n = 1; n < 30; ++n) {
        term *= y / n;
        sum += term;
      }
      sum *= 549755813888.0;
      hi[j] = static_cast<float>(sum);
      lo[j] = static_cast<float>(sum - static_cast<double>(hi[j]));
    }
  }
};
__device__ const Powers kPowers = Powers();

// What turns a logit into a weight 2^-t: 256 t = whole - z c with c = 256 log2(e) / temperature as two floats and an
// integer just above max c, so that weights are at most 1 and the largest is nearly that.  Where max c is not small,
// 256 t = (max - z) c.
struct Scale {
  float max;         // the row's largest logit
  float c_hi, c_lo;  // c
  float d_max;       // differences to the maximum from which on weights are 0
  bool small;
  int whole;         // 255 and the bits of 1.5 2^23 on top
};

// max - z, 0 for equal infinities too.
__device__ __forceinline__ float below_max(float z, const Scale& s) { return z == s.max ? 0.f : s.max - z; }

constexpr float ROUND = 12582912.f;  // 1.5 2^23: adding it rounds to an integer, which the lowest bits then hold
constexpr int ROUND_BITS = 0x4b400000;

// The temperature's scale; without double precision, of which an SM does two operations a cycle.
__device__ __forceinline__ Scale scale_of(float max, float temperature) {
  constexpr double L = 256 * 1.4426950408889634074;  // 256 log2(e)
  constexpr float L_HI = static_cast<float>(L), L_LO = static_cast<float>(L - static_cast<double>(L_HI));
  Scale s;
  s.max = max;
  const float inverse = ptx::rcp_approx(temperature);  // what it is off by goes into the second float
  const float q = L_HI * inverse;
  if (q < 1e37f) {
    s.c_hi = q;
    s.c_lo = (fmaf(-q, temperature, L_HI) + L_LO) * inverse;
    if (!(fabsf(s.c_lo) <= q)) s.c_lo = 0.f;  // an infinite temperature
  } else {  // every difference is too large
    s.c_hi = 1e37f;
    s.c_lo = 0.f;
  }
  s.d_max = T_MAX * 256.f * ptx::rcp_approx(s.c_hi);
  const float m = max * s.c_hi;
  s.small = fabsf(m) < 2097152.f;  // 2^21; false for an infinite maximum
  s.whole = (s.small ? static_cast<int>(ceilf(m)) + 1 : 0) + 255 + ROUND_BITS;
  return s;
}

// The weight as an integer of 2^-39 from n = 255 + the integer part of 256 t and the rest, at most about 1/2 in
// magnitude, of 256 t.  The shift cuts bits off; the lowest bit, always 1, stands for the half that they are on average.
__device__ __forceinline__ uint64_t power(int n, float rest, const float2* powers) {
  constexpr float A = -0.693147180559945309f / 256.f;  // e^(A rest) - 1
  const float q = rest * fmaf(rest, fmaf(rest, A * A * A / 6.f, A * A / 2.f), A);
  const float2 p = powers[n & 255];
  // the table's value, and what comes to it: below 2^31
  const int more = __float2int_rn(fmaf(q, p.x, p.y));
  const unsigned mantissa = (__float_as_uint(p.x) & 0x7fffffu) | 0x800000u;
  const uint64_t m = static_cast<uint64_t>(mantissa) * 65536u + static_cast<uint64_t>(static_cast<int64_t>(more));
  uint64_t w;
  asm("shr.u64 %0, %1, %2;" : "=l"(w) : "l"(m), "r"(n >> 8));  // 0 from 64 on
  return w | 1;
}
// Of a logit from max - d_max on.
__device__ __forceinline__ uint64_t weight_small(float z, const Scale& s, const float2* powers) {
  const float km = fmaf(z, s.c_hi, ROUND);
  const float k = km - ROUND;  // z c rounded to an integer: its difference to z c takes one rounding of a small number
  return power(s.whole - __float_as_int(km), fmaf(-z, s.c_lo, fmaf(-z, s.c_hi, k)), powers);
}
__device__ __noinline__ uint64_t weight_large(float z, const Scale& s, const float2* powers) {
  const float d = below_max(z, s);
  const float th = d * s.c_hi;
  if (!(th < T_MAX * 256.f)) return 0;
  // what rounding took from the difference and from the product
  const float back = d - s.max;
  const float lost = d == 0.f ? 0.f : (s.max - (d - back)) - (z + back);
  const float tl = fmaf(d, s.c_hi, -th) + fmaf(d, s.c_lo, lost * s.c_hi);
  const float nf = rintf(th);
  return power(static_cast<int>(nf) + 255, (th - nf) + tl, powers);
}
__device__ __forceinline__ uint64_t weight(float z, const Scale& s, const float2* powers) {
  return s.small ? weight_small(z, s, powers) : weight_large(z, s, powers);
}

// Logits in an order of unsigned integers; equal logits have equal keys (-0 is 0).
__device__ __forceinline__ unsigned key_of(float z) {
  const unsigned u = __float_as_uint(z + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float logit_of(unsigned key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// ------------------------------------------------------------------------------------ clusters
__device__ __forceinline__ unsigned cluster_size() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void st_cluster_u64(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
// Every thread of the cluster; warps come here converged.
__device__ __forceinline__ void cluster_barrier() {
  __syncwarp();
  ptx::cluster_sync();
}
__device__ __forceinline__ unsigned ld_cluster_u32(uint32_t addr) {
  unsigned v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint64_t ld_cluster_u64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}
// The barrier in two halves.
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ------------------------------------------------------------------------------------ the row
struct SampleArgs {
  const void* logits;
  int64_t ld, V;
  int slice;       // columns of a CTA
  int chunk;       // of them a warp's, in the last pass: a multiple of a vector
  const float* uniform;
  lce_sampling_t set;
  int64_t* tokens;
  float* logprobs;
};

struct Found {  // where a search ended, written by one CTA into all
  uint64_t before;
  unsigned bin;
  float part;
  float count;  // of the bin's tokens, about
};

// What a CTA tells the others about the tokens that it listed.
struct Listed {
  unsigned count, key_min, key_max;
  unsigned all;  // also those that found no room
};

struct alignas(16) Shared {
  float2 powers[256];
  // counts; or weights, low and high words.  In the cluster's first CTA also the candidates of each CTA (key, and the
  // index inverted), which come when no bin is needed any more.
  union {
    struct {
      unsigned lo[BINS], hi[BINS];
    };
    unsigned fine[2 * BINS];  // counts in bins half as wide
    uint64_t room[BINS];
  };
  uint64_t list[LIST], weights[LIST];  // the candidates together
  unsigned own_listed, own_bound, own_share;
  Listed listed[MAX_CLUSTER];
  uint64_t chunk_total[MAX_CLUSTER], kept_total[MAX_CLUSTER], all_total[MAX_CLUSTER], sure_total[MAX_CLUSTER],
      near_total[MAX_CLUSTER];
  float4 extremes[MAX_CLUSTER];  // largest, smallest, NaN seen
  uint2 bound[MAX_CLUSTER];
  Found found;
  uint64_t border;
  unsigned long long middle;
  uint64_t warp_a[WARPS];
  unsigned warp_n[WARPS], equal_total[MAX_CLUSTER];
  float warp_f[3][WARPS];
  unsigned warp_u[2][WARPS];
};

template <typename E>
struct Row {
  static constexpr int V = kVec<E>;
  const E* base;  // 16-byte aligned, `lead` elements before the slice
  E* staged;      // shared memory laid out alike, or null
  int lead, end;  // the slice is [lead, end) there
  int64_t first;  // column of position `lead`

  // 16 bytes at position j (a multiple of V), -inf outside the slice.  What is not staged is read again.
  __device__ __forceinline__ uint4 load_global(int j) const {
    if (j >= lead && j + V <= end) {
      const uint4* q = reinterpret_cast<const uint4*>(base + j);
      return staged ? __ldcs(q) : __ldg(q);
    }
    unsigned w[4];
    constexpr unsigned NEG = sizeof(E) == 2 ? 0xff80u : 0xff800000u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = 0;
#pragma unroll
      for (int k = 0; k < V / 4; ++k) {
        const int at = j + i * (V / 4) + k;
        unsigned e = NEG;
        if (at >= lead && at < end) {
          if constexpr (sizeof(E) == 2) e = reinterpret_cast<const unsigned short*>(base)[at];
          else e = reinterpret_cast<const unsigned*>(base)[at];
        }
        w[i] |= e << (16 * k);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ uint4 load(int j) const {
    return staged ? *reinterpret_cast<const uint4*>(staged + j) : load_global(j);
  }
  __device__ __forceinline__ float at(int j) const {  // inside the slice
    return static_cast<float>(staged ? staged[j] : base[j]);
  }
  __device__ __forceinline__ int64_t column(int j) const { return first + (j - lead); }
  __device__ __forceinline__ unsigned inverted(int j) const {
    return 0xffffffffu - (static_cast<unsigned>(first) + static_cast<unsigned>(j - lead));
  }
};

// The largest of 16 bytes of logits.
template <typename E>
__device__ __forceinline__ float largest(const uint4& q) {
  if constexpr (sizeof(E) == 2) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&q);
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
  } else {
    return fmaxf(fmaxf(__uint_as_float(q.x), __uint_as_float(q.y)), fmaxf(__uint_as_float(q.z), __uint_as_float(q.w)));
  }
}

// f(V logits, their first position) for the logits of this thread's warp's chunk, all lanes of a warp together; -inf
// outside the slice.  Logits below `cut` may be left out: most 16 bytes of a row hold nothing above it and cost an
// instruction a logit.  (A cut that is NaN leaves out nothing.)
template <typename E, typename F>
__device__ __forceinline__ void for_chunk(const Row<E>& row, int chunk, float cut, F&& f) {
  constexpr int V = kVec<E>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int stop = min((warp + 1) * chunk, row.end);
#pragma unroll 2
  for (int j0 = warp * chunk; j0 < stop; j0 += 32 * V) {
    const int j = j0 + lane * V;
    constexpr unsigned NEG = sizeof(E) == 2 ? 0xff80ff80u : 0xff800000u;
    const uint4 q = j < stop ? row.load(j) : make_uint4(NEG, NEG, NEG, NEG);
    if (!__any_sync(0xffffffffu, !(largest<E>(q) < cut))) continue;
    float v[V];
    unpack<E, V>(Raw<E, V>{q}, v);
    f(v, j);
  }
}

// f(position, valid) for the logits among v that `candidate` holds for, one of each lane at a time: where few do, that
// is far less than one after the other.  All lanes call f.
template <int V, typename C, typename F>
__device__ __forceinline__ void for_some(const float (&v)[V], int j, C&& candidate, F&& f) {
  unsigned mask = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) mask |= candidate(v[i]) ? 1u << i : 0u;
  while (__any_sync(0xffffffffu, mask != 0)) {
    f(j + __ffs(mask) - 1, mask != 0);
    mask &= mask - 1;
  }
}

// Exclusive sum over the threads in order; *total over all.
__device__ __forceinline__ uint64_t scan(uint64_t v, uint64_t* sh, uint64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  __syncthreads();  // sh may still be read from the call before
  if (lane == 31) sh[warp] = incl;
  __syncthreads();
  uint64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += sh[w];
    all += sh[w];
  }
  *total = all;
  return before + incl - v;
}

__device__ __forceinline__ int power_of_two(int n) {
  int p = 32;
  while (p < n) p <<= 1;
  return p;
}
// Sorts up to LIST different numbers x, one a thread, 0 where there is none: largest first, 0 behind them.  `size` is a
// power of two that no number lies behind, from 32 on.  All threads of the block come here.
// Up to 256 each number's place is counted, by several threads (0.4 us for 128); comparing all pairs takes longer than
// the 45 steps of a sorting network from 512 on (2.5 us; 128 numbers 2.2).
__device__ __forceinline__ uint64_t sort_down(uint64_t x, int size, uint64_t* sh) {
  const int t = threadIdx.x;
  if (size <= 256) {
    __syncthreads();
    if (t < size) sh[t] = x;
    __syncthreads();
    const int share = THREADS / size;
    const uint64_t mine = sh[t / share];
    int place = 0;
#pragma unroll 4
    for (int j = t & (share - 1); j < size; j += share) place += sh[j] > mine;
    for (int o = 1; o < share; o <<= 1) place += __shfl_xor_sync(0xffffffffu, place, o);
    __syncthreads();
    if (t < size) sh[t] = 0;
    __syncthreads();
    if (mine != 0 && (t & (share - 1)) == 0) sh[place] = mine;
    __syncthreads();
    return t < size ? sh[t] : 0;
  }
  // partners within a warp exchange by shuffles, others through sh
  for (int k = 2; k <= size; k <<= 1) {
    for (int j = k >> 1; j > 0; j >>= 1) {
      uint64_t other;
      if (j >= 32) {
        __syncthreads();
        if (t < size) sh[t] = x;
        __syncthreads();
        other = t < size ? sh[t ^ j] : 0;
      } else {
        other = __shfl_xor_sync(0xffffffffu, x, j);
      }
      // the lower of the two places takes the larger in blocks that go down
      const bool larger = ((t & j) == 0) == ((t & k) == 0);
      if ((x < other) == larger) x = other;
    }
  }
  return x;
}

// Settings of a row.
struct Settings {
  float temperature, top_p, min_p;
  int top_k;
};
__device__ __forceinline__ Settings settings_of(const SampleArgs& a, int64_t row) {
  Settings s;
  s.temperature = a.set.temperatures ? a.set.temperatures[row] : a.set.temperature;
  s.top_p = a.set.top_ps ? a.set.top_ps[row] : a.set.top_p;
  s.min_p = a.set.min_ps ? a.set.min_ps[row] : a.set.min_p;
  s.top_k = a.set.top_ks ? a.set.top_ks[row] : a.set.top_k;
  return s;
}

// x total, rounded down, or up, for x in [0, 1): exact.
__device__ __forceinline__ uint64_t share_of(float x, uint64_t total, bool up) {
  const unsigned u = __float_as_uint(x);
  const int e = static_cast<int>(u >> 23);
  const uint64_t m = e ? (u & 0x7fffffu) | 0x800000u : u & 0x7fffffu;  // x = m 2^-shift
  const int shift = e ? 150 - e : 149;                                 // 24 and more
  const uint64_t lo = m * total, hi = __umul64hi(m, total);            // below 2^86
  uint64_t r, lost;
  if (shift < 64) {
    r = hi << (64 - shift) | lo >> shift;
    lost = lo << (64 - shift);
  } else {
    r = shift < 128 ? hi >> (shift - 64) : 0;
    lost = lo | (shift < 128 ? (shift > 64 ? hi << (128 - shift) : 0) : hi);
  }
  return r + (up && lost != 0);
}
// The number u times a total of weights, as the target that the sums have to pass.
__device__ __forceinline__ uint64_t target_of(float u, uint64_t total) {
  if (!(u > 0.f)) return 0;
  return u < 1.f ? share_of(u, total, false) : total - 1;
}
// The least weight that min-p keeps, of the largest.
__device__ __forceinline__ uint64_t floor_of(float min_p, uint64_t largest) {
  if (!(min_p > 0.f)) return 1;
  return min_p < 1.f ? max(share_of(min_p, largest, true), uint64_t(1)) : largest;
}
// The weight before a token from which on top-p (below 1) drops it; at least 1, so that the first is kept.
__device__ __forceinline__ uint64_t mass_of(float top_p, uint64_t total) {
  return top_p > 0.f ? max(share_of(top_p, total, true), uint64_t(1)) : 1;
}
// The difference to the maximum up to which a token may have the weight `least`, and a little more.  The lowest bit of
// a weight is always set, so that an odd one begins a unit below itself; 1 reaches as far as there are weights.
__device__ __forceinline__ float reach_of(uint64_t least, const Scale& s) {
  const float t = static_cast<float>(WEIGHT_BITS) - __log2f(static_cast<float>(least - 1)) + 0.01f;
  return fminf(s.d_max, t * 256.f * ptx::rcp_approx(s.c_hi));
}
// A logit below which all differences to the maximum are larger than d.
__device__ __forceinline__ float cut_at(float d, const Scale& s) {
  const float z = s.max - d;
  return z - (fabsf(s.max) + fabsf(d)) * 1e-6f;  // -inf for an infinite d, NaN where the maximum is infinite too
}

// A logit above which all differences to the maximum are smaller than d.
__device__ __forceinline__ float above(float d, const Scale& s) {
  const float z = s.max - d;
  const float r = z + (fabsf(s.max) + fabsf(d)) * 1e-6f;
  return r == r ? r : INFINITY;
}

// The tokens kept so far: those of a larger logit, and of this one up to an index.
struct Border {
  float z;
  unsigned inverted;  // 0xffffffff - the last index kept
  __device__ __forceinline__ bool keeps(float v, unsigned inv) const { return v > z || (v == z && inv >= inverted); }
};

// The largest and the smallest logit, and whether there is a NaN: one instruction each for two bf16.
template <typename E>
struct Extremes;
template <>
struct Extremes<__nv_bfloat16> {
  __nv_bfloat162 hi = __float2bfloat162_rn(-INFINITY), lo = __float2bfloat162_rn(INFINITY);
  __device__ __forceinline__ void add(const uint4& q) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&q);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hi = __hmax2_nan(hi, h[i]);  // a NaN stays
      lo = __hmin2(lo, h[i]);
    }
  }
  __device__ __forceinline__ void result(float* largest, float* smallest, bool* nan) const {
    const float a = __low2float(hi), b = __high2float(hi);
    *nan = a != a || b != b;
    *largest = fmaxf(a, b);
    *smallest = fminf(__low2float(lo), __high2float(lo));
  }
};
template <>
struct Extremes<float> {
  float hi = -INFINITY, lo = INFINITY;
  bool bad = false;
  __device__ __forceinline__ void add(const uint4& q) {
    const float v[4] = {__uint_as_float(q.x), __uint_as_float(q.y), __uint_as_float(q.z), __uint_as_float(q.w)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      bad |= v[i] != v[i];
      hi = fmaxf(hi, v[i]);
      lo = fminf(lo, v[i]);
    }
  }
  __device__ __forceinline__ void result(float* largest, float* smallest, bool* nan) const {
    *nan = bad;
    *largest = hi;
    *smallest = lo;
  }
};

// One row's work in a cluster.
template <typename E>
struct Sampler {
  const SampleArgs& a;
  Shared& sh;
  Row<E> row;
  Scale scale;
  float bin_scale;  // bins per unit of difference to the maximum
  unsigned rank, ctas;
  Border border;
  // After nucleus(): the weight of this thread's logits above `sure_above`, all of them kept.
  bool has_sure = false;
  float sure_above = 0.f;
  uint64_t sure = 0;
  // After nucleus_by_value(), where not 0: the weight of each of the logits equal to border.z, of which the first
  // `equal_kept` are kept.
  uint64_t equal_weight = 0, equal_kept = 0;

  __device__ __forceinline__ uint32_t remote(const void* p, unsigned cta) const {
    return ptx::mapa_shared(ptx::smem_addr(p), cta);
  }
  __device__ __forceinline__ unsigned bin_of(float d) const {
    return min(static_cast<unsigned>(fminf(d * bin_scale, static_cast<float>(BINS - 1))), unsigned(BINS - 1));
  }
  __device__ __forceinline__ uint64_t weight_of(float z) const { return weight(z, scale, sh.powers); }
  static constexpr int V = kVec<E>;

  // ------------------------------------------------------------------------ candidates in the first CTA
  // Candidates go into a room of the first CTA, one for each CTA.
  __device__ __forceinline__ int room() const { return BINS / ctas; }
  // Called by whole warps.
  __device__ __forceinline__ void push(bool mine, float z, int j) {
    const unsigned who = __ballot_sync(0xffffffffu, mine);
    if (who == 0) return;
    const int lane = threadIdx.x & 31, leader = __ffs(who) - 1;
    unsigned at = 0;
    if (lane == leader) at = atomicAdd(&sh.own_listed, __popc(who));
    at = __shfl_sync(0xffffffffu, at, leader) + __popc(who & ((1u << lane) - 1u));
    if (mine && at < static_cast<unsigned>(room()))
      st_cluster_u64(remote(&sh.room[rank * room() + at], 0), static_cast<uint64_t>(key_of(z)) << 32 | row.inverted(j));
  }
  // After all have pushed: the count of all CTAs together (more than LIST: there was no room), the smallest and largest
  // key.  The counter is 0 again afterwards.
  __device__ __forceinline__ Listed gather(unsigned kmin, unsigned kmax) {
    kmin = __reduce_min_sync(0xffffffffu, kmin);
    kmax = __reduce_max_sync(0xffffffffu, kmax);
    if ((threadIdx.x & 31) == 0) {
      sh.warp_u[0][threadIdx.x >> 5] = kmin;
      sh.warp_u[1][threadIdx.x >> 5] = kmax;
    }
    __syncthreads();
    if (threadIdx.x < ctas) {
      for (int w = 0; w < WARPS; ++w) {
        kmin = min(kmin, sh.warp_u[0][w]);
        kmax = max(kmax, sh.warp_u[1][w]);
      }
      const uint32_t to = remote(&sh.listed[rank], threadIdx.x);
      ptx::st_shared_cluster(to, sh.own_listed);
      ptx::st_shared_cluster(to + 4, kmin);
      ptx::st_shared_cluster(to + 8, kmax);
    }
    cluster_barrier();
    if (threadIdx.x == 0) sh.own_listed = 0;
    Listed all{0, 0xffffffffu, 0, 0};
    for (unsigned c = 0; c < ctas; ++c) {
      const Listed l = sh.listed[c];
      if (l.count > static_cast<unsigned>(room())) all.count = LIST + 1;
      all.count = min(all.count + l.count, unsigned(LIST + 1));
      all.all += l.count;
      all.key_min = min(all.key_min, l.key_min);
      all.key_max = max(all.key_max, l.key_max);
    }
    return all;
  }
  // In the first CTA: the candidates, n of them, largest first, one a thread; 0 behind them.
  __device__ __forceinline__ uint64_t collect(int n) {
    int at = threadIdx.x, c = 0;
    uint64_t item = 0;
    if (at < n) {
      while (at >= static_cast<int>(sh.listed[c].count)) at -= sh.listed[c++].count;
      item = sh.room[c * room() + at];
    }
    return sort_down(item, power_of_two(n), sh.list);
  }

  // ------------------------------------------------------------------------ top-p of all tokens
  // v summed over the block, in thread 0 .. ctas - 1.
  __device__ __forceinline__ uint64_t block_sum(uint64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh.warp_a[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0;
    if (threadIdx.x < ctas) {
#pragma unroll
      for (int w = 0; w < WARPS; ++w) v += sh.warp_a[w];
    }
    return v;
  }
  // Tokens of the cluster in one of the 4096 bins.
  __device__ __forceinline__ unsigned count_of(int b) const {
    unsigned n[MAX_CLUSTER], count = 0;
#pragma unroll
    for (int c = 0; c < MAX_CLUSTER; ++c) n[c] = c < static_cast<int>(ctas) ? ld_cluster_u32(remote(&sh.fine[b], c)) : 0;
#pragma unroll
    for (int c = 0; c < MAX_CLUSTER; ++c) count += n[c];
    return count;
  }
  // Top-p where no token is dropped yet, with one exact look at every weight instead of two and no atomics on
  // weights: counts in 4096 bins give the bin of the border but for the spread of the weights inside bins
  // (0.4% over the whole range at most, and it averages out); then one pass adds the exact weights of all and of the
  // logits above that bin and its surroundings, and lists those in them.  Where the border turns out not to lie there
  // (one row in a thousand; 3 in 100 with 3/4 of a bin to either side), lower() starts afresh; where too many logits
  // do, it goes on from there.
  __device__ void nucleus(float p) {
    const float fine_scale = 2.f * bin_scale, lowest = fmaxf(scale.max - scale.d_max, -FLT_MAX);
    const float cut = cut_at(scale.d_max, scale);
    for (int i = threadIdx.x; i < 2 * BINS; i += THREADS) sh.fine[i] = 0;
    __syncthreads();
    for_chunk(row, a.chunk, cut, [&](const float (&v)[V], int j) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (v[i] >= lowest)
          atomicAdd(&sh.fine[static_cast<unsigned>(fminf((scale.max - v[i]) * fine_scale, 2 * BINS - 1.f))], 1u);
    });
    cluster_barrier();
    // this CTA's share of the bins: counts over the cluster, times the weight 2^-depth in the middle
    const float depth = ptx::rcp_approx(fine_scale) * scale.c_hi * (1.f / 256.f);
    auto depth_of = [&](int b) { return (static_cast<float>(b) + 0.5f) * depth; };
    constexpr int MOST = 2 * BINS / THREADS;
    const int per_cta = 2 * BINS / ctas, per = per_cta / THREADS, b0 = rank * per_cta + threadIdx.x * per;
    uint64_t v[MOST], sum = 0;
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
      v[i] = 0;
      if (i < per) {
        const unsigned count = count_of(b0 + i);
        v[i] = count ? static_cast<uint64_t>(count * ptx::ex2_approx(static_cast<float>(WEIGHT_BITS) - depth_of(b0 + i))) + 1 : 0;
      }
      sum += v[i];
    }
    uint64_t total;
    uint64_t before = scan(sum, sh.warp_a, &total);
    if (threadIdx.x < ctas) st_cluster_u64(remote(&sh.chunk_total[rank], threadIdx.x), total);
    cluster_barrier();
    uint64_t all = 0;
    for (unsigned c = 0; c < ctas; ++c) {
      if (c == rank) before += all;
      all += sh.chunk_total[c];
    }
    const uint64_t about = mass_of(p, all);
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
      if (v[i] != 0 && before < about && before + v[i] >= about) {
        // where in the bin, if its weights are spread evenly, and how many tokens it has
        const float part = static_cast<float>(about - before) / static_cast<float>(v[i]);
        const float count = static_cast<float>(v[i]) * ptx::ex2_approx(depth_of(b0 + i) - static_cast<float>(WEIGHT_BITS));
        for (unsigned c = 0; c < ctas; ++c) {
          ptx::st_shared_cluster(remote(&sh.found.bin, c), b0 + i);
          ptx::st_shared_cluster(remote(&sh.found.part, c), __float_as_int(part));
          ptx::st_shared_cluster(remote(&sh.found.count, c), __float_as_int(count));
        }
      }
      before += v[i];
    }
    cluster_barrier();
    // that bin, and on either side of the place in it room for 64 tokens or so, 3/4 to 32 bins
    const float chosen = static_cast<float>(sh.found.bin), width = ptx::rcp_approx(fine_scale);
    const float spread = fminf(fmaxf(64.f / sh.found.count, 0.75f), 32.f);
    const float after = fmaxf(1.f, sh.found.part + spread), ahead = fminf(0.f, sh.found.part - spread);
    const float low = fmaxf(fmaxf(cut, cut_at((chosen + after) * width, scale)), lowest);
    const float top = above(fmaxf(chosen + ahead, 0.f) * width, scale);
    uint64_t everything = 0, certain = 0, near = 0;
    unsigned kmin = 0xffffffffu, kmax = 0;
    for_chunk(row, a.chunk, cut, [&](const float (&v)[V], int j) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint64_t w = weight_small(v[i], scale, sh.powers);
        everything += v[i] >= lowest ? w : 0;
        certain += v[i] > top ? w : 0;
      }
      for_some(v, j, [&](float z) { return z >= low && z <= top; }, [&](int at, bool valid) {
        const float z = valid ? row.at(at) : 0.f;
        if (valid) {
          kmin = min(kmin, key_of(z));
          kmax = max(kmax, key_of(z));
          near += weight_of(z);
        }
        push(valid, z, at);
      });
    });
    const uint64_t cta_all = block_sum(everything), cta_sure = block_sum(certain), cta_near = block_sum(near);
    if (threadIdx.x < ctas) {
      st_cluster_u64(remote(&sh.all_total[rank], threadIdx.x), cta_all);
      st_cluster_u64(remote(&sh.sure_total[rank], threadIdx.x), cta_sure);
      st_cluster_u64(remote(&sh.near_total[rank], threadIdx.x), cta_near);
    }
    const Listed listed = gather(kmin, kmax);
    uint64_t base = 0, around = 0;
    all = 0;
    for (unsigned c = 0; c < ctas; ++c) {
      all += sh.all_total[c];
      base += sh.sure_total[c];
      around += sh.near_total[c];
    }
    const uint64_t limit = mass_of(p, all);
    if (base >= limit || base + around < limit) {
      lower<true>(0, p);
      return;
    }
    if (!resolve<true>(listed, base, limit)) lower<true>(0, p, 1, listed.key_min, listed.key_max, base, limit);
    has_sure = true;
    sure_above = top;
    sure = certain;
  }

  // The same for bf16: of its values there are few, with many tokens each, so that counts by value times weights are the
  // exact sums.  Bins are 2048 values from the largest down and 2047 from the smallest with a weight up; the rest,
  // logits next to 0 as a rule, is added up by weights.
  __device__ void nucleus_by_value(float p) {
    const float lowest = fmaxf(scale.max - scale.d_max, -FLT_MAX);
    const int top = key_of(scale.max) >> 16, bottom = key_of(lowest) >> 16;
    for (int i = threadIdx.x; i < 2 * BINS; i += THREADS) sh.fine[i] = 0;
    if (threadIdx.x == 0) sh.middle = 0;
    __syncthreads();
    uint64_t middle = 0;
    for_chunk(row, a.chunk, cut_at(scale.d_max, scale), [&](const float (&v)[V], int j) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (!(v[i] >= lowest)) continue;
        const int key = key_of(v[i]) >> 16, up = key - bottom;
        int b = top - key;
        if (b >= BINS) b = up < BINS - 1 ? 2 * BINS - 1 - up : BINS;
        if (b == BINS) middle += weight_of(v[i]);
        atomicAdd(&sh.fine[b], 1u);
      }
    });
    if (middle) atomicAdd(&sh.middle, static_cast<unsigned long long>(middle));
    cluster_barrier();
    auto value_of = [&](int b) {
      const unsigned key = b < BINS ? top - b : bottom + (2 * BINS - 1 - b);
      return logit_of(key << 16 | (key & 0x8000u ? 0u : 0xffffu));
    };
    constexpr int MOST = 2 * BINS / THREADS;
    const int per_cta = 2 * BINS / ctas, per = per_cta / THREADS, b0 = rank * per_cta + threadIdx.x * per;
    uint64_t v[MOST], sum = 0;
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
      v[i] = 0;
      if (i < per) {
        const unsigned count = count_of(b0 + i);
        if (b0 + i == BINS) {
          uint64_t m[MAX_CLUSTER];  // read at once
#pragma unroll
          for (int c = 0; c < MAX_CLUSTER; ++c) m[c] = c < static_cast<int>(ctas) ? ld_cluster_u64(remote(&sh.middle, c)) : 0;
#pragma unroll
          for (int c = 0; c < MAX_CLUSTER; ++c) v[i] += m[c];
        } else if (count) {
          v[i] = count * weight_of(value_of(b0 + i));
        }
      }
      sum += v[i];
    }
    uint64_t total;
    uint64_t before = scan(sum, sh.warp_a, &total);
    if (threadIdx.x < ctas) st_cluster_u64(remote(&sh.chunk_total[rank], threadIdx.x), total);
    cluster_barrier();
    uint64_t all = 0;
    for (unsigned c = 0; c < ctas; ++c) {
      if (c == rank) before += all;
      all += sh.chunk_total[c];
    }
    const uint64_t limit = mass_of(p, all);
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
      if (v[i] != 0 && before < limit && before + v[i] >= limit) {
        for (unsigned c = 0; c < ctas; ++c) {
          st_cluster_u64(remote(&sh.found.before, c), before);
          ptx::st_shared_cluster(remote(&sh.found.bin, c), b0 + i);
        }
      }
      before += v[i];
    }
    cluster_barrier();
    if (sh.found.bin == BINS) {
      lower<true>(0, p);
      return;
    }
    border.z = value_of(sh.found.bin);
    equal_weight = weight_of(border.z);
    equal_kept = (limit - sh.found.before + equal_weight - 1) / equal_weight;
  }

  // The border among the listed tokens, before which `base` lies; false where they are too many and differ.
  template <bool MASS>
  __device__ bool resolve(const Listed& listed, uint64_t base, uint64_t limit) {
    if (listed.count <= LIST) {
      if (rank == 0) {
        const uint64_t item = collect(listed.count);
        uint64_t w = item != 0;
        if (MASS && item) w = weight_of(logit_of(static_cast<unsigned>(item >> 32)));
        uint64_t unused;
        const uint64_t at = base + scan(w, sh.warp_a, &unused);
        // the last of those before which the limit is not reached
        if (item && at < limit && (threadIdx.x + 1 == listed.count || at + w >= limit)) {
          for (unsigned c = 0; c < ctas; ++c) st_cluster_u64(remote(&sh.border, c), item);
        }
      }
      cluster_barrier();
      border.z = logit_of(static_cast<unsigned>(sh.border >> 32));
      border.inverted = static_cast<unsigned>(sh.border);
      return true;
    }
    if (listed.key_min == listed.key_max) {
      // equal logits: as many of the lowest indices as the limit leaves room for
      const float z0 = logit_of(listed.key_min);
      const uint64_t w = MASS ? weight_of(z0) : 1;
      border = ties(z0, (limit - base + w - 1) / w);
      return true;
    }
    return false;
  }

  // ------------------------------------------------------------------------ limits by bins
  // Lowers the border to where the tokens kept so far reach a limit: their count k (MASS = false), or
  // the share p of their weight.  Leaves it where the limit is not reached.
  // From level 1 on the border is known to lie among the keys key_lo to key_hi, before which `base` lies.
  template <bool MASS>
  __device__ void lower(uint64_t k, float p, int level = 0, unsigned key_lo = 0, unsigned key_hi = 0xffffffffu,
                        uint64_t base = 0, uint64_t limit = 0) {
    float cut = fmaxf(cut_at(scale.d_max, scale), border.z), top = INFINITY;
    if (level == 0) limit = k;
    for (;; ++level) {
      unsigned shift = 0;
      if (level > 0) {
        while ((key_hi - key_lo) >> shift >= BINS) ++shift;
        cut = logit_of(key_lo);
        top = logit_of(key_hi);
      }
      for (int i = threadIdx.x; i < BINS; i += THREADS) sh.lo[i] = sh.hi[i] = 0;
      __syncthreads();
      auto bin = [&](float z, unsigned key) {
        return level == 0 ? bin_of(below_max(z, scale)) : (key_hi - key) >> shift;
      };
      auto member = [&](float z, int j) {
        return below_max(z, scale) <= scale.d_max && border.keeps(z, row.inverted(j));
      };
      auto add = [&](unsigned b, uint64_t w) {
        if constexpr (MASS) {
          const unsigned low = static_cast<unsigned>(w);
          const unsigned old = atomicAdd(&sh.lo[b], low);
          const unsigned high = static_cast<unsigned>(w >> 32) + (old + low < old);
          if (high) atomicAdd(&sh.hi[b], high);
        } else {
          atomicAdd(&sh.lo[b], 1u);
        }
      };
      for_chunk(row, a.chunk, cut, [&](const float (&v)[V], int j) {
        if (level == 0) {  // most of a row
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (member(v[i], j + i)) add(bin_of(below_max(v[i], scale)), MASS ? weight_of(v[i]) : 1);
          return;
        }
        for_some(v, j, [&](float z) { return !(z < cut) && !(z > top); }, [&](int at, bool valid) {
          const float z = valid ? row.at(at) : -INFINITY;
          const unsigned key = key_of(z);
          if (!valid || !member(z, at) || key < key_lo || key > key_hi) return;
          add(bin(z, key), MASS ? weight_of(z) : 1);
        });
      });
      cluster_barrier();
      // this CTA's share of the bins, summed over the cluster
      const int per_cta = BINS / ctas, per = max(1, per_cta / THREADS);
      const int b0 = rank * per_cta + threadIdx.x * per;
      uint64_t v[BINS / THREADS], sum = 0;
#pragma unroll
      for (int i = 0; i < BINS / THREADS; ++i) {
        v[i] = 0;
        if (i < per && static_cast<int>(threadIdx.x) * per < per_cta) {
          unsigned l[MAX_CLUSTER], h[MAX_CLUSTER];
#pragma unroll
          for (int c = 0; c < MAX_CLUSTER; ++c) {
            l[c] = c < static_cast<int>(ctas) ? ld_cluster_u32(remote(&sh.lo[b0 + i], c)) : 0;
            h[c] = MASS && c < static_cast<int>(ctas) ? ld_cluster_u32(remote(&sh.hi[b0 + i], c)) : 0;
          }
#pragma unroll
          for (int c = 0; c < MAX_CLUSTER; ++c) v[i] += (static_cast<uint64_t>(h[c]) << 32) + l[c];
        }
        sum += v[i];
      }
      uint64_t total;
      uint64_t before = scan(sum, sh.warp_a, &total);
      if (threadIdx.x < ctas) st_cluster_u64(remote(&sh.chunk_total[rank], threadIdx.x), total);
      cluster_barrier();
      uint64_t all = 0;
      for (unsigned c = 0; c < ctas; ++c) {
        if (c == rank) before += base + all;
        all += sh.chunk_total[c];
      }
      if (level == 0) {
        if (MASS) limit = mass_of(p, all);
        else if (all <= limit) return;  // in all CTAs alike
      }
#pragma unroll
      for (int i = 0; i < BINS / THREADS; ++i) {
        if (v[i] != 0 && before < limit && before + v[i] >= limit) {
          for (unsigned c = 0; c < ctas; ++c) {
            st_cluster_u64(remote(&sh.found.before, c), before);
            ptx::st_shared_cluster(remote(&sh.found.bin, c), b0 + i);
          }
        }
        before += v[i];
      }
      cluster_barrier();
      const unsigned chosen = sh.found.bin;
      base = sh.found.before;
      // the tokens of that bin
      if (level == 0) {
        cut = fmaxf(cut, cut_at(static_cast<float>(chosen + 1) / bin_scale, scale));
        top = above(static_cast<float>(chosen) / bin_scale, scale);
      }
      unsigned kmin = 0xffffffffu, kmax = 0;
      for_chunk(row, a.chunk, cut, [&](const float (&v)[V], int j) {
        for_some(v, j, [&](float z) { return !(z < cut) && !(z > top); }, [&](int at, bool valid) {
          const float z = valid ? row.at(at) : -INFINITY;
          const unsigned key = key_of(z);
          const bool mine = valid && member(z, at) && key >= key_lo && key <= key_hi && bin(z, key) == chosen;
          if (mine) {
            kmin = min(kmin, key);
            kmax = max(kmax, key);
          }
          push(mine, z, at);
        });
      });
      const Listed listed = gather(kmin, kmax);
      if (resolve<MASS>(listed, base, limit)) return;
      key_lo = listed.key_min;
      key_hi = listed.key_max;
      cluster_barrier();  // the first CTA's room becomes bins again
    }
  }

  // The border behind the first `keep` (at least 1, at most as many as there are) of the kept tokens that
  // equal z0.
  __device__ Border ties(float z0, uint64_t keep) {
    uint64_t mine = 0;
    for_chunk(row, a.chunk, z0, [&](const float (&v)[V], int j) {
#pragma unroll
      for (int i = 0; i < V; ++i) mine += v[i] == z0 && border.keeps(v[i], row.inverted(j + i));
    });
    uint64_t total, chunk_before, inside;
    int warp;
    unsigned none;
    if (locate<false>(mine, 0, keep - 1, sh.chunk_total, &total, &warp, &chunk_before, &none)) {
      const int j0 = max(warp * a.chunk, row.lead), j1 = min((warp + 1) * a.chunk, row.end);
      const int per = (a.chunk + THREADS - 1) / THREADS, t0 = j0 + static_cast<int>(threadIdx.x) * per;
      uint64_t here = 0;
      for (int j = t0; j < min(t0 + per, j1); ++j) {
        const float z = row.at(j);
        here += z == z0 && border.keeps(z, row.inverted(j));
      }
      uint64_t at = chunk_before + scan(here, sh.warp_a, &inside);
      if (at < keep && at + here >= keep) {
        for (int j = t0; j < min(t0 + per, j1); ++j) {
          const float z = row.at(j);
          if (z == z0 && border.keeps(z, row.inverted(j)) && ++at == keep) {
            const uint64_t item = static_cast<uint64_t>(key_of(z0)) << 32 | row.inverted(j);
            for (unsigned c = 0; c < ctas; ++c) st_cluster_u64(remote(&sh.border, c), item);
          }
        }
      }
    }
    cluster_barrier();
    return Border{z0, static_cast<unsigned>(sh.border)};
  }

  // The kept weight of tokens of which `equal` are equal to the border and `more` is the weight of the others.
  template <bool EQUAL = true>
  __device__ __forceinline__ uint64_t with_equal(uint64_t more, unsigned equal) const {
    return EQUAL ? more + equal_weight * min(static_cast<uint64_t>(equal), equal_kept) : more;
  }
  // Sums `mine`, and with EQUAL the count `equal` of logits equal to the border, over the warps' chunks and the CTAs in order; totals:
  // the CTAs' sums, of a room that nobody reads any more.  Where the kept weight passes `target` (a number, or computed
  // from the total) in this CTA: true, the warp whose chunk that is, and the two sums before the chunk.  *total: of the
  // cluster.
  template <bool EQUAL, typename T>
  __device__ bool locate(uint64_t mine, unsigned equal, T&& target_from, uint64_t* totals, uint64_t* total, int* warp,
                         uint64_t* chunk_before, unsigned* equal_before) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (EQUAL) equal = __reduce_add_sync(0xffffffffu, equal);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
      sh.warp_a[threadIdx.x >> 5] = mine;
      if (EQUAL) sh.warp_n[threadIdx.x >> 5] = equal;
    }
    __syncthreads();
    uint64_t cta = 0;
    unsigned cta_equal = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      cta += sh.warp_a[w];
      if (EQUAL) cta_equal += sh.warp_n[w];
    }
    if (threadIdx.x < ctas) {
      st_cluster_u64(remote(&totals[rank], threadIdx.x), cta);
      if (EQUAL) ptx::st_shared_cluster(remote(&sh.equal_total[rank], threadIdx.x), cta_equal);
    }
    cluster_barrier();
    uint64_t before = 0, all = 0;
    unsigned equal_at = 0, equal_all = 0;
    for (unsigned c = 0; c < ctas; ++c) {
      if (c == rank) {
        before = all;
        equal_at = equal_all;
      }
      all += totals[c];
      if (EQUAL) equal_all += sh.equal_total[c];
    }
    all = with_equal<EQUAL>(all, equal_all);
    *total = all;
    uint64_t target;
    if constexpr (std::is_integral<typename std::decay<T>::type>::value) target = target_from;
    else target = target_from(all);
    if (target < with_equal<EQUAL>(before, equal_at) || target >= with_equal<EQUAL>(before + cta, equal_at + cta_equal)) return false;
    int w = 0;
    while (with_equal<EQUAL>(before + sh.warp_a[w], equal_at + sh.warp_n[w]) <= target) {
      before += sh.warp_a[w];
      if (EQUAL) equal_at += sh.warp_n[w];
      ++w;
    }
    *warp = w;
    *chunk_before = before;
    *equal_before = equal_at;
    __syncthreads();  // before warp_a is used again
    return true;
  }

  // ------------------------------------------------------------------------ results
  __device__ __forceinline__ void write(int64_t r, int64_t column, float z, float temperature, uint64_t total) {
    a.tokens[r] = column;
    if (a.logprobs) {
      // x - ln(total / largest weight): two terms of one sign
      const uint64_t largest = weight_of(scale.max);
      const float rest = static_cast<float>(total - largest) / static_cast<float>(largest);
      a.logprobs[r] = -(below_max(z, scale) / temperature + log1pf(rest));
    }
  }

  // The row behind nucleus_by_value().
  __device__ void finish_by_value(int64_t r, const Settings& set, float u) {
    const uint64_t least = floor_of(set.min_p, weight_of(scale.max));
    const float z0 = border.z, cut = fmaxf(cut_at(reach_of(least, scale), scale), z0);
    if (equal_weight < least) equal_weight = 0;
    uint64_t mine = 0, target = 0, total, at, unused;
    unsigned equal = 0, equal_at;
    for_chunk(row, a.chunk, cut, [&](const float (&v)[V], int j) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint64_t w = weight_small(v[i], scale, sh.powers);
        mine += v[i] > z0 && w >= least ? w : 0;
        equal += v[i] == z0;
      }
    });
    int chunk;
    if (!locate<true>(mine, equal, [&](uint64_t t) { return target = target_of(u, t); }, sh.kept_total, &total, &chunk, &at,
                      &equal_at))
      return;
    const int j0 = max(chunk * a.chunk, row.lead), j1 = min((chunk + 1) * a.chunk, row.end);
    const int per = (a.chunk + THREADS - 1) / THREADS, t0 = j0 + static_cast<int>(threadIdx.x) * per;
    mine = 0, equal = 0;
    auto add = [&](float z, uint64_t& more, unsigned& count) {
      const uint64_t w = z > z0 ? weight_of(z) : 0;
      more += w >= least ? w : 0;
      count += z == z0;
    };
    for (int j = t0; j < min(t0 + per, j1); ++j) add(row.at(j), mine, equal);
    at += scan(mine, sh.warp_a, &unused);
    equal_at += static_cast<unsigned>(scan(equal, sh.warp_a, &unused));
    if (with_equal(at, equal_at) > target || target >= with_equal(at + mine, equal_at + equal)) return;
    for (int j = t0;; ++j) {
      const float z = row.at(j);
      add(z, at, equal_at);
      if (with_equal(at, equal_at) > target) {
        write(r, row.column(j), z, set.temperature, total);
        return;
      }
    }
  }

  // The row from the list of the first CTA, which holds every token that top-k may keep (n of them).
  __device__ void finish_list(int64_t r, int n, uint64_t k, const Settings& set, float u) {
    const int t = threadIdx.x;
    const uint64_t item = collect(n);
    const float z = logit_of(static_cast<unsigned>(item >> 32));
    uint64_t w = t < n && static_cast<uint64_t>(t) < k ? weight_of(z) : 0;
    uint64_t total;
    const uint64_t before = scan(w, sh.warp_a, &total);
    if (set.top_p < 1.f && before >= mass_of(set.top_p, total)) w = 0;
    if (w < floor_of(set.min_p, weight_of(scale.max))) w = 0;
    // what is left, in the order of indices
    sh.weights[t] = w;
    const uint64_t by_index = sort_down(w ? (item & 0xffffffffu) << 32 | static_cast<unsigned>(t) : 0, power_of_two(n), sh.list);
    __syncthreads();
    const uint64_t w2 = by_index ? sh.weights[static_cast<unsigned>(by_index)] : 0;
    uint64_t kept;
    const uint64_t at = scan(w2, sh.warp_a, &kept);
    const uint64_t target = target_of(u, kept);
    if (w2 && at <= target && target < at + w2) sh.own_bound = static_cast<unsigned>(by_index);
    __syncthreads();
    if (t == static_cast<int>(sh.own_bound)) write(r, 0xffffffffu - static_cast<unsigned>(item), z, set.temperature, kept);
  }
};

template <typename E>
__global__ void __launch_bounds__(THREADS, 2) sample_kernel(const SampleArgs a, int staged_bytes) {
  extern __shared__ uint4 dynamic[];
  __shared__ Shared sh;
  constexpr int V = kVec<E>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned ctas = cluster_size(), rank = ptx::cluster_ctarank();
  const int64_t r = blockIdx.x / ctas;
  cluster_arrive();  // this CTA has started: its shared memory can be written
  const float2 entry = make_float2(kPowers.hi[threadIdx.x & 255], kPowers.lo[threadIdx.x & 255]);
  if (threadIdx.x == 0) sh.own_listed = 0;
  ptx::wait_for_previous();
  ptx::launch_dependents();
  const Settings set = settings_of(a, r);
  const float u = a.uniform[r];

  // this CTA's columns, into shared memory; their largest and smallest
  Row<E> row;
  row.first = min(static_cast<int64_t>(rank) * a.slice, a.V);
  const int columns = static_cast<int>(min(static_cast<int64_t>(a.slice), a.V - row.first));
  const E* p = static_cast<const E*>(a.logits) + r * a.ld + row.first;
  row.lead = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(E));
  row.base = p - row.lead;
  row.end = row.lead + columns;
  row.staged = staged_bytes ? reinterpret_cast<E*>(dynamic) : nullptr;
  float hi = -INFINITY, lo = INFINITY;
  bool nan;
  {
    constexpr int U = 4;
    const int stop = min((warp + 1) * a.chunk, row.end);
    Extremes<E> x;
    for (int j0 = warp * a.chunk + lane * V; j0 < stop; j0 += 32 * V * U) {
      uint4 q[U];
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (j0 + k * 32 * V < stop) q[k] = row.load_global(j0 + k * 32 * V);
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int j = j0 + k * 32 * V;
        if (j >= stop) break;
        if (row.staged) *reinterpret_cast<uint4*>(row.staged + j) = q[k];
        x.add(q[k]);
      }
    }
    x.result(&hi, &lo, &nan);
  }
  if (threadIdx.x < 256) sh.powers[threadIdx.x] = entry;
  const float own_max = hi;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
  }
  nan = __any_sync(0xffffffffu, nan);
  if (lane == 0) {
    sh.warp_f[0][warp] = hi;
    sh.warp_f[1][warp] = lo;
    sh.warp_f[2][warp] = nan;
  }
  __syncthreads();
  for (int w = 0; w < WARPS; ++w) {
    hi = fmaxf(hi, sh.warp_f[0][w]);
    lo = fminf(lo, sh.warp_f[1][w]);
    nan |= sh.warp_f[2][w] != 0.f;
  }
  cluster_wait();  // every CTA has started
  if (threadIdx.x < ctas) {
    const uint32_t to = ptx::mapa_shared(ptx::smem_addr(&sh.extremes[rank]), threadIdx.x);
    ptx::st_shared_cluster(to, __float_as_int(hi));
    ptx::st_shared_cluster(to + 4, __float_as_int(lo));
    ptx::st_shared_cluster(to + 8, nan);
  }
  cluster_barrier();
  nan = false;
  for (unsigned c = 0; c < ctas; ++c) {
    const float4 x = sh.extremes[c];
    hi = fmaxf(hi, x.x);
    lo = fminf(lo, x.y);
    nan |= __float_as_int(x.z) != 0;
  }
  // from here on every branch that holds a cluster barrier is taken by all threads of the cluster alike
  if (nan || hi == -INFINITY) {
    if (rank == 0 && threadIdx.x == 0) {
      a.tokens[r] = -1;
      if (a.logprobs) a.logprobs[r] = NAN;
    }
    return;
  }
  if (!(set.temperature > 0.f)) {
    // the lowest index of the largest logit
    int64_t first = INT64_MAX;
    for_chunk(row, a.chunk, hi, [&](const float (&v)[V], int j) {
#pragma unroll
      for (int i = V - 1; i >= 0; --i)
        if (v[i] == hi) first = min(first, row.column(j + i));
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) first = min(first, static_cast<int64_t>(__shfl_xor_sync(0xffffffffu, first, o)));
    if (lane == 0) sh.warp_a[warp] = static_cast<uint64_t>(first);
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 0; w < WARPS; ++w) first = min(first, static_cast<int64_t>(sh.warp_a[w]));
      st_cluster_u64(ptx::mapa_shared(ptx::smem_addr(&sh.chunk_total[rank]), 0), static_cast<uint64_t>(first));
    }
    cluster_barrier();
    if (rank == 0 && threadIdx.x == 0) {
      for (unsigned c = 0; c < ctas; ++c) first = min(first, static_cast<int64_t>(sh.chunk_total[c]));
      a.tokens[r] = first;
      if (a.logprobs) a.logprobs[r] = 0.f;
    }
    return;
  }
  const Scale scale = scale_of(hi, set.temperature);
  // bins from the largest to the smallest logit, but not beyond those that have a weight
  const float range = fminf(hi == lo ? 0.f : hi - lo, scale.d_max);
  const float bin_scale = range > 0.f && range < INFINITY ? fminf(BINS * ptx::rcp_approx(range), 3e38f) : 0.f;
  Sampler<E> s{a, sh, row, scale, bin_scale, rank, ctas, Border{-FLT_MAX, 0u}};

  const bool limited = set.top_k > 0 && set.top_k < a.V;
  if (limited) {
    // If k threads of a CTA have a logit in the bins up to b, what lies in later bins is not among the k largest; nor
    // if k / ctas threads of each CTA have.  Bins four at a time here: one a thread.
    if (set.top_k <= LIST) {
      static_assert(BINS == 4 * THREADS, "four bins a thread");
      sh.lo[threadIdx.x] = 0;
      if (threadIdx.x == 0) sh.own_bound = sh.own_share = THREADS - 1;
      __syncthreads();
      const float d = below_max(own_max, scale);
      if (own_max > -INFINITY && d <= scale.d_max) atomicAdd(&sh.lo[s.bin_of(d) / 4], 1u);
      __syncthreads();
      const unsigned here = sh.lo[threadIdx.x];
      unsigned incl = here;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      if (lane == 31) sh.warp_u[0][warp] = incl;
      __syncthreads();
      for (int w = 0; w < warp; ++w) incl += sh.warp_u[0][w];
      const unsigned k = set.top_k, part = (k + ctas - 1) / ctas;
      if (incl >= k && incl - here < k) sh.own_bound = threadIdx.x;
      if (incl >= part && incl - here < part) sh.own_share = threadIdx.x;
      __syncthreads();
      if (threadIdx.x < ctas) {
        const uint32_t to = ptx::mapa_shared(ptx::smem_addr(&sh.bound[rank]), threadIdx.x);
        ptx::st_shared_cluster(to, sh.own_bound);
        ptx::st_shared_cluster(to + 4, sh.own_share);
      }
      cluster_barrier();
      unsigned least = THREADS - 1, most = 0;
      for (unsigned i = 0; i < ctas; ++i) {
        least = min(least, sh.bound[i].x);
        most = max(most, sh.bound[i].y);
      }
      const unsigned bound = min(least, most) * 4 + 3;
      const float cut = cut_at(fminf(scale.d_max, static_cast<float>(bound + 1) / bin_scale), scale);
      for_chunk(row, a.chunk, cut, [&](const float (&v)[V], int j) {
        for_some(v, j, [&](float z) { return !(z < cut) && z > -INFINITY; }, [&](int at, bool valid) {
          const float z = valid ? row.at(at) : -INFINITY, d = below_max(z, scale);
          s.push(valid && d <= scale.d_max && s.bin_of(d) <= bound, z, at);
        });
      });
      const unsigned n = s.gather(0, 0).count;
      if (n <= LIST) {
        if (rank == 0) s.finish_list(r, n, set.top_k, set, u);
        return;
      }
      cluster_barrier();  // the first CTA's room becomes bins again
    }
    s.template lower<false>(set.top_k, 0.f);
  }
  if (set.top_p < 1.f) {
    if (!limited && scale.small && bin_scale > 0.f) {
      if constexpr (sizeof(E) == 2) {
        s.nucleus_by_value(set.top_p);
        if (s.equal_weight) {
          s.finish_by_value(r, set, u);
          return;
        }
      } else {
        s.nucleus(set.top_p);
      }
    } else s.template lower<true>(0, set.top_p);
  }

  // the kept weights, and where the target lies among them
  const uint64_t least = floor_of(set.min_p, s.weight_of(scale.max));
  const float cut = fmaxf(cut_at(reach_of(least, scale), scale), s.border.z);
  uint64_t mine = 0, total, chunk_before, unused;
  unsigned none;
  // at 0: all from d_max on, a comparison a logit
  const bool plain = scale.small && !limited && !(set.top_p < 1.f) && least == 1;
  const float lowest = scale.max - scale.d_max;
  auto kept = [&](float z, int j) -> uint64_t {
    if (plain) return z >= lowest && z > -INFINITY ? weight_small(z, scale, sh.powers) : 0;
    if (!(below_max(z, scale) <= scale.d_max) || !s.border.keeps(z, row.inverted(j))) return 0;
    const uint64_t w = s.weight_of(z);
    return w < least ? 0 : w;
  };
  if (plain) {
    for_chunk(row, a.chunk, cut, [&](const float (&v)[V], int j) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint64_t w = weight_small(v[i], scale, sh.powers);
        mine += v[i] >= lowest && v[i] > -INFINITY ? w : 0;
      }
    });
  } else if (s.has_sure && least == 1) {
    mine = s.sure;
    for_chunk(row, a.chunk, s.border.z, [&](const float (&v)[V], int j) {
      for_some(v, j, [&](float z) { return z >= s.border.z && z <= s.sure_above; }, [&](int at, bool valid) {
        if (valid) mine += kept(row.at(at), at);
      });
    });
  } else {
    for_chunk(row, a.chunk, cut, [&](const float (&v)[V], int j) {
      int n = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) n += !(v[i] < cut);
      if (scale.small && __reduce_max_sync(0xffffffffu, n) > V / 2) {
        // most logits of some lane: all of all lanes
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const uint64_t w = weight_small(v[i], scale, sh.powers);
          const bool keep = below_max(v[i], scale) <= scale.d_max && s.border.keeps(v[i], row.inverted(j + i));
          mine += keep && w >= least ? w : 0;
        }
        return;
      }
      for_some(v, j, [&](float z) { return !(z < cut) && z > -INFINITY; }, [&](int at, bool valid) {
        if (valid) mine += kept(row.at(at), at);
      });
    });
  }
  int w;
  uint64_t target = 0;
  if (!s.template locate<false>(mine, 0, [&](uint64_t t) { return target = target_of(u, t); }, sh.kept_total, &total, &w,
                                &chunk_before, &none))
    return;
  const int j0 = max(w * a.chunk, row.lead), j1 = min((w + 1) * a.chunk, row.end);
  const int per = (a.chunk + THREADS - 1) / THREADS, t0 = j0 + static_cast<int>(threadIdx.x) * per;
  uint64_t here = 0;
  for (int j = t0; j < min(t0 + per, j1); ++j) here += kept(row.at(j), j);
  uint64_t at = chunk_before + scan(here, sh.warp_a, &unused);
  if (at <= target && target < at + here) {
    for (int j = t0;; ++j) {
      const float z = row.at(j);
      at += kept(z, j);
      if (at > target) {
        s.write(r, row.column(j), z, set.temperature, total);
        break;
      }
    }
  }
}

// ---------------------------------------------------------------------------------- host side
bool aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// Shared memory for the row of a CTA where two share an SM, and where each has one of its own.
constexpr int STAGE_TWO = 84 * 1024, STAGE_ONE = 184 * 1024;

struct Plan {
  int ctas, slice, chunk, staged_bytes;
};
template <typename E>
Plan plan(int64_t B, int64_t V, int num_sms) {
  constexpr int VEC = kVec<E>;
  Plan p{1, 0, 0, 0};
  // All rows at once, if two CTAs to an SM can do that: what a row waits for is waited for once.  One to an SM for
  // clusters of 8, of which few find two places to a CTA, and for slices below 16384, which are little work.  64 x 151,936
  // fp32, CTAs a row 1 / 2 / 4 / 8, us: greedy 30 / 18 / 15 / 18, top-k 50 39 / 28 / 25 / 36, top-p 0.9 139 / 81 / 72 /
  // 90; 33 x 151,936 - / - / 8.6 / 9.4, 16 / 25, 42 / 45; 64 x 32,000 7.1 / 6.0 / 6.8 / 12, 15 / 14.5 / 16 / 29, 35 / 27 /
  // 28 / 48; 256 x 50,021 17 / 23 / 28 / 49, 29 / 42 / 59 / 101, 110 / 110 / 125 / 208.
  while (p.ctas < MAX_CLUSTER && V / p.ctas > 4096) {
    const bool alone = B * p.ctas * 2 <= num_sms;
    if (!alone && (B * p.ctas > num_sms || p.ctas * 2 == MAX_CLUSTER || V / (p.ctas * 2) < 16384)) break;
    p.ctas *= 2;
  }
  p.slice = static_cast<int>(((V + p.ctas - 1) / p.ctas + VEC - 1) / VEC * VEC);
  // positions reach from 0 to VEC - 1 behind the slice
  const int span = p.slice + VEC;
  p.chunk = ((span + WARPS - 1) / WARPS + VEC - 1) / VEC * VEC;
  const int64_t need = static_cast<int64_t>(span + VEC) * static_cast<int64_t>(sizeof(E));
  // A row that leaves an SM to one of two CTAs is better read again from L2 (64 x 151,936 fp32 by 4: top-p 0.9 72 us, staged
  // 81); where there is one anyway, staged (33 x 151,936 by 4: 42 us, read again 51).
  const int64_t most = B * p.ctas <= num_sms ? STAGE_ONE : STAGE_TWO;
  p.staged_bytes = need <= most ? static_cast<int>((need + 15) / 16 * 16) : 0;
  return p;
}

template <typename E>
cudaError_t launch_sample(SampleArgs a, int64_t B, int num_sms, cudaStream_t stream) {
  const Plan p = plan<E>(B, a.V, num_sms);
  a.slice = p.slice;
  a.chunk = p.chunk;
  static PerDevice<kMaxDevices> allowed;  // the shared memory, asked for once per device
  int dev = 0, unused;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = allowed.get(dev, [](int* value) {
    *value = 1;
    return cudaFuncSetAttribute(sample_kernel<E>, cudaFuncAttributeMaxDynamicSharedMemorySize, STAGE_ONE);
  }, &unused);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(B * p.ctas));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = static_cast<size_t>(p.staged_bytes);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2] = {dependent_launch(), {}};
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.ctas);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sample_kernel<E>, a, p.staged_bytes);
}

}  // namespace
}  // namespace lce

using namespace lce;

extern "C" {

lce_status_t lce_sample(const void* logits, int64_t ld, int64_t B, int64_t V, lce_dtype_t dtype,
                        const float* uniform, const lce_sampling_t* settings, int64_t* tokens,
                        float* logprobs, void* stream) {
  if ((dtype != LCE_BF16 && dtype != LCE_F32) || !settings) return LCE_ERR_INVALID_ARG;
  const lce_sampling_t& set = *settings;
  if ((!set.temperatures && !(set.temperature >= 0.f)) || (!set.top_ks && set.top_k < 0) ||
      (!set.top_ps && !(set.top_p >= 0.f && set.top_p <= 1.f)) ||
      (!set.min_ps && !(set.min_p >= 0.f && set.min_p <= 1.f)))
    return LCE_ERR_INVALID_ARG;
  if (B < 0 || B > kMaxRows / MAX_CLUSTER || V < 1 || V > kMaxVocabulary || ld < V || ld > (int64_t(1) << 48) ||
      (B > 1 && ld > (int64_t(1) << 61) / B))
    return LCE_ERR_UNSUPPORTED_SHAPE;
  if ((B > 0 && (!logits || !uniform || !tokens)) || !aligned(logits, dtype == LCE_BF16 ? 2 : 4) ||
      !aligned(uniform, 4) || !aligned(tokens, 8) || !aligned(logprobs, 4) || !aligned(set.temperatures, 4) ||
      !aligned(set.top_ps, 4) || !aligned(set.min_ps, 4) || !aligned(set.top_ks, 4))
    return LCE_ERR_INVALID_ARG;
  int num_sms = 0;
  const lce_status_t st = check_device(&num_sms);
  if (st != LCE_OK || B == 0) return st;
  SampleArgs a{};
  a.logits = logits, a.ld = ld, a.V = V, a.uniform = uniform, a.set = set;
  a.tokens = tokens, a.logprobs = logprobs;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t err = traced(K_SAMPLE, s, [&] {
    return dtype == LCE_BF16 ? launch_sample<__nv_bfloat16>(a, B, num_sms, s)
                             : launch_sample<float>(a, B, num_sms, s);
  });
  return err == cudaSuccess ? LCE_OK : LCE_ERR_CUDA;
}

}  // extern "C"
