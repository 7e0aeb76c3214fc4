// The token embedding and its gradient (declared in include/lce.h).
//
//   y_i = scale E[t_i],   dE[v] = scale * sum of dy_i over the positions i with t_i = v
//
// Forward: one gather, bound by memory.  A warp moves up to 4 vectors a lane (2 KB) of one row; of rows that are not
// 16-byte aligned 16 words of 4 bytes, or 16 bf16.
//
// Backward.  The positions are sorted by token (stable, so that the order of each sum is that of the
// positions and nothing depends on timing): passes over digits of at most 10 bits, each of up to 64 blocks
// that count, rank with warp-wide matching and scatter; the counts of the next digit are gathered on
// the way.  Up to 8192 positions one block does it all, and up to 4096 they are placed by counting.  The sorted
// positions are then cut into tiles of equal length whatever the tokens are, so that a token that fills a sixth of the
// batch is spread over many SMs: each tile adds its rows of dy, keeping runs of one token in registers, and writes the
// runs that lie within it to the table's gradient; a run that goes on over a tile's edge leaves a partial sum there, and
// a last launch joins those in order.
// Most of the work for a large vocabulary is writing zeros: the launches of the sort do that beside it, so
// that the memory is busy while they wait for their latencies.  Rows of a token are written twice for that, N of them at
// most; a bitmap of the tokens and zeros beside the sums wrote each once, but left the sort's 25 us bare.
//
// Inside a captured graph: lookup of 32768 x 6144 bf16 79 us (frequent rows come from L2: the 403 MB written alone
// would take 59), 48 x 6144 2.0 us.  Gradient of 32768 x 2048, 151,936 tokens, bf16, Zipf(1.1): 125 us, 0.89 of the copy
// rate over dy and dE; 1999 x 515 fp32, 8,191 tokens 13.8 us (three launches in a row, 3 us of bytes).  Where a smaller table
// leaves the sort bare: 16384 x 512 of 20,000 tokens 31 us (5.5 of bytes), 131072 x 1024 of 50,000 105 (55).
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

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 512;
constexpr int64_t kMaxElements = int64_t(1) << 48;

// ------------------------------------------------------------------------------------ forward
// Vectors a lane moves.
template <typename E, int V>
constexpr int kSegment = V == kVec<E> ? 4 : 16;
constexpr int64_t CHECKED_TOKENS = 8192;  // up to here one block looks all tokens over

struct LookupArgs {
  const int64_t* tokens;
  const void* table;
  void* y;
  int64_t N, V, ldy, ignore_index;
  int64_t items;  // rows x segments
  int d, segments;
  float scale;
  unsigned* flags;
  bool check;     // the last block checks the tokens and writes the flags
};

__global__ void embedding_clear_kernel(unsigned* flags) {
  ptx::wait_for_previous();
  ptx::launch_dependents();
  if (threadIdx.x == 0) *flags = 0u;
}

template <typename E, int V>
__global__ void __launch_bounds__(256) embedding_kernel(const LookupArgs a) {
  ptx::wait_for_previous();
  ptx::launch_dependents();
  if (a.check && blockIdx.x == gridDim.x - 1) {
    int bad = 0;
#pragma unroll 8
    for (int64_t i = threadIdx.x; i < a.N; i += 256) {
      const int64_t t = a.tokens[i];
      bad |= t != a.ignore_index && (t < 0 || t >= a.V);
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *a.flags = bad ? ERR_LABEL : 0u;
    return;
  }
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (item >= a.items) return;
  const int64_t row = a.segments == 1 ? item : item / a.segments;
  constexpr int SEGMENT = kSegment<E, V>;
  const int first = static_cast<int>(item - row * a.segments) * (32 * SEGMENT * V) + (threadIdx.x & 31) * V;
  const int64_t token = a.tokens[row];
  const bool in = token >= 0 && token < a.V;
  const bool use = in && token != a.ignore_index;
  if (!a.check && !in && token != a.ignore_index && first == 0) atomicOr(a.flags, ERR_LABEL);
  const E* src = static_cast<const E*>(a.table) + (use ? token : 0) * a.d;
  E* dst = static_cast<E*>(a.y) + row * a.ldy;
  Raw<E, V> q[SEGMENT];
#pragma unroll
  for (int k = 0; k < SEGMENT; ++k) {
    const int64_t c = first + static_cast<int64_t>(k) * 32 * V;
    q[k] = use && c < a.d ? load_raw<E, V>(src + c) : zero_raw<E, V>();
  }
#pragma unroll
  for (int k = 0; k < SEGMENT; ++k) {
    const int64_t c = first + static_cast<int64_t>(k) * 32 * V;
    if (c >= a.d) continue;
    float v[V];
    unpack<E, V>(q[k], v);
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] *= a.scale;
    if (!use) {  // 0 also where scale is not finite
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = 0.f;
    }
    store_raw<E, V>(dst + c, pack<E, V>(v));
  }
}

// ------------------------------------------------------------------------------------ sorting
constexpr int SORT_THREADS = 1024, SORT_WARPS = 32;
constexpr int MAX_SORT_BLOCKS = 64;
constexpr int MAX_DIGIT_BITS = 10;
constexpr int MAX_BINS = 1 << MAX_DIGIT_BITS;

// Zeros that a launch of the sort writes beside its work: each block behind the sorting ones a contiguous share of a
// part of the gradient.
constexpr int64_t ZERO_SHARE = 256 << 10;  // bytes
struct Zeros {
  char* to;
  int64_t bytes;
};
__device__ __forceinline__ void write_share(const Zeros& z, int64_t block) {
  // shares begin on 16-byte lines; what lies before the first and behind the last is written by two bytes
  const int head = static_cast<int>(min(z.bytes, static_cast<int64_t>(-reinterpret_cast<uintptr_t>(z.to) & 15)));
  char* p = z.to + head;
  const int64_t vectors = (z.bytes - head) / 16;
  const int64_t v0 = block * (ZERO_SHARE / 16), v1 = min(v0 + ZERO_SHARE / 16, vectors);
  for (int64_t i = v0 + threadIdx.x; i < v1; i += blockDim.x)
    __stcs(reinterpret_cast<uint4*>(p) + i, make_uint4(0, 0, 0, 0));
  if (block > 0) return;
  const int tail = static_cast<int>((z.bytes - head) % 16);
  if (static_cast<int>(threadIdx.x) < head / 2) reinterpret_cast<uint16_t*>(z.to)[threadIdx.x] = 0;
  if (static_cast<int>(threadIdx.x) < tail / 2) reinterpret_cast<uint16_t*>(z.to + z.bytes - tail)[threadIdx.x] = 0;
}

struct SortArgs {
  Zeros zeros;
  const int64_t* tokens;       // first pass
  const unsigned* keys;        // later passes: the order so far
  const unsigned* pos;
  unsigned* keys_out;
  unsigned* pos_out;
  const unsigned* counts;      // [blocks][bins] of this digit
  unsigned* counts_next;       // of the next digit, zero before (null in the last pass)
  unsigned* counts_clear;      // zeroed for the digit after that
  unsigned* flags;
  int64_t N, V, ignore_index;
  unsigned tile;               // keys of a block: a multiple of SORT_THREADS
  int blocks, bits, shift, next_bits;
  bool first;
};

// Tokens as keys: those of no row sort behind the others.
__device__ __forceinline__ unsigned key_of(int64_t t, const SortArgs& a) {
  if (t == a.ignore_index) return static_cast<unsigned>(a.V);
  if (t < 0 || t >= a.V) return static_cast<unsigned>(a.V) + 1u;
  return static_cast<unsigned>(t);
}

// Counts of the first digit; clears what later launches count into.
__global__ void __launch_bounds__(SORT_THREADS) embedding_count_kernel(const SortArgs a) {
  __shared__ unsigned bins[MAX_BINS];
  const int n_bins = 1 << a.bits;
  for (int i = threadIdx.x; i < n_bins; i += SORT_THREADS) bins[i] = 0;
  __syncthreads();
  ptx::wait_for_previous();
  ptx::launch_dependents();
  if (static_cast<int>(blockIdx.x) >= a.blocks) {
    write_share(a.zeros, blockIdx.x - a.blocks);
    return;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.flags = 0u;
  for (int i = threadIdx.x; i < MAX_BINS; i += SORT_THREADS)
    a.counts_clear[static_cast<int64_t>(blockIdx.x) * MAX_BINS + i] = 0u;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * a.tile;
  const int64_t i1 = min(i0 + a.tile, a.N);
  // a warp goes on as one, whichever of its lanes are within the tile: all of them take part in the matching
  const int lane = threadIdx.x & 31;
  for (int64_t i = i0 + (threadIdx.x - lane); i < i1; i += SORT_THREADS) {
    const bool in = i + lane < i1;
    const unsigned d = in ? key_of(a.tokens[i + lane], a) & (n_bins - 1) : 0xffffffffu;
    // frequent tokens come many at a time: one addition for each digit of a warp
    const unsigned same = __match_any_sync(0xffffffffu, d);
    if (in && lane == __ffs(same) - 1) atomicAdd(&bins[d], __popc(same));
  }
  __syncthreads();
  unsigned* out = const_cast<unsigned*>(a.counts) + static_cast<int64_t>(blockIdx.x) * MAX_BINS;
  for (int i = threadIdx.x; i < n_bins; i += SORT_THREADS) out[i] = bins[i];
}

// One digit: block b places the keys [b tile, (b + 1) tile) behind those of lower digits, and behind
// equal digits of earlier blocks, warps and lanes.
__global__ void __launch_bounds__(SORT_THREADS) embedding_sort_kernel(const SortArgs a) {
  extern __shared__ unsigned place[];  // [warps][bins]
  __shared__ unsigned warp_sum[SORT_WARPS];
  const int n_bins = 1 << a.bits, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (static_cast<int>(blockIdx.x) < a.blocks) {
    for (int i = threadIdx.x; i < n_bins * SORT_WARPS; i += SORT_THREADS) place[i] = 0u;
  }
  __syncthreads();
  ptx::wait_for_previous();
  ptx::launch_dependents();
  if (static_cast<int>(blockIdx.x) >= a.blocks) {
    write_share(a.zeros, blockIdx.x - a.blocks);
    return;
  }
  if (a.counts_clear)
    for (int i = threadIdx.x; i < MAX_BINS; i += SORT_THREADS)
      a.counts_clear[static_cast<int64_t>(blockIdx.x) * MAX_BINS + i] = 0u;
  // this block's first place for each digit
  unsigned before = 0, total = 0;
  if (threadIdx.x < n_bins) {
#pragma unroll 8
    for (int b = 0; b < a.blocks; ++b) {
      const unsigned c = a.counts[b * MAX_BINS + threadIdx.x];
      if (b < static_cast<int>(blockIdx.x)) before += c;
      total += c;
    }
  }
  unsigned incl = total;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    unsigned v = warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    warp_sum[lane] = v;
  }
  __syncthreads();
  const unsigned base = incl - total + (warp > 0 ? warp_sum[warp - 1] : 0u) + before;
  // counts of each warp's keys, which are contiguous
  unsigned* mine = place + warp * n_bins;
  const int64_t per_warp = a.tile / SORT_WARPS;
  const int64_t w0 = static_cast<int64_t>(blockIdx.x) * a.tile + warp * per_warp;
  const int64_t w1 = min(w0 + per_warp, a.N);
  auto key_at = [&](int64_t i) -> unsigned { return a.first ? key_of(a.tokens[i], a) : a.keys[i]; };
  bool bad = false;
  for (int64_t i = w0; i < w1; i += 32) {
    const bool in = i + lane < w1;
    const unsigned key = in ? key_at(i + lane) : 0u;
    bad |= in && key == static_cast<unsigned>(a.V) + 1u;
    const unsigned d = in ? (key >> a.shift) & (n_bins - 1) : 0xffffffffu;
    const unsigned same = __match_any_sync(0xffffffffu, d);
    if (in && lane == __ffs(same) - 1) mine[d] += __popc(same);
    __syncwarp();
  }
  if (a.first && bad) atomicOr(a.flags, ERR_LABEL);
  __syncthreads();
  if (threadIdx.x < n_bins) {
    unsigned run = base;
#pragma unroll 8
    for (int w = 0; w < SORT_WARPS; ++w) {
      const unsigned c = place[w * n_bins + threadIdx.x];
      place[w * n_bins + threadIdx.x] = run;
      run += c;
    }
  }
  __syncthreads();
  for (int64_t i = w0; i < w1; i += 32) {
    const bool in = i + lane < w1;
    const unsigned key = in ? key_at(i + lane) : 0u;
    const unsigned d = in ? (key >> a.shift) & (n_bins - 1) : 0xffffffffu;
    const unsigned same = __match_any_sync(0xffffffffu, d);
    const unsigned to = in ? mine[d] + __popc(same & ((1u << lane) - 1u)) : 0u;
    __syncwarp();
    if (in && lane == __ffs(same) - 1) mine[d] += __popc(same);
    __syncwarp();
    if (in) {
      a.keys_out[to] = key;
      a.pos_out[to] = a.first ? static_cast<unsigned>(i + lane) : a.pos[i + lane];
    }
    if (a.counts_next) {
      const unsigned slot = in ? (to / a.tile) * MAX_BINS +
                                     ((key >> (a.shift + a.bits)) & ((1u << a.next_bits) - 1u))
                               : 0xffffffffu;
      const unsigned peers = __match_any_sync(0xffffffffu, slot);
      if (in && lane == __ffs(peers) - 1) atomicAdd(&a.counts_next[slot], __popc(peers));
    }
  }
}

// Up to 4096 positions are sorted by counting: the place of a position is the number of smaller keys and of equal ones
// before it.  A block places 32 positions, one a lane; its warps compare them with a share of all the keys each.
// Nothing here waits but for the tokens and one sum over the block; the gradient of 512 x 1024 takes 2.5 us less for it
// than with the digits in one block below, that of 4096 x 256 3.5 us.  At 8192 the N^2 comparisons keep all SMs from
// writing zeros: 54 us against 45 for 8192 x 2048 of 50,000 tokens.
constexpr int RANK_ITEMS = 4;
constexpr int MAX_RANKED = SORT_THREADS * RANK_ITEMS;
__global__ void __launch_bounds__(SORT_THREADS) embedding_rank_kernel(const SortArgs a) {
  __shared__ __align__(16) unsigned keys[MAX_RANKED];
  __shared__ unsigned counted[SORT_WARPS][32];
  ptx::wait_for_previous();
  ptx::launch_dependents();
  if (blockIdx.x >= static_cast<unsigned>(a.blocks)) {
    write_share(a.zeros, blockIdx.x - a.blocks);
    return;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = static_cast<int>(a.N), own = static_cast<int>(blockIdx.x) * 32;
  const int rounds = (n + SORT_THREADS - 1) / SORT_THREADS;
  const int first = warp * rounds * 32;
  constexpr unsigned NONE = 0xffffffffu;
  const unsigned mine = own + lane < n ? key_of(a.tokens[own + lane], a) : NONE;
  bool bad = false;
#pragma unroll
  for (int r = 0; r < RANK_ITEMS; ++r) {
    if (r >= rounds) break;
    const int i = first + r * 32 + lane;
    const unsigned key = i < n ? key_of(a.tokens[i], a) : NONE;
    bad |= key == static_cast<unsigned>(a.V) + 1u;
    keys[i] = key;
  }
  __syncwarp();
  unsigned count = 0;
  for (int r = 0; r < rounds; ++r) {
    const int base = first + r * 32;
    if (base == own) {
#pragma unroll 8
      for (int j = 0; j < 32; ++j) count += keys[base + j] < mine + (j < lane ? 1u : 0u);
    } else {
      const unsigned bound = mine + (base < own ? 1u : 0u);
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const uint4 k = *reinterpret_cast<const uint4*>(keys + base + j);
        count += (k.x < bound) + (k.y < bound) + (k.z < bound) + (k.w < bound);
      }
    }
  }
  counted[warp][lane] = count;
  bad = __syncthreads_or(bad);
  if (warp > 0) return;
  if (own == 0 && lane == 0) *a.flags = bad ? ERR_LABEL : 0u;
  count = 0;
#pragma unroll
  for (int w = 0; w < SORT_WARPS; ++w) count += counted[w][lane];
  if (own + lane < n) {
    a.keys_out[count] = mine;
    a.pos_out[count] = own + lane;
  }
}

// All digits in one block, for more than those, up to SMALL_SORT positions: keys and positions go round through shared memory.
constexpr int SMALL_ITEMS = 8;
constexpr int SMALL_SORT = SORT_THREADS * SMALL_ITEMS;
__global__ void __launch_bounds__(SORT_THREADS) embedding_sort_small_kernel(const SortArgs a, int passes) {
  extern __shared__ unsigned place[];  // [warps][bins], then the keys and positions
  __shared__ unsigned warp_sum[SORT_WARPS];
  const int n_bins = 1 << a.bits, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned* keys = place + n_bins * SORT_WARPS;
  unsigned* pos = keys + SMALL_SORT;
  ptx::wait_for_previous();
  ptx::launch_dependents();
  if (blockIdx.x > 0) {
    write_share(a.zeros, blockIdx.x - 1);
    return;
  }
  const int n = static_cast<int>(a.N);
  // contiguous keys of a warp, as many rounds of 32 as there are for it
  const int rounds = (n + SORT_THREADS - 1) / SORT_THREADS;
  const int first = warp * rounds * 32 + lane;
  unsigned key[SMALL_ITEMS], at[SMALL_ITEMS];
  bool bad = false;
#pragma unroll
  for (int r = 0; r < SMALL_ITEMS; ++r) {
    const int i = first + r * 32;
    key[r] = 0xffffffffu;
    at[r] = i;
    if (r < rounds && i < n) {
      key[r] = key_of(a.tokens[i], a);
      bad |= key[r] == static_cast<unsigned>(a.V) + 1u;
    }
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) *a.flags = bad ? ERR_LABEL : 0u;
  unsigned* mine = place + warp * n_bins;
  for (int p = 0; p < passes; ++p) {
    for (int i = threadIdx.x; i < n_bins * SORT_WARPS / 4; i += SORT_THREADS)
      reinterpret_cast<uint4*>(place)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    unsigned rank[SMALL_ITEMS];
#pragma unroll
    for (int r = 0; r < SMALL_ITEMS; ++r) {
      if (r >= rounds) break;
      const bool in = first + r * 32 < n;
      const unsigned d = in ? (key[r] >> (p * a.bits)) & (n_bins - 1) : 0xffffffffu;
      const unsigned same = __match_any_sync(0xffffffffu, d);
      rank[r] = in ? mine[d] + __popc(same & ((1u << lane) - 1u)) : 0u;
      __syncwarp();
      if (in && lane == __ffs(same) - 1) mine[d] += __popc(same);
      __syncwarp();
    }
    __syncthreads();
    // counts of a digit over the warps, then over the digits
    unsigned total = 0;
    if (threadIdx.x < n_bins) {
#pragma unroll 8
      for (int w = 0; w < SORT_WARPS; ++w) {
        const unsigned c = place[w * n_bins + threadIdx.x];
        place[w * n_bins + threadIdx.x] = total;
        total += c;
      }
    }
    unsigned incl = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    unsigned before = 0;
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    before += incl - total;
    if (threadIdx.x < n_bins) {
#pragma unroll 8
      for (int w = 0; w < SORT_WARPS; ++w) place[w * n_bins + threadIdx.x] += before;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < SMALL_ITEMS; ++r) {
      if (r >= rounds) break;
      if (first + r * 32 >= n) continue;
      const unsigned to = rank[r] + mine[(key[r] >> (p * a.bits)) & (n_bins - 1)];
      keys[to] = key[r];
      pos[to] = at[r];
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < SMALL_ITEMS; ++r) {
      const int i = first + r * 32;
      if (r < rounds && i < n) {
        key[r] = keys[i];
        at[r] = pos[i];
      }
    }
  }
  for (int i = threadIdx.x; i < n; i += SORT_THREADS) {
    a.keys_out[i] = keys[i];
    a.pos_out[i] = pos[i];
  }
}

// ------------------------------------------------------------------------------------ sums
constexpr int MAX_TILE = 64;    // sorted positions of a tile

struct SumArgs {
  const unsigned* keys;
  const unsigned* pos;
  const void* dy;
  void* out;
  float* part;                // [tiles][2][d]: of a run from the tile before, of one into the next
  int64_t N, V, ldy;
  int d, tile;
  unsigned tiles, chunks;     // column chunks of blockDim.x vectors
  float scale;
  bool accumulate;
};

// V values of type G: 16 bytes at a time, or as many as there are.
template <typename G, int V>
__device__ __forceinline__ void store_vec(G* p, const float (&v)[V]) {
  constexpr int STEP = V < kVec<G> ? (V < kWord<G> ? 1 : kWord<G>) : kVec<G>;
#pragma unroll
  for (int i = 0; i < V; i += STEP) {
    float u[STEP];
#pragma unroll
    for (int j = 0; j < STEP; ++j) u[j] = v[i + j];
    store_raw<G, STEP>(p + i, pack<G, STEP>(u));
  }
}
template <typename G, int V>
__device__ __forceinline__ void load_vec(const G* p, float (&v)[V]) {
  constexpr int STEP = V < kVec<G> ? (V < kWord<G> ? 1 : kWord<G>) : kVec<G>;
#pragma unroll
  for (int i = 0; i < V; i += STEP) {
    float u[STEP];
    unpack<G, STEP>(load_raw<G, STEP>(p + i), u);
#pragma unroll
    for (int j = 0; j < STEP; ++j) v[i + j] = u[j];
  }
}
// The finished sum of one token's rows.
template <typename G, int V>
__device__ __forceinline__ void write_sum(G* p, float (&s)[V], float scale, bool accumulate) {
  if (accumulate) {
    float old[V];
    load_vec<G, V>(p, old);
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] = fmaf(s[j], scale, old[j]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] *= scale;
  }
  store_vec<G, V>(p, s);
}

template <typename E, typename G, int V>
__global__ void __launch_bounds__(256) embedding_grad_kernel(const SumArgs a) {
  __shared__ unsigned found[2 * MAX_TILE], place[2 * MAX_TILE];
  ptx::wait_for_previous();
  ptx::launch_dependents();
  const unsigned tile = blockIdx.x / a.chunks;
  constexpr unsigned NONE = 0xffffffffu;
  const int64_t r0 = static_cast<int64_t>(tile) * a.tile;
  const int spare = a.tile / 4;
  for (int i = threadIdx.x; i < a.tile + spare + 2; i += blockDim.x) {
    const int64_t r = r0 - 1 + i;
    const bool in = r >= 0 && r < a.N;
    found[i] = in ? a.keys[r] : NONE;
    place[i] = in ? a.pos[r] : 0u;
  }
  __syncthreads();
  // a run that goes on over an edge of the tile by `spare` rows at most belongs to the tile before the edge
  auto moved = [&](int edge) {  // edge: place in found of the first row behind it
    int m = 0;
    while (m <= spare && found[edge + m] == found[edge - 1]) ++m;
    return m <= spare ? m : 0;
  };
  const int64_t end = min(r0 + a.tile, a.N);
  const int from = r0 > 0 ? moved(1) : 0;
  const int to = static_cast<int>(end - r0) + (end < a.N ? moved(1 + a.tile) : 0);
  const int n = to - from;
  const unsigned* keys = found + from;  // of the row before the first, then of the rows, then of the one behind
  const unsigned* pos = place + from + 1;
  const int64_t c = (static_cast<int64_t>(blockIdx.x % a.chunks) * blockDim.x + threadIdx.x) * V;
  if (c >= a.d) return;
  const E* dy = static_cast<const E*>(a.dy) + c;
  constexpr int U = V == kVec<E> ? 8 : 16;  // rows in flight
  float s[V];
#pragma unroll
  for (int j = 0; j < V; ++j) s[j] = 0.f;
  const unsigned vocabulary = static_cast<unsigned>(a.V);
  bool whole = keys[0] != keys[1];  // the run began in this tile
  for (int r = 0; r < n; r += U) {
    Raw<E, V> q[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = r + u < n && keys[r + u + 1] < vocabulary;
      q[u] = in ? load_raw_once<E, V>(dy + static_cast<int64_t>(pos[r + u]) * a.ldy) : zero_raw<E, V>();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (r + u >= n) break;
      const unsigned key = keys[r + u + 1];
      if (key >= vocabulary) return;  // the rest is of no row
      float v[V];
      unpack<E, V>(q[u], v);
#pragma unroll
      for (int j = 0; j < V; ++j) s[j] += v[j];
      const bool goes_on = keys[r + u + 2] == key;
      if (goes_on && r + u + 1 < n) continue;
      // the run ends here, or the tile does
      if (!whole) store_vec<float, V>(a.part + static_cast<int64_t>(tile) * 2 * a.d + c, s);
      else if (goes_on) store_vec<float, V>(a.part + (static_cast<int64_t>(tile) * 2 + 1) * a.d + c, s);
      else write_sum<G, V>(static_cast<G*>(a.out) + static_cast<int64_t>(key) * a.d + c, s, a.scale, a.accumulate);
      whole = true;
#pragma unroll
      for (int j = 0; j < V; ++j) s[j] = 0.f;
    }
  }
}

// Joins the partial sums of the run that begins in tile t and goes on after it: that of its beginning, then
// one of each following tile it reaches.  A warp a column chunk of 32 vectors and every eighth partial.
template <typename G, int V>
__global__ void __launch_bounds__(256) embedding_join_kernel(const SumArgs a) {
  __shared__ float sh[8][32 * V];
  ptx::wait_for_previous();
  ptx::launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = blockIdx.x / a.chunks;
  const int64_t r0 = t * a.tile, r1 = r0 + a.tile;
  const int spare = a.tile / 4;
  if (r1 + spare >= a.N) return;
  // what decides, and the first keys that count the tiles, are read at once
  auto key_at = [&](int64_t r) { return r >= 0 && r < a.N ? a.keys[r] : 0xffffffffu; };
  auto reached = [&](int64_t count) { return key_at((t + 1 + count + lane) * a.tile + spare); };
  const unsigned key = a.keys[r1 - 1], behind = a.keys[r1 + spare], before = key_at(r0 - 1);
  unsigned next = reached(1);
  // not a run that goes on by more than the tile takes over, or one that began before
  if ((key >= static_cast<unsigned>(a.V)) | (behind != key) | (before == key)) return;
  int64_t count = 1;  // tiles after t that it reaches
  while (true) {
    const unsigned on = __ballot_sync(0xffffffffu, next == key);
    const int more = on == 0xffffffffu ? 32 : __ffs(~on) - 1;
    count += more;
    if (more < 32) break;
    next = reached(count);
  }
  const int64_t c = (static_cast<int64_t>(blockIdx.x % a.chunks) * 32 + lane) * V;
  float s[V];
#pragma unroll
  for (int j = 0; j < V; ++j) s[j] = 0.f;
  if (c < a.d) {
#pragma unroll 4
    for (int64_t k = warp; k <= count; k += 8) {
      float v[V];
      load_vec<float, V>(a.part + ((t + k) * 2 + (k == 0 ? 1 : 0)) * a.d + c, v);
#pragma unroll
      for (int j = 0; j < V; ++j) s[j] += v[j];
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) sh[warp][j * 32 + lane] = s[j];
  __syncthreads();
  if (warp == 0 && c < a.d) {
#pragma unroll
    for (int w = 1; w < 8; ++w) {
#pragma unroll
      for (int j = 0; j < V; ++j) s[j] += sh[w][j * 32 + lane];
    }
    write_sum<G, V>(static_cast<G*>(a.out) + static_cast<int64_t>(key) * a.d + c, s, a.scale, a.accumulate);
  }
}

// ---------------------------------------------------------------------------------- host side
bool aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool dtype_ok(lce_dtype_t dt) { return dt == LCE_BF16 || dt == LCE_F32; }
size_t elem(lce_dtype_t dt) { return dt == LCE_BF16 ? 2 : 4; }
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
bool dim_ok(int64_t n, int64_t least) { return n >= least && n <= kMaxDim; }
bool sizes_ok(int64_t N, int64_t d, int64_t V) {
  return dim_ok(N, 0) && dim_ok(d, 1) && dim_ok(V, 1) && N * d <= kMaxElements && V * d <= kMaxElements;
}
bool stride_ok(int64_t ld, int64_t d, int64_t N) {
  return ld >= d && ld <= kMaxElements && (N <= 1 || ld <= (int64_t(1) << 62) / N);
}

// Sorted positions of a tile: long enough that joining is little work, short enough that there are warps for the SMs,
// with as many positions to fetch one after the other.  Added to an fp32 gradient, us for 8 / 16 / 64: 512 x 1024
// 8.5 / 10.9 / 27, 1999 x 515 15 / 15 / 31 (written: 15.3 / 13.6 / 22), 4096 x 2048 18 / 21.5 / 36, 17523 x 368 32 / 28 /
// 43, 32768 x 512 47 / 37 / 46, 32768 x 2048 98 / 76 / 71, 65536 x 64 68 / 49 / 50 (written: 69 / 49 / 43).
int tile_rows(int64_t N, int64_t d) {
  if (N <= 1024 || (N <= 4096 && N * d <= (int64_t(1) << 19))) return 8;
  return N < 65536 && N * d < (int64_t(1) << 25) ? 16 : 64;
}

// As many tiles as N positions or fewer may have: a workspace does for smaller calls too.
int64_t most_tiles(int64_t N, int64_t d) {
  const int64_t by8 = std::min(N, std::max<int64_t>(1024, std::min<int64_t>(4096, (int64_t(1) << 19) / d)));
  const int64_t by16 = std::min({N, int64_t(65535), ((int64_t(1) << 25) - 1) / d});
  return std::max({(N + 63) / 64, (by16 + 15) / 16, (by8 + 7) / 8});
}

struct Layout {
  size_t keys[2], pos[2], counts[3], part, total;
  int64_t tiles;
};
Layout layout(int64_t N, int64_t d) {
  Layout l{};
  size_t off = WS_HEADER_BYTES;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += align256(bytes);
    return at;
  };
  for (int i = 0; i < 2; ++i) {
    l.keys[i] = take(static_cast<size_t>(N) * 4);
    l.pos[i] = take(static_cast<size_t>(N) * 4);
  }
  for (int i = 0; i < 3; ++i) l.counts[i] = take(sizeof(unsigned) * MAX_SORT_BLOCKS * MAX_BINS);
  const int rows = tile_rows(N, d);
  l.tiles = (N + rows - 1) / rows;
  l.part = take(static_cast<size_t>(most_tiles(N, d)) * 2 * static_cast<size_t>(d) * sizeof(float));
  l.total = off;
  return l;
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), unsigned grid, int threads, size_t smem, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {dependent_launch()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

unsigned zero_blocks(int64_t bytes) { return static_cast<unsigned>((bytes + ZERO_SHARE - 1) / ZERO_SHARE); }

// Lets a kernel use so much shared memory on the current device; asked once of each.
template <typename K>
cudaError_t allow(K kernel, size_t smem, PerDevice<kMaxDevices>& allowed) {
  int dev = 0, unused;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess)
    e = allowed.get(dev, [&](int* value) {
      *value = 1;
      return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    }, &unused);
  return note(e);
}

// Sorts the positions by token; *result: which of the two pairs of arrays holds them.  Its launches also write zeros to
// all bytes of out, a share each: the memory is busy while the sort waits for its latencies.
cudaError_t sort_positions(SortArgs a, char* ws, const Layout& l, char* out, int64_t bytes, int* result, cudaStream_t s) {
  int bits = 1;
  while (bits < 32 && (uint64_t(1) << bits) < static_cast<uint64_t>(a.V) + 2) ++bits;
  const int passes = (bits + MAX_DIGIT_BITS - 1) / MAX_DIGIT_BITS;
  const int digit = (bits + passes - 1) / passes;
  if (a.N <= MAX_RANKED) {
    a.blocks = static_cast<int>((a.N + 31) / 32);
    a.keys_out = reinterpret_cast<unsigned*>(ws + l.keys[0]);
    a.pos_out = reinterpret_cast<unsigned*>(ws + l.pos[0]);
    a.zeros = Zeros{out, bytes};
    *result = 0;
    return traced(K_EMBED_SORT, s, [&] {
      return launch(embedding_rank_kernel, a.blocks + zero_blocks(bytes), SORT_THREADS, 0, s, a);
    });
  }
  if (a.N <= SMALL_SORT) {
    a.bits = digit;
    a.keys_out = reinterpret_cast<unsigned*>(ws + l.keys[0]);
    a.pos_out = reinterpret_cast<unsigned*>(ws + l.pos[0]);
    a.zeros = Zeros{out, bytes};
    *result = 0;
    const size_t smem = ((size_t(1) << digit) * SORT_WARPS + 2 * SMALL_SORT) * sizeof(unsigned);
    static PerDevice<kMaxDevices> allowed;
    const cudaError_t e = allow(embedding_sort_small_kernel, (MAX_BINS * SORT_WARPS + 2 * SMALL_SORT) * sizeof(unsigned), allowed);
    if (e != cudaSuccess) return e;
    return traced(K_EMBED_SORT, s, [&] {
      return launch(embedding_sort_small_kernel, 1 + zero_blocks(bytes), SORT_THREADS, smem, s, a,
                    passes);
    });
  }
  const int64_t least = (a.N + MAX_SORT_BLOCKS - 1) / MAX_SORT_BLOCKS;
  a.tile = static_cast<unsigned>((least + SORT_THREADS - 1) / SORT_THREADS * SORT_THREADS);
  a.blocks = static_cast<int>((a.N + a.tile - 1) / a.tile);
  auto at = [&](size_t off) { return reinterpret_cast<unsigned*>(ws + off); };
  // what is left of the zeros, shared among what is left of the launches
  auto take_zeros = [&](int launches) {
    const int64_t n = launches == 1 ? bytes : bytes / launches / 256 * 256;
    a.zeros = Zeros{out, n};
    out += n;
    bytes -= n;
    return a.blocks + zero_blocks(n);
  };
  a.bits = a.next_bits = digit;
  a.counts = at(l.counts[0]);
  a.counts_clear = at(l.counts[1]);
  cudaError_t e = traced(K_EMBED_SORT, s, [&] {
    const unsigned grid = take_zeros(passes + 1);
    return launch(embedding_count_kernel, grid, SORT_THREADS, 0, s, a);
  });
  const size_t smem = (size_t(1) << digit) * SORT_WARPS * sizeof(unsigned);
  static PerDevice<kMaxDevices> allowed;
  if (e == cudaSuccess) e = allow(embedding_sort_kernel, MAX_BINS * SORT_WARPS * sizeof(unsigned), allowed);
  for (int p = 0; p < passes && e == cudaSuccess; ++p) {
    a.first = p == 0;
    const bool last = p == passes - 1;
    a.shift = p * digit;
    a.counts = at(l.counts[p % 3]);
    a.counts_next = last ? nullptr : at(l.counts[(p + 1) % 3]);
    a.counts_clear = last ? nullptr : at(l.counts[(p + 2) % 3]);
    a.keys_out = at(l.keys[p & 1]);
    a.pos_out = at(l.pos[p & 1]);
    const unsigned grid = take_zeros(passes - p);
    e = traced(K_EMBED_SORT, s, [&] { return launch(embedding_sort_kernel, grid, SORT_THREADS, smem, s, a); });
    a.keys = a.keys_out;
    a.pos = a.pos_out;
    *result = p & 1;
  }
  return e;
}

template <typename E, typename G, int V>
cudaError_t sum_rows(SumArgs a, cudaStream_t s) {
  const int64_t nv = (a.d + V - 1) / V;
  const int threads = static_cast<int>(std::min<int64_t>(256, (nv + 31) / 32 * 32));
  a.chunks = static_cast<unsigned>((nv + threads - 1) / threads);
  const int64_t grid = static_cast<int64_t>(a.tiles) * a.chunks;
  if (grid > kMaxDim) return cudaErrorInvalidConfiguration;
  cudaError_t e = traced(K_EMBED_GRAD, s, [&] {
    return launch(embedding_grad_kernel<E, G, V>, static_cast<unsigned>(grid), threads, 0, s, a);
  });
  if (e != cudaSuccess || a.tiles < 2) return e;
  a.chunks = static_cast<unsigned>((nv + 31) / 32);
  return traced(K_EMBED_JOIN, s, [&] {
    return launch(embedding_join_kernel<G, V>, a.tiles * a.chunks, 256, 0, s, a);
  });
}

}  // namespace
}  // namespace lce

using namespace lce;

extern "C" {

size_t lce_embedding_workspace_size(int64_t N, int64_t d, int64_t V, int32_t backward) {
  if (!sizes_ok(N, d, V) || (backward != 0 && backward != 1)) return 0;
  if (!backward) return WS_HEADER_BYTES;
  const Layout l = layout(N, d);
  // blocks of the launches of sums and of zeros
  if (l.tiles * ((d + 31) / 32) > kMaxDim || V * d > (kMaxDim - MAX_SORT_BLOCKS) * (ZERO_SHARE / 4)) return 0;
  return l.total;
}

lce_status_t lce_embedding_forward(const int64_t* tokens, const void* table, int64_t N, int64_t d,
                                   int64_t V, float scale, int64_t ignore_index, lce_dtype_t dtype,
                                   void* Y, int64_t ldy, void* workspace, size_t ws_bytes,
                                   void* stream) {
  if (!dtype_ok(dtype)) return LCE_ERR_INVALID_ARG;
  if (!sizes_ok(N, d, V) || !stride_ok(ldy, d, N)) return LCE_ERR_UNSUPPORTED_SHAPE;
  const size_t e = elem(dtype);
  if (!table || (N > 0 && (!tokens || !Y)) || !workspace || !aligned(workspace, 16) || !aligned(tokens, 8) ||
      !aligned(table, e) || !aligned(Y, e))
    return LCE_ERR_INVALID_ARG;
  if (ws_bytes < WS_HEADER_BYTES) return LCE_ERR_WORKSPACE_TOO_SMALL;
  LookupArgs a{};
  a.tokens = tokens, a.table = table, a.y = Y, a.N = N, a.V = V, a.ldy = ldy, a.ignore_index = ignore_index;
  a.d = static_cast<int>(d), a.scale = scale, a.flags = static_cast<unsigned*>(workspace);
  a.check = N <= CHECKED_TOKENS;
  auto whole = [&](size_t n) {
    return aligned(table, n) && aligned(Y, n) && d * e % n == 0 && (N <= 1 || ldy * e % n == 0);
  };
  const bool by16 = whole(16), by4 = whole(4);
  const int64_t width = 32 * (by16 ? 4 * (16 / static_cast<int64_t>(e)) : 16 * (by4 ? 4 / static_cast<int64_t>(e) : 1));
  a.segments = static_cast<int>((d + width - 1) / width);
  a.items = N * a.segments;
  const int64_t blocks = (a.items + 7) / 8 + (a.check ? 1 : 0);
  if (blocks > kMaxDim) return LCE_ERR_UNSUPPORTED_SHAPE;
  int num_sms = 0;
  const lce_status_t st = check_device(&num_sms);
  if (st != LCE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!a.check && traced(K_EMBED, s, [&] {
        return launch_kernel(embedding_clear_kernel, dim3(1), 32, s, a.flags);
      }) != cudaSuccess)
    return LCE_ERR_CUDA;
  const cudaError_t err = traced(K_EMBED, s, [&] {
    const dim3 grid(static_cast<unsigned>(blocks));
    if (dtype == LCE_BF16)
      return by16  ? launch_kernel(embedding_kernel<__nv_bfloat16, 8>, grid, 256, s, a)
             : by4 ? launch_kernel(embedding_kernel<__nv_bfloat16, 2>, grid, 256, s, a)
                   : launch_kernel(embedding_kernel<__nv_bfloat16, 1>, grid, 256, s, a);
    return by16 ? launch_kernel(embedding_kernel<float, 4>, grid, 256, s, a)
                : launch_kernel(embedding_kernel<float, 1>, grid, 256, s, a);
  });
  return err == cudaSuccess ? LCE_OK : LCE_ERR_CUDA;
}

lce_status_t lce_embedding_backward(const int64_t* tokens, const void* dY, int64_t ldy, int64_t N,
                                    int64_t d, int64_t V, float scale, int64_t ignore_index,
                                    lce_dtype_t dtype, lce_dtype_t grad_dtype, int32_t accumulate,
                                    void* dtable, void* workspace, size_t ws_bytes, void* stream) {
  if (!dtype_ok(dtype) || (grad_dtype != dtype && grad_dtype != LCE_F32) ||
      (accumulate != 0 && accumulate != 1))
    return LCE_ERR_INVALID_ARG;
  const size_t need = lce_embedding_workspace_size(N, d, V, 1);
  if (need == 0 || !stride_ok(ldy, d, N)) return LCE_ERR_UNSUPPORTED_SHAPE;
  const size_t e = elem(dtype), ge = elem(grad_dtype);
  if (!dtable || (N > 0 && (!tokens || !dY)) || !workspace || !aligned(workspace, 16) || !aligned(tokens, 8) ||
      !aligned(dY, e) || !aligned(dtable, ge))
    return LCE_ERR_INVALID_ARG;
  if (ws_bytes < need) return LCE_ERR_WORKSPACE_TOO_SMALL;
  int num_sms = 0;
  const lce_status_t st = check_device(&num_sms);
  if (st != LCE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  if (N == 0) {
    cudaError_t err = cudaMemsetAsync(ws, 0, sizeof(unsigned), s);
    if (err == cudaSuccess && !accumulate)
      err = cudaMemsetAsync(dtable, 0, static_cast<size_t>(V) * static_cast<size_t>(d) * ge, s);
    return note(err) == cudaSuccess ? LCE_OK : LCE_ERR_CUDA;
  }
  const Layout l = layout(N, d);
  SortArgs so{};
  so.tokens = tokens, so.flags = reinterpret_cast<unsigned*>(ws), so.N = N, so.V = V;
  so.ignore_index = ignore_index;
  int which = 0;
  SumArgs a{};
  if (sort_positions(so, ws, l, static_cast<char*>(dtable), accumulate ? 0 : V * d * static_cast<int64_t>(ge), &which, s) !=
      cudaSuccess)
    return LCE_ERR_CUDA;
  a.keys = reinterpret_cast<unsigned*>(ws + l.keys[which]);
  a.pos = reinterpret_cast<unsigned*>(ws + l.pos[which]);
  a.dy = dY, a.out = dtable, a.part = reinterpret_cast<float*>(ws + l.part);
  a.N = N, a.V = V, a.ldy = ldy, a.d = static_cast<int>(d), a.tile = tile_rows(N, d);
  a.tiles = static_cast<unsigned>(l.tiles), a.scale = scale, a.accumulate = accumulate != 0;
  auto whole = [&](size_t n) {
    return aligned(dY, n) && aligned(dtable, n) && d * e % n == 0 && (N <= 1 || ldy * e % n == 0);
  };
  const bool by16 = whole(16), by4 = whole(4);
  cudaError_t err;
  if (dtype == LCE_F32)
    err = by16 ? sum_rows<float, float, 4>(a, s) : sum_rows<float, float, 1>(a, s);
  else if (grad_dtype == LCE_F32)
    err = by16  ? sum_rows<__nv_bfloat16, float, 8>(a, s)
          : by4 ? sum_rows<__nv_bfloat16, float, 2>(a, s)
                : sum_rows<__nv_bfloat16, float, 1>(a, s);
  else
    err = by16  ? sum_rows<__nv_bfloat16, __nv_bfloat16, 8>(a, s)
          : by4 ? sum_rows<__nv_bfloat16, __nv_bfloat16, 2>(a, s)
                : sum_rows<__nv_bfloat16, __nv_bfloat16, 1>(a, s);
  return err == cudaSuccess ? LCE_OK : LCE_ERR_CUDA;
}

}  // extern "C"
