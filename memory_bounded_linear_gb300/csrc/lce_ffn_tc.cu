// Feed-forward products on the tensor cores of sm_103a (tcgen05 + TMEM + TMA).
//
// One persistent, warp-specialised kernel on CTA pairs; a pair computes a tile of 256 x bn
// accumulators (bn = 256, or 128 for small products) with cta_group::2 MMAs, CTA r holding its rows
// 128 r .. 128 r + 127:
//   warp 0      TMA producer and tile scheduler (as in lce_tc.cu)
//   warp 1      MMA issuer; two 128 x 256 fp32 accumulators in TMEM, one filled while the other
//               is drained
//   warps 2..9  epilogue: warp w reads the 32 TMEM lanes of its quadrant, one half of the columns
//
// Modes (FfnMode):
//   LINEAR     C = act(Z + bias) + R            Z = A B^T, operands K-major
//   LINEAR_DZ  C = D act'(Z + bias)
//   GATED      C = act(G) U                     the pair's first CTA loads bn/2 rows of Wg, the second
//   GATED_DGU  C = D U act'(G), C2 = D act(G)   the same rows of Wu: the bn accumulator columns are
//                                               G | U of bn/2 output columns, and one thread holds
//                                               both values of an element
//   GRADS      up to three products per launch: dW = dZ^T X (both operands MN-major, read from their
//              row-major arrays) and dX = dZ W (+ dZ2 W2, the K loop running over both pairs)
//
// fp32 operands come as three bf16 parts x = p0 + p1 + p2 (8 bits each, together the 24 of x), and
// a product is the sum of six part products, smallest first: p2 q0, p0 q2, p1 q1, p1 q0, p0 q1,
// p0 q0; the three that are left out are below 2^-24 of the product.  To the kernel that is a K
// loop six times as long, the part being the third coordinate of the operand's tensor map.  The
// tensor cores cut each addition into an accumulator off rather than round it, an error that grows
// with the number of additions (2.6e-6 of a sum of 2008 products); so an fp32 tile is summed in
// steps of F32_STEP k-blocks, each into a fresh accumulator, which the epilogue warps add up in
// registers (4e-7 there, for a drain of about 1,000 cycles per 12,000 of products).
//
// With few tiles (SPLIT) a cluster of 2 or 4 pairs computes each: every pair sums a piece of the K
// loop, puts its partial sums into its ring's memory, and finishes some of the tile's boxes from all
// of them, read through distributed shared memory in the order of the pieces.
//
// The outgoing gradient D and the residual R enter, and C leaves, through 4 KB boxes of the epilogue
// warps (32 rows x 128 bytes, 128-byte swizzle): 16-byte copies by the warp's lanes, each thread
// rewrites its own row, TMA store.  (Boxes loaded by TMA held up the operands behind them in its
// queue: tiles of 4096 x 2048 -> 8192 took 22,000 cycles instead of 17,000.)  Modes that load boxes
// have two per warp, both fetched while the products of their tile run, and a ring of five 32 KB
// stages; so have the others while K is short, where the epilogue decides (a warp then fills one box
// while the other leaves); with long K they have one box and six stages.
//
// Bound: tensor pipe for many tokens (products hide the epilogue from K = 1024 on; at K = 512 a tile's
// epilogue takes 11,000 cycles, its products 4,100).  Measured inside a captured graph, and as single
// calls: gated backward 16384 x 4096 -> 16384 7.0-7.1 ms (1,850-1,880 TFLOP/s) and 7.7-7.8, linear 4096 x
// 8192 -> 2048 83 us (1,650: 128 tiles on 76 pairs) and 93, gated forward 777 x 4096 -> 10952 96 us (1,450:
// four row tiles for 3.04) and 111.
// Ragged edges: TMA zero-fills loads and clips stores.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "bf16_parts.cuh"
#include "lce_act.cuh"
#include "lce_ffn.h"
#include "lce_internal.h"
#include "per_device.h"
#include "ptx.cuh"
#include "tc_common.cuh"

namespace lce {
namespace {

constexpr int TILE = 256;               // rows of a pair's tile, and its accumulator columns at most
constexpr int BK = 64;                  // K elements per stage (one 128-byte swizzle span)
constexpr int A_BYTES = BM * 128;
constexpr int STAGE_BYTES = 2 * A_BYTES;
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 64 + 32 * EPI_WARPS;
constexpr uint32_t TMEM_COLS = 2 * TILE;
constexpr int CTL_BYTES = 512;
constexpr int MAX_STAGES = 6;
constexpr int FFN_LINEAR_RES = 5;       // FFN_LINEAR with a residual, a kernel of its own

template <int MODE>
struct Cfg {
  static constexpr bool GATED = MODE == FFN_GATED || MODE == FFN_GATED_DGU;
  static constexpr bool DZ = MODE == FFN_LINEAR_DZ || MODE == FFN_GATED_DGU;
  static constexpr bool LOADS = DZ || MODE == FFN_LINEAR_RES;  // boxes of D or R are loaded
};

// Shared memory: the stages of the ring, then the boxes of the eight epilogue warps: six stages and
// one box per warp, or five and two.
constexpr int RING_AND_BOXES = 6 * STAGE_BYTES + EPI_WARPS * STAGE_BUF_BYTES;
constexpr int SMEM_BYTES = RING_AND_BOXES + 1024 + CTL_BYTES;
static_assert(5 * STAGE_BYTES + 2 * EPI_WARPS * STAGE_BUF_BYTES == RING_AND_BOXES, "one size");
static_assert(SMEM_BYTES <= 232448, "227 KB of shared memory per CTA");
// a tile's partial sums (SPLIT) fit in the ring
static_assert(5 * STAGE_BYTES >= TILE * BM * 4, "ring smaller than an accumulator");
// K-blocks of a tile up to which two boxes are worth a stage.
constexpr int SHORT_K = 12;
constexpr int RASTER = 8;               // row tiles per rasterisation group (as in lce_tc.cu)
constexpr int MAX_JOBS = 3;
constexpr int MAX_SPLIT = 4;             // pairs that may sum one tile: clusters of 8 CTAs
// Tiles per pair up to which they are dealt out without a scheduler counter: in launches of one
// product, and of several, whose tiles take different times.
constexpr int DEALT_WAVES = 20;
constexpr int DEALT_WAVES_MIXED = 2;
constexpr int F32_STEP = 4;             // k-blocks per accumulator of an fp32 tile
struct Ctl {
  uint64_t full[MAX_STAGES];
  uint64_t empty[MAX_STAGES];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t drain;
  uint64_t tq_full[TQ];
  uint64_t tq_empty[TQ];
  int tq[TQ];
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(Ctl) <= CTL_BYTES, "control block too large");

struct Job {
  int tiles_m, tiles_n, num_tiles;
  int nkb;      // k-blocks of one operand pair and part product
  int pairs;    // operand pairs summed (1 or 2)
  int mn;       // both operands MN-major (dW), else A K-major (and B MN-major in GRADS)
  int c_cols;
  int whole;    // SPLIT: a cluster sums one tile; else each of its pairs computes a tile of its own
};

struct KParams {
  Job job[MAX_JOBS];
  int njobs, total_tiles;
  int act;
  int split;               // pairs per cluster
  int bn;                  // accumulator columns of a tile: 256 or 128
  int boxes;               // per epilogue warp, modes that load none: 1 or 2
  const void* bias;
  const char* d;           // R or D, row stride in bytes
  int64_t d_stride;
  int64_t m_rows;          // rows of Z
  // fp32 pre-activation gradients are written as parts, from registers
  __nv_bfloat16* parts[2];
  int64_t part_ld, part_stride;
  unsigned* err;
  unsigned* sched;         // scheduler counters, or null: tiles are dealt out round-robin
  int clear_flags;         // the first CTA clears the error flags
  int withhold;            // test hook (lce_test_inject_stall): no operand is loaded
};

struct FMaps {
  CUtensorMap a[MAX_JOBS][2];
  CUtensorMap b[MAX_JOBS][2];
  CUtensorMap c[MAX_JOBS];
  CUtensorMap c2;
};

// The six part products, smallest first: operand parts of A and B.
__device__ __forceinline__ int part_a(int s) { return (0x201100 >> (4 * (5 - s))) & 15; }
__device__ __forceinline__ int part_b(int s) { return (0x021010 >> (4 * (5 - s))) & 15; }

struct TilePos {
  int job, tm, tn;
};
__device__ __forceinline__ TilePos locate(const KParams& p, int t) {
  int j = 0;
  while (j + 1 < p.njobs && t >= p.job[j].num_tiles) {
    t -= p.job[j].num_tiles;
    ++j;
  }
  TilePos r;
  r.job = j;
  tile_coords(t, p.job[j].tiles_m, p.job[j].tiles_n, RASTER, r.tm, r.tn);
  return r;
}

// A tile's K loop as steps: single k-blocks for bf16, F32_STEP k-blocks of one operand pair (all six
// part products) for fp32.  bf16 sums every step into one accumulator, fp32 each into its own.
template <bool F32>
__host__ __device__ __forceinline__ int steps_per_pair(int nkb) {
  return F32 ? (nkb + F32_STEP - 1) / F32_STEP : nkb;
}

// The steps of a tile that a CTA pair sums: all, or the part `piece` of `split` (see SPLIT below).
struct Range {
  int lo, hi;
};
__device__ __forceinline__ Range piece_of(int steps, int piece, int split) {
  return Range{static_cast<int>(static_cast<int64_t>(steps) * piece / split),
               static_cast<int>(static_cast<int64_t>(steps) * (piece + 1) / split)};
}

// SPLIT: the work of pair `piece` of cluster `unit`; tm < 0 when there is none.
__device__ __forceinline__ TilePos locate_split(const KParams& p, int unit, int piece) {
  int j = 0;
  while (true) {
    const Job& jb = p.job[j];
    const int clusters = jb.whole ? jb.num_tiles : (jb.num_tiles + p.split - 1) / p.split;
    if (j + 1 == p.njobs || unit < clusters) break;
    unit -= clusters;
    ++j;
  }
  const int tile = p.job[j].whole ? unit : unit * p.split + piece;
  TilePos r{j, -1, -1};
  if (tile < p.job[j].num_tiles)
    tile_coords(tile, p.job[j].tiles_m, p.job[j].tiles_n, RASTER, r.tm, r.tn);
  return r;
}

// Producer side of one tile.  A_MN, B_MN: the operand is MN-major.
template <bool A_MN, bool B_MN, bool F32>
__device__ __forceinline__ bool produce_tile(int nkb, int pairs, Range range, const CUtensorMap* mA,
                                             const CUtensorMap* mB, int m0, int n0, uint32_t base,
                                             Ctl* ctl, Ring& r, volatile int* abort_flag,
                                             unsigned* err, uint32_t rank, uint32_t leader,
                                             int bn, int stages) {
  auto block = [&](const CUtensorMap* a, const CUtensorMap* b, int k0, int za, int zb) {
    const uint32_t full_local = ptx::smem_addr(&ctl->full[r.stage]);
    if (!wait_bar(ptx::smem_addr(&ctl->empty[r.stage]), r.ph ^ 1u, abort_flag, err)) return false;
    const uint32_t full = ptx::mapa_shared(full_local, leader);
    if (rank == 0) ptx::mbar_arrive_expect_tx(full_local, 2 * A_BYTES + bn * 128);
    const uint32_t sa = base + r.stage * STAGE_BYTES, sb = sa + A_BYTES;
    if (A_MN) {
#pragma unroll
      for (int c = 0; c < BM / MN_BOX_ELEMS; ++c)
        ptx::tma_load_3d_pair(sa + c * MN_BOX_BYTES, a, m0 + c * MN_BOX_ELEMS, k0, za, full);
    } else {
      ptx::tma_load_3d_pair(sa, a, k0, m0, za, full);
    }
    if (B_MN) {
      ptx::tma_load_3d_pair(sb, b, n0, k0, zb, full);
      if (bn == TILE)
        ptx::tma_load_3d_pair(sb + MN_BOX_BYTES, b, n0 + MN_BOX_ELEMS, k0, zb, full);
    } else {
      ptx::tma_load_3d_pair(sb, b, k0, n0, zb, full);
    }
    if (++r.stage == stages) { r.stage = 0; r.ph ^= 1u; }
    return true;
  };
  const int per_pair = steps_per_pair<F32>(nkb);
  for (int pr = 0; pr < pairs; ++pr) {
    const CUtensorMap* a = &mA[pr];
    const CUtensorMap* b = &mB[pr];
    const int lo = max(range.lo - pr * per_pair, 0), hi = min(range.hi - pr * per_pair, per_pair);
    for (int st = lo; st < hi; ++st) {
      if (!F32) {
        if (!block(a, b, st * BK, 0, 0)) return false;
      } else {
        const int end = min(nkb, (st + 1) * F32_STEP);
        for (int s = 0; s < 6; ++s)
          for (int kb = st * F32_STEP; kb < end; ++kb)
            if (!block(a, b, kb * BK, part_a(s), part_b(s))) return false;
      }
    }
  }
  return true;
}

template <bool A_MN, bool B_MN>
__device__ __forceinline__ bool mma_tile(int blocks, uint32_t d_tmem, uint32_t base, Ctl* ctl, Ring& r,
                                         volatile int* abort_flag, unsigned* err, uint16_t pair_mask,
                                         int bn, int stages) {
  const uint32_t idesc = bn == TILE ? ptx::idesc_bf16_f32(TILE, TILE, A_MN, B_MN)
                                    : ptx::idesc_bf16_f32(TILE, TILE / 2, A_MN, B_MN);
  for (int kb = 0; kb < blocks; ++kb) {
    if (!wait_bar(ptx::smem_addr(&ctl->full[r.stage]), r.ph, abort_flag, err)) return false;
    ptx::tc_fence_after();
    const uint32_t sa = base + r.stage * STAGE_BYTES, sb = sa + A_BYTES;
#pragma unroll
    for (int k = 0; k < BK / 16; ++k)
      ptx::tc_mma_f16_pair(d_tmem, A_MN ? desc_mnmajor(sa, k) : desc_kmajor(sa, k),
                           B_MN ? desc_mnmajor(sb, k) : desc_kmajor(sb, k), idesc, (kb | k) != 0);
    ptx::tc_commit_pair(ptx::smem_addr(&ctl->empty[r.stage]), pair_mask);
    if (++r.stage == stages) { r.stage = 0; r.ph ^= 1u; }
  }
  return true;
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float lo16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi16(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// The 32-column groups (4, or 2 where bn = 128) of accumulator columns that a warp of column half
// `half` copies.
template <bool GATED>
__device__ __forceinline__ int half_col(int half, int h, int bn) {
  const int groups = bn / 64;
  return GATED ? (h >= groups / 2) * (bn / 2) + half * (bn / 4) + (h & (groups / 2 - 1)) * 32
               : half * (bn / 2) + h * 32;
}

// Element values of `E` per 16-byte chunk.
template <bool F32>
constexpr int CHUNK = F32 ? 4 : 8;

template <bool F32>
__device__ __forceinline__ void unpack(const uint4& q, float* v) {
  if (F32) {
    v[0] = __uint_as_float(q.x); v[1] = __uint_as_float(q.y);
    v[2] = __uint_as_float(q.z); v[3] = __uint_as_float(q.w);
  } else {
    v[0] = lo16(q.x); v[1] = hi16(q.x); v[2] = lo16(q.y); v[3] = hi16(q.y);
    v[4] = lo16(q.z); v[5] = hi16(q.z); v[6] = lo16(q.w); v[7] = hi16(q.w);
  }
}
template <bool F32>
__device__ __forceinline__ uint4 pack(const float* v) {
  if (F32)
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3]));
  return make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}

// 16 columns of one thread's row: z (and u) in registers, D or R read from and the result written to
// the thread's row of the box (chunks first, first + 1, ...).  GATED_DGU: dU goes to the same place of
// the row at row2.  fp32 pre-activation gradients stay in registers: dZ or dG in z, dU in u.
// (16 columns and a loop around them, not a whole box unrolled: the fp32 GELU gradient of 32 columns
// was 70 KB of code, and a short launch spent most of its time fetching it.)
template <int MODE, int ACT, bool F32>
__device__ __forceinline__ void epilogue16(float (&z)[16], float (&u)[16], uint32_t row, uint32_t row2,
                                           uint32_t sw, int first, int col, int c_cols,
                                           const void* bias) {
  constexpr int CH = CHUNK<F32>;
  constexpr bool LINEAR = MODE == FFN_LINEAR || MODE == FFN_LINEAR_RES;
  constexpr bool DZ = Cfg<MODE>::DZ;
#pragma unroll
  for (int q = 0; q < 16 / CH; ++q) {
    const uint32_t place = (static_cast<uint32_t>(first + q) ^ sw) << 4;
    float d[CH], o[CH], b[CH], du[CH];
    if (LINEAR || MODE == FFN_LINEAR_DZ) {
#pragma unroll
      for (int i = 0; i < CH; ++i) b[i] = 0.f;
      if (bias != nullptr && col + q * CH < c_cols) {
        const char* pb = static_cast<const char*>(bias) +
                         static_cast<size_t>(col + q * CH) * (F32 ? 4 : 2);
        unpack<F32>(__ldg(reinterpret_cast<const uint4*>(pb)), b);
      }
    }
    if (Cfg<MODE>::LOADS) unpack<F32>(ptx::ld_shared_v4(row + place), d);
#pragma unroll
    for (int i = 0; i < CH; i += 2) {
      auto two = [](float* x) { return make_float2(x[0], x[1]); };
      auto put = [](float* x, float2 v) { x[0] = v.x; x[1] = v.y; };
      float2 v = two(z + q * CH + i);
      if constexpr (MODE == FFN_GRADS) {
        put(o + i, v);
      } else if constexpr (LINEAR) {
        v = act<ACT, !F32>(vadd(v, two(b + i)));
        if (MODE == FFN_LINEAR_RES) v = vadd(v, two(d + i));
        put(o + i, v);
      } else if constexpr (MODE == FFN_GATED) {
        put(o + i, vmul(act<ACT, !F32>(v), two(u + q * CH + i)));
      } else {
        float2 a, g;
        if (MODE == FFN_LINEAR_DZ) v = vadd(v, two(b + i));
        act_grad<ACT, !F32>(v, a, g);
        float2 r = two(d + i);
        if constexpr (MODE == FFN_GATED_DGU) {
          a = vmul(r, a);
          r = vmul(r, two(u + q * CH + i));
          put(du + i, a);
        }
        r = chain<ACT>(r, g);
        put(o + i, r);
        if (F32) {
          put(z + q * CH + i, r);
          if (MODE == FFN_GATED_DGU) put(u + q * CH + i, a);
        }
      }
    }
    if constexpr (!(F32 && DZ)) {
      uint4 w = pack<F32>(o);
      ptx::st_shared_v4(row + place, w.x, w.y, w.z, w.w);
      if constexpr (MODE == FFN_GATED_DGU) {
        w = pack<F32>(du);
        ptx::st_shared_v4(row2 + place, w.x, w.y, w.z, w.w);
      }
    }
  }
}

// 16 columns of a warp's 32 rows, fp32 values of one row per thread, as three bf16 parts.  Lanes
// exchange halves in pairs, so that two lanes write the 32 bytes (a sector) of one row of a part
// together.  out: the box's first row, at these columns; rows, cols: what exists from there on.  The
// padding of a row to a multiple of 8 columns may be written, nothing reads it.
__device__ __forceinline__ void store_parts(const float (&v)[16], __nv_bfloat16* out, int64_t ld,
                                            int64_t stride, int64_t rows, int cols) {
  const int lane = threadIdx.x & 31;
  const bool odd = lane & 1;
  uint32_t w[3][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a[3], b[3];
    split_bf16(v[2 * i], a);
    split_bf16(v[2 * i + 1], b);
#pragma unroll
    for (int s = 0; s < 3; ++s) w[s][i] = pack2(a[s], b[s]);
  }
  const int row = lane & ~1, c = odd ? 8 : 0;  // rows row and row + 1; this lane writes columns c ..
#pragma unroll
  for (int s = 0; s < 3; ++s) {
    uint32_t got[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      got[i] = __shfl_xor_sync(0xffffffffu, odd ? w[s][i] : w[s][4 + i], 1);
    const uint4 even_row = odd ? make_uint4(got[0], got[1], got[2], got[3])
                               : make_uint4(w[s][0], w[s][1], w[s][2], w[s][3]);
    const uint4 odd_row = odd ? make_uint4(w[s][4], w[s][5], w[s][6], w[s][7])
                              : make_uint4(got[0], got[1], got[2], got[3]);
    __nv_bfloat16* o = out + s * stride + row * ld + c;
    if (c < cols && row < rows) *reinterpret_cast<uint4*>(o) = even_row;
    if (c < cols && row + 1 < rows) *reinterpret_cast<uint4*>(o + ld) = odd_row;
  }
}

// Tickets of one role: from the queue, or where no counters are used dealt out round-robin, which every
// role of both CTAs works out for itself.
struct Tickets {
  TileQueue<true, Ctl> tq;
  bool dealt;
  int next, units, total;
  __device__ __forceinline__ int take(unsigned mask) {
    if (!dealt) return tq.take(mask);
    const int t = next < total ? next : -1;
    next += units;
    return t;
  }
};

template <int MODE, bool F32, bool SPLIT>
__global__ void __launch_bounds__(THREADS, 1)
    ffn_tc_kernel(const __grid_constant__ FMaps maps, const KParams p) {
  using Cf = Cfg<MODE>;
  constexpr bool GATED = Cf::GATED, DZ = Cf::DZ;
  const int nboxes = Cf::LOADS ? 2 : p.boxes;  // per epilogue warp
  const int stages = 7 - nboxes;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = ptx::smem_addr(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;  // 128B-swizzled tiles need 1024B alignment
  uint8_t* smem = smem_raw + (base - raw_addr);
  const uint32_t boxes = base + stages * STAGE_BYTES;
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + RING_AND_BOXES);
  volatile int* abort_flag = &ctl->abort_flag;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  // A cluster is one pair, or with SPLIT several, each summing a piece of the same tile's K loop.
  const uint32_t crank = ptx::cluster_ctarank();
  const uint32_t rank = SPLIT ? crank & 1u : crank;  // 0 = the pair's MMA issuer
  const uint32_t leader = SPLIT ? crank & ~1u : 0u;  // cluster rank of the issuer
  const uint16_t pair_mask = static_cast<uint16_t>(0x3u << leader);
  const int split = SPLIT ? p.split : 1, piece = static_cast<int>(leader >> 1);
  const int units = static_cast<int>(gridDim.x >> 1) / split;
  const int unit = static_cast<int>(blockIdx.x >> 1) / split;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      ptx::mbar_init(ptx::smem_addr(&ctl->full[s]), 1);
      ptx::mbar_init(ptx::smem_addr(&ctl->empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(ptx::smem_addr(&ctl->tfull[b]), 1);
      ptx::mbar_init(ptx::smem_addr(&ctl->tempty[b]), 2 * EPI_WARPS);
    }
    ptx::mbar_init(ptx::smem_addr(&ctl->drain), 1);
    for (int i = 0; i < TQ; ++i) {
      ptx::mbar_init(ptx::smem_addr(&ctl->tq_full[i]), 1);
      // readers: MMA issuer, the second CTA's producer, the epilogue warps of both
      ptx::mbar_init(ptx::smem_addr(&ctl->tq_empty[i]), 2 + 2 * EPI_WARPS);
    }
    ctl->abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(ptx::smem_addr(&ctl->tmem_base), TMEM_COLS);
    ptx::tmem_relinquish_pair();
    ptx::tc_fence_before();
  }
  if (warp == 0 && lane == 0) {
    for (int j = 0; j < p.njobs; ++j) {
      ptx::prefetch_tmap(&maps.a[j][0]);
      ptx::prefetch_tmap(&maps.b[j][0]);
    }
  }
  ptx::wait_for_previous();  // no memory of the caller is touched before this
  // the first CTA is among the first to run, and a wait gives up only WAIT_LIMIT_NS after that
  if (threadIdx.x == 0 && blockIdx.x == 0 && p.clear_flags) *p.err = 0u;
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem_base = ctl->tmem_base;

  // Epilogue warps: the warp's boxes, and the work on one box of results.
  const int e = (warp + 6) & 7;  // warps 2..9
  const int q = warp & 3;        // TMEM lane quadrant the warp may access
  const int half = e >> 2;       // which half of the columns it drains
  constexpr int UC = F32 ? 32 : 64;          // columns of one box
  const int cols = GATED ? p.bn / 2 : p.bn;  // output columns of a tile
  const int nbox = cols / UC;                // its boxes: the first half of them (at least one) for
  const int per_half = max(nbox / 2, 1);     // the warps of column half 0, the rest for half 1
  const int groups = p.bn / 64;              // 32-column groups of accumulators per warp
  const uint32_t my_boxes = boxes + e * nboxes * STAGE_BUF_BYTES;
  const uint32_t sw = lane & 7;
  uint32_t in_flight = 0;              // boxes being loaded, a bit each
  int turn = 0;                        // boxes stored so far, modes that load none
  int split_tile = -1;                 // SPLIT: the cluster whose tile is finished together
  // R or D of one box of results into box i, once the stores from the boxes have been read: eight lanes
  // copy a row's 128 bytes; zeros outside the result.
  auto fetch = [&](int i, int c_cols, int col, int box_row) {
    if (lane == 0) ptx::bulk_wait_read<0>();
    __syncwarp();
    const int c = lane & 7;
    const bool col_ok = col + c * CHUNK<F32> < c_cols;
    const int64_t at = static_cast<int64_t>(col) * (F32 ? 4 : 2) + c * 16;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int r = k * 4 + (lane >> 3);
      const bool ok = col_ok && box_row + r < p.m_rows;
      ptx::copy16_async(my_boxes + i * STAGE_BUF_BYTES + r * 128 + ((c ^ (r & 7)) << 4),
                        p.d + (ok ? (box_row + r) * p.d_stride + at : 0), ok);
    }
    ptx::copy_commit();
    in_flight |= 1u << i;
  };
  // One box of results through box `slot` (modes that load none: through the boxes in turn, whatever
  // the tile): columns col .., rows box_row .. + 31.  load(c, z, u) gives 16 accumulator columns of the
  // thread's row from the box's column c on; loaded() is called once all have been read.
  auto process = [&](int slot, const CUtensorMap* mC, int c_cols, int col, int box_row, auto&& load,
                     auto&& loaded) {
    const int i = Cf::LOADS ? slot : turn++ & (nboxes - 1);
    const uint32_t box = my_boxes + i * STAGE_BUF_BYTES, row_addr = box + lane * 128;
    // dU leaves through the other box: a bf16 tile has one box of D per warp
    const uint32_t box2 = my_boxes + (i ^ 1) * STAGE_BUF_BYTES, row2 = box2 + lane * 128;
    if (Cf::LOADS) {
      // the other box, if it is being loaded, was asked for later
      in_flight &= ~(1u << i);
      if (in_flight) ptx::copy_wait<1>();
      else ptx::copy_wait<0>();
    } else if (lane == 0) {  // the box's last store, the one before the latest if there are two, is read
      if (nboxes == 2) ptx::bulk_wait_read<1>();
      else ptx::bulk_wait_read<0>();
    }
    __syncwarp();
    auto columns = [&](auto tag) {
#pragma unroll 1
      for (int c = 0; c < UC; c += 16) {
        float z[16], u[16];
        load(c, z, u);
        if (c + 16 == UC) loaded();
        epilogue16<MODE, decltype(tag)::value, F32>(z, u, row_addr, row2, sw, c / CHUNK<F32>, col + c,
                                                    c_cols, p.bias);
        if constexpr (DZ && F32) {
          const int64_t off = box_row * p.part_ld + col + c, rows = p.m_rows - box_row;
          store_parts(z, p.parts[0] + off, p.part_ld, p.part_stride, rows, c_cols - col - c);
          if (GATED)
            store_parts(u, p.parts[1] + off, p.part_ld, p.part_stride, rows, c_cols - col - c);
        }
      }
    };
    if constexpr (MODE == FFN_GRADS) columns(ActTag<LCE_ACT_NONE>{});
    else dispatch_act(p.act, columns);
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if constexpr (!(DZ && F32)) {
      if (lane == 0) {
        ptx::tma_store_2d(mC, box, col, box_row);
        if (MODE == FFN_GATED_DGU) ptx::tma_store_2d(&maps.c2, box2, col, box_row);
        ptx::bulk_commit();
      }
    }
  };

  auto role_tickets = [&](bool remote) {
    return Tickets{TileQueue<true, Ctl>{ctl, abort_flag, p.err, 0, 0u, remote, leader}, p.sched == nullptr,
                   unit, units, p.total_tiles};
  };

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    if (lane == 0) {
      bool ok = !p.withhold;
      Ring ring{0, 0u};
      Tickets tickets = role_tickets(rank != 0);
      TileQueue<true, Ctl>& tq = tickets.tq;
      const bool posts = p.sched && rank == 0;  // this thread hands the tickets out
      unsigned next = 0u;
      int upcoming = -1;
      if (posts) {
        next = atomicAdd(&p.sched[0], 1u);
        upcoming = tq.post(next, p.sched, p.total_tiles, units);
        if (upcoming >= 0) next = atomicAdd(&p.sched[0], 1u);
      }
      while (ok) {
        int tile;
        if (posts) {
          tile = upcoming;
          if (tile < 0) break;
          upcoming = tq.post(next, p.sched, p.total_tiles, units);
          if (upcoming >= 0) next = atomicAdd(&p.sched[0], 1u);
        } else {
          tile = tickets.take(1u);
        }
        if (tile < 0) break;
        const TilePos tp = SPLIT ? locate_split(p, tile, piece) : locate(p, tile);
        if (SPLIT && tp.tm < 0) continue;
        const Job& jb = p.job[tp.job];
        const bool whole = SPLIT && jb.whole;
        const int m0 = tp.tm * TILE + static_cast<int>(rank) * BM;
        const Range range =
            piece_of(steps_per_pair<F32>(jb.nkb) * jb.pairs, whole ? piece : 0, whole ? split : 1);
        if constexpr (GATED) {
          // CTA 0 loads its columns' rows of Wg, CTA 1 the same rows of Wu
          ok = produce_tile<false, false, F32>(jb.nkb, 1, range, maps.a[0], &maps.b[0][rank], m0,
                                               tp.tn * (p.bn / 2), base, ctl, ring, abort_flag, p.err,
                                               rank, leader, p.bn, stages);
        } else {
          const int n0 = tp.tn * p.bn + static_cast<int>(rank) * (p.bn / 2);
          if constexpr (MODE == FFN_GRADS) {
            if (jb.mn)
              ok = produce_tile<true, true, F32>(jb.nkb, jb.pairs, range, maps.a[tp.job],
                                                 maps.b[tp.job], m0, n0, base, ctl, ring, abort_flag,
                                                 p.err, rank, leader, p.bn, stages);
            else
              ok = produce_tile<false, true, F32>(jb.nkb, jb.pairs, range, maps.a[tp.job],
                                                  maps.b[tp.job], m0, n0, base, ctl, ring,
                                                  abort_flag, p.err, rank, leader, p.bn, stages);
          } else {
            ok = produce_tile<false, false, F32>(jb.nkb, 1, range, maps.a[0], maps.b[0], m0, n0, base,
                                                 ctl, ring, abort_flag, p.err, rank, leader, p.bn,
                                                 stages);
          }
        }
      }
      ptx::launch_dependents();
      if (!ok) {
        // Let copies already in flight land before the CTA can exit.
        const uint64_t t0 = ptx::globaltimer();
        while (ptx::globaltimer() - t0 < 2000000ull) {}
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0 && rank == 0) {
      bool ok = true;
      Ring ring{0, 0u};
      int acc = 0;
      uint32_t aph = 0;
      Tickets tickets = role_tickets(false);
      while (ok) {
        const int tile = tickets.take(1u);
        if (tile < 0) break;
        const TilePos tp = SPLIT ? locate_split(p, tile, piece) : locate(p, tile);
        if (SPLIT && tp.tm < 0) continue;
        const Job& jb = p.job[tp.job];
        const bool whole = SPLIT && jb.whole;
        const int per_pair = steps_per_pair<F32>(jb.nkb);
        const Range range = piece_of(per_pair * jb.pairs, whole ? piece : 0, whole ? split : 1);
        for (int st = range.lo; ok && (st < range.hi || st == range.lo); ++st) {
          // an empty piece still hands its accumulator over; no one reads it
          const int blocks = range.hi == range.lo ? 0
                             : F32 ? 6 * min(F32_STEP, jb.nkb - (st % per_pair) * F32_STEP)
                                   : range.hi - range.lo;
          if (!wait_bar(ptx::smem_addr(&ctl->tempty[acc]), aph ^ 1u, abort_flag, p.err)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t d_tmem = tmem_base + acc * TILE;
          if constexpr (MODE == FFN_GRADS) {
            if (jb.mn)
              ok = mma_tile<true, true>(blocks, d_tmem, base, ctl, ring, abort_flag, p.err, pair_mask,
                                        p.bn, stages);
            else
              ok = mma_tile<false, true>(blocks, d_tmem, base, ctl, ring, abort_flag, p.err, pair_mask,
                                         p.bn, stages);
          } else {
            ok = mma_tile<false, false>(blocks, d_tmem, base, ctl, ring, abort_flag, p.err, pair_mask,
                                        p.bn, stages);
          }
          if (!ok) break;
          ptx::tc_commit_pair(ptx::smem_addr(&ctl->tfull[acc]), pair_mask);
          acc ^= 1;
          if (acc == 0) aph ^= 1u;
          if (!F32) break;  // one accumulator for the whole range
        }
      }
      if (!ok) {
        // Make sure no MMA is still writing TMEM before it is released.
        ptx::tc_commit_pair(ptx::smem_addr(&ctl->drain), static_cast<uint16_t>(1u << leader));
        wait_bar_drain(ptx::smem_addr(&ctl->drain), 0, 100000000ull);
      }
    }
  } else {
    // ------------------------------------------------------------------ epilogue (warps 2..9)
    Tickets tickets = role_tickets(rank != 0);
    int acc = 0;
    uint32_t aph = 0;
    bool ok = true;
    while (ok) {
      const int tile = tickets.take(0xffffffffu);
      if (tile < 0) break;
      const TilePos tp = SPLIT ? locate_split(p, tile, piece) : locate(p, tile);
      if (SPLIT && tp.tm < 0) continue;
      const Job& jb = p.job[tp.job];
      const bool whole = SPLIT && jb.whole;
      const uint32_t lanes = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
      const Range range =
          piece_of(steps_per_pair<F32>(jb.nkb) * jb.pairs, whole ? piece : 0, whole ? split : 1);
      const int box_row = tp.tm * TILE + static_cast<int>(rank) * BM + q * 32;
      const int col0 = tp.tn * cols + half * per_half * UC;
      // the n-th box of this warp: its first column.  Boxes of a tile that a cluster finishes together:
      // box b belongs to pair b % split, there to the warps of column half (b / split) % 2.
      auto box_col = [&](int n) {
        return whole ? tp.tn * cols + (piece + split * (half + 2 * n)) * UC : col0 + n * UC;
      };
      // columns end with the result, the tile, or (direct) the half's boxes
      const int col_end = min(min(jb.c_cols, (tp.tn + 1) * cols),
                              whole ? jb.c_cols : col0 + per_half * UC);
      if (Cf::LOADS) {  // R or D of the first boxes, while the products run
        for (int n = 0; n < nboxes; ++n)
          if (box_col(n) < col_end) fetch(n, jb.c_cols, box_col(n), box_row);
      }
      // hand the accumulator back to the MMA issuer (in the pair's first CTA)
      auto release = [&]() {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) {  // nothing but the tensor memory is handed over
          const uint32_t empty = ptx::smem_addr(&ctl->tempty[acc]);
          if (rank == 0) ptx::mbar_arrive(empty);
          else ptx::mbar_arrive_cluster_relaxed(ptx::mapa_shared(empty, leader));
        }
        acc ^= 1;
        if (acc == 0) aph ^= 1u;
      };
      const int steps = F32 ? max(range.hi - range.lo, 1) : 1;
      if (F32 && steps > 1) {
        // sum the steps' accumulators; the total goes back into the last one's columns
        float sum[4][32];
#pragma unroll
        for (int i = 0; i < 128; ++i) sum[i >> 5][i & 31] = 0.f;
#pragma unroll 1
        for (int st = 0; st < steps; ++st) {
          if (!wait_bar(ptx::smem_addr(&ctl->tfull[acc]), aph, abort_flag, p.err)) { ok = false; break; }
          ptx::tc_fence_after();
#pragma unroll
          for (int h = 0; h < 8; ++h) {
            if (h >= 2 * groups) break;
            ptx::tmem_add16(lanes + acc * TILE + half_col<GATED>(half, h >> 1, p.bn) + (h & 1) * 16,
                            &sum[h >> 1][(h & 1) * 16]);
          }
          if (st + 1 < steps) release();
        }
        if (!ok) break;
#pragma unroll
        for (int h = 0; h < 4; ++h)
          if (h < groups) ptx::tmem_store32(lanes + acc * TILE + half_col<GATED>(half, h, p.bn), sum[h]);
      } else if (!wait_bar(ptx::smem_addr(&ctl->tfull[acc]), aph, abort_flag, p.err)) {
        break;
      }
      ptx::tc_fence_after();
      const uint32_t tbase = lanes + acc * TILE;
      if (whole) {
        // This pair's partial sums into shared memory, four columns of a row together: every MMA is
        // done, so the ring is free.  The boxes follow below, once all pairs are here.
#pragma unroll 1
        for (int h = 0; h < groups; ++h) {
          const int c = half_col<GATED>(half, h, p.bn);
          float v[32];
          ptx::tmem_load32(tbase + c, v);
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            ptx::st_shared_v4(base + (((c + i) >> 2) * BM + q * 32 + lane) * 16, __float_as_uint(v[i]),
                              __float_as_uint(v[i + 1]), __float_as_uint(v[i + 2]),
                              __float_as_uint(v[i + 3]));
        }
        split_tile = tile;
        release();
      } else {
        if (col0 >= col_end) release();  // no box for this warp
#pragma unroll 1
        for (int un = 0;; ++un) {
          const int col = col0 + un * UC;
          if (col >= col_end) break;  // same for every thread of the warp
          const int at = (half * per_half + un) * UC;  // accumulator column
          process(un & (nboxes - 1), &maps.c[tp.job], jb.c_cols, col, box_row,
                  [&](int c, float (&z)[16], float (&u)[16]) {
                    ptx::tmem_load16(tbase + at + c, z);
                    if (GATED) ptx::tmem_load16(tbase + p.bn / 2 + at + c, u);
                  },
                  [&] { if (col + UC >= col_end) release(); });
          if (Cf::LOADS && col + nboxes * UC < col_end)
            fetch(un & (nboxes - 1), jb.c_cols, col + nboxes * UC, box_row);
        }
      }
    }
  }

  if constexpr (SPLIT) {
    __syncwarp();
    ptx::cluster_sync();  // every pair's partial sums are written
    if (warp >= 2 && split_tile >= 0) {
      const TilePos tp = locate_split(p, split_tile, piece);
      const Job& jb = p.job[tp.job];
      const int steps = steps_per_pair<F32>(jb.nkb) * jb.pairs;
      const int box_row = tp.tm * TILE + static_cast<int>(rank) * BM + q * 32;
      const int col_end = min(jb.c_cols, (tp.tn + 1) * cols);
      // 16 columns from all pairs, in the order of the pieces
      auto gather = [&](int c, float (&v)[16]) {
        const uint32_t at = base + ((c >> 2) * BM + q * 32 + lane) * 16;
        float4 t[MAX_SPLIT][4];
#pragma unroll
        for (int s = 0; s < MAX_SPLIT; ++s) {
          const Range r = piece_of(steps, s, split);
          const bool some = s < split && r.lo < r.hi;
          const uint32_t peer = ptx::mapa_shared(at, some ? 2 * s + rank : crank);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            t[s][i] = some ? ptx::ld_shared_cluster_v4(peer + i * BM * 16) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float4 x = t[0][i];
#pragma unroll
          for (int s = 1; s < MAX_SPLIT; ++s) {
            x.x += t[s][i].x; x.y += t[s][i].y; x.z += t[s][i].z; x.w += t[s][i].w;
          }
          v[4 * i] = x.x; v[4 * i + 1] = x.y; v[4 * i + 2] = x.z; v[4 * i + 3] = x.w;
        }
      };
#pragma unroll 1
      for (int n = 0;; ++n) {
        const int b = piece + split * (half + 2 * n);
        const int col = tp.tn * cols + b * UC;
        if (col >= col_end) break;
        process(n & (nboxes - 1), &maps.c[tp.job], jb.c_cols, col, box_row,
                [&](int c, float (&z)[16], float (&u)[16]) {
                  gather(b * UC + c, z);
                  if (GATED) gather(p.bn / 2 + b * UC + c, u);
                },
                [] {});
        const int next = col + nboxes * 2 * split * UC;
        if (Cf::LOADS && next < col_end) fetch(n & (nboxes - 1), jb.c_cols, next, box_row);
      }
    }
  }
  if (warp >= 2) {
    if (Cf::LOADS) ptx::copy_wait<0>();
    if (lane == 0) ptx::bulk_wait<0>();  // this warp's output stores have landed
    __syncwarp();
  }

  // Every role of both CTAs is done before TMEM is released and the CTAs exit.
  ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

// ------------------------------------------------------------------------------ host side

// Tensor map over a row-major [outer x inner] array (row stride ld elements), 128-byte swizzle,
// zero fill outside.  parts > 1: so many of them, part_stride elements apart (a third dimension).
bool make_map(CUtensorMap* m, const void* ptr, uint64_t inner, uint64_t outer, uint64_t ld,
              uint32_t box_inner, uint32_t box_outer, bool fp32, int dims_n, uint64_t parts,
              uint64_t part_stride, const char* what) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) {
    set_error_detail("cuTensorMapEncodeTiled entry point unavailable");
    return false;
  }
  const uint64_t e = fp32 ? 4 : 2;
  const cuuint64_t dims[3] = {inner, outer, parts};
  const cuuint64_t strides[2] = {ld * e, part_stride * e};
  const cuuint32_t box[3] = {box_inner, box_outer, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r =
      enc(m, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dims_n,
          const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error_detail("tensor map of a feed-forward operand (%s) refused (CUresult %d; %llu x %llu"
                     " elements, row stride %llu, box %u x %u, address %p)",
                     what, static_cast<int>(r), static_cast<unsigned long long>(outer),
                     static_cast<unsigned long long>(inner), static_cast<unsigned long long>(ld),
                     box_outer, box_inner, ptr);
    return false;
  }
  return true;
}

// An operand [.. x K] (K-major, boxes of `rows` rows), or stored [K x ..] (MN-major): 3-D, the parts
// last.
bool operand(CUtensorMap* m, const FfnOperand& o, bool mn, int rows, const char* what) {
  const uint64_t ps = o.parts > 1 ? o.part_stride : static_cast<uint64_t>(o.ld) * o.stored_rows;
  return make_map(m, o.ptr, o.stored_cols, o.stored_rows, o.ld, BK, mn ? BK : rows, false, 3, o.parts,
                  ps, what);
}

// The device that is current, one that this library keeps state for.
cudaError_t current_device(int* dev) {
  const cudaError_t e = cudaGetDevice(dev);
  if (e != cudaSuccess) return e;
  return *dev >= 0 && *dev < kMaxDevices ? cudaSuccess : cudaErrorInvalidDevice;
}

// Largest number of clusters of 1 .. MAX_SPLIT CTA pairs that the device holds at once (every mode's
// kernel takes the same room), for the powers of two.
struct ClusterLimits {
  int of[MAX_SPLIT + 1] = {};
};
template <bool F32>
cudaError_t cluster_limits(int dev, ClusterLimits* limits) {
  static PerDevice<kMaxDevices> cached[MAX_SPLIT + 1];
  for (int pairs = 2; pairs <= MAX_SPLIT; pairs *= 2) {
    auto query = [&](int* n) {
      const auto kernel = ffn_tc_kernel<FFN_GRADS, F32, true>;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(2 * pairs, 1, 1);
      cfg.blockDim = dim3(THREADS, 1, 1);
      cfg.dynamicSmemBytes = SMEM_BYTES;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 2 * pairs;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
      if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(n, kernel, &cfg);
      if (e != cudaSuccess)
        set_error_detail("clusters of %d CTAs of a feed-forward kernel: %s", 2 * pairs, cudaGetErrorName(e));
      return e;
    };
    const cudaError_t e = cached[pairs].get(dev, query, &limits->of[pairs]);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// How a launch's tiles and sums are cut.  It is chosen from all products of the launch, asked for or
// not, so that a result is the same bits whichever others are computed with it.
struct Plan {
  int bn = TILE, split = 1;
  bool whole[MAX_JOBS] = {};
  double cost = 0.0;  // estimate, SM cycles
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The cheapest of the tile widths and cluster sizes by an estimate in SM cycles, from measured parts: a
// k-block costs 528 cycles in a 256 x 256 tile and about 390 in one of half the width (its operands
// then bound it), finishing a 256 x 256 tile 3,000, and joining the pieces of one the transfer of its
// partial sums at 14 bytes per cycle and SM (the rate distributed shared memory showed: 5 us for a
// tile cut in four) after about 1,500 of synchronisation.
template <bool F32>
Plan choose_plan(const FfnTc* jobs, int njobs, bool gated, int units, const ClusterLimits& limits) {
  Plan best;
  for (int bn = TILE; bn >= TILE / 2; bn /= 2) {
    const double step_cost = (bn == TILE ? 528.0 : 390.0) * (F32 ? 6 * F32_STEP : 1);
    const double finish = 3000.0 * bn / TILE * (F32 ? 2 : 1);
    int64_t tiles[MAX_JOBS], steps[MAX_JOBS], all = 0;
    double work = 0.0, longest = 0.0;
    for (int j = 0; j < njobs; ++j) {
      const FfnTc& g = jobs[j];
      tiles[j] = ceil_div(g.M, TILE) * ceil_div(g.Ncols, gated ? bn / 2 : bn);
      steps[j] = steps_per_pair<F32>(static_cast<int>(ceil_div(g.K, BK))) * (!gated && g.A2.ptr ? 2 : 1);
      all += tiles[j];
      work += static_cast<double>(tiles[j]) * steps[j] * step_cost;
      longest = std::max(longest, steps[j] * step_cost);
    }
    // pairs on their own: waves of one product's tiles; several products fill each other's gaps
    double cost = all <= units ? longest
                  : njobs == 1 ? ceil_div(all, units) * longest
                               : work / units + longest / 2;
    cost += finish;
    if (best.cost == 0.0 || cost < best.cost) {
      best = Plan{};
      best.bn = bn;
      best.cost = cost;
    }
    for (int k = 2; k <= MAX_SPLIT; k *= 2) {
      // products are cut from `least` steps per piece on; the others' tiles lie side by side
      for (const int least : {1, F32 ? 2 : 6}) {
        int64_t clusters = 0;
        double slowest = 0.0;
        bool whole[MAX_JOBS] = {}, any = false;
        for (int j = 0; j < njobs; ++j) {
          whole[j] = steps[j] >= static_cast<int64_t>(least) * k;
          any |= whole[j];
          clusters += whole[j] ? tiles[j] : ceil_div(tiles[j], k);
          const double join = 1500.0 + bn * BM * 4.0 * (k - 1) / k / 14.0;
          slowest = std::max(slowest, whole[j] ? ceil_div(steps[j], k) * step_cost + join + finish / k
                                               : steps[j] * step_cost + finish);
        }
        if (!any || clusters > limits.of[k] || slowest >= best.cost) continue;
        best.cost = slowest;
        best.bn = bn;
        best.split = k;
        for (int j = 0; j < njobs; ++j) best.whole[j] = whole[j];
      }
    }
  }
  return best;
}

template <int MODE, bool F32>
cudaError_t launch(const FMaps& maps, KParams& p, int num_sms, cudaStream_t stream) {
  static PerDevice<kMaxDevices> attr_set;
  int dev = 0, set = 0;
  cudaError_t e = current_device(&dev);
  if (e != cudaSuccess) return e;
  e = attr_set.get(dev, [](int* done) {
    *done = 1;
    cudaError_t r = cudaFuncSetAttribute(ffn_tc_kernel<MODE, F32, false>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (r == cudaSuccess)
      r = cudaFuncSetAttribute(ffn_tc_kernel<MODE, F32, true>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (r != cudaSuccess)
      set_error_detail("shared-memory attribute of a feed-forward kernel: %s", cudaGetErrorName(r));
    return r;
  }, &set);
  if (e != cudaSuccess) return e;
  int clusters = 0;
  for (int j = 0; j < p.njobs; ++j)
    clusters += static_cast<int>(p.job[j].whole ? p.job[j].num_tiles : ceil_div(p.job[j].num_tiles, p.split));
  const int units = num_sms / 2;
  cudaLaunchConfig_t cfg = {};
  if (p.split > 1) p.total_tiles = clusters;  // a ticket is a cluster's work
  cfg.gridDim = dim3(2 * (p.split > 1 ? clusters * p.split : std::min(p.total_tiles, units)), 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2 * p.split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1] = dependent_launch();
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = p.split > 1 ? cudaLaunchKernelEx(&cfg, ffn_tc_kernel<MODE, F32, true>, maps, p)
                  : cudaLaunchKernelEx(&cfg, ffn_tc_kernel<MODE, F32, false>, maps, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess)
    set_error_detail("launch of a feed-forward product (mode %d, %d tiles, split %d): %s", MODE,
                     p.total_tiles, p.split, cudaGetErrorName(e));
  return e;
}

template <bool F32>
cudaError_t run(const FfnTc* jobs, int njobs, const Plan& plan, unsigned* header, CallState* state,
                int num_sms, cudaStream_t stream) {
  FMaps maps;
  memset(&maps, 0, sizeof(maps));
  KParams p{};
  const int mode = jobs[0].mode;
  const bool gated = mode == FFN_GATED || mode == FFN_GATED_DGU;
  const bool dz = mode == FFN_LINEAR_DZ || mode == FFN_GATED_DGU;
  const uint32_t uc = F32 ? 32 : 64;
  p.split = plan.split;
  p.bn = plan.bn;
  int64_t longest = 0;
  for (int i = 0; i < njobs; ++i) longest = std::max(longest, ceil_div(jobs[i].K, BK) * (jobs[i].A2.ptr ? 2 : 1));
  p.boxes = !F32 && longest <= SHORT_K ? 2 : 1;
  int n = 0;
  for (int i = 0; i < njobs; ++i) {
    const FfnTc& g = jobs[i];
    Job jb{};
    if (!g.C) continue;  // a result that is not asked for counts in the plan only
    const int64_t tm = ceil_div(g.M, TILE), tn = ceil_div(g.Ncols, gated ? p.bn / 2 : p.bn);
    if (tm * tn > (int64_t(1) << 28)) {
      set_error_detail("feed-forward product of %lld x %lld tiles: beyond the scheduler's range",
                       static_cast<long long>(tm), static_cast<long long>(tn));
      return cudaErrorInvalidValue;
    }
    jb.tiles_m = static_cast<int>(tm);
    jb.tiles_n = static_cast<int>(tn);
    jb.num_tiles = jb.tiles_m * jb.tiles_n;
    jb.nkb = static_cast<int>(ceil_div(g.K, BK));
    jb.pairs = (!gated && g.A2.ptr) ? 2 : 1;
    jb.mn = g.a_mn;
    jb.c_cols = static_cast<int>(g.Ncols);
    jb.whole = plan.split > 1 && plan.whole[i];
    const int j = n++;
    p.job[j] = jb;
    p.total_tiles += jb.num_tiles;
    const int b_rows = p.bn / 2;
    if (!operand(&maps.a[j][0], g.A, g.a_mn, BM, "A") ||
        !operand(&maps.b[j][0], g.B, g.b_mn, b_rows, "B") ||
        (jb.pairs == 2 && !operand(&maps.a[j][1], g.A2, g.a_mn, BM, "A2")) ||
        ((gated || jb.pairs == 2) && !operand(&maps.b[j][1], g.B2, g.b_mn, b_rows, "B2")))
      return cudaErrorInvalidResourceHandle;
    if (!(dz && F32)) {
      if (!make_map(&maps.c[j], g.C, g.Ncols, g.M, g.ldc, uc, 32, F32, 2, 1, 0, "C"))
        return cudaErrorInvalidResourceHandle;
      if (mode == FFN_GATED_DGU &&
          !make_map(&maps.c2, g.C2, g.Ncols, g.M, g.ldc, uc, 32, F32, 2, 1, 0, "C2"))
        return cudaErrorInvalidResourceHandle;
    }
  }
  if (n == 0) return cudaSuccess;
  const FfnTc& g = jobs[0];
  p.njobs = n;
  p.act = g.act;
  p.bias = g.bias;
  p.m_rows = g.M;
  const void* d = dz ? g.D : (mode == FFN_LINEAR ? g.R : nullptr);
  p.d = static_cast<const char*>(d);
  p.d_stride = (dz ? g.ldd : g.ldr) * (F32 ? 4 : 2);
  if (dz && F32) {
    p.parts[0] = static_cast<__nv_bfloat16*>(g.C);
    p.parts[1] = static_cast<__nv_bfloat16*>(g.C2);
    p.part_ld = g.ldc;
    p.part_stride = g.part_stride;
  }
  p.err = header;
  // Tiles are dealt out round-robin, or taken as tickets from the counters in the header.  Dealing needs
  // nothing cleared beforehand and no hand-over between the roles (4096 x 512 x 8192: 32 us, 40 with
  // tickets; x 2048: 77, 85); tickets even out tiles of different lengths (backward products of 512 x
  // 4096 x 8192: 58 us, 67 dealt) and keep tiles that share operands together over long launches
  // (gated backward 16384 x 4096 x 16384: 7.06 ms, 7.25 dealt).
  if (p.total_tiles > (njobs == 1 ? DEALT_WAVES : DEALT_WAVES_MIXED) * (num_sms / 2)) {
    p.sched = header + WS_SCHED_WORD;
    const size_t from = state->flags ? WS_SCHED_WORD * sizeof(unsigned) : 0;
    if (!state->sched) {
      cudaError_t e = cudaMemsetAsync(reinterpret_cast<char*>(header) + from, 0, WS_HEADER_BYTES - from,
                                      stream);
      if (e != cudaSuccess) return e;
      state->flags = state->sched = true;  // the launch leaves the counters at zero
    }
  }
  p.clear_flags = !state->flags;
  p.withhold = g_inject_stall;  // one launch only
  g_inject_stall = 0;
  state->flags = true;
  switch (mode) {
    case FFN_LINEAR:
      return d ? launch<FFN_LINEAR_RES, F32>(maps, p, num_sms, stream)
               : launch<FFN_LINEAR, F32>(maps, p, num_sms, stream);
    case FFN_GATED: return launch<FFN_GATED, F32>(maps, p, num_sms, stream);
    case FFN_LINEAR_DZ: return launch<FFN_LINEAR_DZ, F32>(maps, p, num_sms, stream);
    case FFN_GATED_DGU: return launch<FFN_GATED_DGU, F32>(maps, p, num_sms, stream);
    default: return launch<FFN_GRADS, F32>(maps, p, num_sms, stream);
  }
}

// A launch of all products, or one of the weight gradients and one of the others: sums over very many
// tokens make few and long tiles, which only a launch of their own can cut for all SMs (backward of
// 16384 x 512 -> 1024: 8 tiles of 256 k-blocks beside 128 of 16).
template <bool F32>
cudaError_t run_planned(const FfnTc* jobs, int njobs, unsigned* header, CallState* state, int num_sms,
                        cudaStream_t stream) {
  constexpr double kLaunch = 5000.0;  // cycles that another launch costs
  const bool gated = jobs[0].mode == FFN_GATED || jobs[0].mode == FFN_GATED_DGU;
  for (int i = 0; i < njobs; ++i)
    if (ceil_div(jobs[i].K, BK) > (1 << 25)) return cudaErrorInvalidValue;  // widths end at 2^31
  int dev = 0;
  ClusterLimits limits;
  cudaError_t e = current_device(&dev);
  if (e == cudaSuccess) e = cluster_limits<F32>(dev, &limits);
  if (e != cudaSuccess) return e;
  const Plan all = choose_plan<F32>(jobs, njobs, gated, num_sms / 2, limits);
  if (njobs > 1) {
    FfnTc group[2][MAX_JOBS];
    int n[2] = {0, 0};
    for (int i = 0; i < njobs; ++i) {
      const int k = jobs[i].a_mn ? 0 : 1;
      group[k][n[k]++] = jobs[i];
    }
    if (n[0] && n[1]) {
      const Plan plan[2] = {choose_plan<F32>(group[0], n[0], gated, num_sms / 2, limits),
                            choose_plan<F32>(group[1], n[1], gated, num_sms / 2, limits)};
      if (plan[0].cost + plan[1].cost + kLaunch < all.cost) {
        int launches = 0;
        for (int k = 0; k < 2; ++k) {
          bool asked = false;
          for (int i = 0; i < n[k]; ++i) asked |= group[k][i].C != nullptr;
          if (!asked) continue;
          e = run<F32>(group[k], n[k], plan[k], header, state, num_sms, stream);
          if (e != cudaSuccess) return e;
          ++launches;
        }
        g_extra_kernels += launches - 1;
        return cudaSuccess;
      }
    }
  }
  return run<F32>(jobs, njobs, all, header, state, num_sms, stream);
}

}  // namespace

cudaError_t launch_ffn_tc(const FfnTc* jobs, int njobs, lce_dtype_t dtype, unsigned* header,
                          CallState* state, int num_sms, cudaStream_t stream) {
  if (njobs < 1 || njobs > MAX_JOBS) return cudaErrorInvalidValue;
  return dtype == LCE_BF16 ? run_planned<false>(jobs, njobs, header, state, num_sms, stream)
                           : run_planned<true>(jobs, njobs, header, state, num_sms, stream);
}

}  // namespace lce
