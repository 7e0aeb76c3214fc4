// Feed-forward products on the tensor cores of sm_103a (tcgen05 + TMEM + TMA).
//
// One persistent, warp-specialised kernel on CTA pairs; a pair computes a 256 x 256 tile of
// accumulators with cta_group::2 MMAs, CTA r holding its rows 128 r .. 128 r + 127:
//   warp 0      TMA producer and tile scheduler (as in lce_tc.cu)
//   warp 1      MMA issuer; two 128 x 256 fp32 accumulators in TMEM, one filled while the other
//               is drained
//   warps 2..9  epilogue: warp w reads the 32 TMEM lanes of its quadrant, one half of the columns
//
// Modes (FfnMode):
//   LINEAR     C = act(Z + bias) + R            Z = A B^T, operands K-major
//   LINEAR_DZ  C = D act'(Z + bias)
//   GATED      C = act(G) U                     the pair's first CTA loads 128 rows of Wg, the second
//   GATED_DGU  C = D U act'(G), C2 = D act(G)   the same 128 rows of Wu: the 256 accumulator columns
//                                               are G | U of 128 output columns, and one thread
//                                               holds both values of an element
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
// The outgoing gradient D and the residual R enter, and C leaves, through one 4 KB box per epilogue
// warp (32 rows x 128 bytes, 128-byte swizzle): TMA load, each thread rewrites its own row, TMA
// store.  Six 32 KB stages and eight boxes fill the shared memory.
//
// Bound: tensor pipe for many tokens.  Ragged edges: TMA zero-fills loads and clips stores.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "bf16_parts.cuh"
#include "lce_act.cuh"
#include "lce_ffn.h"
#include "lce_internal.h"
#include "ptx.cuh"
#include "tc_common.cuh"

namespace lce {
namespace {

constexpr int TILE = 256;               // rows and accumulator columns of a pair's tile
constexpr int HALF = 128;               // B rows per CTA; output columns of a gated tile
constexpr int BK = 64;                  // K elements per stage (one 128-byte swizzle span)
constexpr int STAGES = 6;
constexpr int A_BYTES = BM * 128;
constexpr int STAGE_BYTES = 2 * A_BYTES;
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 64 + 32 * EPI_WARPS;
constexpr uint32_t TMEM_COLS = 2 * TILE;
constexpr int CTL_BYTES = 512;
constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + EPI_WARPS * STAGE_BUF_BYTES + 1024 + CTL_BYTES;
constexpr int RASTER = 8;               // row tiles per rasterisation group (as in lce_tc.cu)
constexpr int MAX_JOBS = 3;
constexpr int F32_STEP = 4;             // k-blocks per accumulator of an fp32 tile
static_assert(SMEM_BYTES <= 232448, "227 KB of shared memory per CTA");

struct Ctl {
  uint64_t full[STAGES];
  uint64_t empty[STAGES];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t drain;
  uint64_t tq_full[TQ];
  uint64_t tq_empty[TQ];
  uint64_t box[EPI_WARPS];
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
};

struct KParams {
  Job job[MAX_JOBS];
  int njobs, total_tiles;
  int act;
  int has_d;               // a box of R or D is loaded
  const void* bias;
  int64_t m_rows;          // rows of Z
  // fp32 pre-activation gradients are written as parts, from registers
  __nv_bfloat16* parts[2];
  int64_t part_ld, part_stride;
  unsigned* err;
  unsigned* sched;
};

struct FMaps {
  CUtensorMap a[MAX_JOBS][2];
  CUtensorMap b[MAX_JOBS][2];
  CUtensorMap c[MAX_JOBS];
  CUtensorMap c2;
  CUtensorMap d;
};

// The six part products, smallest first: operand parts of A and B.
__device__ __forceinline__ int part_a(int s) { return (0x201100 >> (4 * (5 - s))) & 15; }
__device__ __forceinline__ int part_b(int s) { return (0x021010 >> (4 * (5 - s))) & 15; }

template <int MODE>
constexpr bool kGated = MODE == FFN_GATED || MODE == FFN_GATED_DGU;

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

// A tile's K loop as steps, one accumulator each: bf16 a single step over all operand pairs, fp32
// F32_STEP k-blocks of one pair at a time.
template <bool F32>
__device__ __forceinline__ int steps_of(int nkb, int pairs) {
  return F32 ? pairs * ((nkb + F32_STEP - 1) / F32_STEP) : 1;
}

// Producer side of one tile.  A_MN, B_MN: the operand is MN-major.
template <bool A_MN, bool B_MN, bool F32>
__device__ __forceinline__ bool produce_tile(int nkb, int pairs, const CUtensorMap* mA,
                                             const CUtensorMap* mB, int m0, int n0, uint32_t base,
                                             Ctl* ctl, Ring& r, volatile int* abort_flag,
                                             unsigned* err, uint32_t rank) {
  auto block = [&](const CUtensorMap* a, const CUtensorMap* b, int k0, int za, int zb) {
    const uint32_t full_local = ptx::smem_addr(&ctl->full[r.stage]);
    if (!wait_bar(ptx::smem_addr(&ctl->empty[r.stage]), r.ph ^ 1u, abort_flag, err)) return false;
    const uint32_t full = ptx::mapa_shared(full_local, 0);
    if (rank == 0) ptx::mbar_arrive_expect_tx(full_local, 2 * STAGE_BYTES);
    const uint32_t sa = base + r.stage * STAGE_BYTES, sb = sa + A_BYTES;
    if (A_MN) {
#pragma unroll
      for (int c = 0; c < BM / MN_BOX_ELEMS; ++c)
        ptx::tma_load_3d_pair(sa + c * MN_BOX_BYTES, a, m0 + c * MN_BOX_ELEMS, k0, za, full);
    } else {
      ptx::tma_load_3d_pair(sa, a, k0, m0, za, full);
    }
    if (B_MN) {
#pragma unroll
      for (int c = 0; c < HALF / MN_BOX_ELEMS; ++c)
        ptx::tma_load_3d_pair(sb + c * MN_BOX_BYTES, b, n0 + c * MN_BOX_ELEMS, k0, zb, full);
    } else {
      ptx::tma_load_3d_pair(sb, b, k0, n0, zb, full);
    }
    if (++r.stage == STAGES) { r.stage = 0; r.ph ^= 1u; }
    return true;
  };
  for (int pr = 0; pr < pairs; ++pr) {
    const CUtensorMap* a = &mA[pr];
    const CUtensorMap* b = &mB[pr];
    if (!F32) {
      for (int kb = 0; kb < nkb; ++kb)
        if (!block(a, b, kb * BK, 0, 0)) return false;
    } else {
      for (int kb0 = 0; kb0 < nkb; kb0 += F32_STEP)
        for (int s = 0; s < 6; ++s)
          for (int kb = kb0; kb < min(nkb, kb0 + F32_STEP); ++kb)
            if (!block(a, b, kb * BK, part_a(s), part_b(s))) return false;
    }
  }
  return true;
}

template <bool A_MN, bool B_MN>
__device__ __forceinline__ bool mma_tile(int blocks, uint32_t d_tmem, uint32_t base, Ctl* ctl, Ring& r,
                                         volatile int* abort_flag, unsigned* err) {
  constexpr uint32_t IDESC = ptx::idesc_bf16_f32(TILE, TILE, A_MN, B_MN);
  for (int kb = 0; kb < blocks; ++kb) {
    if (!wait_bar(ptx::smem_addr(&ctl->full[r.stage]), r.ph, abort_flag, err)) return false;
    ptx::tc_fence_after();
    const uint32_t sa = base + r.stage * STAGE_BYTES, sb = sa + A_BYTES;
#pragma unroll
    for (int k = 0; k < BK / 16; ++k)
      ptx::tc_mma_f16_pair(d_tmem, A_MN ? desc_mnmajor(sa, k) : desc_kmajor(sa, k),
                           B_MN ? desc_mnmajor(sb, k) : desc_kmajor(sb, k), IDESC, (kb | k) != 0);
    ptx::tc_commit_pair(ptx::smem_addr(&ctl->empty[r.stage]), 0x3);
    if (++r.stage == STAGES) { r.stage = 0; r.ph ^= 1u; }
  }
  return true;
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float lo16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi16(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// The four 32-column groups of accumulator columns that a warp of column half `half` drains.
template <bool GATED>
__device__ __forceinline__ int half_col(int half, int h) {
  return GATED ? (h >> 1) * HALF + half * (HALF / 2) + (h & 1) * 32 : half * HALF + h * 32;
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

// 32 columns of one thread's row: z (and u) in registers, D or R read from and the result written to
// the thread's row of the box (chunks first, first + 1, ...).  For GATED_DGU z keeps dG in the box
// and the dU values in z; for fp32 pre-activation gradients both stay in registers (z, u).
template <int MODE, int ACT, bool F32>
__device__ __forceinline__ void epilogue32(float (&z)[32], float (&u)[32], uint32_t row, uint32_t sw,
                                           int first, int col, int c_cols, const void* bias,
                                           bool has_d) {
  constexpr int CH = CHUNK<F32>;
#pragma unroll
  for (int q = 0; q < 32 / CH; ++q) {
    const uint32_t addr = row + ((static_cast<uint32_t>(first + q) ^ sw) << 4);
    float d[CH], o[CH], b[CH];
    if ((MODE == FFN_LINEAR || MODE == FFN_LINEAR_DZ)) {
#pragma unroll
      for (int i = 0; i < CH; ++i) b[i] = 0.f;
      if (bias != nullptr && col + q * CH < c_cols) {
        const char* pb = static_cast<const char*>(bias) +
                         static_cast<size_t>(col + q * CH) * (F32 ? 4 : 2);
        unpack<F32>(__ldg(reinterpret_cast<const uint4*>(pb)), b);
      }
    }
    const bool read = MODE == FFN_LINEAR_DZ || MODE == FFN_GATED_DGU || (MODE == FFN_LINEAR && has_d);
    if (read) unpack<F32>(ptx::ld_shared_v4(addr), d);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const float v = z[q * CH + i];
      if constexpr (MODE == FFN_GRADS) {
        o[i] = v;
      } else if constexpr (MODE == FFN_LINEAR) {
        o[i] = act<ACT, !F32>(v + b[i]);
        if (has_d) o[i] += d[i];
      } else if constexpr (MODE == FFN_GATED) {
        o[i] = act<ACT, !F32>(v) * u[q * CH + i];
      } else {
        float a, g;
        act_grad<ACT, !F32>(MODE == FFN_LINEAR_DZ ? v + b[i] : v, a, g);
        if constexpr (MODE == FFN_GATED_DGU) {
          o[i] = d[i] * u[q * CH + i] * g;
          if (F32) { z[q * CH + i] = o[i]; u[q * CH + i] = d[i] * a; }
          else z[q * CH + i] = d[i] * a;
        } else {
          o[i] = d[i] * g;
          if (F32) z[q * CH + i] = o[i];
        }
      }
    }
    if (!(F32 && (MODE == FFN_LINEAR_DZ || MODE == FFN_GATED_DGU))) {
      const uint4 w = pack<F32>(o);
      ptx::st_shared_v4(addr, w.x, w.y, w.z, w.w);
    }
  }
}

// fp32 values of one row as three bf16 parts, 64 bytes per part.
__device__ __forceinline__ void store_parts(const float (&v)[32], __nv_bfloat16* out, int64_t stride,
                                            int cols) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t w[3][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float p[2][3];
#pragma unroll
      for (int e = 0; e < 2; ++e) split_bf16(v[q * 8 + 2 * i + e], p[e]);
#pragma unroll
      for (int s = 0; s < 3; ++s) w[s][i] = pack2(p[0][s], p[1][s]);
    }
    // the row's padding to a multiple of 8 columns may be written: nothing reads it
    if (q * 8 < cols) {
#pragma unroll
      for (int s = 0; s < 3; ++s)
        *reinterpret_cast<uint4*>(out + s * stride + q * 8) =
            make_uint4(w[s][0], w[s][1], w[s][2], w[s][3]);
    }
  }
}

template <int MODE, bool F32>
__global__ void __launch_bounds__(THREADS, 1)
    ffn_tc_kernel(const __grid_constant__ FMaps maps, const KParams p) {
  constexpr bool GATED = kGated<MODE>;
  constexpr bool DZ = MODE == FFN_LINEAR_DZ || MODE == FFN_GATED_DGU;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = ptx::smem_addr(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;  // 128B-swizzled tiles need 1024B alignment
  uint8_t* smem = smem_raw + (base - raw_addr);
  const uint32_t boxes = base + STAGES * STAGE_BYTES;
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + STAGES * STAGE_BYTES + EPI_WARPS * STAGE_BUF_BYTES);
  volatile int* abort_flag = &ctl->abort_flag;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();  // 0 = the pair's MMA issuer
  const int units = static_cast<int>(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
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
    for (int i = 0; i < EPI_WARPS; ++i) ptx::mbar_init(ptx::smem_addr(&ctl->box[i]), 1);
    ctl->abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(ptx::smem_addr(&ctl->tmem_base), TMEM_COLS);
    ptx::tmem_relinquish_pair();
    ptx::tc_fence_before();
  }
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem_base = ctl->tmem_base;

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    if (lane == 0) {
      bool ok = true;
      Ring ring{0, 0u};
      TileQueue<true, Ctl> tq{ctl, abort_flag, p.err, 0, 0u, rank != 0};
      unsigned next = 0u;
      int upcoming = -1;
      if (rank == 0) {
        next = atomicAdd(&p.sched[0], 1u);
        upcoming = tq.post(next, p.sched, p.total_tiles, units);
        if (upcoming >= 0) next = atomicAdd(&p.sched[0], 1u);
      }
      while (ok) {
        int tile;
        if (rank == 0) {
          tile = upcoming;
          if (tile < 0) break;
          upcoming = tq.post(next, p.sched, p.total_tiles, units);
          if (upcoming >= 0) next = atomicAdd(&p.sched[0], 1u);
        } else {
          tile = tq.take(1u);
        }
        if (tile < 0) break;
        const TilePos tp = locate(p, tile);
        const Job& jb = p.job[tp.job];
        const int m0 = tp.tm * TILE + static_cast<int>(rank) * BM;
        if constexpr (GATED) {
          // CTA 0 loads its columns' rows of Wg, CTA 1 the same rows of Wu
          ok = produce_tile<false, false, F32>(jb.nkb, 1, maps.a[0], &maps.b[0][rank], m0,
                                               tp.tn * HALF, base, ctl, ring, abort_flag, p.err,
                                               rank);
        } else {
          const int n0 = tp.tn * TILE + static_cast<int>(rank) * HALF;
          if constexpr (MODE == FFN_GRADS) {
            if (jb.mn)
              ok = produce_tile<true, true, F32>(jb.nkb, jb.pairs, maps.a[tp.job], maps.b[tp.job], m0,
                                                 n0, base, ctl, ring, abort_flag, p.err, rank);
            else
              ok = produce_tile<false, true, F32>(jb.nkb, jb.pairs, maps.a[tp.job], maps.b[tp.job],
                                                  m0, n0, base, ctl, ring, abort_flag, p.err, rank);
          } else {
            ok = produce_tile<false, false, F32>(jb.nkb, 1, maps.a[0], maps.b[0], m0, n0, base, ctl,
                                                 ring, abort_flag, p.err, rank);
          }
        }
      }
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
      TileQueue<true, Ctl> tq{ctl, abort_flag, p.err, 0, 0u, false};
      while (ok) {
        const int tile = tq.take(1u);
        if (tile < 0) break;
        const TilePos tp = locate(p, tile);
        const Job& jb = p.job[tp.job];
        const int steps = steps_of<F32>(jb.nkb, jb.pairs), per_pair = steps / jb.pairs;
        for (int st = 0; ok && st < steps; ++st) {
          const int blocks =
              F32 ? 6 * min(F32_STEP, jb.nkb - (st % per_pair) * F32_STEP) : jb.nkb * jb.pairs;
          if (!wait_bar(ptx::smem_addr(&ctl->tempty[acc]), aph ^ 1u, abort_flag, p.err)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t d_tmem = tmem_base + acc * TILE;
          if constexpr (MODE == FFN_GRADS) {
            if (jb.mn) ok = mma_tile<true, true>(blocks, d_tmem, base, ctl, ring, abort_flag, p.err);
            else ok = mma_tile<false, true>(blocks, d_tmem, base, ctl, ring, abort_flag, p.err);
          } else {
            ok = mma_tile<false, false>(blocks, d_tmem, base, ctl, ring, abort_flag, p.err);
          }
          if (!ok) break;
          ptx::tc_commit_pair(ptx::smem_addr(&ctl->tfull[acc]), 0x3);
          acc ^= 1;
          if (acc == 0) aph ^= 1u;
        }
      }
      if (!ok) {
        // Make sure no MMA is still writing TMEM before it is released.
        ptx::tc_commit_pair(ptx::smem_addr(&ctl->drain), 0x1);
        wait_bar_drain(ptx::smem_addr(&ctl->drain), 0, 100000000ull);
      }
    }
  } else {
    // ------------------------------------------------------------------ epilogue (warps 2..9)
    const int e = warp - 2;
    const int q = warp & 3;       // TMEM lane quadrant this warp may access
    const int half = e >> 2;      // which half of the columns
    constexpr int UC = F32 ? 32 : 64;          // columns of one box
    constexpr int COLS = GATED ? HALF : TILE;  // output columns of a tile
    constexpr int UNITS = COLS / 2 / UC;       // boxes per warp and tile
    const uint32_t box = boxes + e * STAGE_BUF_BYTES;
    const uint32_t box_bar = ptx::smem_addr(&ctl->box[e]);
    const uint32_t row_addr = box + lane * 128, sw = lane & 7;
    const bool has_d = DZ || (MODE == FFN_LINEAR && p.has_d);
    uint32_t box_ph = 0;
    int acc = 0;
    uint32_t aph = 0;
    bool ok = true, in_flight = false;
    TileQueue<true, Ctl> tq{ctl, abort_flag, p.err, 0, 0u, rank != 0};
    while (ok) {
      const int tile = tq.take(0xffffffffu);
      if (tile < 0) break;
      const TilePos tp = locate(p, tile);
      const Job& jb = p.job[tp.job];
      const CUtensorMap* mC = &maps.c[tp.job];
      const uint32_t lanes = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
      const int box_row = tp.tm * TILE + static_cast<int>(rank) * BM + q * 32;
      const int col0 = tp.tn * COLS + half * (COLS / 2);
      // R or D of a unit into the box, once the store before it has been read
      auto fetch = [&](int col) {
        if (lane == 0) {
          ptx::bulk_wait_read<0>();
          ptx::mbar_arrive_expect_tx(box_bar, STAGE_BUF_BYTES);
          ptx::tma_load_2d(box, &maps.d, col, box_row, box_bar);
        }
        in_flight = true;
      };
      if (has_d && col0 < jb.c_cols) fetch(col0);
      // hand the accumulator back to the MMA issuer (in the pair's first CTA)
      auto release = [&]() {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0)
          ptx::mbar_arrive_cluster(ptx::mapa_shared(ptx::smem_addr(&ctl->tempty[acc]), 0));
        acc ^= 1;
        if (acc == 0) aph ^= 1u;
      };
      if (F32) {
        // sum the steps' accumulators; the total goes back into the last one's columns
        const int steps = steps_of<F32>(jb.nkb, jb.pairs);
        if (steps > 1) {
          float sum[4][32];
#pragma unroll
          for (int i = 0; i < 128; ++i) sum[i >> 5][i & 31] = 0.f;
#pragma unroll 1
          for (int st = 0; st < steps; ++st) {
            if (!wait_bar(ptx::smem_addr(&ctl->tfull[acc]), aph, abort_flag, p.err)) { ok = false; break; }
            ptx::tc_fence_after();
#pragma unroll
            for (int h = 0; h < 8; ++h)
              ptx::tmem_add16(lanes + acc * TILE + half_col<GATED>(half, h >> 1) + (h & 1) * 16,
                              &sum[h >> 1][(h & 1) * 16]);
            if (st + 1 < steps) release();
          }
          if (!ok) break;
#pragma unroll
          for (int h = 0; h < 4; ++h)
            ptx::tmem_store32(lanes + acc * TILE + half_col<GATED>(half, h), sum[h]);
        }
      }
      if (!(F32 && steps_of<F32>(jb.nkb, jb.pairs) > 1) &&
          !wait_bar(ptx::smem_addr(&ctl->tfull[acc]), aph, abort_flag, p.err))
        break;
      ptx::tc_fence_after();
      const uint32_t tbase = lanes + acc * TILE;
#pragma unroll 1
      for (int un = 0; un < UNITS; ++un) {
        const int col = col0 + un * UC;
        if (col >= jb.c_cols) break;  // same for every thread of the warp
        if (has_d) {
          if (un > 0) fetch(col);
          if (!wait_bar(box_bar, box_ph, abort_flag, p.err)) { ok = false; break; }
          in_flight = false;
          box_ph ^= 1u;
        } else {
          if (lane == 0) ptx::bulk_wait_read<0>();
          __syncwarp();
        }
        uint32_t keep[MODE == FFN_GATED_DGU && !F32 ? 32 : 1];
#pragma unroll
        for (int h = 0; h < UC / 32; ++h) {
          const int at = half * (COLS / 2) + un * UC + h * 32;  // accumulator column
          float z[32], u[32];
          ptx::tmem_load32(tbase + at, z);
          if (GATED) ptx::tmem_load32(tbase + HALF + at, u);
          if constexpr (MODE == FFN_GRADS)
            epilogue32<MODE, LCE_ACT_NONE, F32>(z, u, row_addr, sw, h * 4, col + h * 32, jb.c_cols,
                                                nullptr, false);
          else
            dispatch_act(p.act, [&](auto tag) {
              epilogue32<MODE, decltype(tag)::value, F32>(z, u, row_addr, sw, h * 4, col + h * 32,
                                                          jb.c_cols, p.bias, has_d);
            });
          if constexpr (MODE == FFN_GATED_DGU && !F32) {
#pragma unroll
            for (int i = 0; i < 16; ++i) keep[h * 16 + i] = pack2(z[2 * i], z[2 * i + 1]);
          }
          if constexpr (DZ && F32) {
            const int64_t row = box_row + lane;
            if (row < p.m_rows) {
              const int64_t off = row * p.part_ld + col;
              store_parts(z, p.parts[0] + off, p.part_stride, jb.c_cols - col);
              if (GATED) store_parts(u, p.parts[1] + off, p.part_stride, jb.c_cols - col);
            }
          }
        }
        if constexpr (!(DZ && F32)) {
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            ptx::tma_store_2d(mC, box, col, box_row);
            ptx::bulk_commit();
          }
          if constexpr (MODE == FFN_GATED_DGU) {
            if (lane == 0) ptx::bulk_wait_read<0>();
            __syncwarp();
#pragma unroll
            for (int c = 0; c < 8; ++c)
              ptx::st_shared_v4(row_addr + ((static_cast<uint32_t>(c) ^ sw) << 4), keep[4 * c],
                                keep[4 * c + 1], keep[4 * c + 2], keep[4 * c + 3]);
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              ptx::tma_store_2d(&maps.c2, box, col, box_row);
              ptx::bulk_commit();
            }
          }
        } else {
          // every lane has read its row before the next box may land on it
          ptx::fence_proxy_async_smem();
          __syncwarp();
        }
      }
      if (!ok) break;
      release();
    }
    if (in_flight) wait_bar_drain(box_bar, box_ph, 100000000ull);
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

// An operand [rows x K] (K-major), or stored [K x rows] (MN-major): 3-D, the parts last.
bool operand(CUtensorMap* m, const FfnOperand& o, bool mn, const char* what) {
  const uint64_t ps = o.parts > 1 ? o.part_stride : static_cast<uint64_t>(o.ld) * o.stored_rows;
  return make_map(m, o.ptr, o.stored_cols, o.stored_rows, o.ld, BK, mn ? BK : BM, false, 3, o.parts,
                  ps, what);
}

template <int MODE, bool F32>
cudaError_t launch(const FMaps& maps, const KParams& p, int num_sms, cudaStream_t stream) {
  static bool attr_set = false;
  if (!attr_set) {
    cudaError_t e = cudaFuncSetAttribute(ffn_tc_kernel<MODE, F32>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (e != cudaSuccess) {
      set_error_detail("shared-memory attribute of a feed-forward kernel: %s", cudaGetErrorName(e));
      return e;
    }
    attr_set = true;
  }
  const int units = num_sms / 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (p.total_tiles < units ? p.total_tiles : units), 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, ffn_tc_kernel<MODE, F32>, maps, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess)
    set_error_detail("launch of a feed-forward product (mode %d, %d tiles): %s", MODE, p.total_tiles,
                     cudaGetErrorName(e));
  return e;
}

template <bool F32>
cudaError_t run(const FfnTc* jobs, int njobs, unsigned* header, int num_sms, cudaStream_t stream) {
  FMaps maps;
  memset(&maps, 0, sizeof(maps));
  KParams p{};
  const int mode = jobs[0].mode;
  const bool gated = mode == FFN_GATED || mode == FFN_GATED_DGU;
  const bool dz = mode == FFN_LINEAR_DZ || mode == FFN_GATED_DGU;
  const uint32_t uc = F32 ? 32 : 64;
  for (int j = 0; j < njobs; ++j) {
    const FfnTc& g = jobs[j];
    Job& jb = p.job[j];
    const int64_t cols = gated ? HALF : TILE;
    const int64_t tm = (g.M + TILE - 1) / TILE, tn = (g.Ncols + cols - 1) / cols;
    const int64_t nkb = (g.K + BK - 1) / BK;
    if (tm * tn > (int64_t(1) << 28) || p.total_tiles + tm * tn > (int64_t(1) << 29) || nkb > (1 << 25)) {
      set_error_detail("feed-forward product of %lld x %lld tiles: beyond the scheduler's range",
                       static_cast<long long>(tm), static_cast<long long>(tn));
      return cudaErrorInvalidValue;
    }
    jb.tiles_m = static_cast<int>(tm);
    jb.tiles_n = static_cast<int>(tn);
    jb.num_tiles = jb.tiles_m * jb.tiles_n;
    jb.nkb = static_cast<int>(nkb);
    jb.pairs = (!gated && g.A2.ptr) ? 2 : 1;
    jb.mn = g.a_mn;
    jb.c_cols = static_cast<int>(g.Ncols);
    p.total_tiles += jb.num_tiles;
    if (!operand(&maps.a[j][0], g.A, g.a_mn, "A") || !operand(&maps.b[j][0], g.B, g.b_mn, "B"))
      return cudaErrorInvalidResourceHandle;
    if (gated && !operand(&maps.b[j][1], g.B2, g.b_mn, "B2")) return cudaErrorInvalidResourceHandle;
    if (jb.pairs == 2 && (!operand(&maps.a[j][1], g.A2, g.a_mn, "A2") ||
                          !operand(&maps.b[j][1], g.B2, g.b_mn, "B2")))
      return cudaErrorInvalidResourceHandle;
    if (!(dz && F32)) {
      if (!make_map(&maps.c[j], g.C, g.Ncols, g.M, g.ldc, uc, 32, F32, 2, 1, 0, "C"))
        return cudaErrorInvalidResourceHandle;
      if (mode == FFN_GATED_DGU &&
          !make_map(&maps.c2, g.C2, g.Ncols, g.M, g.ldc, uc, 32, F32, 2, 1, 0, "C2"))
        return cudaErrorInvalidResourceHandle;
    }
  }
  const FfnTc& g = jobs[0];
  p.njobs = njobs;
  p.act = g.act;
  p.bias = g.bias;
  p.m_rows = g.M;
  const void* d = dz ? g.D : (mode == FFN_LINEAR ? g.R : nullptr);
  p.has_d = d != nullptr;
  if (d && !make_map(&maps.d, d, g.Ncols, g.M, dz ? g.ldd : g.ldr, uc, 32, F32, 2, 1, 0, "D"))
    return cudaErrorInvalidResourceHandle;
  if (dz && F32) {
    p.parts[0] = static_cast<__nv_bfloat16*>(g.C);
    p.parts[1] = static_cast<__nv_bfloat16*>(g.C2);
    p.part_ld = g.ldc;
    p.part_stride = g.part_stride;
  }
  p.err = header;
  p.sched = header + WS_SCHED_WORD;
  switch (mode) {
    case FFN_LINEAR: return launch<FFN_LINEAR, F32>(maps, p, num_sms, stream);
    case FFN_GATED: return launch<FFN_GATED, F32>(maps, p, num_sms, stream);
    case FFN_LINEAR_DZ: return launch<FFN_LINEAR_DZ, F32>(maps, p, num_sms, stream);
    case FFN_GATED_DGU: return launch<FFN_GATED_DGU, F32>(maps, p, num_sms, stream);
    default: return launch<FFN_GRADS, F32>(maps, p, num_sms, stream);
  }
}

}  // namespace

cudaError_t launch_ffn_tc(const FfnTc* jobs, int njobs, lce_dtype_t dtype, unsigned* header,
                          int num_sms, cudaStream_t stream) {
  if (njobs < 1 || njobs > MAX_JOBS) return cudaErrorInvalidValue;
  return dtype == LCE_BF16 ? run<false>(jobs, njobs, header, num_sms, stream)
                           : run<true>(jobs, njobs, header, num_sms, stream);
}

}  // namespace lce
