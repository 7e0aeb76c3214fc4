// Parts shared by the tensor-core kernels (lce_tc.cu, lce_ffn_tc.cu): bounded barrier waits, the
// dynamic tile scheduler, operand descriptors of the 128-byte-swizzled shared-memory tiles, and the
// driver's tensor-map encoder.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "lce_internal.h"
#include "ptx.cuh"

namespace lce {

constexpr int BM = 128;     // accumulator rows held by one CTA (TMEM lanes)
// bf16 MN-major operands: 64(MN) x 64(K) boxes of 8 KB
constexpr int MN_BOX_ELEMS = 64;
constexpr int MN_BOX_BYTES = 64 * 64 * 2;
constexpr int STAGE_BUF_BYTES = 32 * 128;  // a 32-row x 128-byte epilogue box
constexpr uint64_t WAIT_LIMIT_NS = 2000000000ull;  // a wait longer than 2 s is treated as a hang

// Tiles handed out by the dynamic scheduler wait in a small ring until every role has read them.
constexpr int TQ = 4;

// Suspend-time hint of every barrier wait (ns): a waiting thread sleeps in the try_wait until the
// phase completes, up to this long, instead of returning early and polling again.  Measured 1.0-
// 1.5% faster steps than the instruction's default, with or without the power cap.
#ifndef LCE_WAIT_HINT_NS
#define LCE_WAIT_HINT_NS 20000
#endif

// Bounded wait on an mbarrier phase.  Gives up after WAIT_LIMIT_NS (or at once when another role
// already gave up), raising the CTA's abort flag and the workspace timeout bit.
template <bool CLUSTER_ACQUIRE = false>
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                         unsigned* err) {
  auto try_once = [&]() {
    return CLUSTER_ACQUIRE ? ptx::mbar_try_wait_cluster(bar, parity, LCE_WAIT_HINT_NS)
                           : ptx::mbar_try_wait(bar, parity, LCE_WAIT_HINT_NS);
  };
  if (try_once()) return true;
  const uint64_t t0 = ptx::globaltimer();
  while (true) {
    if (*abort_flag) return false;
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (try_once()) return true;
    if (ptx::globaltimer() - t0 > WAIT_LIMIT_NS) {
      *abort_flag = 1;
      atomicOr(err, ERR_TIMEOUT);
      return false;
    }
  }
}

// Wait on a barrier regardless of the abort flag, for at most `limit_ns` (used while draining).
__device__ __forceinline__ void wait_bar_drain(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  const uint64_t t0 = ptx::globaltimer();
  while (!ptx::mbar_try_wait(bar, parity, LCE_WAIT_HINT_NS))
    if (ptx::globaltimer() - t0 > limit_ns) return;
}

// Grouped rasterisation: `group` row tiles sweep the column tiles together, so the tiles
// resident at one time share a few A row-blocks and B column-blocks through L2.
__device__ __forceinline__ void tile_coords(int tile, int tiles_m, int tiles_n, int group, int& tm,
                                            int& tn) {
  const int per_group = group * tiles_n;
  const int g = tile / per_group;
  const int first_m = g * group;
  const int gm = min(tiles_m - first_m, group);
  const int r = tile - g * per_group;
  tm = first_m + r % gm;
  tn = r / gm;
}

// Dynamic tile scheduler.  The producer thread of the (first) CTA takes tickets from a global
// counter -- tiles come out in job and raster order, so the tiles in flight at any moment stay
// together however unevenly the SMs progress, and operands keep being shared through L2 -- and
// posts each ticket into the ring `tq` of both CTAs of a pair.  Every other role reads the
// tickets from its own CTA's ring and hands the slot back.  -1 ends the sequence.  The producer
// takes the ticket of its next tile from the counter as soon as it has posted the current one, so
// the atomic's round trip overlaps the current tile's loads instead of opening a gap in the
// operand stream at every tile boundary.
template <bool PAIR, class Ctl>
struct TileQueue {
  Ctl* ctl;
  volatile int* abort_flag;
  unsigned* err;
  int slot;
  uint32_t ph;
  // a reader in the second CTA of a pair: it hands slots back to the first CTA's barrier with a
  // cluster-scope release; readers in the first CTA hand back locally with a CTA-scope release,
  // which does not make them wait the way the cluster-scope one does (measured: the MMA thread
  // spent 5-14% of its time in a cluster-scope hand-back)
  bool remote;
  uint32_t leader = 0;  // cluster rank of the pair's first CTA

  __device__ __forceinline__ void advance() {
    if (++slot == TQ) { slot = 0; ph ^= 1u; }
  }

  // Scheduler: posts `ticket` (taken from the counter sched[0] beforehand) to both CTAs, or -1
  // when it is past the last tile.  Returns what was posted (-1 also after a timeout); the last
  // unit to receive -1 clears the counters for the next launch.
  __device__ __forceinline__ int post(unsigned ticket, unsigned* sched, int num_tiles, int units) {
    const uint32_t empty = ptx::smem_addr(&ctl->tq_empty[slot]);
    if (!wait_bar<PAIR>(empty, ph ^ 1u, abort_flag, err)) return -1;
    const int t = (ticket < static_cast<unsigned>(num_tiles)) ? static_cast<int>(ticket) : -1;
    ctl->tq[slot] = t;
    const uint32_t full = ptx::smem_addr(&ctl->tq_full[slot]);
    if (PAIR) {
      ptx::st_shared_cluster(ptx::mapa_shared(ptx::smem_addr(&ctl->tq[slot]), leader + 1), t);
      ptx::mbar_arrive_cluster(ptx::mapa_shared(full, leader + 1));
    }
    ptx::mbar_arrive(full);
    advance();
    if (t < 0 && atomicAdd(&sched[1], 1u) == static_cast<unsigned>(units - 1)) {
      atomicExch(&sched[0], 0u);
      atomicExch(&sched[1], 0u);
    }
    return t;
  }

  // Reader: the next ticket of this CTA's ring.  `mask` names the lanes of the calling warp that
  // read it together; the slot is handed back (once per warp) after all of them have.
  __device__ __forceinline__ int take(unsigned mask) {
    const uint32_t full = ptx::smem_addr(&ctl->tq_full[slot]);
    int t = -1;
    if (wait_bar<PAIR>(full, ph, abort_flag, err)) t = ctl->tq[slot];
    __syncwarp(mask);
    if ((threadIdx.x & 31) == static_cast<unsigned>(__ffs(mask) - 1)) {
      const uint32_t empty = ptx::smem_addr(&ctl->tq_empty[slot]);
      if (remote) ptx::mbar_arrive_cluster(ptx::mapa_shared(empty, leader));
      else ptx::mbar_arrive(empty);
    }
    advance();
    return t;
  }
};

__device__ __forceinline__ uint64_t desc_kmajor(uint32_t tile_base, int k) {
  // K-major, 128B swizzle: rows of 128 bytes, 8-row swizzle atoms 1024 bytes apart; the k-th
  // MMA slice (16 bf16 or 8 tf32 elements) starts 32 bytes further into the row.
  return ptx::sw128_desc(tile_base + k * 32, 16, 1024);
}
__device__ __forceinline__ uint64_t desc_mnmajor(uint32_t tile_base, int k16) {
  // bf16 MN-major, 128B swizzle: each 64-wide MN box holds 64 rows (one per k) of 128 bytes;
  // boxes are MN_BOX_BYTES apart (leading byte offset), groups of 8 k-rows 1024 bytes apart
  // (stride byte offset); the k-th 16-row slice starts 16 * 128 bytes further.
  return ptx::sw128_desc(tile_base + k16 * 16 * 128, MN_BOX_BYTES, 1024);
}

// Position in a shared-memory ring (stage index and phase parity).
struct Ring {
  int stage;
  uint32_t ph;
};

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  if (!fn) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(f);
  }
  return fn;
}

}  // namespace lce
