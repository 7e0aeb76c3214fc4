// Feed-forward products of a few tokens (decoding), bf16: Y = act(X W^T + b) + R and
// H = act(X Wg^T) * (X Wu^T) for at most FFN_FEW_TOKENS rows of X.
//
// The weights are read once and little else, so the kernel is a weight stream: bound by HBM.  The
// tensor cores take the weights as their 128-row operand and the tokens as the columns
// (D[128 features x nt tokens] = W_tile X^T, nt = N rounded up to 16, the tokens past N zero-filled
// by TMA), so one kernel serves one token and a hundred at the same bytes.
//   warp 0      TMA producer: k-blocks of 64 of the weight rows (of Wg and Wu both) and of X through
//               a ring of up to 218 KB, or two CTAs per SM of 110 KB: 200 KB in flight per SM
//   warp 1      MMA issuer (tcgen05, cta_group::1, M = 128, N = nt), accumulators in TMEM
//   warps 2..5  epilogue: thread = feature, so a token's results leave as 64 contiguous bytes a warp
// With few row tiles the K loop is split over a cluster of S = 2, 4 or 8 CTAs; each puts its fp32
// partial sums into its shared memory and adds up every S-th token from all of them, in rank order,
// through distributed shared memory: no second launch, no atomics, a fixed order.
//
// Measured inside a captured graph: gated 48 x 6144 -> 16384 65 us (6.2 TB/s of weights), linear 4 x 16384
// -> 4096 23 us (5.8), gated 1 x 2048 -> 8192 13 us (5.1): about 3 us of each are the launch, the first loads
// and the join; a call on its own takes 0.7 to 1.0 us more.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "lce_act.cuh"
#include "lce_ffn.h"
#include "lce_internal.h"
#include "per_device.h"
#include "ptx.cuh"
#include "tc_common.cuh"

namespace lce {
namespace {

constexpr int BK = 64;
constexpr int THREADS = 192;
constexpr int MAX_STAGES = 12;
constexpr int CTL_BYTES = 256;
constexpr int MAX_SPLIT = 8;
constexpr int W_BYTES = BM * 128;  // one k-block of 128 weight rows
// Shared memory of a CTA (ring or partial sums, alignment, control block) with two or one per SM.
constexpr int SMEM_TWO = 112 * 1024;
constexpr int SMEM_ONE = 220 * 1024;

struct Ctl {
  uint64_t full[MAX_STAGES];
  uint64_t empty[MAX_STAGES];
  uint64_t done;
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(Ctl) <= CTL_BYTES, "control block too large");

struct Maps {
  CUtensorMap w, w2, x;
};

struct Params {
  int N, nt, width, nkb, split;
  int stages, stage_bytes, ring_bytes;
  uint32_t tmem_cols, idesc;
  int act;
  const __nv_bfloat16* bias;
  const __nv_bfloat16* R; int64_t ldr;
  __nv_bfloat16* Y; int64_t ldy;
  unsigned* err;
  int withhold;  // test hook (lce_test_inject_stall): no operand is loaded
};

// One result: feature f of token t.
template <int ACT, bool GATED>
__device__ __forceinline__ void finish(const Params& p, int t, int f, float z, float u, float b) {
  float v;
  if (GATED) {
    v = act<ACT, true>(z) * u;
  } else {
    v = act<ACT, true>(z + b);
    if (p.R) v += __bfloat162float(p.R[t * p.ldr + f]);
  }
  p.Y[t * p.ldy + f] = __float2bfloat16_rn(v);
}

template <bool GATED>
__global__ void __launch_bounds__(THREADS) ffn_few_kernel(const __grid_constant__ Maps maps,
                                                          const Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = ptx::smem_addr(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw_addr);
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + p.ring_bytes);
  const int x_off = (GATED ? 2 : 1) * W_BYTES;  // X's k-block in a stage
  volatile int* abort_flag = &ctl->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(blockIdx.x) % p.split, tile = static_cast<int>(blockIdx.x) / p.split;
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.nkb) * rank / p.split);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.nkb) * (rank + 1) / p.split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      ptx::mbar_init(ptx::smem_addr(&ctl->full[s]), 1);
      ptx::mbar_init(ptx::smem_addr(&ctl->empty[s]), 1);
    }
    ptx::mbar_init(ptx::smem_addr(&ctl->done), 1);
    ctl->abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_addr(&ctl->tmem_base), p.tmem_cols);
    ptx::tmem_relinquish();
    ptx::tc_fence_before();
  }
  if (warp == 0 && lane == 0) {
    ptx::prefetch_tmap(&maps.w);
    ptx::prefetch_tmap(&maps.x);
    if (GATED) ptx::prefetch_tmap(&maps.w2);
  }
  ptx::wait_for_previous();  // no memory of the caller is touched before this
  // The workspace's error flags: the first CTA is among the first to run, and a wait gives up only
  // WAIT_LIMIT_NS after that.
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.err = 0u;
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = ctl->tmem_base;

  if (warp == 0) {
    if (lane == 0) {
      Ring r{0, 0u};
      bool ok = !p.withhold;
      for (int kb = kb0; ok && kb < kb1; ++kb) {
        const uint32_t full = ptx::smem_addr(&ctl->full[r.stage]);
        if (!wait_bar(ptx::smem_addr(&ctl->empty[r.stage]), r.ph ^ 1u, abort_flag, p.err)) {
          ok = false;
          break;
        }
        ptx::mbar_arrive_expect_tx(full, p.stage_bytes);
        const uint32_t s0 = base + r.stage * p.stage_bytes;
        ptx::tma_load_2d(s0, &maps.w, kb * BK, tile * BM, full);
        if (GATED) ptx::tma_load_2d(s0 + W_BYTES, &maps.w2, kb * BK, tile * BM, full);
        ptx::tma_load_2d(s0 + x_off, &maps.x, kb * BK, 0, full);
        if (++r.stage == p.stages) { r.stage = 0; r.ph ^= 1u; }
      }
      // only now: CTAs of the next launch that came earlier would take places next to slower ones of this
      ptx::launch_dependents();
      if (!ok) {  // let copies already in flight land before the CTA can exit
        const uint64_t t0 = ptx::globaltimer();
        while (ptx::globaltimer() - t0 < 2000000ull) {}
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      Ring r{0, 0u};
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!wait_bar(ptx::smem_addr(&ctl->full[r.stage]), r.ph, abort_flag, p.err)) break;
        ptx::tc_fence_after();
        const uint32_t s0 = base + r.stage * p.stage_bytes;
        const uint32_t sx = s0 + x_off;
#pragma unroll
        for (int k = 0; k < BK / 16; ++k) {
          const uint32_t acc = (kb != kb0 || k != 0) ? 1u : 0u;
          ptx::tc_mma_f16(tmem_base, desc_kmajor(s0, k), desc_kmajor(sx, k), p.idesc, acc);
          if (GATED)
            ptx::tc_mma_f16(tmem_base + p.nt, desc_kmajor(s0 + W_BYTES, k), desc_kmajor(sx, k),
                            p.idesc, acc);
        }
        ptx::tc_commit(ptx::smem_addr(&ctl->empty[r.stage]));
        if (++r.stage == p.stages) { r.stage = 0; r.ph ^= 1u; }
      }
      // the accumulators are complete (after a timeout: no MMA is still writing them)
      ptx::tc_commit(ptx::smem_addr(&ctl->done));
    }
    __syncwarp();
  }

  const int q = warp & 3;
  const int feature = q * 32 + lane;
  const int f = tile * BM + feature;
  const bool epilogue = warp >= 2;
  const uint32_t tbase = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
  float b = 0.f;
  if (epilogue) {
    if (!GATED && p.bias && f < p.width) b = __bfloat162float(p.bias[f]);
    // bounded like every wait; after an abort the results are worthless, the flag says so
    wait_bar_drain(ptx::smem_addr(&ctl->done), 0, WAIT_LIMIT_NS + WAIT_LIMIT_NS / 2);
    ptx::tc_fence_after();
    if (p.split == 1) {
      dispatch_act(p.act, [&](auto tag) {
#pragma unroll 1
        for (int c = 0; c < p.N; c += 16) {
          float z[16], u[16];
          ptx::tmem_load16(tbase + c, z);
          if (GATED) ptx::tmem_load16(tbase + p.nt + c, u);
          if (f < p.width) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (c + j < p.N)
                finish<decltype(tag)::value, GATED>(p, c + j, f, z[j], GATED ? u[j] : 0.f, b);
          }
        }
      });
    } else {
      // every load of the ring has been read by an MMA: its memory holds the partial sums now
      float* part = reinterpret_cast<float*>(smem);
#pragma unroll 1
      for (int c = 0; c < p.N; c += 16) {
        float z[16];
#pragma unroll
        for (int g = 0; g < (GATED ? 2 : 1); ++g) {
          ptx::tmem_load16(tbase + g * p.nt + c, z);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (c + j < p.N) part[(g * p.N + c + j) * BM + feature] = z[j];
        }
      }
    }
  }
  if (p.split > 1) {
    __syncwarp();
    ptx::cluster_sync();
    if (epilogue && f < p.width) {
      uint32_t peer[MAX_SPLIT];
#pragma unroll
      for (int s = 0; s < MAX_SPLIT; ++s)
        peer[s] = ptx::mapa_shared(base + feature * 4, s < p.split ? s : 0);
      dispatch_act(p.act, [&](auto tag) {
#pragma unroll 1
        for (int t = rank; t < p.N; t += p.split) {
          float v[GATED ? 2 : 1][MAX_SPLIT];
#pragma unroll
          for (int g = 0; g < (GATED ? 2 : 1); ++g)
#pragma unroll
            for (int s = 0; s < MAX_SPLIT; ++s)
              v[g][s] = s < p.split ? ptx::ld_shared_cluster(peer[s] + (g * p.N + t) * BM * 4) : 0.f;
          float z = 0.f, u = 0.f;
#pragma unroll
          for (int s = 0; s < MAX_SPLIT; ++s) {
            z += v[0][s];
            if (GATED) u += v[GATED ? 1 : 0][s];
          }
          finish<decltype(tag)::value, GATED>(p, t, f, z, u, b);
        }
      });
    }
    __syncwarp();
    ptx::cluster_sync();  // no CTA leaves while another reads its partial sums
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, p.tmem_cols);
  }
}

// ------------------------------------------------------------------------------ host side

bool make_map(CUtensorMap* m, const void* ptr, int64_t inner, int64_t outer, int64_t ld, int box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) {
    set_error_detail("cuTensorMapEncodeTiled entry point unavailable");
    return false;
  }
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[2] = {BK, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides,
                         box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error_detail("tensor map of a few-token operand refused (CUresult %d; %lld x %lld elements,"
                     " row stride %lld, address %p)",
                     static_cast<int>(r), static_cast<long long>(outer),
                     static_cast<long long>(inner), static_cast<long long>(ld), ptr);
    return false;
  }
  return true;
}

template <bool GATED>
cudaError_t launch(const FfnGemm& g, unsigned* err, int num_sms, cudaStream_t stream) {
  static PerDevice<kMaxDevices> attr_set;
  int dev = 0, set = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  cudaError_t e = attr_set.get(dev, [](int* done) {
    *done = 1;
    const cudaError_t r = cudaFuncSetAttribute(ffn_few_kernel<GATED>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_ONE);
    if (r != cudaSuccess)
      set_error_detail("shared-memory attribute of the few-token kernel: %s", cudaGetErrorName(r));
    return r;
  }, &set);
  if (e != cudaSuccess) return e;
  constexpr int W = GATED ? 2 : 1;
  Params p{};
  p.N = static_cast<int>(g.M);
  p.nt = (p.N + 15) / 16 * 16;
  p.width = static_cast<int>(g.Ncols);
  p.nkb = static_cast<int>((g.K + BK - 1) / BK);
  p.act = g.act;
  p.bias = static_cast<const __nv_bfloat16*>(g.bias);
  p.R = static_cast<const __nv_bfloat16*>(g.R); p.ldr = g.ldr;
  p.Y = static_cast<__nv_bfloat16*>(g.C); p.ldy = g.ldc;
  p.err = err;
  p.withhold = g_inject_stall;  // one launch only
  g_inject_stall = 0;
  p.idesc = ptx::idesc_bf16_f32(BM, p.nt, false, false);
  p.tmem_cols = 32;
  while (p.tmem_cols < static_cast<uint32_t>(W * p.nt)) p.tmem_cols *= 2;
  p.stage_bytes = W * W_BYTES + p.nt * 128;
  // Tiles for more than half the SMs but not more than one each: one CTA per SM with a deep ring and its
  // whole K loop (48 x 6144 x 16384 gated: 64 us, 70 with 256 CTAs on half the ring and half of K each;
  // 128 x 4096 x 11008: 40 and 58).  Otherwise two CTAs per SM, where two k-blocks fit in half its shared
  // memory and the accumulators in half its tensor memory, and K split until those places are filled,
  // with at least four k-blocks for each CTA and the partial sums of a tile within the budget.  (The
  // CTAs an SM holds never need more than its 512 columns together: a CTA of a cluster that waited for
  // them could be waited for in turn.)
  const int64_t tiles = (g.Ncols + BM - 1) / BM;
  const bool one_each = 2 * tiles > num_sms && tiles <= num_sms;
  const bool two = !one_each && 2 * p.stage_bytes + 1024 + CTL_BYTES <= SMEM_TWO &&
                   p.tmem_cols <= 256;
  const int budget = (two ? SMEM_TWO : SMEM_ONE) - 1024 - CTL_BYTES;
  const int64_t places = (two ? 2 : 1) * num_sms;
  const int part_bytes = W * p.N * BM * 4;
  p.split = 1;
  while (p.split < MAX_SPLIT && part_bytes <= budget && tiles * p.split * 2 <= places &&
         p.nkb >= 8 * p.split)
    p.split *= 2;
  p.stages = std::min(MAX_STAGES, budget / p.stage_bytes);
  p.ring_bytes = p.stages * p.stage_bytes;
  if (p.split > 1) p.ring_bytes = std::max(p.ring_bytes, part_bytes);
  Maps maps;
  memset(&maps, 0, sizeof(maps));
  if (!make_map(&maps.w, g.B, g.K, g.Ncols, g.ldb, BM) ||
      !make_map(&maps.x, g.A, g.K, g.M, g.lda, p.nt) ||
      (GATED && !make_map(&maps.w2, g.B2, g.K, g.Ncols, g.ldb, BM)))
    return cudaErrorInvalidResourceHandle;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * p.split), 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = p.ring_bytes + 1024 + CTL_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1] = dependent_launch();
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, ffn_few_kernel<GATED>, maps, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess)
    set_error_detail("launch of the few-token kernel (%lld tiles, split %d): %s",
                     static_cast<long long>(tiles), p.split, cudaGetErrorName(e));
  return e;
}

}  // namespace

cudaError_t launch_ffn_few(const FfnGemm& g, unsigned* err, int num_sms, cudaStream_t stream) {
  return g.mode == FFN_GATED ? launch<true>(g, err, num_sms, stream)
                             : launch<false>(g, err, num_sms, stream);
}

}  // namespace lce
