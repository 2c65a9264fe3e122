// What the 8-bit product and the weight gradient share: the list of row tiles
// of experts' rows, a tile's way from TMEM to global memory, and the sum of a
// cluster's partial tiles.
//
// Both put the long, regular axis (weight rows, or weight columns) on the MMA's
// M side, 128 TMEM lanes, and the ragged one on its N side, whose width an
// instruction chooses: a tile of few rows then costs few columns, and a warp
// stores a TMEM column as one contiguous run of an output row, whatever the
// row's alignment.
#pragma once

#include <algorithm>

#include "qmoe_ops.cuh"
#include "qmoe_tma.cuh"

namespace qmoe {

constexpr int kTileM = 128;

__device__ __forceinline__ void tma_3d_elect(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n\t}" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// ----------------------------------------------------------------------------
// Pairs of CTAs (cta_group::2): one MMA of M = 256, each CTA with its half of M,
// half of the rows of N in its shared memory and an accumulator of all N columns
// in its TMEM.  The first CTA of a pair issues the MMAs; both CTAs' copies
// complete on its barriers.
//
// What such a kernel lives by, as measured with the waits of every role timed:
// - the TMA unit takes a row of 128 bytes in two to three cycles, and a copy of few
//   rows hardly less than one of many: a tile of 128 x 192 (320 rows in 384 cycles
//   of MMAs) is bound by that, a pair's 256 x 224 (240 rows an SM in 448) is not;
// - a wait that parks takes some 230 cycles where its phase is complete already, a
//   poll 60, so a producer thread does one copy a stage and the issuing warp asks
//   for its next stage before it issues the one it has;
// - arrivals and waits at cluster scope that release and acquire memory take some
//   700 cycles each, relaxed ones no more than those within a CTA.
// ----------------------------------------------------------------------------
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// This CTA of its pair.
__device__ __forceinline__ int pair_rank() {
  uint32_t rank;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  return (int)rank;
}
// Arrives, when the MMAs issued so far are done, on the barrier of both CTAs.
__device__ __forceinline__ void tc_commit_pair_elect(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// All threads of all CTAs of the cluster.
__device__ __forceinline__ void cluster_sync_all() {
  __syncwarp();   // the barrier is the whole warp's, and lanes leave a wait one by one
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Last of a pair, behind a barrier of the CTA.  Both CTAs wait for every commit that
// arrives in them (see drain_ring): a producer for the last phase of each stage's
// barrier and a scale warp for that of each group's, the epilogue for every
// accumulator, and here the second CTA for the issuer's last commit, as the issuer did.
// (After a wait that ran out the phases to come are not known: what the issuer did
// commit arrives within the limits of these waits, thousands of MMAs long.)
// Arrivals by threads come before their own arrival at the cluster's barrier, behind
// which neither CTA leaves before the other.
__device__ __forceinline__ void pair_end(uint64_t* drain_bar, int rank, int* status) {
  const WaitCfg drain{status, kDrainWaitLimit};
  if (rank == 1 && threadIdx.x < 32) mbar_wait_bounded(drain_bar, 0, drain);
  __syncthreads();
  cluster_sync_all();
}
// A barrier's address in the first CTA.
__device__ __forceinline__ uint32_t first_cta_bar(uint64_t* bar) {
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(at) : "r"(smem_u32(bar)));
  return at;
}
// Arrivals of threads of both CTAs.  What they stand for is tensor memory read or
// written (an accumulator that is free, scales that are there) and nothing in shared
// or global memory, so the arrival and the wait are relaxed: the fences
// tcgen05.fence::before_thread_sync and ::after_thread_sync order tensor memory
// accesses against the instructions that order execution, of which an arrival and the
// wait that observes it are one pair, relaxed or not; release and acquire would add
// the order of ordinary memory (some 700 cycles each).
__device__ __forceinline__ void cluster_bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool cluster_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
// A copy to this CTA's shared memory that completes on a barrier of either, by one
// thread.
__device__ __forceinline__ void tma_3d_pair(void* dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// A producer's wait, by one thread: a poll that does not park first (a parked one
// takes some 230 cycles where the phase is complete already).
__device__ __forceinline__ bool poll_or_wait(uint64_t* bar, uint32_t parity, const WaitCfg& w, volatile int* abort_flag) {
  return mbar_test_wait(bar, parity) || wait_or_abort(bar, parity, w, abort_flag);
}
// A slot of a ring of S and the parity of its phase.
template <int S>
struct RingAt {
  int s = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void step() {
    if (++s == S) {
      s = 0;
      ph ^= 1u;
    }
  }
};
// spin_or_abort for such a phase: one answer for the whole warp.
__device__ __forceinline__ bool warp_spin_cluster(uint64_t* bar, uint32_t parity, const WaitCfg& w, volatile int* abort_flag) {
  const long long limit = w.limit * 64;
  for (long long i = 0; i < limit; ++i) {
    if (__shfl_sync(0xffffffffu, cluster_test_wait(bar, parity), 0)) return true;
    if ((i & 255) == 255 && __shfl_sync(0xffffffffu, *abort_flag, 0)) return false;
  }
  atomicExch(w.status, DEV_TIMEOUT);
  *abort_flag = 1;
  return false;
}

// Shared-memory matrix descriptor of an operand that lies along M or N (the
// reduction down the rows): rows of 128 bytes in the 128-byte swizzle, eight rows
// to the next 1024 bytes, panels of 128 bytes `panel` bytes apart.
__device__ __forceinline__ uint64_t smem_desc_mn128(uint32_t addr, uint32_t panel) {
  uint64_t d = 0;
  d |= (uint64_t)((addr & 0x3FFFF) >> 4);
  d |= (uint64_t)(panel >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// First row of group e (0 .. E; group E is the rows without a route).  Clamped
// to the rows there are, so that no offsets make a role leave its operands.
__device__ __forceinline__ int group_first_row(const int* offsets, int E, int64_t R, int e) {
  if (e <= 0) return 0;
  if (!offsets || e > E) return (int)R;
  return min(max(offsets[e], 0), (int)R);
}

// First row tile (of `bn` rows) and first row of every group, by a whole warp:
// tp[e], tp[E + 1] their number, row0[e].
__device__ __forceinline__ void group_tiles(const int* offsets, int E, int64_t R, int bn, int* tp, int* row0) {
  const int lane = threadIdx.x & 31;
  int first = 0;
  for (int e0 = 0; e0 <= E; e0 += 32) {
    const int e = e0 + lane;
    int n = 0;
    if (e <= E) {
      const int lo = group_first_row(offsets, E, R, e), hi = group_first_row(offsets, E, R, e + 1);
      n = hi > lo ? (hi - lo + bn - 1) / bn : 0;
      row0[e] = lo;
    }
    int run = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += up;
    }
    if (e <= E) tp[e] = first + run - n;
    first += __shfl_sync(0xffffffffu, run, 31);
  }
  if (lane == 0) {
    tp[E + 1] = first;
    row0[E + 1] = (int)R;
  }
}
struct RowTile {
  int e, start, rows;   // e == E: rows without a route (zeros)
};
__device__ __forceinline__ RowTile row_tile(int E, const int* tp, const int* row0, int bn, int mt) {
  int lo = 0, hi = E;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tp[mid] <= mt) lo = mid;
    else hi = mid - 1;
  }
  RowTile t;
  t.e = lo;
  t.start = row0[lo] + (mt - tp[lo]) * bn;
  t.rows = min(bn, row0[lo + 1] - t.start);
  return t;
}

// Two warps take a quarter of a tile's lanes, every other 32 columns each.  With
// one, and an address and a test for every store, the epilogue was what bounded
// both kernels (16 instructions a column; a tile of the weight gradient over 512
// rows took 7000 cycles, its MMAs 4350).
constexpr int kEpiWarps = 8;

// Columns of a warp's quarter of a tile to rows 0 .. n of the output, a lane an
// element of each (`in`: the lane has one).  `out`: the lane's element of the
// first row; half: which of the two warps.
template <int OUT>
__device__ __forceinline__ void store_tile(uint32_t taddr, typename ElemT<OUT>::t* out, int64_t ld, int n, bool in, int half) {
  using T = typename ElemT<OUT>::t;
  out += (size_t)(half * 32) * ld;
  for (int c0 = half * 32; c0 < n; c0 += 64, out += (size_t)64 * ld) {
    uint32_t v[32];
    __syncwarp();   // lanes outside left the last round early; the load is the whole warp's
    TC_LD32(taddr + c0, v);
    tc_wait_ld();
    if (!in) continue;
    T* p = out;
    if (c0 + 32 <= n) {
#pragma unroll
      for (int c = 0; c < 32; ++c, p += ld) store_d<OUT>(p, 0, __uint_as_float(v[c]));
    } else {
#pragma unroll
      for (int c = 0; c < 32; ++c, p += ld)
        if (c0 + c < n) store_d<OUT>(p, 0, __uint_as_float(v[c]));
    }
  }
}
// The same added to what is there (32-bit results).  The tensor core cuts off what
// an addition to its accumulator leaves over, always towards zero, so that a long
// sum falls short by a share that grows with its length (an MMA of normal 16-bit
// values 2^-25.6 of it, of 8-bit ones 2^-27.8, of 8-bit values of one sign 2^-25):
// 32-bit results of long reductions are summed in pieces, and the pieces here, to
// nearest, by the thread that stored the first one.
__device__ __forceinline__ void add_tile(uint32_t taddr, float* out, int64_t ld, int n, bool in, int half) {
  out += (size_t)(half * 32) * ld;
  for (int c0 = half * 32; c0 < n; c0 += 64, out += (size_t)64 * ld) {
    uint32_t v[32];
    __syncwarp();   // lanes outside left the last round early; the load is the whole warp's
    TC_LD32(taddr + c0, v);
    tc_wait_ld();
    if (!in) continue;
    float* p = out;
#pragma unroll
    for (int b = 0; b < 32; b += 16) {   // sixteen loads under way
      float was[16];
      float* q = p;
#pragma unroll
      for (int c = 0; c < 16; ++c, q += ld) was[c] = c0 + b + c < n ? *q : 0.f;
#pragma unroll
      for (int c = 0; c < 16; ++c, p += ld)
        if (c0 + b + c < n) *p = was[c] + __uint_as_float(v[b + c]);
    }
  }
}
// sum = piece, or sum + piece, to nearest, of a warp's share of a tile's columns, in
// TMEM, where there is room for both.
__device__ __forceinline__ void add_pieces(uint32_t sum, uint32_t piece, int n, int half, bool first) {
  for (int c0 = half * 32; c0 < n; c0 += 64) {
    uint32_t v[32];
    TC_LD32(piece + c0, v);
    if (!first) {
      uint32_t w[32];
      TC_LD32(sum + c0, w);
      tc_wait_ld();
#pragma unroll
      for (int c = 0; c < 32; ++c) v[c] = __float_as_uint(__uint_as_float(w[c]) + __uint_as_float(v[c]));
    } else {
      tc_wait_ld();
    }
    TC_ST32(sum + c0, v);
  }
  tc_wait_st();
}
template <int OUT>
__device__ __forceinline__ void store_zeros(typename ElemT<OUT>::t* out, int64_t ld, int n, bool in, int half) {
  if (in)
    for (int c = half; c < n; c += 2) store_d<OUT>(out + (size_t)c * ld, 0, 0.f);
}

// A tile whose reduction is split over the CTAs of a cluster: each CTA's
// partial sums to its own shared memory, [column][128] ...
__device__ __forceinline__ void put_partial(uint32_t taddr, float* part, int q, int n, int half) {
  const int lane = threadIdx.x & 31;
  for (int c0 = half * 32; c0 < n; c0 += 64) {
    uint32_t v[32];
    TC_LD32(taddr + c0, v);
    tc_wait_ld();
#pragma unroll
    for (int c = 0; c < 32; ++c)
      if (c0 + c < n) part[(c0 + c) * kTileM + q * 32 + lane] = __uint_as_float(v[c]);
  }
}
// ... and, after a barrier of the cluster, every CTA adds up its share of the
// columns in the order of the ranks and stores them.
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr, int rank) {
  uint32_t at;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}
// Four columns' loads from every rank are under way at once: each takes some 250
// cycles, and added up one by one they were most of a small call's time (weight
// gradient of 777 rows, 1001 x 513, in four parts: 27.7 us, so 18.4).
template <int OUT>
__device__ __forceinline__ void store_sum(const float* part, int q, typename ElemT<OUT>::t* out, int64_t ld, int n, bool in,
                                          int rank, int ranks, int half) {
  constexpr int most = 8, cols = 4;   // ranks, columns
  const int lane = threadIdx.x & 31;
  for (int c0 = rank + half * ranks * cols; c0 < n; c0 += 2 * ranks * cols) {
    float v[cols][most];
#pragma unroll
    for (int u = 0; u < cols; ++u) {
      const uint32_t at = smem_u32(part + min(c0 + u * ranks, n - 1) * kTileM + q * 32 + lane);
#pragma unroll
      for (int r = 0; r < most; ++r) v[u][r] = r < ranks ? ld_cluster_f32(at, r) : 0.f;
    }
#pragma unroll
    for (int u = 0; u < cols; ++u) {
      float sum = 0.f;
#pragma unroll
      for (int r = 0; r < most; ++r) sum += v[u][r];
      if (in && c0 + u * ranks < n) store_d<OUT>(out + (size_t)(c0 + u * ranks) * ld, 0, sum);
    }
  }
}

// Rows [rows, inner] of `size`-byte elements, `matrices` of them, rows `pitch`
// bytes apart: boxes of 128 bytes by box_rows rows, 128-byte swizzle, zeros outside.
inline bool encode_tiles(CUtensorMap* m, CUtensorMapDataType type, int size, const void* base, int64_t inner, int64_t rows,
                         int64_t matrices, int64_t pitch, int box_rows) {
  const EncodeFn f = encoder();
  if (!f) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)matrices};
  const cuuint64_t strides[2] = {(cuuint64_t)pitch, (cuuint64_t)(pitch * rows)};
  const cuuint32_t box[3] = {(cuuint32_t)(128 / size), (cuuint32_t)box_rows, 1};
  const cuuint32_t ones[3] = {1, 1, 1};
  return f(m, type, 3, const_cast<void*>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The launch of a tile kernel: clusters of `cluster` CTAs, dependent on the kernel before.
template <typename... Params, typename... Args>
cudaError_t launch_tiles(void (*kern)(Params...), int64_t ctas, int cluster, int threads, int smem, cudaStream_t s, const Args&... args) {
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)cluster, 1, 1};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace qmoe
