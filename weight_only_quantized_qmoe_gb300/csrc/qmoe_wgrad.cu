// Gradient of the experts' weights:
//
//   dw[e, n, k] = sum over rows i in [offsets[e], offsets[e + 1]) of dy[i, n] x[i, k]
//
// 16-bit operands, fp32 accumulation, one rounding to the output type.
//
// GB300 form: tcgen05.mma kind::f16 with both operands read along M and N: the
// reduction goes down the rows, so tiles of dy and x are used as they lie in
// memory, nothing is transposed.  The MMA's M side is 128 columns of x, its N
// side up to BN columns of dy, so that a TMEM column is a run of a row of dw; a
// ring stage holds 64 rows of both, in panels of 64 columns (128-byte rows,
// swizzled) copied by TMA.  An expert's rows start and end anywhere: the last
// stage runs as many K = 16 MMAs as there are rows, and the rows past the last in
// the last of them are overwritten with zeros in both operands (they belong to the
// next expert, and may hold anything).
//   warp 0    TMA producer (one elected lane)
//   warp 1    MMA issuer, zeros past the last row
//   warp 3    first rows of the experts
//   warps 4-11 epilogue: TMEM columns to rows of dw
// Two accumulators alternate; long sums are taken in pieces, the first of which stays
// in one and gets the others' added through the other.  CTAs are persistent over the
// (expert, tile) list.
// Where there are few tiles, the CTAs of a cluster share a tile's rows and add up
// their parts in a fixed order.  Operands that TMA cannot read (rows that do not
// start on 16 bytes) are copied to rows that do first.
//
// That is the form for few tiles (rows of 7 experts, 429 each, 1001 x 513: 9.5 us, and
// 4.6 for the aligned copies; the launch, one round of the ring and the stores bound
// it); more take pairs of CTAs, further down.
//
// Waits are bounded as in the 8-bit products' kernels.
#include "qmoe_tile.cuh"

namespace qmoe {

constexpr int kWgRows = 64;                     // rows a stage
constexpr int kWgPanel = 64;                    // columns of a panel (128 bytes)
constexpr int kWgPanelBytes = kWgRows * 128;
constexpr int kWgThreads = 128 + 32 * kEpiWarps;
constexpr int kWgBN = 256;
// Rows summed in the tensor core at a time, whole stages (see add_tile; of normal
// values, relative error of 1024 rows in one piece 1.2e-6, of 32768 3.8e-5): for
// 16-bit results as many as leave out a sixth of their own rounding (2^-11 for f16).
template <int OUT>
__device__ __forceinline__ int piece_end(int from, int hi) {
  constexpr int piece = OUT == QMOE_F32 ? 5 * 128 : 1 << 16;
  return hi - from > piece ? from + piece : hi;
}
// The accumulator of a piece where the pieces of a tile are added up in TMEM: the
// first one, which the others are added to, keeps a tile's `home`, the others go
// through the other one.  A tile of one piece leaves the other free for the next.
struct WgAccs {
  int home = 0;
  uint32_t used = 0;   // a bit each: parity of the uses so far
  __device__ __forceinline__ int of(bool first) const { return first ? home : home ^ 1; }
  __device__ __forceinline__ uint32_t parity(int ab) const { return used >> ab & 1u; }
  __device__ __forceinline__ void step(int ab) { used ^= 1u << ab; }
};

struct WgRing {
  static constexpr int stages = 4;
  static constexpr int x_panels = kTileM / kWgPanel, dy_panels = kWgBN / kWgPanel;
  static constexpr int x_bytes = x_panels * kWgPanelBytes;
  static constexpr int dy_bytes = dy_panels * kWgPanelBytes;
  static constexpr int x_off = 0;
  static constexpr int dy_off = x_off + stages * x_bytes;
  static constexpr int bar_off = dy_off + stages * dy_bytes;
  static constexpr int row_off = bar_off + 512;                 // first row of each expert
  static constexpr int total = row_off + (kSortMaxExperts + 1) * 4;
  static constexpr int tmem_cols = 2 * kWgBN;
  static_assert(total > kAloneBytes && total + 1024 <= 227 * 1024, "shared memory");
  static_assert(kWgBN * kTileM * 4 <= bar_off, "a partial tile fits the ring");
};

// Zeros from row `rows` of a stage to the end of its 16, in `panels` panels, by a
// whole warp.
__device__ __forceinline__ void zero_rows(uint8_t* base, int panels, int rows) {
  const int n = (((rows + 15) & ~15) - rows) * 8;   // 16-byte pieces a panel
  for (int p = 0; p < panels; ++p)
    for (int i = threadIdx.x & 31; i < n; i += 32)
      reinterpret_cast<uint4*>(base + p * kWgPanelBytes + rows * 128)[i] = make_uint4(0, 0, 0, 0);
}

// Up to four K = 16 MMAs of 64 rows, and the commit that frees their stage if they
// are its last, by one elected lane of a CTA or of the first CTA of a pair; 16 rows
// on is 2048 bytes in either operand.
template <int CTAS>
__device__ __forceinline__ void wg_stage_elect(uint32_t d, uint64_t x, uint64_t dy, uint32_t idesc, uint32_t acc, int nk, uint64_t* empty) {
  if constexpr (CTAS == 1) {
    asm volatile(
        "{\n\t.reg .pred e, p0, p1, q1, q2, q3;\n\t.reg .b64 y1, y2, y3, z1, z2, z3;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p0, %4, 0;\n\tsetp.eq.b32 p1, %4, %4;\n\t"
        "setp.gt.and.s32 q1, %5, 1, e;\n\tsetp.gt.and.s32 q2, %5, 2, e;\n\tsetp.gt.and.s32 q3, %5, 3, e;\n\t"
        "add.u64 y1, %1, 128;\n\tadd.u64 y2, %1, 256;\n\tadd.u64 y3, %1, 384;\n\t"
        "add.u64 z1, %2, 128;\n\tadd.u64 z2, %2, 256;\n\tadd.u64 z3, %2, 384;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p0;\n\t"
        "@q1 tcgen05.mma.cta_group::1.kind::f16 [%0], y1, z1, %3, p1;\n\t"
        "@q2 tcgen05.mma.cta_group::1.kind::f16 [%0], y2, z2, %3, p1;\n\t"
        "@q3 tcgen05.mma.cta_group::1.kind::f16 [%0], y3, z3, %3, p1;\n\t}" ::"r"(d),
        "l"(x), "l"(dy), "r"(idesc), "r"(acc), "r"(nk)
        : "memory");
    if (empty) tc_commit_elect(empty);
  } else {
    asm volatile(
        "{\n\t.reg .pred e, p0, p1, q1, q2, q3;\n\t.reg .b64 y1, y2, y3, z1, z2, z3;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p0, %4, 0;\n\tsetp.eq.b32 p1, %4, %4;\n\t"
        "setp.gt.and.s32 q1, %5, 1, e;\n\tsetp.gt.and.s32 q2, %5, 2, e;\n\tsetp.gt.and.s32 q3, %5, 3, e;\n\t"
        "add.u64 y1, %1, 128;\n\tadd.u64 y2, %1, 256;\n\tadd.u64 y3, %1, 384;\n\t"
        "add.u64 z1, %2, 128;\n\tadd.u64 z2, %2, 256;\n\tadd.u64 z3, %2, 384;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p0;\n\t"
        "@q1 tcgen05.mma.cta_group::2.kind::f16 [%0], y1, z1, %3, p1;\n\t"
        "@q2 tcgen05.mma.cta_group::2.kind::f16 [%0], y2, z2, %3, p1;\n\t"
        "@q3 tcgen05.mma.cta_group::2.kind::f16 [%0], y3, z3, %3, p1;\n\t}" ::"r"(d),
        "l"(x), "l"(dy), "r"(idesc), "r"(acc), "r"(nk)
        : "memory");
    if (empty) tc_commit_pair_elect(empty);
  }
}

// Instruction descriptor, kind::f16: D f32, both operands f16 or both bf16,
// both along M and N (bits 15 and 16).
__device__ __forceinline__ uint32_t idesc_wgrad(int bf16, int M, int N) {
  return 1u << 4 | (uint32_t)bf16 << 7 | (uint32_t)bf16 << 10 | 1u << 15 | 1u << 16 | (uint32_t)(N >> 3) << 17 | (uint32_t)(M >> 4) << 24;
}

struct WgKernelArgs {
  WgradArgs a;
  int inject_stall;
};
struct WgTile {
  int e, n0, k0, lo, hi;   // this CTA's rows of it
};

// SPLIT: a cluster shares each tile's rows, and there is one tile a cluster at
// most.
template <int OUT, bool SPLIT>
__global__ void __launch_bounds__(kWgThreads, 1)
    weight_grad_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_dy, const WgKernelArgs args) {
  using RG = WgRing;
  using T = typename ElemT<OUT>::t;
  constexpr int S = RG::stages;
  extern __shared__ __align__(1024) uint8_t wg_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(wg_smem_raw) + 1023) & ~uintptr_t(1023));
  const WgradArgs& a = args.a;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + RG::bar_off);
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain_bar = acc_empty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* row0 = reinterpret_cast<int*>(smem + RG::row_off);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], kEpiWarps);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, RG::tmem_cols);
    tmem_relinquish();
  }
  op_begin();   // the operands and offsets may come from the kernel before
  if (warp == 3)
    for (int e = lane; e <= a.E; e += 32) row0[e] = a.offsets ? min(max(a.offsets[e], 0), (int)a.R) : (e ? (int)a.R : 0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const int ntn = (a.N + kWgBN - 1) / kWgBN, ntk = (a.K + kTileM - 1) / kTileM;
  const int total = a.E * ntn * ntk;
  int ranks = 1, rank = 0, first = blockIdx.x, stride = gridDim.x;
  if constexpr (SPLIT) {
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ranks));
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    first = blockIdx.x / ranks;
    stride = gridDim.x / ranks;
  }
  // whole stages to each rank; the first ranks have rows where there are few
  auto tile_of = [&](int tile) {
    WgTile t;
    const int kt = tile % ntk, rest = tile / ntk, nt = rest % ntn;
    t.e = rest / ntn;
    t.n0 = nt * kWgBN;
    t.k0 = kt * kTileM;
    const int lo = row0[t.e], hi = max(row0[t.e + 1], lo);
    const int steps = (hi - lo + kWgRows - 1) / kWgRows, each = (steps + ranks - 1) / ranks;
    // (their ends may lie past hi, by less than 512 rows: rows are below 2^31 - 512)
    t.lo = min(lo + rank * each * kWgRows, hi);
    t.hi = min(t.lo + each * kWgRows, hi);
    return t;
  };

  if (warp == 0) {
    // ---------------- producer ----------------
    int it = 0;
    bool ok = true;
    for (int tile = first; tile < total && ok; tile += stride) {
      const WgTile t = tile_of(tile);
      const int panels = min(RG::dy_panels, (a.N - t.n0 + kWgPanel - 1) / kWgPanel);
      for (int r = t.lo; r < t.hi; r += kWgRows, ++it) {
        const int s = it % S;
        ok = wait_or_abort(&empty[s], ((it / S) & 1) ^ 1, a.wait, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        mbar_arrive_expect_tx_elect(&full[s], (uint32_t)((RG::x_panels + panels) * kWgPanelBytes));
        // Test hook: the first stage's barrier is armed, its copies are never issued.
        if (args.inject_stall && it == 0) continue;
#pragma unroll
        for (int p = 0; p < RG::x_panels; ++p)
          tma_3d_elect(smem + RG::x_off + s * RG::x_bytes + p * kWgPanelBytes, &map_x, t.k0 + p * kWgPanel, r, 0, &full[s]);
        for (int p = 0; p < panels; ++p)
          tma_3d_elect(smem + RG::dy_off + s * RG::dy_bytes + p * kWgPanelBytes, &map_dy, t.n0 + p * kWgPanel, r, 0, &full[s]);
      }
    }
    if (!ok) drain_ring<S>(full, it, a.wait.status, kDrainPolls);
    drain_ring<S>(empty, it, a.wait.status, ok ? kDrainWaitLimit : kDrainPolls);
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    const uint64_t xdesc0 = smem_desc_mn128(smem_u32(smem + RG::x_off), kWgPanelBytes);
    const uint64_t dydesc0 = smem_desc_mn128(smem_u32(smem + RG::dy_off), kWgPanelBytes);
    int it = 0;
    WgAccs accs;
    bool ok = true;
    for (int tile = first; tile < total && ok; tile += stride) {
      const WgTile t = tile_of(tile);
      if (t.lo >= t.hi) continue;
      const uint32_t idesc = idesc_wgrad(a.dtype == QMOE_BF16, kTileM, (min(kWgBN, a.N - t.n0) + 15) & ~15);
      for (int lo = t.lo, end; lo < t.hi && ok; lo = end) {
        end = piece_end<OUT>(lo, t.hi);
        const int ab = accs.of(lo == t.lo);
        ok = spin_or_abort(&acc_empty[ab], accs.parity(ab) ^ 1u, a.wait, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        for (int r = lo; r < end && ok; r += kWgRows, ++it) {
          const int s = it % S;
          if (!warp_test_wait(&full[s], (it / S) & 1)) {
            ok = spin_or_abort(&full[s], (it / S) & 1, a.wait, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
          }
          const int rows = min(kWgRows, end - r);
          if (rows & 15) {
            zero_rows(smem + RG::x_off + s * RG::x_bytes, RG::x_panels, rows);
            zero_rows(smem + RG::dy_off + s * RG::dy_bytes, min(RG::dy_panels, (a.N - t.n0 + kWgPanel - 1) / kWgPanel), rows);
            fence_proxy_async_smem();
            __syncwarp();
          }
          tc_fence_after();
          wg_stage_elect<1>(tmem + ab * kWgBN, xdesc0 + (uint64_t)((s * RG::x_bytes) >> 4), dydesc0 + (uint64_t)((s * RG::dy_bytes) >> 4),
                            idesc, r != lo ? 1u : 0u, (rows + 15) / 16, &empty[s]);
        }
        if (ok) tc_commit_elect(&acc_full[ab]);
        accs.step(ab);
      }
      accs.home ^= 1;
    }
    tc_commit_elect(drain_bar);
    const WaitCfg drain{a.wait.status, kDrainWaitLimit};
    mbar_wait_bounded(drain_bar, 0, drain);
  } else if (warp >= 4) {
    // ---------------- epilogue ----------------
    const int q = warp & 3, half = (warp >> 2) - 1;
    WgAccs accs;
    bool ok = true;
    for (int tile = first; tile < total && ok; tile += stride) {
      const WgTile t = tile_of(tile);
      const int col = t.k0 + q * 32 + lane, n = min(kWgBN, a.N - t.n0);
      const bool in = col < a.K;
      T* out = static_cast<T*>(a.dw) + ((size_t)t.e * a.N + t.n0) * a.K + col;
      if (t.lo >= t.hi) {
        if constexpr (SPLIT) {
          float* part = reinterpret_cast<float*>(smem);
          for (int c = half; c < n; c += 2) part[c * kTileM + q * 32 + lane] = 0.f;
        } else {
          store_zeros<OUT>(out, a.K, n, in, half);
        }
        continue;
      }
      const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16), sum = lanes + accs.home * kWgBN;
      auto release = [&](int ab) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[ab]);
      };
      for (int lo = t.lo, end; lo < t.hi; lo = end) {
        end = piece_end<OUT>(lo, t.hi);
        const int ab = accs.of(lo == t.lo);
        ok = wait_or_abort(&acc_full[ab], accs.parity(ab), a.wait, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        accs.step(ab);
        if (lo != t.lo) {
          add_pieces(sum, lanes + ab * kWgBN, n, half, false);
          release(ab);
        }
      }
      if (!ok) break;
      if constexpr (SPLIT) put_partial(sum, reinterpret_cast<float*>(smem), q, n, half);   // the ring is empty
      else store_tile<OUT>(sum, out, a.K, n, in, half);
      release(accs.home);
      accs.home ^= 1;
    }
  }
  if constexpr (SPLIT) {
    __syncwarp();
    cluster_sync_all();
    if (warp >= 4 && first < total) {
      const WgTile t = tile_of(first);
      const int q = warp & 3, col = t.k0 + q * 32 + lane;
      store_sum<OUT>(reinterpret_cast<const float*>(smem), q, static_cast<T*>(a.dw) + ((size_t)t.e * a.N + t.n0) * a.K + col, a.K,
                     min(kWgBN, a.N - t.n0), col < a.K, rank, ranks, (warp >> 2) - 1);
    }
    __syncwarp();
    cluster_sync_all();   // no CTA leaves while another may still read its part
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  __syncwarp();   // the lanes of warp 1 leave its last wait one by one
  if (warp == 1) tmem_dealloc(tmem, RG::tmem_cols);
}

// The same with pairs of CTAs: tiles of 256 columns of x by up to 256 of dy, of
// which each CTA loads half, 128 rows a stage: a copy of 64 rows hardly takes the
// TMA unit less time than one of 128.  Nothing is overwritten with zeros here:
// copies of an expert's rows go by tensor maps whose rows end with the expert's, so
// that what lies behind reads as zeros (a warp of each CTA that wrote the zeros, and
// their arrival at the first CTA, took 3000 cycles a tile).  A kernel before this
// one makes them, two for each expert (4 us alone).
//
// Bound: the MMAs, the copies at 2.4 cycles a row of 128 bytes and, with few rows an
// expert, the stores (8192 rows of 8192 x 8192: 652 us, 1.69 PFLOP/s, 89 % of the
// measured bf16 rate; 32768 rows of 64 experts, 4096 x 1536: 290 us, 1.42 PFLOP/s and
// 4.0 TB/s of what has to move).
constexpr int kWgPairRows = 128;
struct WgMaps {
  CUtensorMap x, dy;   // copies of 64 columns by 128 rows
};
struct WgPairRing {
  static constexpr int stages = 3;
  static constexpr int panels = 2;                              // of x, and of a half of dy's columns
  static constexpr int panel_bytes = kWgPairRows * 128;
  static constexpr int x_bytes = panels * panel_bytes;
  static constexpr int dy_bytes = panels * panel_bytes;
  static constexpr int x_off = 0;
  static constexpr int dy_off = x_off + stages * x_bytes;
  static constexpr int bar_off = dy_off + stages * dy_bytes;
  static constexpr int row_off = bar_off + 512;
  static constexpr int total = row_off + (kSortMaxExperts + 1) * 4;
  static_assert(total > kAloneBytes && total + 1024 <= 227 * 1024, "shared memory");
};

// The maps of every expert with rows: those of all rows, ended at its last.  A warp
// an expert.
__global__ void __launch_bounds__(32) weight_grad_maps_kernel(const __grid_constant__ WgMaps maps, const int* offsets, int64_t R, WgMaps* out) {
  op_begin();
  __shared__ __align__(128) WgMaps mine;
  const int e = blockIdx.x, lane = threadIdx.x;
  const int hi = min(max(offsets[e + 1], 0), (int)R);
  if (hi == 0) return;
  static_assert(sizeof(WgMaps) == 32 * sizeof(uint2), "a piece a lane");
  reinterpret_cast<uint2*>(&mine)[lane] = reinterpret_cast<const uint2*>(&maps)[lane];
  __syncwarp();
  if (lane < 2)
    asm volatile("tensormap.replace.tile.global_dim.shared::cta.b1024.b32 [%0], 1, %1;" ::"r"(smem_u32(&mine) + lane * 128), "r"(hi) : "memory");
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 2; ++i)
    asm volatile("tensormap.cp_fenceproxy.global.shared::cta.tensormap::generic.release.gpu.sync.aligned [%0], [%1], 128;" ::"l"(
                     reinterpret_cast<uint8_t*>(out + e) + i * 128),
                 "r"(smem_u32(&mine) + i * 128)
                 : "memory");
}
// Before a map of that kernel is used.
__device__ __forceinline__ void acquire_map(const CUtensorMap* map) {
  asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(map) : "memory");
}

template <int OUT>
__global__ void __launch_bounds__(kWgThreads, 1)
    weight_grad_pair_kernel(const __grid_constant__ WgMaps maps, const WgMaps* by_expert, const WgKernelArgs args) {
  using RG = WgPairRing;
  using T = typename ElemT<OUT>::t;
  constexpr int S = RG::stages;
  // 32-bit results' pieces are many: both accumulators take them in turn, and they are
  // added up where the results are
  constexpr bool kAddInMemory = OUT == QMOE_F32;
  extern __shared__ __align__(1024) uint8_t wg_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(wg_smem_raw) + 1023) & ~uintptr_t(1023));
  const WgradArgs& a = args.a;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + RG::bar_off);   // the first CTA's count for both
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;
  uint64_t* acc_empty = acc_full + 2;                                 // the first CTA's count for both
  uint64_t* drain_bar = acc_empty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* row0 = reinterpret_cast<int*>(smem + RG::row_off);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = pair_rank();
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 2 * kEpiWarps);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncwarp();
  if (warp == 1) tmem_alloc_pair(tmem_holder, 2 * kWgBN);
  op_begin();   // the operands and offsets may come from the kernel before
  if (warp == 3)
    for (int e = lane; e <= a.E; e += 32) row0[e] = a.offsets ? min(max(a.offsets[e], 0), (int)a.R) : (e ? (int)a.R : 0);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // the other CTA's barriers and TMEM are there
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const int ntn = (a.N + kWgBN - 1) / kWgBN, ntk = (a.K + 2 * kTileM - 1) / (2 * kTileM);
  const int total = a.E * ntn * ntk, first = blockIdx.x / 2, stride = gridDim.x / 2;
  auto tile_of = [&](int tile) {
    WgTile t;
    const int kt = tile % ntk, rest = tile / ntk;
    t.e = rest / ntn;
    t.n0 = (rest % ntn) * kWgBN;
    t.k0 = (kt * 2 + rank) * kTileM;
    t.lo = row0[t.e];
    t.hi = max(row0[t.e + 1], t.lo);
    return t;
  };
  // columns of dy of each CTA: half of the tile's, in whole sixteens
  auto half_of = [&](const WgTile& t) { return ((min(kWgBN, a.N - t.n0) + 31) & ~31) / 2; };

  if (warp == 0 || warp == 2) {
    // ---------------- producers: x, and dy ----------------
    if (lane == 0) {   // one thread each, as in the products' kernel
      RingAt<S> at;
      int it = 0;
      bool ok = true;
      for (int tile = first; tile < total && ok; tile += stride) {
        const WgTile t = tile_of(tile);
        const int half = half_of(t), panels = (half + kWgPanel - 1) / kWgPanel, col0 = t.n0 + rank * half;
        const uint32_t bytes = (uint32_t)(2 * (RG::panels + panels) * RG::panel_bytes);
        const WgMaps* m = by_expert ? by_expert + t.e : &maps;
        // warp 0's operand, or warp 2's
        const CUtensorMap* map = warp == 0 ? &m->x : &m->dy;
        const int from = warp == 0 ? t.k0 : col0, copies = warp == 0 ? RG::panels : panels;
        if (by_expert && t.lo < t.hi) acquire_map(map);
        for (int r = t.lo; r < t.hi; r += kWgPairRows, ++it, at.step()) {
          const int s = at.s;
          ok = poll_or_wait(&empty[s], at.ph ^ 1u, a.wait, abort_flag);
          if (!ok) break;
          const uint32_t bar = first_cta_bar(&full[s]);
          if (warp == 0 && rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
          // Test hook: the first stage's barrier is armed, its copies are never issued.
          if (args.inject_stall && it == 0) continue;
          uint8_t* dst = warp == 0 ? smem + RG::x_off + s * RG::x_bytes : smem + RG::dy_off + s * RG::dy_bytes;
          for (int p = 0; p < copies; ++p) tma_3d_pair(dst + p * RG::panel_bytes, map, from + p * kWgPanel, r, 0, bar);
        }
      }
      // (both CTAs' copies count on the first one's barriers; the second one's own
      // never complete, so it waits for as long as the limit says)
      if (!ok) drain_ring<S>(full, it, a.wait.status, kDrainPolls);
      if (warp == 0) drain_ring<S>(empty, it, a.wait.status, ok ? kDrainWaitLimit : kDrainPolls);
    }
  } else if (warp == 1 && rank == 0) {
    // ---------------- MMA issuer ----------------
    const uint64_t xdesc0 = smem_desc_mn128(smem_u32(smem + RG::x_off), RG::panel_bytes);
    const uint64_t dydesc0 = smem_desc_mn128(smem_u32(smem + RG::dy_off), RG::panel_bytes);
    RingAt<S> at;
    WgAccs accs;
    bool ok = true;
    bool there = mbar_test_wait(&full[0], 0);   // the next stage, asked ahead as in the products' kernel
    for (int tile = first; tile < total && ok; tile += stride) {
      const WgTile t = tile_of(tile);
      if (t.lo >= t.hi) continue;
      const int half = half_of(t);
      const uint32_t idesc = idesc_wgrad(a.dtype == QMOE_BF16, 2 * kTileM, 2 * half);
      for (int lo = t.lo, end; lo < t.hi && ok; lo = end) {
        end = piece_end<OUT>(lo, t.hi);
        const int ab = accs.of(kAddInMemory || lo == t.lo);
        ok = warp_spin_cluster(&acc_empty[ab], accs.parity(ab) ^ 1u, a.wait, abort_flag);
        for (int r = lo; r < end && ok; r += kWgPairRows) {
          const int s = at.s, rows = min(kWgPairRows, end - r);
          if (!__shfl_sync(0xffffffffu, there, 0)) {
            ok = spin_or_abort(&full[s], at.ph, a.wait, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
          }
          at.step();
          there = mbar_test_wait(&full[at.s], at.ph);
          tc_fence_after();
          const uint64_t xd = xdesc0 + (uint32_t)((s * RG::x_bytes) >> 4), dyd = dydesc0 + (uint32_t)((s * RG::dy_bytes) >> 4);
          constexpr uint32_t on = (kWgRows * 128) >> 4;   // 64 rows
          wg_stage_elect<2>(tmem + ab * kWgBN, xd, dyd, idesc, r != lo ? 1u : 0u, (min(rows, kWgRows) + 15) / 16,
                            rows > kWgRows ? nullptr : &empty[s]);
          if (rows > kWgRows) wg_stage_elect<2>(tmem + ab * kWgBN, xd + on, dyd + on, idesc, 1u, (rows - kWgRows + 15) / 16, &empty[s]);
        }
        if (ok) tc_commit_pair_elect(&acc_full[ab]);
        accs.step(ab);
        if (kAddInMemory || end == t.hi) accs.home ^= 1;
      }
    }
    tc_commit_pair_elect(drain_bar);
    const WaitCfg drain{a.wait.status, kDrainWaitLimit};
    mbar_wait_bounded(drain_bar, 0, drain);
  } else if (warp >= 4) {
    // ---------------- epilogue ----------------
    const int q = warp & 3, half = (warp >> 2) - 1;
    WgAccs accs;
    bool ok = true;
    for (int tile = first; tile < total && ok; tile += stride) {
      const WgTile t = tile_of(tile);
      const int col = t.k0 + q * 32 + lane, n = min(kWgBN, a.N - t.n0);
      const bool in = col < a.K;
      T* out = static_cast<T*>(a.dw) + ((size_t)t.e * a.N + t.n0) * a.K + col;
      if (t.lo >= t.hi) {
        store_zeros<OUT>(out, a.K, n, in, half);
        continue;
      }
      const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
      auto release = [&](int ab) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) cluster_bar_arrive(first_cta_bar(&acc_empty[ab]));
      };
      for (int lo = t.lo, end; lo < t.hi; lo = end) {
        end = piece_end<OUT>(lo, t.hi);
        const int ab = accs.of(kAddInMemory || lo == t.lo);
        ok = wait_or_abort(&acc_full[ab], accs.parity(ab), a.wait, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        accs.step(ab);
        const uint32_t acc = lanes + ab * kWgBN, sum = lanes + accs.home * kWgBN;
        if constexpr (kAddInMemory) {
          if (lo != t.lo) add_tile(acc, reinterpret_cast<float*>(out), a.K, n, in, half);
          else store_tile<OUT>(acc, out, a.K, n, in, half);
        } else {
          if (lo != t.lo) {
            add_pieces(sum, acc, n, half, false);
            release(ab);
          }
          if (end < t.hi) continue;
          store_tile<OUT>(sum, out, a.K, n, in, half);
        }
        release(accs.home);
        accs.home ^= 1;
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  pair_end(drain_bar, rank, a.wait.status);   // neither CTA leaves, or frees TMEM, while the other may still use it
  tc_fence_after();
  __syncwarp();
  if (warp == 1) tmem_dealloc_pair(tmem, 2 * kWgBN);
}

// Rows that start on any element to rows that start on 16 bytes, of both
// operands in one launch.  A thread writes 16 bytes: it loads the aligned 16
// bytes that hold its first element and the following ones (words that are not
// wholly inside the tensor element by element) and shifts.
struct AlignArgs {
  const uint16_t* src[2];
  int64_t ld[2], pitch[2];
  uint16_t* dst[2];
  int width[2], groups[2];   // of 8 elements a row; 0: nothing to copy
  int64_t rows;
};
constexpr int kAlignThreads = 256;
__device__ __forceinline__ uint4 load_inside(const uint16_t* x, int64_t from, int64_t size) {
  if (from >= 0 && from + 8 <= size) return ld_once_v4(x + from);
  uint32_t v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = from + j >= 0 && from + j < size ? x[from + j] : 0u;
  return make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
}
__global__ void __launch_bounds__(kAlignThreads) align_rows_kernel(const AlignArgs a) {
  op_begin();
  const int per_row = a.groups[0] + a.groups[1];
  const int64_t n = a.rows * per_row;
  for (int64_t i = blockIdx.x * (int64_t)kAlignThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kAlignThreads) {
    const int64_t r = i / per_row;
    int g = (int)(i - r * per_row);
    const int which = g >= a.groups[0] ? 1 : 0;
    g -= which ? a.groups[0] : 0;
    const uint16_t* x = which ? a.src[1] : a.src[0];
    const int64_t ld = which ? a.ld[1] : a.ld[0], row0 = r * ld, size = (a.rows - 1) * ld + (which ? a.width[1] : a.width[0]);
    const int m = (int)((reinterpret_cast<uintptr_t>(x + row0) & 15) >> 1), c = g * 8;
    const uint4 lo = load_inside(x, row0 + c - m, size), hi = m ? load_inside(x, row0 + c - m + 8, size) : lo;
    uint32_t u[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int j = 0; j < 6; ++j) u[j] = (m & 4) ? u[j + 2] : u[j];
#pragma unroll
    for (int j = 0; j < 5; ++j) u[j] = (m & 2) ? u[j + 1] : u[j];
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = (m & 1) ? __funnelshift_r(u[j], u[j + 1], 16) : u[j];
    *reinterpret_cast<uint4*>((which ? a.dst[1] : a.dst[0]) + r * (which ? a.pitch[1] : a.pitch[0]) + c) = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

// ----------------------------------------------------------------------------
// Host side
// ----------------------------------------------------------------------------
namespace {

int64_t wgrad_tiles(int64_t E, int64_t N, int64_t K) { return E * ((N + kWgBN - 1) / kWgBN) * ((K + kTileM - 1) / kTileM); }
// Pairs of CTAs once every multiprocessor has a tile.
bool wgrad_pairs(int64_t E, int64_t N, int64_t K) { return wgrad_tiles(E, N, K) > kSms && K > kTileM; }

// TMA reads rows that start on 16 bytes, 16-byte multiples apart.
bool tma_rows(const void* p, int64_t ld) { return aligned16(p) && ld % 8 == 0; }
size_t align_bytes(const void* p, int64_t ld, int64_t R, int64_t width) {
  return tma_rows(p, ld) ? 0 : (size_t)R * (size_t)((width + 7) / 8 * 8) * 2;
}

// Copies what TMA cannot read into the workspace, and points the arguments there.
cudaError_t align_operands(WgradArgs& a, cudaStream_t s) {
  AlignArgs c{};
  c.rows = a.R;
  uint8_t* work = a.workspace + (wgrad_pairs(a.E, a.N, a.K) ? a.E * sizeof(WgMaps) : 0);
  auto take = [&](int i, const void*& p, int64_t& ld, int width) {
    if (tma_rows(p, ld)) return;
    c.src[i] = static_cast<const uint16_t*>(p);
    c.ld[i] = ld;
    c.width[i] = width;
    c.groups[i] = (width + 7) / 8;
    c.pitch[i] = (int64_t)c.groups[i] * 8;
    c.dst[i] = reinterpret_cast<uint16_t*>(work);
    work += (size_t)a.R * c.pitch[i] * 2;
    p = c.dst[i];
    ld = c.pitch[i];
  };
  take(0, a.dy, a.ld_dy, a.N);
  take(1, a.x, a.ld_x, a.K);
  const int64_t n = a.R * (c.groups[0] + c.groups[1]);
  if (n == 0) return cudaSuccess;
  const unsigned blocks = (unsigned)std::min<int64_t>((n + kAlignThreads - 1) / kAlignThreads, kSms * 8);
  return launch_op(align_rows_kernel, dim3(blocks), dim3(kAlignThreads), 0, s, c);
}

template <int OUT>
cudaError_t launch_wg(const WgKernelArgs& args, cudaStream_t s) {
  const WgradArgs& a = args.a;
  WgMaps maps;
  const auto type = a.dtype == QMOE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const bool pairs = wgrad_pairs(a.E, a.N, a.K);
  const int box = pairs ? kWgPairRows : kWgRows;
  if (!encode_tiles(&maps.x, type, 2, a.x, a.K, a.R, 1, a.ld_x * 2, box) ||
      !encode_tiles(&maps.dy, type, 2, a.dy, a.N, a.R, 1, a.ld_dy * 2, box))
    return cudaErrorInvalidValue;
  const int64_t tiles = wgrad_tiles(a.E, a.N, a.K);
  if (pairs) {
    WgMaps* by_expert = a.offsets ? reinterpret_cast<WgMaps*>(a.workspace) : nullptr;
    if (by_expert) {
      const cudaError_t e = launch_op(weight_grad_maps_kernel, dim3((unsigned)a.E), dim3(32), 0, s, maps, a.offsets, a.R, by_expert);
      if (e != cudaSuccess) return e;
    }
    const WgMaps* by = by_expert;
    return launch_tiles(weight_grad_pair_kernel<OUT>, kSms, 2, kWgThreads, WgPairRing::total + 1024, s, maps, by, args);
  }
  constexpr int smem = WgRing::total + 1024;   // + alignment slack
  // A tile's rows over the CTAs of a cluster while there are CTAs without a tile, if
  // the rows, spread evenly, fill 24 stages (us with / without: 2048 rows of 256 x
  // 256, in 8 parts, 10.2 / 17.2; 4000 of 1024 x 1024, in 4, 17.0 / 30.9; 32768 of
  // 64 x 64, in 8, 23.5 / 153; but 1000 of 1024 x 1024, 16 stages in 4, 11.9 / 11.1.
  // Uneven spreads are not told apart: 32768 rows over 16 experts of 256 x 256, even 15,
  // all of one expert, in 4, 66; dense, in 8, 37).
  const int64_t steps = (a.R / a.E + kWgRows - 1) / kWgRows;
  int split = 1;
  while (steps >= 24 && split < 8 && tiles * split * 2 <= kSms && split * 8 <= steps) split *= 2;
  if (split > 1) return launch_tiles(weight_grad_kernel<OUT, true>, tiles * split, split, kWgThreads, smem, s, maps.x, maps.dy, args);
  return launch_tiles(weight_grad_kernel<OUT, false>, std::min<int64_t>(tiles, kSms), 1, kWgThreads, smem, s, maps.x, maps.dy, args);
}

}  // namespace

// The maps of every expert, then the aligned copies.
size_t weight_grad_workspace(const void* dy, int64_t ld_dy, const void* x, int64_t ld_x, int64_t R, int64_t E, int64_t N, int64_t K) {
  return (wgrad_pairs(E, N, K) ? (size_t)E * sizeof(WgMaps) : 0) + align_bytes(dy, ld_dy, R, N) + align_bytes(x, ld_x, R, K);
}

cudaError_t launch_weight_grad(const WgradArgs& a, int inject_stall, cudaStream_t s) {
  if (wgrad_tiles(a.E, a.N, a.K) > 0x7fffffff) return cudaErrorInvalidValue;
  WgKernelArgs args{a, inject_stall};
  const cudaError_t e = align_operands(args.a, s);
  if (e != cudaSuccess) return e;
  if (a.out_dtype == QMOE_F32) return launch_wg<QMOE_F32>(args, s);
  if (a.out_dtype == QMOE_F16) return launch_wg<QMOE_F16>(args, s);
  return launch_wg<QMOE_BF16>(args, s);
}

}  // namespace qmoe
