// Product of microscaled 4-bit rows with microscaled 4-bit weights, dense or
// grouped by expert:
//
//   out[i, n] = sum_d A[i, d] * W[e, n, d]   for rows i in [offsets[e], offsets[e + 1])
//
// with A and W the values of their codes and scales (qmoe_mx4.cu).  A product
// of two E2M1 values and two power-of-two scales is exact, so the fp32
// accumulation and the one rounding to the output type are the only ones.
//
// GB300 form: tcgen05.mma kind::mxf4.block_scale reads both operands as
// packed codes from shared memory and both scale sets from TMEM, so nothing is
// dequantised anywhere.  A tile is 128 rows of A (the MMA's M, TMEM lanes) by
// BN weight rows; a ring stage holds 256 values along K of both: 128-byte rows
// (one 128-byte swizzle atom), copied by TMA tensor maps, and the scale bytes
// of 8 blocks a row, copied four bytes a row by cp.async (a panel of scales
// holds the four scales of 128 values for consecutive rows side by side, so a
// warp's copy is one contiguous line) straight into the 32 x 16-byte order
// that tcgen05.cp spreads over TMEM.
//   warp 0    TMA producer (one elected lane)
//   warp 1    MMA issuer: scales to TMEM, then four K = 64 MMAs a stage
//   warps 2-3 scale loaders
//   warps 4-7 epilogue: TMEM -> registers -> shared memory -> whole rows
// Two accumulators of BN columns alternate, so the epilogue of one tile runs
// under the MMAs of the next.  CTAs are persistent over the (expert, row tile,
// weight tile) list, which every CTA derives from the device offsets.
//
// Bound: at few rows an expert the weight bytes (17/32 byte a weight; 256 rows
// of 2048 to 1536 over 128 experts, 99 of which have rows, 166 MB: 33 us, 5.0
// TB/s); at many the way of a stage round the ring, about 4000 cycles for four
// stages of 384 cycles of MMAs (32768 rows of 1536 to 4096 over 64 experts: 122
// us, 3.4 PFLOP/s, 4.2 TB/s of its bytes; the same copies without MMAs, scales and
// stores take 107).  BN = 192 is what two accumulators and the scales leave of
// TMEM; BN = 64 puts more multiprocessors to work where there are few tiles.
//
// Every wait on an mbarrier is bounded; a timeout aborts all roles, drains what is in
// flight, frees TMEM and is reported by qmoe_op_poll_status.  (Not so the waits for the
// kernel before and for tensor memory, and the barriers that every warp comes to.)
#include <algorithm>

#include "qmoe_ops.cuh"
#include "qmoe_tma.cuh"

namespace qmoe {

constexpr int kMxRows = 128;                   // rows of A a tile
constexpr int kMxBoxRows = 32;                 // rows of A a copy where a tile is not full
constexpr int kMxStageK = 256;                 // values along K a stage
constexpr int kMxRowBytes = kMxStageK / 2;     // 128: one swizzle atom
constexpr int kMxTmemCols = 512;
constexpr int kMxThreads = 256;
constexpr int kMxEpiPitch = 144;               // bytes of a staged output row (128 + 16: banks)
constexpr int kMxMaxExperts = 1024;

template <int BN>
struct MxRing {
  static constexpr int stages = BN == 192 ? 4 : 7;
  static constexpr int groups = (BN + 127) / 128;                 // 128-row scale groups of W
  static constexpr int a_bytes = kMxRows * kMxRowBytes;
  static constexpr int b_bytes = BN * kMxRowBytes;
  static constexpr int sfa_bytes = 2 * 512;                       // two 128-value chunks
  static constexpr int sfb_bytes = 2 * 512 * groups;
  static constexpr int a_off = 0;
  static constexpr int b_off = a_off + stages * a_bytes;
  static constexpr int sfa_off = b_off + stages * b_bytes;
  static constexpr int sfb_off = sfa_off + stages * sfa_bytes;
  static constexpr int epi_off = sfb_off + stages * sfb_bytes;
  static constexpr int bar_off = epi_off + 4 * 32 * kMxEpiPitch;
  static constexpr int tp_off = bar_off + 512;                    // first row tile and first row of each expert
  static constexpr int total = tp_off + 2 * (kMxMaxExperts + 2) * 4;
  // TMEM columns: two accumulators, then per stage the scales of A and W
  static constexpr int sf_col0 = 2 * BN;
  static constexpr int sf_cols = 8 + 8 * groups;
  static_assert(sf_col0 + stages * sf_cols <= kMxTmemCols, "TMEM columns");
  static_assert(total > kAloneBytes && total + 1024 <= 227 * 1024, "shared memory");
  static_assert(b_bytes % 1024 == 0 && a_bytes % 1024 == 0, "swizzle atoms");
};

// ----------------------------------------------------------------------------
// Instructions
// ----------------------------------------------------------------------------
// One stage, issued by one elected lane: the scales of A (two chunks of 512
// bytes) and of W (two per 128-row group) to TMEM, four columns each and the
// same in every quarter of the lanes, then up to four K = 64 MMAs of E2M1
// operands with E8M0 scales of 32 values, then the commit that frees the
// stage.  One block of instructions with one elect: the issue of a stage has
// to take less time than its MMAs (four of 96 cycles at 192 columns), and with
// an elect and operand moves per instruction it took three times as long.
template <int GROUPS>
__device__ __forceinline__ void mx_stage_elect(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sf, uint64_t sa,
                                               uint64_t sb, uint32_t acc, int nk, uint64_t* empty) {
  static_assert(GROUPS == 1 || GROUPS == 2, "row groups of W");
  if constexpr (GROUPS == 2) {
    asm volatile(
        "{\n\t.reg .pred e, p0, p1, q1, q2, q3;\n\t"
        ".reg .b32 t<6>, i2;\n\t.reg .b64 x<6>, y<4>, z<4>;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p0, %7, 0;\n\tsetp.eq.b32 p1, %7, %7;\n\t"
        "setp.gt.and.s32 q1, %8, 1, e;\n\tsetp.gt.and.s32 q2, %8, 2, e;\n\tsetp.gt.and.s32 q3, %8, 3, e;\n\t"
        "add.u32 t1, %4, 4;\n\tadd.u32 t2, %4, 8;\n\tadd.u32 t3, %4, 12;\n\tadd.u32 t4, %4, 16;\n\tadd.u32 t5, %4, 20;\n\t"
        "add.u64 x1, %5, 32;\n\tadd.u64 x3, %6, 32;\n\tadd.u64 x4, %6, 64;\n\tadd.u64 x5, %6, 96;\n\t"
        "add.u64 y1, %1, 2;\n\tadd.u64 y2, %1, 4;\n\tadd.u64 y3, %1, 6;\n\t"
        "add.u64 z1, %2, 2;\n\tadd.u64 z2, %2, 4;\n\tadd.u64 z3, %2, 6;\n\t"
        "or.b32 i2, %3, 0x40000020;\n\t"
        "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%4], %5;\n\t"
        "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [t2], %6;\n\t"
        "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [t3], x3;\n\t"
        "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [t1], x1;\n\t"
        "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [t4], x4;\n\t"
        "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [t5], x5;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [t2], p0;\n\t"
        "@q1 tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], y1, z1, i2, [%4], [t2], p1;\n\t"
        "@q2 tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], y2, z2, %3, [t1], [t4], p1;\n\t"
        "@q3 tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], y3, z3, i2, [t1], [t4], p1;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%9];\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sf), "l"(sa), "l"(sb), "r"(acc), "r"(nk), "r"(smem_u32(empty))
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred e, p0, p1, q1, q2, q3;\n\t"
        ".reg .b32 t<4>, i2;\n\t.reg .b64 x<4>, y<4>, z<4>;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p0, %7, 0;\n\tsetp.eq.b32 p1, %7, %7;\n\t"
        "setp.gt.and.s32 q1, %8, 1, e;\n\tsetp.gt.and.s32 q2, %8, 2, e;\n\tsetp.gt.and.s32 q3, %8, 3, e;\n\t"
        "add.u32 t1, %4, 4;\n\tadd.u32 t2, %4, 8;\n\tadd.u32 t3, %4, 12;\n\t"
        "add.u64 x1, %5, 32;\n\tadd.u64 x3, %6, 32;\n\t"
        "add.u64 y1, %1, 2;\n\tadd.u64 y2, %1, 4;\n\tadd.u64 y3, %1, 6;\n\t"
        "add.u64 z1, %2, 2;\n\tadd.u64 z2, %2, 4;\n\tadd.u64 z3, %2, 6;\n\t"
        "or.b32 i2, %3, 0x40000020;\n\t"
        "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%4], %5;\n\t"
        "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [t2], %6;\n\t"
        "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [t1], x1;\n\t"
        "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [t3], x3;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [t2], p0;\n\t"
        "@q1 tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], y1, z1, i2, [%4], [t2], p1;\n\t"
        "@q2 tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], y2, z2, %3, [t1], [t3], p1;\n\t"
        "@q3 tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], y3, z3, i2, [t1], [t3], p1;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%9];\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sf), "l"(sa), "l"(sb), "r"(acc), "r"(nk), "r"(smem_u32(empty))
        : "memory");
  }
}
// Instruction descriptor, kind::mxf4: both operands E2M1, scales E8M0, M =
// 128, K = 64.  The scale ids (bits 29-30 and 4-5) name the byte pair of a
// 32-bit scale word that an MMA's two blocks use: 0, or 2 for every second MMA.
__device__ __forceinline__ uint32_t idesc_mxf4(int N) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(kMxRows >> 7) << 27);
}

// ----------------------------------------------------------------------------
// Kernel
// ----------------------------------------------------------------------------
struct MxTile {
  int e, start, rows, n0;   // e == E: rows without a route (zeros)
};

struct MxKernelArgs {
  Mx4MatmulArgs a;
  int inject_stall;
  int vec_out;              // 16-byte output stores
};

// First row of group e (0 .. E; group E is the rows without a route).  Clamped
// to the rows there are, so that no offsets make a role leave its operands.
__device__ __forceinline__ int mx_first_row(const Mx4MatmulArgs& a, int e) {
  if (e <= 0) return 0;
  if (!a.offsets || e > a.E) return (int)a.R;
  return min(max(a.offsets[e], 0), (int)a.R);
}

// Tile index -> expert, rows and weight columns.  tp[e] is the first row tile
// of group e, tp[E + 1] their number, and its first row is row0[e].
__device__ __forceinline__ MxTile mx_tile(const Mx4MatmulArgs& a, const int* tp, const int* row0, int ntn, int bn, int tile) {
  const int mt = tile / ntn;
  int lo = 0, hi = a.E;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tp[mid] <= mt) lo = mid;
    else hi = mid - 1;
  }
  MxTile t;
  t.e = lo;
  t.start = row0[lo] + (mt - tp[lo]) * kMxRows;
  t.rows = min(kMxRows, row0[lo + 1] - t.start);
  t.n0 = (tile - mt * ntn) * bn;
  return t;
}

template <int BN, int OUT>
__global__ void __launch_bounds__(kMxThreads, 1)
    mx4_matmul_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_a32,
                      const __grid_constant__ CUtensorMap map_w, const MxKernelArgs args) {
  using RG = MxRing<BN>;
  constexpr int S = RG::stages;
  extern __shared__ __align__(1024) uint8_t mx_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(mx_smem_raw) + 1023) & ~uintptr_t(1023));
  const Mx4MatmulArgs& a = args.a;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + RG::bar_off);
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain_bar = acc_empty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* tp = reinterpret_cast<int*>(smem + RG::tp_off);
  int* row0 = tp + kMxMaxExperts + 2;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      // one barrier tells the MMA warp that a stage is there (a poll takes 120
      // cycles, a stage's MMAs 384): the announced bytes and the 64 lanes of the
      // scale loaders
      mbar_init(&full[i], 1 + 64);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 4);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, kMxTmemCols);
    tmem_relinquish();
  }
  op_begin();   // the operands and offsets may come from the kernel before
  if (warp == 3) {
    // first row tile of each group: E experts, then the rows without a route
    int first = 0;
    for (int e0 = 0; e0 <= a.E; e0 += 32) {
      const int e = e0 + lane;
      int n = 0;
      if (e <= a.E) {
        const int lo = mx_first_row(a, e), hi = mx_first_row(a, e + 1);
        n = hi > lo ? (hi - lo + kMxRows - 1) / kMxRows : 0;
        row0[e] = lo;
      }
      int run = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += up;
      }
      if (e <= a.E) tp[e] = first + run - n;
      first += __shfl_sync(0xffffffffu, run, 31);
    }
    if (lane == 0) {
      tp[a.E + 1] = first;
      row0[a.E + 1] = (int)a.R;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const int ntn = (a.N + BN - 1) / BN;
  const int total = tp[a.E + 1] * ntn;
  const int nb = (a.K + 31) / 32, nq = (nb + 3) / 4;
  const int ksteps = (nb + 7) / 8;

  if (warp == 0) {
    // ---------------- producer ----------------
    int it = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
      const MxTile t = mx_tile(a, tp, row0, ntn, BN, tile);
      if (t.e == a.E) continue;
      // the rows in one copy if they are many, else in copies of 32
      const int boxes = (max(t.rows, 0) + kMxBoxRows - 1) / kMxBoxRows;
      for (int ks = 0; ks < ksteps; ++ks, ++it) {
        const int s = it % S;
        ok = wait_or_abort(&empty[s], ((it / S) & 1) ^ 1, a.wait, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        mbar_arrive_expect_tx_elect(&full[s], (uint32_t)(boxes * kMxBoxRows * kMxRowBytes + RG::b_bytes));
        // Test hook: the first stage's barrier is armed, its copies are never issued.
        if (args.inject_stall && it == 0) continue;
        if (boxes == kMxRows / kMxBoxRows)
          tma_2d_elect(smem + RG::a_off + s * RG::a_bytes, &map_a, ks * kMxRowBytes, t.start, &full[s]);
        else
          for (int b = 0; b < boxes; ++b)
            tma_2d_elect(smem + RG::a_off + s * RG::a_bytes + b * kMxBoxRows * kMxRowBytes, &map_a32, ks * kMxRowBytes,
                         t.start + b * kMxBoxRows, &full[s]);
        tma_2d_elect(smem + RG::b_off + s * RG::b_bytes, &map_w, ks * kMxRowBytes, t.e * a.N + t.n0, &full[s]);
      }
    }
    // (after a wait that ran out the scale loaders may have left the stages short)
    if (!ok) drain_ring<S>(full, it, a.wait.status, kDrainPolls);
    drain_ring<S>(empty, it, a.wait.status, ok ? kDrainWaitLimit : kDrainPolls);
  } else if (warp == 2 || warp == 3) {
    // ---------------- scale loaders: warp 2 + h takes the 128-value chunk h of each stage ----------------
    // Row 32 j + lane of a 128-row group goes to bytes lane * 16 + j * 4 of its
    // chunk.  Pointers are set up once a tile and step from panel to panel.
    // Padding scales (past nb, in the last panel's words) are kept out: with an
    // odd number of blocks the last MMA meets one, and NaN times a zero code is NaN.
    const int h = warp - 2;
    const uint32_t sfa0 = smem_u32(smem + RG::sfa_off) + h * 512 + lane * 16;
    const uint32_t sfb0 = smem_u32(smem + RG::sfb_off) + h * RG::groups * 512 + lane * 16;
    const size_t step_a = (size_t)a.R * 8, step_w = (size_t)a.N * 8;   // two panels on
    int it = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
      const MxTile t = mx_tile(a, tp, row0, ntn, BN, tile);
      if (t.e == a.E) continue;
      const uint8_t* pa = a.a_scales + ((size_t)h * a.R + t.start + lane) * 4;
      const uint8_t* pw = a.w_scales + (((size_t)t.e * nq + h) * a.N + t.n0 + lane) * 4;
      const int na = (int)a.R - t.start - lane, nw = a.N - t.n0 - lane;   // row 32 j exists: 32 j < n
      const bool inside = t.start + kMxRows <= (int)a.R && t.n0 + BN <= a.N;
      for (int ks = 0; ks < ksteps; ++ks, ++it, pa += step_a, pw += step_w) {
        const int s = it % S;
        ok = wait_or_abort(&empty[s], ((it / S) & 1) ^ 1, a.wait, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t da = sfa0 + s * RG::sfa_bytes, db = sfb0 + s * RG::sfb_bytes;
        const int bytes = min(4, nb - 4 * (2 * ks + h));   // scales of this chunk, none if it is not above zero
        if (inside && bytes > (nb & 1 ? 3 : 0)) {   // every row exists: no tests between the copies
#pragma unroll
          for (int j = 0; j < kMxRows / 32; ++j) cp_async4(da + j * 4, pa + j * 128);
#pragma unroll
          for (int j = 0; j < BN / 32; ++j) cp_async4(db + (j / 4) * 512 + (j & 3) * 4, pw + j * 128);
        } else {
          const bool in = bytes > 0;
#pragma unroll
          for (int j = 0; j < kMxRows / 32; ++j) {
            const bool real = in && 32 * j < na;
            cp_async4_or_zero(da + j * 4, real ? pa + j * 128 : a.a_scales, real ? bytes : 0);
          }
#pragma unroll
          for (int j = 0; j < BN / 32; ++j) {
            const bool real = in && 32 * j < nw;
            cp_async4_or_zero(db + (j / 4) * 512 + (j & 3) * 4, real ? pw + j * 128 : a.w_scales, real ? bytes : 0);
          }
        }
        cp_async_arrive(&full[s]);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    // The tiles that hold rows come first, so their number is all this warp
    // needs to know.  The stage loop is unrolled over the ring: every stage's
    // operands are compile-time offsets from a few bases.
    const uint64_t adesc0 = smem_desc_sw128(smem_u32(smem + RG::a_off));
    const uint64_t bdesc0 = smem_desc_sw128(smem_u32(smem + RG::b_off));
    const uint64_t sadesc0 = smem_desc_scales(smem_u32(smem + RG::sfa_off));
    const uint64_t sbdesc0 = smem_desc_scales(smem_u32(smem + RG::sfb_off));
    const uint32_t idesc = idesc_mxf4(BN);
    const int real = tp[a.E] * ntn;
    const int tail = (nb * 32 - (ksteps - 1) * kMxStageK + 63) / 64;   // MMAs of a tile's last stage
    int st = 0, tc = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < real && ok; tile += gridDim.x, ++tc) {
      const int ab = tc & 1;
      ok = spin_or_abort(&acc_empty[ab], ((tc >> 1) & 1) ^ 1, a.wait, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t dacc = tmem + ab * BN;
      int ks = 0;
      while (ks < ksteps && ok) {
#pragma unroll
        for (int u = 0; u < S; ++u) {
          if (u == st && ks < ksteps && ok) {
            if (!warp_test_wait(&full[u], ph)) {
              ok = spin_or_abort(&full[u], ph, a.wait, abort_flag);
              ok = __all_sync(0xffffffffu, ok);
            }
            if (ok) {
              tc_fence_after();
              fence_proxy_async_smem();   // the scale loader's copies are generic-proxy writes
              mx_stage_elect<RG::groups>(dacc, adesc0 + (uint64_t)((u * RG::a_bytes) >> 4),
                                         bdesc0 + (uint64_t)((u * RG::b_bytes) >> 4), idesc,
                                         tmem + RG::sf_col0 + u * RG::sf_cols, sadesc0 + (uint64_t)((u * RG::sfa_bytes) >> 4),
                                         sbdesc0 + (uint64_t)((u * RG::sfb_bytes) >> 4), ks != 0 ? 1u : 0u,
                                         ks + 1 < ksteps ? 4 : tail, &empty[u]);
              ++ks;
              if (++st == S) {
                st = 0;
                ph ^= 1u;
              }
            }
          }
        }
      }
      if (ok) tc_commit_elect(&acc_full[ab]);
    }
    tc_commit_elect(drain_bar);
    const WaitCfg drain{a.wait.status, kDrainWaitLimit};
    mbar_wait_bounded(drain_bar, 0, drain);
  } else if (warp >= 4) {
    // ---------------- epilogue ----------------
    const int q = warp & 3;
    constexpr int esz = OUT == QMOE_F32 ? 4 : 2;
    constexpr int cols = 128 / esz;              // columns of a staged row
    uint8_t* stage = smem + RG::epi_off + q * 32 * kMxEpiPitch;
    int tc = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
      const MxTile t = mx_tile(a, tp, row0, ntn, BN, tile);
      const bool zero = t.e == a.E;
      const int ab = tc & 1;
      if (!zero) {
        ok = wait_or_abort(&acc_full[ab], (tc >> 1) & 1, a.wait, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
      }
      const int wrows = min(32, t.rows - q * 32);   // rows of this warp (may be <= 0)
      for (int c0 = 0; c0 < BN; c0 += cols) {
        const int ncols = min(cols, a.N - (t.n0 + c0));
        if (ncols <= 0 || wrows <= 0) break;        // the same for the whole warp
#pragma unroll
        for (int u = 0; u < cols / 32; ++u) {
          uint32_t v[32];
          if (!zero) {
            TC_LD32(tmem + ((uint32_t)(q * 32) << 16) + ab * BN + c0 + 32 * u, v);
            tc_wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0u;
          }
          uint4* dst = reinterpret_cast<uint4*>(stage + lane * kMxEpiPitch + u * 64);
          if constexpr (OUT == QMOE_F32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) dst[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          } else {
            auto f = [&](int i) { return pack2<OUT>(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])); };
#pragma unroll
            for (int i = 0; i < 4; ++i) dst[i] = make_uint4(f(4 * i), f(4 * i + 1), f(4 * i + 2), f(4 * i + 3));
          }
        }
        __syncwarp();
        uint8_t* out = static_cast<uint8_t*>(a.out) + ((size_t)(t.start + q * 32) * a.ld_out + t.n0 + c0) * esz;
        if (args.vec_out && ncols == cols) {
          // eight lanes a row: 128-byte runs
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + (lane >> 3);
            if (r < wrows)
              *reinterpret_cast<uint4*>(out + (size_t)r * a.ld_out * esz + (lane & 7) * 16) =
                  *reinterpret_cast<const uint4*>(stage + r * kMxEpiPitch + (lane & 7) * 16);
          }
        } else {
          using T = typename ElemT<OUT>::t;
          for (int r = 0; r < wrows; ++r)
            for (int c = lane; c < ncols; c += 32)
              reinterpret_cast<T*>(out)[(size_t)r * a.ld_out + c] = reinterpret_cast<const T*>(stage + r * kMxEpiPitch)[c];
        }
        __syncwarp();
      }
      if (!zero) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[ab]);
        ++tc;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  __syncwarp();   // the lanes of warp 1 leave its last wait one by one
  if (warp == 1) tmem_dealloc(tmem, kMxTmemCols);
}

// ----------------------------------------------------------------------------
// Host side
// ----------------------------------------------------------------------------
namespace {

// Rows of codes: boxes of `box_rows` rows by 128 bytes, 128-byte swizzle,
// zeros outside.
bool encode_rows(CUtensorMap* m, const uint8_t* codes, int64_t rows, int64_t pitch, int box_rows) {
  const EncodeFn f = encoder();
  if (!f) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)pitch, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)pitch};
  const cuuint32_t box[2] = {(cuuint32_t)kMxRowBytes, (cuuint32_t)box_rows};
  const cuuint32_t ones[2] = {1, 1};
  return f(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dims, strides, box, ones,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, int OUT>
cudaError_t launch_mx(const MxKernelArgs& args, int64_t tiles, cudaStream_t s) {
  const Mx4MatmulArgs& a = args.a;
  const int64_t pitch = (int64_t)((a.K + 31) / 32) * 16;
  CUtensorMap map_a, map_a32, map_w;
  if (!encode_rows(&map_a, a.a_codes, a.R, pitch, kMxRows) || !encode_rows(&map_a32, a.a_codes, a.R, pitch, kMxBoxRows) ||
      !encode_rows(&map_w, a.w_codes, (int64_t)a.E * a.N, pitch, BN))
    return cudaErrorInvalidValue;
  constexpr int smem = MxRing<BN>::total + 1024;   // + alignment slack
  auto kern = mx4_matmul_kernel<BN, OUT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(tiles, kSms));
  cfg.blockDim = dim3(kMxThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, map_a, map_a32, map_w, args);
}

// Output tiles there can be at most (the device offsets decide how many there are).
int64_t most_tiles(const Mx4MatmulArgs& a, int bn) {
  const int64_t groups = a.offsets ? std::min<int64_t>((int64_t)a.E + 1, a.R) : 1;
  return (a.R / kMxRows + groups) * ((a.N + bn - 1) / bn);
}

}  // namespace

cudaError_t launch_mx4_matmul(const Mx4MatmulArgs& a, int inject_stall, cudaStream_t s) {
  MxKernelArgs args{a, inject_stall, 0};
  args.vec_out = rows_aligned16(a.out, a.ld_out, a.out_dtype) ? 1 : 0;
  auto run = [&](auto bn, int64_t tiles) {
    constexpr int BN = decltype(bn)::value;
    if (a.out_dtype == QMOE_F32) return launch_mx<BN, QMOE_F32>(args, tiles, s);
    if (a.out_dtype == QMOE_F16) return launch_mx<BN, QMOE_F16>(args, tiles, s);
    return launch_mx<BN, QMOE_BF16>(args, tiles, s);
  };
  // narrow tiles while they are all under way at once, wide ones from then on
  // (us, narrow / wide: 64 x 4096 x 4096, 64 narrow tiles, 9.4 / 10.3; 1 x 8192 x
  // 2048, 128, 7.9 / 8.0; 512 x 4096 x 4096, 320, 13.9 / 9.9; 2048 x 4096 x 4096,
  // 1088, 38.9 / 20.8)
  const int64_t narrow = most_tiles(a, 64);
  return narrow <= kSms ? run(std::integral_constant<int, 64>{}, narrow)
                        : run(std::integral_constant<int, 192>{}, most_tiles(a, 192));
}

}  // namespace qmoe
