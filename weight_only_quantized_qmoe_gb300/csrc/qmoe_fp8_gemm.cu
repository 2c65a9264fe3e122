// Product of 8-bit rows with 8-bit weights, dense or grouped by expert:
//
//   out[i, n] = sum_k A[i, k] W[e, n, k]     rows i in [offsets[e], offsets[e + 1])
//   out[i, k] = sum_n A[i, n] W[e, n, k]     (back: the gradient of the rows)
//
// with A and W the values of their codes and scales (qmoe_fp8.cu).  A product
// of two E4M3 values and two power-of-two scales is exact in fp32, so the fp32
// accumulation and the one rounding to the output type are the only ones.
//
// GB300 form: tcgen05.mma kind::mxf8f6f4.block_scale reads both operands as
// codes from shared memory and the scales from TMEM.  Its scale blocks are 32
// values, ours four of them: all four MMAs of 128 values name the same byte of
// the scale words.  The MMA's M side is 128 weight rows (back: weight columns, the
// same codes read along M), its N side up to 32 rows of A; a ring stage holds 128
// reduction values of both, 128-byte rows copied by TMA.
//   warp 0    TMA producer (one elected lane)
//   warp 1    MMA issuer: scales to TMEM, then four K = 32 MMAs a stage
//   warp 2    scales of A's rows: four bytes a row by cp.async (512 values' worth)
//   warp 3    scale of the weight block: one byte, spread over 512
//   warps 4-11 epilogue: TMEM columns to rows of the output
// Two accumulators of 32 columns alternate, so the epilogue of one tile runs
// under the MMAs of the next.  CTAs are persistent over the (expert, row tile,
// weight tile) list, which every CTA derives from the device offsets.  Where
// there are few tiles, the CTAs of a cluster share a tile's reduction and add up
// their parts in a fixed order.
//
// That is the form for few rows (1 x 2048 x 2048: 5.9 us; 32 tokens to 8 of 128
// experts of 1536 x 2048: 51 to 56 us, 6 TB/s of the weights of those that have
// rows, which bound it; 16 x 8192 x 16384 25.3, with a 32-bit result in pieces 25.5).
// Many rows take pairs of CTAs, further down.
//
// Every wait on an mbarrier is bounded; a timeout aborts all roles, drains what is in
// flight, frees TMEM and is reported by qmoe_op_poll_status.  Three waits have no limit
// of their own: for the kernel before (op_begin); at the barriers of the CTA and of the
// cluster, which every warp comes to, whatever its waits gave; and for tensor memory,
// which is free (kAloneBytes).
#include "qmoe_tile.cuh"

namespace qmoe {

constexpr int kF8StageK = 128;                 // values along the reduction a stage: one swizzle atom
constexpr int kF8Threads = 128 + 32 * kEpiWarps;

struct F8Ring {
  static constexpr int bn = 32;                                   // rows of A a tile
  static constexpr int stages = 10;
  static constexpr int w_bytes = kTileM * kF8StageK;
  static constexpr int a_bytes = bn * kF8StageK;
  static constexpr int sfw_bytes = 512;
  static constexpr int sfa_bytes = 512;                           // a group of 128 rows
  static constexpr int w_off = 0;
  static constexpr int a_off = w_off + stages * w_bytes;
  static constexpr int sfw_off = a_off + stages * a_bytes;
  static constexpr int sfa_off = sfw_off + stages * sfw_bytes;
  static constexpr int bar_off = sfa_off + stages * sfa_bytes;
  static constexpr int tp_off = bar_off + 512;                    // first row tile and first row of each expert
  static constexpr int total = tp_off + 2 * (kSortMaxExperts + 2) * 4;
  // TMEM columns: two accumulators, then per stage the scales of W and A
  static constexpr int sf_col0 = 2 * bn;
  static constexpr int sf_cols = 8;
  static constexpr int sum_col0 = sf_col0 + stages * sf_cols;     // the sum of the pieces of 32-bit results
  static constexpr int tmem_cols = 256;
  static_assert(sum_col0 + bn <= tmem_cols, "TMEM columns");
  static_assert(total > kAloneBytes && total + 1024 <= 227 * 1024, "shared memory");
  static_assert(a_bytes % 1024 == 0, "swizzle atoms");
  static_assert(bn * kTileM * 4 <= stages * w_bytes, "a partial tile fits the ring");
};

// Stages summed in the tensor core at a time, for 32-bit results (see add_tile;
// relative error of 16384 values in one piece 1.2e-6, in three 4e-7): for pairs whole
// groups of four stages, which share a word of scales.
constexpr int kF8Piece = 48;
template <int OUT>
__device__ __forceinline__ int f8_piece_end(int from, int end) {
  return OUT == QMOE_F32 && end - from > kF8Piece ? from + kF8Piece : end;
}

// One stage, issued by one elected lane: the scales of W and of A's rows to TMEM, up
// to four K = 32 MMAs, the commit that frees the stage.
__device__ __forceinline__ void f8_stage_elect(uint32_t d, uint64_t w, uint64_t wstep, uint64_t a, uint32_t idesc, uint32_t sf,
                                               uint64_t sw, uint64_t sa, uint32_t acc, int nk, uint64_t* empty) {
  asm volatile(
      "{\n\t.reg .pred e, p0, p1, q1, q2, q3;\n\t"
      ".reg .b32 t1;\n\t.reg .b64 y1, y2, y3, z1, z2, z3;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p0, %8, 0;\n\tsetp.eq.b32 p1, %8, %8;\n\t"
      "setp.gt.and.s32 q1, %9, 1, e;\n\tsetp.gt.and.s32 q2, %9, 2, e;\n\tsetp.gt.and.s32 q3, %9, 3, e;\n\t"
      "add.u32 t1, %5, 4;\n\t"
      "add.u64 y1, %1, %2;\n\tadd.u64 y2, y1, %2;\n\tadd.u64 y3, y2, %2;\n\t"
      "add.u64 z1, %3, 2;\n\tadd.u64 z2, %3, 4;\n\tadd.u64 z3, %3, 6;\n\t"
      "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%5], %6;\n\t"
      "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [t1], %7;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %3, %4, [%5], [t1], p0;\n\t"
      "@q1 tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], y1, z1, %4, [%5], [t1], p1;\n\t"
      "@q2 tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], y2, z2, %4, [%5], [t1], p1;\n\t"
      "@q3 tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], y3, z3, %4, [%5], [t1], p1;\n\t}" ::"r"(d),
      "l"(w), "l"(wstep), "l"(a), "r"(idesc), "r"(sf), "l"(sw), "l"(sa), "r"(acc), "r"(nk)
      : "memory");
  tc_commit_elect(empty);
}

// Instruction descriptor, kind::mxf8f6f4: both operands E4M3, scales E8M0; W
// along K, or along M (bit 15).  The scale ids (bits 29-30 and 4-5) name
// the byte of a 32-bit scale word.
__device__ __forceinline__ uint32_t idesc_mxf8(int M, int N, int back) {
  return ((uint32_t)back << 15) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 7) << 27);
}

struct F8KernelArgs {
  Fp8MatmulArgs a;
  int inject_stall;
  int bn;                   // rows of A a tile, of pairs: 32 i
};

// SPLIT: a cluster shares each tile's reduction, and there is one tile a cluster
// at most.
template <int OUT, bool SPLIT>
__global__ void __launch_bounds__(kF8Threads, 1)
    fp8_matmul_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w, const F8KernelArgs args) {
  using RG = F8Ring;
  using T = typename ElemT<OUT>::t;
  constexpr int S = RG::stages, BN = RG::bn;
  extern __shared__ __align__(1024) uint8_t f8_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(f8_smem_raw) + 1023) & ~uintptr_t(1023));
  const Fp8MatmulArgs& a = args.a;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + RG::bar_off);
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain_bar = acc_empty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* tp = reinterpret_cast<int*>(smem + RG::tp_off);
  int* row0 = tp + kSortMaxExperts + 2;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1 + 32 + 1);   // the announced bytes, the lanes of A's scales, the weight's scale
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
  if (warp == 3) group_tiles(a.offsets, a.E, a.R, BN, tp, row0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const int inner = a.back ? a.N : a.K, width = a.back ? a.K : a.N;   // of A's rows, of the output's
  const int ntw = (width + kTileM - 1) / kTileM;
  const int total = tp[a.E + 1] * ntw;
  const int nbn = (a.N + kF8StageK - 1) / kF8StageK, nbk = (a.K + kF8StageK - 1) / kF8StageK;
  const int ksteps = a.back ? nbn : nbk;
  int ranks = 1, rank = 0, first = blockIdx.x, stride = gridDim.x;
  if constexpr (SPLIT) {
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ranks));
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    first = blockIdx.x / ranks;
    stride = gridDim.x / ranks;
  }
  const int ks0 = (int)((int64_t)ksteps * rank / ranks), ks1 = (int)((int64_t)ksteps * (rank + 1) / ranks);
  auto tile_of = [&](int tile, int& n0) {
    const int mt = tile / ntw;
    n0 = (tile - mt * ntw) * kTileM;
    return row_tile(a.E, tp, row0, BN, mt);
  };

  if (warp == 0) {
    // ---------------- producer ----------------
    int it = 0;
    bool ok = true;
    for (int tile = first; tile < total && ok; tile += stride) {
      int n0;
      const RowTile t = tile_of(tile, n0);
      if (t.e == a.E) continue;
      for (int ks = ks0; ks < ks1; ++ks, ++it) {
        const int s = it % S;
        ok = wait_or_abort(&empty[s], ((it / S) & 1) ^ 1, a.wait, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        mbar_arrive_expect_tx_elect(&full[s], (uint32_t)(RG::a_bytes + RG::w_bytes));
        // Test hook: the first stage's barrier is armed, its copies are never issued.
        if (args.inject_stall && it == 0) continue;
        tma_3d_elect(smem + RG::a_off + s * RG::a_bytes, &map_a, ks * kF8StageK, t.start, 0, &full[s]);
        uint8_t* dw = smem + RG::w_off + s * RG::w_bytes;
        if (a.back) tma_3d_elect(dw, &map_w, n0, ks * kF8StageK, t.e, &full[s]);
        else tma_3d_elect(dw, &map_w, ks * kF8StageK, n0, t.e, &full[s]);
      }
    }
    // (after a wait that ran out the scale warps may have left the stages short)
    if (!ok) drain_ring<S>(full, it, a.wait.status, kDrainPolls);
    drain_ring<S>(empty, it, a.wait.status, ok ? kDrainWaitLimit : kDrainPolls);
  } else if (warp == 2) {
    // ---------------- scales of A's rows ----------------
    // Row `lane` goes to bytes lane * 16 of the chunk: the four bytes of 512 values, of
    // which a stage's MMAs name one.
    const uint32_t dst0 = smem_u32(smem + RG::sfa_off) + lane * 16;
    int it = 0;
    bool ok = true;
    for (int tile = first; tile < total && ok; tile += stride) {
      int n0;
      const RowTile t = tile_of(tile, n0);
      if (t.e == a.E) continue;
      const bool real = t.start + lane < a.R;
      for (int ks = ks0; ks < ks1; ++ks, ++it) {
        const int s = it % S;
        ok = wait_or_abort(&empty[s], ((it / S) & 1) ^ 1, a.wait, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint8_t* src = a.a_scales + ((size_t)(ks >> 2) * a.R + t.start + lane) * 4;
        cp_async4_or_zero(dst0 + s * RG::sfa_bytes, real ? src : a.a_scales, real ? 4 : 0);
        cp_async_arrive(&full[s]);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == 3) {
    // ---------------- scale of the weight block ----------------
    uint8_t* dst = smem + RG::sfw_off + lane * 16;
    int it = 0;
    bool ok = true;
    for (int tile = first; tile < total && ok; tile += stride) {
      int n0;
      const RowTile t = tile_of(tile, n0);
      if (t.e == a.E) continue;
      const int ob = n0 / kTileM;
      const uint8_t* src = a.w_scales + (size_t)t.e * nbn * nbk + (a.back ? ob : (size_t)ob * nbk);
      const size_t step = a.back ? nbk : 1;
      uint32_t next = src[ks0 * step];
      for (int ks = ks0; ks < ks1; ++ks, ++it) {
        const uint32_t word = next * 0x01010101u;
        if (ks + 1 < ks1) next = src[(ks + 1) * step];
        const int s = it % S;
        ok = wait_or_abort(&empty[s], ((it / S) & 1) ^ 1, a.wait, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        *reinterpret_cast<uint4*>(dst + s * RG::sfw_bytes) = make_uint4(word, word, word, word);
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    // The tiles that hold rows come first, so their number is all this warp
    // needs to know beside their rows.
    const uint64_t wdesc0 = a.back ? smem_desc_mn128(smem_u32(smem + RG::w_off), RG::w_bytes) : smem_desc_sw128(smem_u32(smem + RG::w_off));
    const uint64_t wstep = a.back ? (32 * 128) >> 4 : 32 >> 4;   // 32 reduction values on: 32 rows, or 32 bytes
    const uint64_t adesc0 = smem_desc_sw128(smem_u32(smem + RG::a_off));
    const uint64_t swdesc0 = smem_desc_scales(smem_u32(smem + RG::sfw_off));
    const uint64_t sadesc0 = smem_desc_scales(smem_u32(smem + RG::sfa_off));
    const int real = tp[a.E] * ntw;
    const int tail = (inner - (ksteps - 1) * kF8StageK + 31) / 32;   // MMAs of the last stage
    int st = 0, tc = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int tile = first; tile < real && ok; tile += stride) {
      int n0;
      const RowTile t = tile_of(tile, n0);
      const uint32_t idesc0 = idesc_mxf8(kTileM, (t.rows + 15) & ~15, a.back);
      for (int from = ks0, to; from < ks1 && ok; from = to, ++tc) {
        to = f8_piece_end<OUT>(from, ks1);
        const int ab = tc & 1;
        ok = spin_or_abort(&acc_empty[ab], ((tc >> 1) & 1) ^ 1, a.wait, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t dacc = tmem + ab * BN;
        int ks = from;
        while (ks < to && ok) {
#pragma unroll
          for (int u = 0; u < S; ++u) {
            if (u == st && ks < to && ok) {
              if (!warp_test_wait(&full[u], ph)) {
                ok = spin_or_abort(&full[u], ph, a.wait, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
              }
              if (ok) {
                tc_fence_after();
                fence_proxy_async_smem();   // the scales were written through the generic proxy
                f8_stage_elect(dacc, wdesc0 + (uint64_t)((u * RG::w_bytes) >> 4), wstep, adesc0 + (uint64_t)((u * RG::a_bytes) >> 4),
                               idesc0 | (uint32_t)(ks & 3) << 29 | (uint32_t)(ks & 3) << 4, tmem + RG::sf_col0 + u * RG::sf_cols,
                               swdesc0 + (uint64_t)((u * RG::sfw_bytes) >> 4), sadesc0 + (uint64_t)((u * RG::sfa_bytes) >> 4),
                               ks != from ? 1u : 0u, ks + 1 < ksteps ? 4 : tail, &empty[u]);
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
    }
    tc_commit_elect(drain_bar);
    const WaitCfg drain{a.wait.status, kDrainWaitLimit};
    mbar_wait_bounded(drain_bar, 0, drain);
  } else if (warp >= 4) {
    // ---------------- epilogue ----------------
    const int q = warp & 3, half = (warp >> 2) - 1;
    int tc = 0;
    bool ok = true;
    for (int tile = first; tile < total && ok; tile += stride) {
      int n0;
      const RowTile t = tile_of(tile, n0);
      const int col = n0 + q * 32 + lane;
      const bool in = col < width;
      T* out = static_cast<T*>(a.out) + (size_t)t.start * a.ld_out + col;
      if (t.e == a.E) {
        if (rank == 0) store_zeros<OUT>(out, a.ld_out, t.rows, in, half);
        continue;
      }
      for (int from = ks0, to; from < ks1; from = to, ++tc) {
        to = f8_piece_end<OUT>(from, ks1);
        const int ab = tc & 1;
        ok = wait_or_abort(&acc_full[ab], (tc >> 1) & 1, a.wait, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
        uint32_t acc = lanes + ab * BN;
        if (OUT == QMOE_F32 && (from != ks0 || to < ks1)) {   // in pieces
          add_pieces(lanes + RG::sum_col0, acc, t.rows, half, from == ks0);
          acc = lanes + RG::sum_col0;
        }
        if (to == ks1) {
          if constexpr (SPLIT) put_partial(acc, reinterpret_cast<float*>(smem + RG::w_off), q, t.rows, half);   // the ring is empty
          else store_tile<OUT>(acc, out, a.ld_out, t.rows, in, half);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[ab]);
      }
    }
  }
  if constexpr (SPLIT) {
    __syncwarp();
    cluster_sync_all();
    if (warp >= 4 && first < total) {
      int n0;
      const RowTile t = tile_of(first, n0);
      const int q = warp & 3, col = n0 + q * 32 + lane;
      if (t.e != a.E)
        store_sum<OUT>(reinterpret_cast<const float*>(smem + RG::w_off), q, static_cast<T*>(a.out) + (size_t)t.start * a.ld_out + col,
                       a.ld_out, t.rows, col < width, rank, ranks, (warp >> 2) - 1);
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

// ----------------------------------------------------------------------------
// Pairs of CTAs, for many rows: tiles of 256 weight rows (back: columns) by up to
// 224 rows of A, of which each CTA loads half.  Scales do not pass through shared
// memory: four warps a CTA, one for each quarter of the TMEM lanes, load the
// words of 512 reduction values (all rows of A, this CTA's weight block) and
// write them to TMEM, every quarter the same, and arrive on the first CTA's
// barrier once in four stages.
//   warp 0      copies of W, the announcement of a stage
//   warp 1      MMA issuer (first CTA)
//   warp 2      copies of A's rows
//   warp 3      tile table
//   warps 4-7   scales
//   warps 8-15  epilogue
// Bound: the MMAs and what an SM takes in (8192 x 8192 x 8192: 321 us, 3.4 PFLOP/s,
// 1.8 times the measured bf16 rate, a stage in some 500 cycles of 448 of MMAs; 32768 x
// 4096 x 1536 over 64 experts: 172 us, 2.4 PFLOP/s, of which the stores, 2 bytes a lane,
// are 20, and back, 4096 to 1536, 155 us).
// ----------------------------------------------------------------------------
struct F8PairRing {
  static constexpr int bn = 224;
  static constexpr int stages = 7;
  static constexpr int sf_groups = 5;                             // scales of four stages each
  static constexpr int w_bytes = kTileM * kF8StageK;
  static constexpr int a_bytes = bn / 2 * kF8StageK;
  static constexpr int w_off = 0;
  static constexpr int a_off = w_off + stages * w_bytes;
  static constexpr int bar_off = a_off + stages * a_bytes;
  static constexpr int tp_off = bar_off + 512;
  static constexpr int total = tp_off + 2 * (kSortMaxExperts + 2) * 4;
  static constexpr int sf_col0 = 2 * bn;
  static constexpr int sf_cols = 12;                              // W's four columns, then A's eight
  static_assert(sf_col0 + sf_groups * sf_cols <= 512, "TMEM columns");
  static_assert(total > kAloneBytes && total + 1024 <= 227 * 1024, "shared memory");
  static_assert(a_bytes % 1024 == 0, "swizzle atoms");
};
// Copies of A's rows of every size that a tile has, 16 to 112 rows a CTA, so that a
// stage is one copy (with copies of 8 rows the tiles that are not full took twice
// as long as the others: 32768 rows over 64 experts 210 us, now 172).
struct F8RowMaps {
  CUtensorMap of[F8PairRing::bn / 32];
};
constexpr int kF8PairThreads = 256 + 32 * kEpiWarps;

// One stage: up to four K = 32 MMAs of the pair and the commit that frees it.
__device__ __forceinline__ void f8_pair_stage_elect(uint32_t d, uint64_t w, uint64_t wstep, uint64_t a, uint32_t idesc, uint32_t sfw,
                                                    uint32_t sfa, uint32_t acc, int nk, uint64_t* empty) {
  asm volatile(
      "{\n\t.reg .pred e, p0, p1, q1, q2, q3;\n\t.reg .b64 y1, y2, y3, z1, z2, z3;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p0, %7, 0;\n\tsetp.eq.b32 p1, %7, %7;\n\t"
      "setp.gt.and.s32 q1, %8, 1, e;\n\tsetp.gt.and.s32 q2, %8, 2, e;\n\tsetp.gt.and.s32 q3, %8, 3, e;\n\t"
      "add.u64 y1, %1, %2;\n\tadd.u64 y2, y1, %2;\n\tadd.u64 y3, y2, %2;\n\t"
      "add.u64 z1, %3, 2;\n\tadd.u64 z2, %3, 4;\n\tadd.u64 z3, %3, 6;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %3, %4, [%5], [%6], p0;\n\t"
      "@q1 tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], y1, z1, %4, [%5], [%6], p1;\n\t"
      "@q2 tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], y2, z2, %4, [%5], [%6], p1;\n\t"
      "@q3 tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], y3, z3, %4, [%5], [%6], p1;\n\t}" ::"r"(d),
      "l"(w), "l"(wstep), "l"(a), "r"(idesc), "r"(sfw), "r"(sfa), "r"(acc), "r"(nk)
      : "memory");
  tc_commit_pair_elect(empty);
}
__device__ __forceinline__ void tmem_store_x4(uint32_t taddr, uint32_t v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%1,%1,%1};" ::"r"(taddr), "r"(v) : "memory");
}
__device__ __forceinline__ void tmem_store_x8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

template <int OUT>
__global__ void __launch_bounds__(kF8PairThreads, 1)
    fp8_matmul_pair_kernel(const __grid_constant__ F8RowMaps map_a, const __grid_constant__ CUtensorMap map_w, const F8KernelArgs args) {
  using RG = F8PairRing;
  using T = typename ElemT<OUT>::t;
  constexpr int S = RG::stages, G = RG::sf_groups, BN = RG::bn;
  extern __shared__ __align__(1024) uint8_t f8_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(f8_smem_raw) + 1023) & ~uintptr_t(1023));
  const Fp8MatmulArgs& a = args.a;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + RG::bar_off);   // the first CTA's count for both
  uint64_t* empty = full + S;
  uint64_t* sf_full = empty + S;                                      // the first CTA's count for both
  uint64_t* sf_empty = sf_full + G;
  uint64_t* acc_full = sf_empty + G;
  uint64_t* acc_empty = acc_full + 2;                                 // the first CTA's count for both
  uint64_t* drain_bar = acc_empty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* tp = reinterpret_cast<int*>(smem + RG::tp_off);
  int* row0 = tp + kSortMaxExperts + 2;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = pair_rank();
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < G; ++i) {
      mbar_init(&sf_full[i], 8);    // four warps of each CTA
      mbar_init(&sf_empty[i], 1);
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
  if (warp == 1) tmem_alloc_pair(tmem_holder, 512);
  op_begin();   // the operands and offsets may come from the kernel before
  if (warp == 3) group_tiles(a.offsets, a.E, a.R, args.bn, tp, row0);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // the other CTA's barriers and TMEM are there
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const int inner = a.back ? a.N : a.K, width = a.back ? a.K : a.N;   // of A's rows, of the output's
  const int ntw = (width + 2 * kTileM - 1) / (2 * kTileM);
  const int total = tp[a.E + 1] * ntw, real = tp[a.E] * ntw;          // with and without the rows that have no route
  const int nbn = (a.N + kF8StageK - 1) / kF8StageK, nbk = (a.K + kF8StageK - 1) / kF8StageK;
  const int ksteps = a.back ? nbn : nbk, first = blockIdx.x / 2, stride = gridDim.x / 2;
  auto tile_of = [&](int tile, int& n0) {
    const int mt = tile / ntw;
    n0 = ((tile - mt * ntw) * 2 + rank) * kTileM;
    return row_tile(a.E, tp, row0, args.bn, mt);
  };
  // stages summed in the tensor core at a time: whole groups of scales (see add_tile)
  const int piece = OUT == QMOE_F32 ? kF8Piece : ksteps;
  // rows of A of each CTA: half of the tile's, in whole sixteens
  auto half_of = [&](const RowTile& t) { return ((t.rows + 31) & ~31) / 2; };

  if (warp == 0 || warp == 2) {
    // ---------------- producers: W, and A's rows ----------------
    // One thread each: a stage's wait, announcement and two copies by one warp
    // took 740 cycles, its MMAs 448.
    if (lane == 0) {
      RingAt<S> at;
      int it = 0;
      bool ok = true;
      for (int tile = first; tile < real && ok; tile += stride) {
        int n0;
        const RowTile t = tile_of(tile, n0);
        const int half = half_of(t);
        for (int ks = 0; ks < ksteps; ++ks, ++it, at.step()) {
          const int s = at.s;
          ok = poll_or_wait(&empty[s], at.ph ^ 1u, a.wait, abort_flag);
          if (!ok) break;
          const uint32_t bar = first_cta_bar(&full[s]);
          if (warp == 0 && rank == 0) mbar_arrive_expect_tx(&full[s], (uint32_t)(2 * (half * kF8StageK + RG::w_bytes)));
          // Test hook: the first stage's barrier is armed, its copies are never issued.
          if (args.inject_stall && it == 0) continue;
          if (warp == 0) {
            uint8_t* dw = smem + RG::w_off + s * RG::w_bytes;
            if (a.back) tma_3d_pair(dw, &map_w, n0, ks * kF8StageK, t.e, bar);
            else tma_3d_pair(dw, &map_w, ks * kF8StageK, n0, t.e, bar);
            continue;
          }
          tma_3d_pair(smem + RG::a_off + s * RG::a_bytes, &map_a.of[half / 16 - 1], ks * kF8StageK, t.start + rank * half, 0, bar);
        }
      }
      // (both CTAs' copies count on the first one's barriers; the second one's own
      // never complete, so it waits for as long as the limit says)
      if (!ok) drain_ring<S>(full, it, a.wait.status, kDrainPolls);
      if (warp == 0) drain_ring<S>(empty, it, a.wait.status, ok ? kDrainWaitLimit : kDrainPolls);
    }
  } else if (warp == 1 && rank == 0) {
    // ---------------- MMA issuer ----------------
    const uint64_t wdesc0 = a.back ? smem_desc_mn128(smem_u32(smem + RG::w_off), RG::w_bytes) : smem_desc_sw128(smem_u32(smem + RG::w_off));
    const uint64_t wstep = a.back ? (32 * 128) >> 4 : 32 >> 4;   // 32 reduction values on: 32 rows, or 32 bytes
    const uint64_t adesc0 = smem_desc_sw128(smem_u32(smem + RG::a_off));
    const int tail = (inner - (ksteps - 1) * kF8StageK + 31) / 32;   // MMAs of the last stage
    RingAt<S> at;
    RingAt<G> sf;
    int tc = 0;
    bool ok = true;
    // whether the next stage is there, asked before the MMAs of the one before
    // are issued
    bool there = mbar_test_wait(&full[0], 0), sf_there = false;
    for (int tile = first; tile < real && ok; tile += stride, ++tc) {
      int n0;
      const RowTile t = tile_of(tile, n0);
      const uint32_t idesc0 = idesc_mxf8(2 * kTileM, 2 * half_of(t), a.back);
      int left = 0;   // stages of this piece
      for (int ks = 0; ks < ksteps && ok; ++ks, --left) {
        const int id = ks & 3, s = at.s;
        if (left == 0) {
          if (ks) {
            tc_commit_pair_elect(&acc_full[tc & 1]);
            ++tc;
          }
          left = piece;
          ok = warp_spin_cluster(&acc_empty[tc & 1], ((tc >> 1) & 1) ^ 1, a.wait, abort_flag);
          if (!ok) break;
        }
        if (id == 0) {
          // (asked for ahead as well)
          ok = __shfl_sync(0xffffffffu, sf_there, 0) || warp_spin_cluster(&sf_full[sf.s], sf.ph, a.wait, abort_flag);
          if (!ok) break;
        }
        if (!__shfl_sync(0xffffffffu, there, 0)) {
          ok = spin_or_abort(&full[s], at.ph, a.wait, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
        }
        at.step();
        there = mbar_test_wait(&full[at.s], at.ph);
        tc_fence_after();
        const uint32_t sft = tmem + RG::sf_col0 + sf.s * RG::sf_cols;
        f8_pair_stage_elect(tmem + (tc & 1) * BN, wdesc0 + (uint32_t)((s * RG::w_bytes) >> 4), wstep, adesc0 + (uint32_t)((s * RG::a_bytes) >> 4),
                            idesc0 | (uint32_t)id << 29 | (uint32_t)id << 4, sft, sft + 4, left != piece ? 1u : 0u, ks + 1 < ksteps ? 4 : tail,
                            &empty[s]);
        if (id == 3 || ks + 1 == ksteps) {
          tc_commit_pair_elect(&sf_empty[sf.s]);
          sf.step();
          sf_there = cluster_test_wait(&sf_full[sf.s], sf.ph);
        }
      }
      if (ok) tc_commit_pair_elect(&acc_full[tc & 1]);
    }
    tc_commit_pair_elect(drain_bar);
    const WaitCfg drain{a.wait.status, kDrainWaitLimit};
    mbar_wait_bounded(drain_bar, 0, drain);
  } else if (warp >= 4 && warp < 8) {
    // ---------------- scales ----------------
    // Row 32 j + lane's word of A goes to column 4 + j of this quarter's lane; the
    // weight block's word, the same for every row, to columns 0 to 3.
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    RingAt<G> sf;
    int groups = 0;
    bool ok = true;
    for (int tile = first; tile < real && ok; tile += stride) {
      int n0;
      const RowTile t = tile_of(tile, n0);
      const int left = min((int)a.R - t.start, args.bn) - lane;   // row 32 j exists: 32 j < left
      const int ob = min(n0, width - 1) / kTileM;
      const uint8_t* w0 = a.w_scales + (size_t)t.e * nbn * nbk + (a.back ? ob : (size_t)ob * nbk);
      const size_t wstep = a.back ? nbk : 1;
      uint32_t next[8], next_w = 0;   // on their way while the ones before are written
      auto fetch = [&](int ks) {
        const uint8_t* src = a.a_scales + ((size_t)(ks >> 2) * a.R + t.start + lane) * 4;
#pragma unroll
        for (int j = 0; j < 8; ++j) next[j] = 32 * j < left ? *reinterpret_cast<const uint32_t*>(src + j * 128) : 0u;
        next_w = lane < 4 && ks + lane < ksteps ? (uint32_t)w0[(ks + lane) * wstep] << (8 * lane) : 0u;
      };
      fetch(0);
      for (int ks = 0; ks < ksteps; ks += 4, ++groups, sf.step()) {
        uint32_t word[8], w = next_w;
#pragma unroll
        for (int j = 0; j < 8; ++j) word[j] = next[j];
        if (ks + 4 < ksteps) fetch(ks + 4);
        w |= __shfl_xor_sync(0xffffffffu, w, 1);
        w |= __shfl_xor_sync(0xffffffffu, w, 2);
        const uint32_t every = __shfl_sync(0xffffffffu, w, 0);
        ok = wait_or_abort(&sf_empty[sf.s], sf.ph ^ 1u, a.wait, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t at = tmem + lanes + RG::sf_col0 + sf.s * RG::sf_cols;
        tmem_store_x4(at, every);
        tmem_store_x8(at + 4, word);
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) cluster_bar_arrive(first_cta_bar(&sf_full[sf.s]));
      }
    }
    if (warp == 4) drain_ring<G>(sf_empty, groups, a.wait.status, ok ? kDrainWaitLimit : kDrainPolls);
  } else if (warp >= 8) {
    // ---------------- epilogue ----------------
    const int q = warp & 3, half = (warp >> 2) - 2;
    int tc = 0;
    bool ok = true;
    for (int tile = first; tile < total && ok; tile += stride) {
      int n0;
      const RowTile t = tile_of(tile, n0);
      const int col = n0 + q * 32 + lane;
      const bool in = col < width;
      T* out = static_cast<T*>(a.out) + (size_t)t.start * a.ld_out + col;
      if (t.e == a.E) {
        store_zeros<OUT>(out, a.ld_out, t.rows, in, half);
        continue;
      }
      for (int ks = 0; ks < ksteps; ks += piece, ++tc) {
        const int ab = tc & 1;
        ok = wait_or_abort(&acc_full[ab], (tc >> 1) & 1, a.wait, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + ab * BN;
        if (OUT == QMOE_F32 && ks) add_tile(acc, reinterpret_cast<float*>(out), a.ld_out, t.rows, in, half);
        else store_tile<OUT>(acc, out, a.ld_out, t.rows, in, half);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) cluster_bar_arrive(first_cta_bar(&acc_empty[ab]));
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  pair_end(drain_bar, rank, a.wait.status);   // neither CTA leaves, or frees TMEM, while the other may still use it
  tc_fence_after();
  __syncwarp();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// ----------------------------------------------------------------------------
// Host side
// ----------------------------------------------------------------------------
namespace {

template <int OUT>
cudaError_t launch_f8(const F8KernelArgs& args, bool pairs, int64_t tiles, int split, cudaStream_t s) {
  const Fp8MatmulArgs& a = args.a;
  const int64_t inner = a.back ? a.N : a.K, pitch = fp8_pitch(inner);
  CUtensorMap map_w;
  constexpr auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  if (!encode_tiles(&map_w, u8, 1, a.w_codes, a.K, a.N, a.E, fp8_pitch(a.K), kTileM)) return cudaErrorInvalidValue;
  constexpr int slack = 1024;   // of the alignment
  if (pairs) {
    F8RowMaps map_a;
    for (int i = 0; i < F8PairRing::bn / 32; ++i)
      if (!encode_tiles(&map_a.of[i], u8, 1, a.a_codes, inner, a.R, 1, pitch, 16 * (i + 1))) return cudaErrorInvalidValue;
    return launch_tiles(fp8_matmul_pair_kernel<OUT>, std::min<int64_t>(2 * tiles, kSms), 2, kF8PairThreads, F8PairRing::total + slack, s, map_a,
                        map_w, args);
  }
  CUtensorMap map_a;
  if (!encode_tiles(&map_a, u8, 1, a.a_codes, inner, a.R, 1, pitch, F8Ring::bn)) return cudaErrorInvalidValue;
  if (split > 1)
    return launch_tiles(fp8_matmul_kernel<OUT, true>, tiles * split, split, kF8Threads, F8Ring::total + slack, s, map_a, map_w, args);
  return launch_tiles(fp8_matmul_kernel<OUT, false>, std::min<int64_t>(tiles, kSms), 1, kF8Threads, F8Ring::total + slack, s, map_a, map_w, args);
}

// Output tiles there can be at most (the device offsets decide how many there
// are): of bn rows of A by `wide` weight rows.
int64_t most_tiles(const Fp8MatmulArgs& a, int bn, int wide) {
  const int64_t rows = a.offsets ? a.R / bn + std::min<int64_t>((int64_t)a.E + 1, a.R) : (a.R + bn - 1) / bn;
  return rows * (((a.back ? a.K : a.N) + wide - 1) / wide);
}

// Rows of A a tile of pairs.  Dense: those that take the least rounds of 76 pairs
// times a stage's time, some 265 cycles and one more a row (8192 x 8192 x 8192, us:
// 224 rows 321, 160 rows 384; those of the rule / 224: 512 x 4096 x 4096 12.6 /
// 13.1, 2001 x 2880 x 5761 34.9 / 37.3).  Grouped: as many as there can
// be, as experts' rows are uneven and a remainder costs a tile of its own (32768
// rows over 64 experts 175 us, by the rule for an even spread 186).
int pair_rows(const Fp8MatmulArgs& a) {
  int best = F8PairRing::bn;
  if (a.offsets) return best;
  const int64_t wide = ((a.back ? a.K : a.N) + 2 * kTileM - 1) / (2 * kTileM);
  int64_t least = INT64_MAX;
  for (int bn = F8PairRing::bn; bn >= 64; bn -= 32) {
    const int64_t tiles = (a.R + bn - 1) / bn * wide, time = (tiles + kSms / 2 - 1) / (kSms / 2) * (265 + bn);
    if (time < least) {
      least = time;
      best = bn;
    }
  }
  return best;
}

}  // namespace

cudaError_t launch_fp8_matmul(const Fp8MatmulArgs& a, int inject_stall, cudaStream_t s) {
  F8KernelArgs args{a, inject_stall, F8Ring::bn};
  const int64_t ksteps = ((a.back ? a.N : a.K) + kF8StageK - 1) / kF8StageK, narrow = most_tiles(a, F8Ring::bn, kTileM);
  auto run = [&](bool pairs, int64_t tiles, int split) {
    if (a.out_dtype == QMOE_F32) return launch_f8<QMOE_F32>(args, pairs, tiles, split, s);
    if (a.out_dtype == QMOE_F16) return launch_f8<QMOE_F16>(args, pairs, tiles, split, s);
    return launch_f8<QMOE_BF16>(args, pairs, tiles, split, s);
  };
  const int64_t rows = a.offsets ? a.R / std::min<int64_t>(a.E, a.R) : a.R;   // of an expert, if they are spread evenly
  // tiles of 32 rows while they are all under way at once, or an expert has few rows
  // (us, narrow / pairs: 64 x 2048 x 2048 over all 7.7 / 7.4, 300 rows 13.5 / 8.0;
  // experts of 1536 x 2048, 2 rows each of 128 50.8 / 52.0, 16 of 64 38.9 / 39.1, 32
  // of 64 48.9 / 40.3; uneven spreads are not told apart: 4096 rows over 256 experts in
  // narrow tiles, even 133, half of them one expert's 157, all 65, where the dense
  // product of as many rows takes 15)
  if (narrow > kSms && rows >= 24) {
    args.bn = pair_rows(a);
    return run(true, most_tiles(a, args.bn, 2 * kTileM), 1);
  }
  // A tile's reduction over the CTAs of a cluster while there are CTAs without a
  // tile, at least two stages each, up to four: eight CTAs' parts take longer to add
  // up than four's to make (1 x 2048 x 2048 in 1, 2, 4, 8 parts: 7.8, 6.5, 5.9, 9.9 us).
  int split = 1;
  while (split < 4 && narrow * split * 2 <= kSms && split * 4 <= ksteps) split *= 2;
  return run(false, narrow, split);
}

}  // namespace qmoe
