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
// same codes read along M), its N side up to BN rows of A; a ring stage holds 128
// reduction values of both, 128-byte rows copied by TMA.
//   warp 0    TMA producer (one elected lane)
//   warp 1    MMA issuer: scales to TMEM, then four K = 32 MMAs a stage
//   warp 2    scales of A's rows: four bytes a row by cp.async (512 values' worth)
//   warp 3    scale of the weight block: one byte, spread over 512
//   warps 4-11 epilogue: TMEM columns to rows of the output
// Two accumulators of BN columns alternate, so the epilogue of one tile runs
// under the MMAs of the next.  CTAs are persistent over the (expert, row tile,
// weight tile) list, which every CTA derives from the device offsets.  Where
// there are few tiles, the CTAs of a cluster share a tile's reduction and add up
// their parts in a fixed order.
//
// Every wait is bounded; a timeout aborts all roles, drains what is in
// flight, frees TMEM and is reported by qmoe_op_poll_status.
#include "qmoe_tile.cuh"

namespace qmoe {

constexpr int kF8StageK = 128;                 // values along the reduction a stage: one swizzle atom
constexpr int kF8BoxRows = 32;                 // rows of A a copy where a tile is not full
constexpr int kF8Threads = 128 + 32 * kEpiWarps;
constexpr long long kF8DrainPolls = 4096;      // parked polls (about 4 ms) a copy in flight is given to land

template <int BN>
struct F8Ring {
  static constexpr int stages = BN == 192 ? 5 : 10;
  static constexpr int groups = (BN + 127) / 128;                 // 128-row scale groups of A
  static constexpr int w_bytes = kTileM * kF8StageK;
  static constexpr int a_bytes = BN * kF8StageK;
  static constexpr int sfw_bytes = 512;
  static constexpr int sfa_bytes = 512 * groups;
  static constexpr int w_off = 0;
  static constexpr int a_off = w_off + stages * w_bytes;
  static constexpr int sfw_off = a_off + stages * a_bytes;
  static constexpr int sfa_off = sfw_off + stages * sfw_bytes;
  static constexpr int bar_off = sfa_off + stages * sfa_bytes;
  static constexpr int tp_off = bar_off + 512;                    // first row tile and first row of each expert
  static constexpr int total = tp_off + 2 * (kSortMaxExperts + 2) * 4;
  // TMEM columns: two accumulators, then per stage the scales of W and A
  static constexpr int sf_col0 = 2 * BN;
  static constexpr int sf_cols = 4 + 4 * groups;
  static constexpr int tmem_cols = sf_col0 + stages * sf_cols <= 256 ? 256 : 512;
  static_assert(sf_col0 + stages * sf_cols <= tmem_cols, "TMEM columns");
  static_assert(total + 1024 <= 227 * 1024, "shared memory");
  static_assert(a_bytes % 1024 == 0, "swizzle atoms");
  static_assert(BN * kTileM * 4 <= stages * w_bytes || BN == 192, "a partial tile fits the ring");
};

// One stage, issued by one elected lane: the scales of W and of A's row groups
// to TMEM, up to four K = 32 MMAs, the commit that frees the stage.
template <int GROUPS, int MC>
__device__ __forceinline__ void f8_stage_elect(uint32_t d, uint64_t w, uint64_t wstep, uint64_t a, uint32_t idesc, uint32_t sf,
                                               uint64_t sw, uint64_t sa, uint32_t acc, int nk, uint64_t* empty) {
  static_assert(GROUPS == 1 || GROUPS == 2, "row groups of A");
  asm volatile(
      "{\n\t.reg .pred e, p0, p1, q1, q2, q3, g2;\n\t"
      ".reg .b32 t1, t2;\n\t.reg .b64 x1, y1, y2, y3, z1, z2, z3;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p0, %8, 0;\n\tsetp.eq.b32 p1, %8, %8;\n\t"
      "setp.gt.and.s32 q1, %9, 1, e;\n\tsetp.gt.and.s32 q2, %9, 2, e;\n\tsetp.gt.and.s32 q3, %9, 3, e;\n\t"
      "setp.gt.and.s32 g2, %10, 1, e;\n\t"
      "add.u32 t1, %5, 4;\n\tadd.u32 t2, %5, 8;\n\tadd.u64 x1, %7, 32;\n\t"
      "add.u64 y1, %1, %2;\n\tadd.u64 y2, y1, %2;\n\tadd.u64 y3, y2, %2;\n\t"
      "add.u64 z1, %3, 2;\n\tadd.u64 z2, %3, 4;\n\tadd.u64 z3, %3, 6;\n\t"
      "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%5], %6;\n\t"
      "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [t1], %7;\n\t"
      "@g2 tcgen05.cp.cta_group::1.32x128b.warpx4 [t2], x1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %3, %4, [%5], [t1], p0;\n\t"
      "@q1 tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], y1, z1, %4, [%5], [t1], p1;\n\t"
      "@q2 tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], y2, z2, %4, [%5], [t1], p1;\n\t"
      "@q3 tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], y3, z3, %4, [%5], [t1], p1;\n\t}" ::"r"(d),
      "l"(w), "l"(wstep), "l"(a), "r"(idesc), "r"(sf), "l"(sw), "l"(sa), "r"(acc), "r"(nk), "n"(GROUPS)
      : "memory");
  if constexpr (MC > 1) tc_commit_pair_elect(empty);
  else tc_commit_elect(empty);
}

// Instruction descriptor, kind::mxf8f6f4: both operands E4M3, scales E8M0, M =
// 128; W along K, or along M (bit 15).  The scale ids (bits 29-30 and 4-5) name
// the byte of a 32-bit scale word.
__device__ __forceinline__ uint32_t idesc_mxf8(int N, int back) {
  return ((uint32_t)back << 15) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(kTileM >> 7) << 27);
}

struct F8KernelArgs {
  Fp8MatmulArgs a;
  int inject_stall;
};

// SPLIT: a cluster shares each tile's reduction, and there is one tile a cluster
// at most.  MC = 2: the CTAs of a pair take neighbouring weight rows with the
// same rows of A; each loads half of the latter and sends it to both.
template <int BN, int OUT, bool SPLIT, int MC>
__global__ void __launch_bounds__(kF8Threads, 1)
    fp8_matmul_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_a32,
                      const __grid_constant__ CUtensorMap map_w, const F8KernelArgs args) {
  using RG = F8Ring<BN>;
  using T = typename ElemT<OUT>::t;
  constexpr int S = RG::stages;
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
      mbar_init(&empty[i], MC);
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
  if constexpr (MC > 1) cluster_sync_all();   // the other CTA's barriers are there
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const int inner = a.back ? a.N : a.K, width = a.back ? a.K : a.N;   // of A's rows, of the output's
  const int ntw = (width + MC * kTileM - 1) / (MC * kTileM);   // of the CTAs that go together
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
  const int mc = MC > 1 ? blockIdx.x % MC : 0;   // this CTA in its pair
  if constexpr (MC > 1) {
    first = blockIdx.x / MC;
    stride = gridDim.x / MC;
  }
  const int ks0 = (int)((int64_t)ksteps * rank / ranks), ks1 = (int)((int64_t)ksteps * (rank + 1) / ranks);
  auto tile_of = [&](int tile, int& n0) {
    const int mt = tile / ntw;
    n0 = ((tile - mt * ntw) * MC + mc) * kTileM;
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
      // the rows in one copy if they are many, else in copies of 32
      const int boxes = (t.rows + kF8BoxRows - 1) / kF8BoxRows;
      for (int ks = ks0; ks < ks1; ++ks, ++it) {
        const int s = it % S;
        ok = wait_or_abort(&empty[s], ((it / S) & 1) ^ 1, a.wait, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        mbar_arrive_expect_tx_elect(&full[s], (uint32_t)(boxes * kF8BoxRows * kF8StageK + RG::w_bytes));
        // Test hook: the first stage's barrier is armed, its copies are never issued.
        if (args.inject_stall && it == 0) continue;
        uint8_t* da = smem + RG::a_off + s * RG::a_bytes;
        if constexpr (MC > 1) {
          if (boxes == BN / kF8BoxRows)
            tma_3d_pair_elect(da + mc * (BN / MC) * kF8StageK, &map_a, ks * kF8StageK, t.start + mc * (BN / MC), 0, &full[s]);
          else
            for (int b = mc; b < boxes; b += MC)
              tma_3d_pair_elect(da + b * kF8BoxRows * kF8StageK, &map_a32, ks * kF8StageK, t.start + b * kF8BoxRows, 0, &full[s]);
        } else if (boxes == BN / kF8BoxRows) {
          tma_3d_elect(da, &map_a, ks * kF8StageK, t.start, 0, &full[s]);
        } else {
          for (int b = 0; b < boxes; ++b)
            tma_3d_elect(da + b * kF8BoxRows * kF8StageK, &map_a32, ks * kF8StageK, t.start + b * kF8BoxRows, 0, &full[s]);
        }
        uint8_t* dw = smem + RG::w_off + s * RG::w_bytes;
        if (a.back) tma_3d_elect(dw, &map_w, n0, ks * kF8StageK, t.e, &full[s]);
        else tma_3d_elect(dw, &map_w, ks * kF8StageK, n0, t.e, &full[s]);
      }
    }
    if (!ok) {
      // After a wait that ran out the copies in flight must land before the CTA
      // leaves: wait for the last stages' barriers, with a limit, as the scale
      // warps may have left them short.
      const WaitCfg drain{a.wait.status, kF8DrainPolls};
      for (int i = it > S ? it - S : 0; i < it; ++i) mbar_wait_bounded(&full[i % S], (i / S) & 1, drain);
    }
  } else if (warp == 2) {
    // ---------------- scales of A's rows ----------------
    // Row 32 j + lane of a 128-row group goes to bytes lane * 16 + j * 4 of its
    // chunk: the four bytes of 512 values, of which a stage's MMAs name one.
    const uint32_t dst0 = smem_u32(smem + RG::sfa_off) + lane * 16;
    int it = 0;
    bool ok = true;
    for (int tile = first; tile < total && ok; tile += stride) {
      int n0;
      const RowTile t = tile_of(tile, n0);
      if (t.e == a.E) continue;
      const int left = (int)a.R - t.start - lane;   // row 32 j exists: 32 j < left
      for (int ks = ks0; ks < ks1; ++ks, ++it) {
        const int s = it % S;
        ok = wait_or_abort(&empty[s], ((it / S) & 1) ^ 1, a.wait, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint8_t* src = a.a_scales + ((size_t)(ks >> 2) * a.R + t.start + lane) * 4;
        const uint32_t dst = dst0 + s * RG::sfa_bytes;
#pragma unroll
        for (int j = 0; j < BN / 32; ++j) {
          const bool real = 32 * j < left;
          cp_async4_or_zero(dst + (j / 4) * 512 + (j & 3) * 4, real ? src + j * 128 : a.a_scales, real ? 4 : 0);
        }
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
      const int ob = min(n0, width - 1) / kTileM;
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
    for (int tile = first; tile < real && ok; tile += stride, ++tc) {
      int n0;
      const RowTile t = tile_of(tile, n0);
      const uint32_t idesc0 = idesc_mxf8((t.rows + 15) & ~15, a.back);
      const int ab = tc & 1;
      ok = spin_or_abort(&acc_empty[ab], ((tc >> 1) & 1) ^ 1, a.wait, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t dacc = tmem + ab * BN;
      int ks = ks0;
      while (ks < ks1 && ok) {
#pragma unroll
        for (int u = 0; u < S; ++u) {
          if (u == st && ks < ks1 && ok) {
            if (!warp_test_wait(&full[u], ph)) {
              ok = spin_or_abort(&full[u], ph, a.wait, abort_flag);
              ok = __all_sync(0xffffffffu, ok);
            }
            if (ok) {
              tc_fence_after();
              fence_proxy_async_smem();   // the scales were written through the generic proxy
              f8_stage_elect<RG::groups, MC>(dacc, wdesc0 + (uint64_t)((u * RG::w_bytes) >> 4), wstep,
                                         adesc0 + (uint64_t)((u * RG::a_bytes) >> 4),
                                         idesc0 | (uint32_t)(ks & 3) << 29 | (uint32_t)(ks & 3) << 4, tmem + RG::sf_col0 + u * RG::sf_cols,
                                         swdesc0 + (uint64_t)((u * RG::sfw_bytes) >> 4), sadesc0 + (uint64_t)((u * RG::sfa_bytes) >> 4),
                                         ks != ks0 ? 1u : 0u, ks + 1 < ksteps ? 4 : tail, &empty[u]);
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
      const int ab = tc & 1;
      ok = wait_or_abort(&acc_full[ab], (tc >> 1) & 1, a.wait, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + ab * BN;
      if constexpr (SPLIT) put_partial(acc, reinterpret_cast<float*>(smem + RG::w_off), q, t.rows, half);   // the ring is empty
      else store_tile<OUT>(acc, out, a.ld_out, t.rows, in, half);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[ab]);
      ++tc;
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
  if constexpr (MC > 1) {
    __syncwarp();
    cluster_sync_all();   // no CTA leaves while the other may still send to it
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, RG::tmem_cols);
}

// ----------------------------------------------------------------------------
// Host side
// ----------------------------------------------------------------------------
namespace {

template <int BN, int OUT>
cudaError_t launch_f8(const F8KernelArgs& args, int64_t tiles, int split, bool pairs, cudaStream_t s) {
  const Fp8MatmulArgs& a = args.a;
  const int64_t inner = a.back ? a.N : a.K;
  CUtensorMap map_a, map_a32, map_w;
  constexpr auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  if (!encode_tiles(&map_a, u8, 1, a.a_codes, inner, a.R, 1, fp8_pitch(inner), pairs ? BN / 2 : BN) ||
      !encode_tiles(&map_a32, u8, 1, a.a_codes, inner, a.R, 1, fp8_pitch(inner), kF8BoxRows) ||
      !encode_tiles(&map_w, u8, 1, a.w_codes, a.K, a.N, a.E, fp8_pitch(a.K), kTileM))
    return cudaErrorInvalidValue;
  constexpr int smem = F8Ring<BN>::total + 1024;   // + alignment slack
  if constexpr (BN == 32)
    if (split > 1) return launch_tiles(fp8_matmul_kernel<BN, OUT, true, 1>, tiles * split, split, kF8Threads, smem, s, map_a, map_a32, map_w, args);
  if constexpr (BN == 192)
    if (pairs) return launch_tiles(fp8_matmul_kernel<BN, OUT, false, 2>, kSms, 2, kF8Threads, smem, s, map_a, map_a32, map_w, args);
  return launch_tiles(fp8_matmul_kernel<BN, OUT, false, 1>, std::min<int64_t>(tiles, kSms), 1, kF8Threads, smem, s, map_a, map_a32, map_w, args);
}

// Output tiles there can be at most (the device offsets decide how many there are).
int64_t most_tiles(const Fp8MatmulArgs& a, int bn) {
  const int64_t groups = a.offsets ? std::min<int64_t>((int64_t)a.E + 1, a.R) : 1;
  return (a.R / bn + groups) * (((a.back ? a.K : a.N) + kTileM - 1) / kTileM);
}

}  // namespace

cudaError_t launch_fp8_matmul(const Fp8MatmulArgs& a, int inject_stall, cudaStream_t s) {
  const F8KernelArgs args{a, inject_stall};
  const int64_t ksteps = ((a.back ? a.N : a.K) + kF8StageK - 1) / kF8StageK, narrow = most_tiles(a, 32);
  auto run = [&](auto bn, int64_t tiles, int split) {
    constexpr int BN = decltype(bn)::value;
    const bool pairs = BN == 192 && tiles > kSms && (a.back ? a.K : a.N) > kTileM;
    if (a.out_dtype == QMOE_F32) return launch_f8<BN, QMOE_F32>(args, tiles, split, pairs, s);
    if (a.out_dtype == QMOE_F16) return launch_f8<BN, QMOE_F16>(args, tiles, split, pairs, s);
    return launch_f8<BN, QMOE_BF16>(args, tiles, split, pairs, s);
  };
  const int64_t rows = a.offsets ? a.R / std::min<int64_t>(a.E, a.R) : a.R;   // of an expert, if they are spread evenly
  if (narrow > kSms && rows > 32) return run(std::integral_constant<int, 192>{}, most_tiles(a, 192), 1);
  // a tile's reduction over the CTAs of a cluster while there are CTAs without a
  // tile, at least two stages each
  int split = 1;
  while (split < 8 && narrow * split * 2 <= kSms && split * 4 <= ksteps) split *= 2;
  return run(std::integral_constant<int, 32>{}, narrow, split);
}

}  // namespace qmoe
