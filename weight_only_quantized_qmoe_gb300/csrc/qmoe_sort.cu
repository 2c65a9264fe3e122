// Tokens sorted by expert and back, with weights applied, and the gradients.
//
//   sort:     route r = t * k + j goes to expert ids[t, j]; pos[r] is its row
//             in the stable order by expert, perm the inverse, offsets[e] the
//             first row of expert e.  A route whose id is outside [0, E) is
//             dropped: pos -1, no row; rows past offsets[E] have perm -1.
//   dispatch: xs[pos[t, j]] = x[t]
//   combine:  out[t] = sum_j w[t, j] * y[pos[t, j]], in slot order, fp32
//   their gradients: dx[t] = sum_j dxs[pos[t, j]] (combine with unit weights);
//             dy[pos[t, j]] = w[t, j] * dout[t], dw[t, j] = <dout[t], y[pos[t, j]]>
//
// All of them run in token order: a token's row is read (or written) once and
// its k rows in expert order once each, so every row crosses the memory
// exactly once, whole.  No atomics: every result has one owner and one order.
// Bound by those bytes (bf16, 4096 tokens to 8 experts, rows of 4096: dispatch
// 45 us, 6.7 TB/s; combine 56 us, 5.4 TB/s; 6001 to 4, rows of 2880: gradient of
// the combine 50 us, 6.2 TB/s).
#include <cooperative_groups.h>

#include <algorithm>

#include "qmoe_ops.cuh"

namespace cg = cooperative_groups;

namespace qmoe {

// ----------------------------------------------------------------------------
// Sort
// ----------------------------------------------------------------------------
// One launch of one cluster: every warp owns a contiguous run of routes, counts
// it per expert in shared memory, the counts of all warps of all CTAs become
// first rows (distributed shared memory between the CTAs), and the warps walk
// their runs again in order.  No workspace and no second launch: at the sizes
// a layer sorts (up to some 10^5 routes) the time is latency, not bandwidth.
constexpr int kSortCluster = 8;

template <typename ID>
__global__ void __launch_bounds__(1024) expert_sort_kernel(const SortArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), c = (int)cluster.block_rank();
  const int W = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = a.E, pitch = E | 1;    // an odd pitch: a warp reads a column of counters without bank conflicts
  extern __shared__ int sort_smem[];
  int* cnt = sort_smem;                 // [W][pitch]: counts, then the warp's next rank within the CTA
  int* tot = cnt + (size_t)W * pitch;   // [E]: this CTA's counts (read by the other CTAs)
  int* base = tot + E;                  // [E]: routes of earlier CTAs
  int* off = base + E;                  // [E + 1]: all counts, then first rows
  for (int i = threadIdx.x; i < W * pitch; i += blockDim.x) cnt[i] = 0;
  op_begin();
  __syncthreads();

  const ID* ids = static_cast<const ID*>(a.ids);
  const bool dense = a.ld_ids == a.k;
  auto id_of = [&](int64_t r) -> int {
    const ID v = ids[dense ? r : (r / a.k) * a.ld_ids + r % a.k];
    return v >= 0 && v < (ID)E ? (int)v : -1;
  };
  // routes [r0, r1) of this warp, a multiple of 32 each but the last
  const int64_t per = ((a.R + (int64_t)C * W - 1) / ((int64_t)C * W) + 31) / 32 * 32;
  const int64_t r0 = std::min<int64_t>(a.R, per * ((int64_t)c * W + warp)), r1 = std::min<int64_t>(a.R, r0 + per);
  int* mine = cnt + (size_t)warp * pitch;
  constexpr int U = 4;                  // ids in flight per lane
  int e[U];
  auto fetch = [&](int64_t b) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = b + 32 * u + lane;
      e[u] = r < r1 ? id_of(r) : -1;
    }
  };
  for (int64_t b = r0; b < r1; b += 32 * U) {
    fetch(b);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (e[u] >= 0) atomicAdd(mine + e[u], 1);
  }
  __syncthreads();
  // a warp takes an expert at a time, a lane the counter of a warp: counts
  // become ranks within the CTA
  for (int x = warp; x < E; x += W) {
    const int n = lane < W ? cnt[(size_t)lane * pitch + x] : 0;
    int run = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += up;
    }
    if (lane < W) cnt[(size_t)lane * pitch + x] = run - n;
    if (lane == 31) tot[x] = run;
  }
  if (C > 1) cluster.sync();
  else __syncthreads();
  for (int x = threadIdx.x; x < E; x += blockDim.x) {
    int before = 0, all = 0;
    if (C > 1) {
#pragma unroll
      for (int q = 0; q < kSortCluster; ++q) {
        const int n = cluster.map_shared_rank(tot, q)[x];
        before += q < c ? n : 0;
        all += n;
      }
    } else {
      all = tot[x];
    }
    base[x] = before;
    off[x] = all;
  }
  __syncthreads();
  if (warp == 0) {
    // exclusive scan of the expert counts: a contiguous run of experts a lane
    const int per_lane = (E + 31) / 32, e0 = std::min(E, lane * per_lane), e1 = std::min(E, e0 + per_lane);
    int sum = 0;
    for (int x = e0; x < e1; ++x) sum += off[x];
    int run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += up;
    }
    int first = run - sum;
    for (int x = e0; x < e1; ++x) {
      const int n = off[x];
      off[x] = first;
      first += n;
    }
    if (lane == 31) off[E] = run;
  }
  __syncthreads();
  const int used = off[E];
  if (c == 0)
    for (int x = threadIdx.x; x <= E; x += blockDim.x) a.offsets[x] = off[x];
  // rows without a route
  for (int64_t i = used + (int64_t)c * blockDim.x + threadIdx.x; i < a.R; i += (int64_t)C * blockDim.x) a.perm[i] = -1;

  const bool again = r1 - r0 > 32 * U;  // else the ids are still in registers
  for (int64_t b = r0; b < r1; b += 32 * U) {
    if (again) fetch(b);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = b + 32 * u + lane;
      // lanes with the same expert take consecutive rows in lane order
      const unsigned peers = __match_any_sync(0xffffffffu, e[u]);
      const int rank = __popc(peers & ((1u << lane) - 1u));
      int p = -1;
      if (e[u] >= 0) p = off[e[u]] + base[e[u]] + mine[e[u]] + rank;
      __syncwarp();
      if (e[u] >= 0 && rank == 0) mine[e[u]] += __popc(peers);
      __syncwarp();
      if (r < r1) {
        a.pos[r] = p;
        if (p >= 0) a.perm[p] = (int)r;
      }
    }
  }
  if (C > 1) cluster.sync();   // no CTA leaves while another may still read its counts
}

// Shared memory of W warps: their counters, three values an expert and the end.
static constexpr size_t sort_shared(int W, int E) { return ((size_t)W * (E | 1) + 3 * (size_t)E + 1) * sizeof(int); }

cudaError_t launch_expert_sort(const SortArgs& a, cudaStream_t s) {
  // One CTA for a few routes, else a cluster of eight, whose two barriers cost
  // about a microsecond (us, one / eight CTAs: 256 routes 6.0 / 7.0, 512 6.2 /
  // 6.1, 4096 to 256 experts 8.9 / 6.6, 32768 to 64 35.4 / 8.4).
  const int C = a.R <= 256 ? 1 : kSortCluster;
  const int64_t passes = (a.R + 32 * C - 1) / (32 * C);
  const int W = (int)std::max<int64_t>(1, std::min<int64_t>(32, passes));
  const size_t smem = sort_shared(W, a.E);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)C, 1, 1};
  cfg.gridDim = dim3(C);
  cfg.blockDim = dim3(32 * W);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 2 : 1;   // a single CTA is its own cluster
  auto run = [&](auto kern) {
    const cudaError_t err = allow_shared(kern, smem, (int)sort_shared(32, kSortMaxExperts));
    if (err != cudaSuccess) return err;
    return cudaLaunchKernelEx(&cfg, kern, a);
  };
  return a.id_bytes == 8 ? run(expert_sort_kernel<long long>) : run(expert_sort_kernel<int>);
}

// ----------------------------------------------------------------------------
// Row copies and sums
// ----------------------------------------------------------------------------
// A row takes blockDim.x threads, blockDim.y rows a CTA (row_shape).  Rows are
// held as they are in memory until they are added, and the slots of a token
// (SLOTS of them, 1 to 8, the least that holds top_k; more than 8 in turns) are
// in flight together: with eight rows unpacked to 32 bits ahead of their use
// a thread took 128 registers and the sum ran at a quarter of the bandwidth.
// Rows pass by the L1, as each is read once (sum of 4096 x 8 rows of 4096: 56 us,
// through it 60).

// Threads of a row at most, and CTAs a multiprocessor the registers are cut
// for: many short CTAs, whose loads, sums and stores fall at different times
// (gradient of 6001 x 4 rows of 2880: 56 us with 128 threads and 8 CTAs, 60
// with 256 and 4, 91 with 256 and 2; eight slots need 85 registers, 4096 x 8
// rows of 4096: 95 us with 6 CTAs, 107 with 8).
constexpr int kRowThreads = 128;
constexpr int row_ctas(int slots) { return slots == 8 ? 6 : 8; }

// The row of a slot, -1 where it has none.
__device__ __forceinline__ int slot_row(const RowsArgs& a, int p) { return p < a.T * a.k ? p : -1; }

// Rows offsets[E] .. T * k - 1 of dst, which no route fills: zeros, spread
// over the rows of the grid.
template <int DT, bool VECTOR>
__device__ __forceinline__ void zero_unused_rows(const RowsArgs& a, int64_t t) {
  using F = Frag<DT, VECTOR>;
  const int H = (int)a.H;
  const int64_t R = a.T * a.k, used = max(a.offsets[a.E], 0);
  float z[F::n];
#pragma unroll
  for (int i = 0; i < F::n; ++i) z[i] = 0.f;
  F f;
  f.set(z);
  for (int64_t i = used + t; i < R; i += a.T)
    for (int c = F::first(threadIdx.x); c < H; c += F::step(blockDim.x))
      f.store(static_cast<typename ElemT<DT>::t*>(a.dst) + i * a.H + c, H - c, blockDim.x);
}

template <int DT, bool VECTOR>
__global__ void __launch_bounds__(kRowThreads) dispatch_kernel(const RowsArgs a) {
  op_begin();
  using F = Frag<DT, VECTOR>;
  const int H = (int)a.H;
  const int64_t t = blockIdx.x * (int64_t)blockDim.y + threadIdx.y;
  if (t >= a.T) return;
  const int* pos = a.pos + t * a.k;
  for (int c = F::first(threadIdx.x); c < H; c += F::step(blockDim.x)) {
    F f;
    f.load_once(static_cast<const typename ElemT<DT>::t*>(a.src) + t * a.ld_src + c, H - c, blockDim.x);
    for (int j = 0; j < a.k; ++j) {
      const int64_t p = slot_row(a, pos[j]);
      if (p >= 0) f.store(static_cast<typename ElemT<DT>::t*>(a.dst) + p * a.H + c, H - c, blockDim.x);
    }
  }
  zero_unused_rows<DT, VECTOR>(a, t);
}

template <int DT, bool VECTOR, int SLOTS>
__global__ void __launch_bounds__(kRowThreads, row_ctas(SLOTS)) combine_kernel(const RowsArgs a) {
  op_begin();
  using F = Frag<DT, VECTOR>;
  const int H = (int)a.H;
  const int64_t t = blockIdx.x * (int64_t)blockDim.y + threadIdx.y;
  if (t >= a.T) return;
  const int* pos = a.pos + t * a.k;
  for (int c = F::first(threadIdx.x); c < H; c += F::step(blockDim.x)) {
    float acc[F::n];
#pragma unroll
    for (int i = 0; i < F::n; ++i) acc[i] = 0.f;
    for (int j0 = 0; j0 < a.k; j0 += SLOTS) {
      F f[SLOTS];
      float w[SLOTS];
      int p[SLOTS];
#pragma unroll
      for (int u = 0; u < SLOTS; ++u) {
        p[u] = j0 + u < a.k ? slot_row(a, pos[j0 + u]) : -1;
        w[u] = a.w && j0 + u < a.k ? a.w[t * a.k + j0 + u] : 1.f;
      }
#pragma unroll
      for (int u = 0; u < SLOTS; ++u)
        if (p[u] >= 0) f[u].load_once(static_cast<const typename ElemT<DT>::t*>(a.src) + (int64_t)p[u] * a.ld_src + c, H - c, blockDim.x);
#pragma unroll
      for (int u = 0; u < SLOTS; ++u)
        if (p[u] >= 0) {
          float v[F::n];
          f[u].get(v);
#pragma unroll
          for (int i = 0; i < F::n; ++i) acc[i] = fmaf(w[u], v[i], acc[i]);
        }
    }
    F out;
    out.set(acc);
    out.store(static_cast<typename ElemT<DT>::t*>(a.dst) + t * a.H + c, H - c, blockDim.x);
  }
}

// Sums v[0 .. N - 1] over the 32 lanes of a warp: lane l ends with the sum of
// entry slot(l) in v[0].  Each of the first steps halves what a lane still
// carries, so N sums take N + 4 - log2(N) exchanges or fewer instead of 5 N.
template <int N>
__device__ __forceinline__ int warp_sums(float (&v)[N]) {
  const int lane = threadIdx.x & 31;
  int slot = 0, o = 16;
#pragma unroll
  for (int n = N / 2; n >= 1; n /= 2, o /= 2) {
    const bool up = lane & o;
    slot += up ? n : 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  for (; o >= 1; o /= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  return slot;
}

template <int DT, bool VECTOR, int SLOTS>
__global__ void __launch_bounds__(kRowThreads, row_ctas(SLOTS)) combine_grad_kernel(const RowsArgs a) {
  op_begin();
  using F = Frag<DT, VECTOR>;
  const int H = (int)a.H;
  __shared__ float part[kRowThreads / 32][SLOTS];
  const int64_t t = blockIdx.x * (int64_t)blockDim.y + threadIdx.y;
  const bool live = t < a.T;
  const int tid = threadIdx.y * blockDim.x + threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int* pos = a.pos + (live ? t : 0) * a.k;
  for (int j0 = 0; j0 < a.k; j0 += SLOTS) {
    int p[SLOTS];
    float w[SLOTS], dot[SLOTS];
#pragma unroll
    for (int u = 0; u < SLOTS; ++u) {
      p[u] = live && j0 + u < a.k ? slot_row(a, pos[j0 + u]) : -1;
      w[u] = p[u] >= 0 && a.w ? a.w[t * a.k + j0 + u] : 1.f;
      dot[u] = 0.f;
    }
    if (live) {
      for (int c = F::first(threadIdx.x); c < H; c += F::step(blockDim.x)) {
        F fg, f[SLOTS];
        fg.load_once(static_cast<const typename ElemT<DT>::t*>(a.src) + t * a.ld_src + c, H - c, blockDim.x);
        if (a.dw) {
#pragma unroll
          for (int u = 0; u < SLOTS; ++u)
            if (p[u] >= 0) f[u].load_once(static_cast<const typename ElemT<DT>::t*>(a.y) + (int64_t)p[u] * a.ld_y + c, H - c, blockDim.x);
        }
        float g[F::n];
        fg.get(g);
#pragma unroll
        for (int u = 0; u < SLOTS; ++u) {
          if (p[u] < 0) continue;
          float v[F::n];
          if (a.dw) {
            f[u].get(v);
#pragma unroll
            for (int i = 0; i < F::n; ++i) dot[u] = fmaf(g[i], v[i], dot[u]);
          }
          if (a.dst) {
#pragma unroll
            for (int i = 0; i < F::n; ++i) v[i] = w[u] * g[i];
            F out;
            out.set(v);
            out.store(static_cast<typename ElemT<DT>::t*>(a.dst) + (int64_t)p[u] * a.H + c, H - c, blockDim.x);
          }
        }
      }
    }
    if (!a.dw) continue;
    if (blockDim.x >= 32) {
      const int slot = warp_sums<SLOTS>(dot);
      if ((lane & (32 / SLOTS - 1)) == 0) part[warp][slot] = dot[0];
      __syncthreads();
      if (threadIdx.x < SLOTS) {
        float sum = 0.f;
        const int nw = blockDim.x >> 5, w0 = threadIdx.y * nw;
        for (int q = 0; q < nw; ++q) sum += part[w0 + q][threadIdx.x];
        if (live && j0 + (int)threadIdx.x < a.k) a.dw[t * a.k + j0 + threadIdx.x] = sum;
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int u = 0; u < SLOTS; ++u) {
        for (int o = blockDim.x >> 1; o > 0; o >>= 1) dot[u] += __shfl_xor_sync(0xffffffffu, dot[u], o);
        if (threadIdx.x == 0 && live && j0 + u < a.k) a.dw[t * a.k + j0 + u] = dot[u];
      }
    }
  }
  if (live && a.dst) zero_unused_rows<DT, VECTOR>(a, t);
}

// Calls f(type, 16-byte accesses?, slots in flight).
template <int DT, bool VECTOR, typename F>
static cudaError_t by_slots(int k, F&& f) {
  using D = std::integral_constant<int, DT>;
  using V = std::integral_constant<bool, VECTOR>;
  if (k <= 1) return f(D{}, V{}, std::integral_constant<int, 1>{});
  if (k <= 2) return f(D{}, V{}, std::integral_constant<int, 2>{});
  if (k <= 4) return f(D{}, V{}, std::integral_constant<int, 4>{});
  return f(D{}, V{}, std::integral_constant<int, 8>{});
}
// 16-byte accesses need every row of every operand on a 16-byte boundary and
// whole vectors a row; anything else moves element by element.
template <typename F>
static cudaError_t by_rows(const RowsArgs& a, F&& f) {
  const bool vec = a.H % (16 / dtype_size(a.dtype)) == 0 && rows_aligned16(a.src, a.ld_src, a.dtype) &&
                   rows_aligned16(a.y, a.ld_y, a.dtype) && rows_aligned16(a.dst, a.H, a.dtype);
  if (a.dtype == QMOE_F32) return vec ? by_slots<QMOE_F32, true>(a.k, f) : by_slots<QMOE_F32, false>(a.k, f);
  if (a.dtype == QMOE_F16) return vec ? by_slots<QMOE_F16, true>(a.k, f) : by_slots<QMOE_F16, false>(a.k, f);
  return vec ? by_slots<QMOE_BF16, true>(a.k, f) : by_slots<QMOE_BF16, false>(a.k, f);
}
template <int DT, bool VECTOR>
static RowShape rows_of(const RowsArgs& a, dim3* grid) {
  const RowShape r = row_shape(a.H, Frag<DT, VECTOR>::n, kRowThreads);
  *grid = dim3((unsigned)((a.T + r.rpb - 1) / r.rpb));
  return r;
}

cudaError_t launch_dispatch(const RowsArgs& a, cudaStream_t s) {
  return by_rows(a, [&](auto dt, auto vec, auto) {
    dim3 grid;
    const RowShape r = rows_of<dt, vec>(a, &grid);
    return launch_op(dispatch_kernel<dt, vec>, grid, dim3(r.tpr, r.rpb), 0, s, a);
  });
}

cudaError_t launch_combine(const RowsArgs& a, cudaStream_t s) {
  return by_rows(a, [&](auto dt, auto vec, auto slots) {
    dim3 grid;
    const RowShape r = rows_of<dt, vec>(a, &grid);
    return launch_op(combine_kernel<dt, vec, slots>, grid, dim3(r.tpr, r.rpb), 0, s, a);
  });
}

cudaError_t launch_combine_grad(const RowsArgs& a, cudaStream_t s) {
  return by_rows(a, [&](auto dt, auto vec, auto slots) {
    dim3 grid;
    const RowShape r = rows_of<dt, vec>(a, &grid);
    return launch_op(combine_grad_kernel<dt, vec, slots>, grid, dim3(r.tpr, r.rpb), 0, s, a);
  });
}

}  // namespace qmoe
