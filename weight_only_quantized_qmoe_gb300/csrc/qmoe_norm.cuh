// What the forward and the backward of the block norms share (qmoe_norm.cu,
// qmoe_norm_grad.cu): the sums of a row, the ring of rows on their way, and
// the choice of a kernel by type, alignment and row length.
#pragma once

#include <algorithm>

#include "qmoe_ops.cuh"

namespace qmoe {

// Multiprocessors of the one GPU these kernels are built for: persistent CTAs
// are counted in them.
constexpr int kNormSms = 152;

// Sums of v over the threads of a row (blockDim.x of them: 8, 16 or whole
// warps; every thread of the block calls it).  `red` holds 2 x 16 x N floats
// and `turn` alternates between its halves: a half is written again only after
// the barrier of the sum in between, which its readers have passed.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* red, int& turn) {
  const int width = min((int)blockDim.x, 32);
#pragma unroll
  for (int i = 0; i < N; ++i)
    for (int o = width >> 1; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (blockDim.x <= 32) return;
  const int tid = threadIdx.y * blockDim.x + threadIdx.x, warp = tid >> 5;
  const int nw = blockDim.x >> 5, w0 = threadIdx.y * nw;
  float* half = red + turn * 16 * N;
  turn ^= 1;
  if ((tid & 31) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) half[i * 16 + warp] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float s = 0.f;
    for (int q = 0; q < nw; ++q) s += half[i * 16 + w0 + q];
    v[i] = s;
  }
}

// Rows on their way from memory.  With 16-byte rows a thread copies its own
// vectors of the next rows into shared memory (cp.async) while it works on
// this one; nobody else reads them, so there is no barrier to wait at.
// Otherwise rows are loaded when they are used.
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Column of a thread's vector p, and whether the row has it.
template <int DT, bool VECTOR>
__device__ __forceinline__ int64_t norm_column(int p) {
  using F = Frag<DT, VECTOR>;
  return F::first(threadIdx.x) + p * F::step(blockDim.x);
}

// The weights or the channel gate of a thread's columns, or ones.
template <int DT, bool VECTOR>
__device__ __forceinline__ void load_columns(const void* p, int64_t c, int64_t H, float (&v)[Frag<DT, VECTOR>::n]) {
  if (p) {
    Frag<DT, VECTOR> f;
    f.load(p, 0, c, H, blockDim.x);
    f.get(v);
  } else {
#pragma unroll
    for (int i = 0; i < Frag<DT, VECTOR>::n; ++i) v[i] = 1.f;
  }
}

inline bool norm_vec(const NormArgs& a) {
  const void* whole[] = {a.w_post, a.w_pre, a.r, a.h, a.dx, a.d_o};
  for (const void* p : whole)
    if (p && !aligned16(p)) return false;
  if (a.gate && a.gate_kind != QMOE_GATE_TOKEN && !aligned16(a.gate)) return false;
  if (a.dgate && a.gate_kind == QMOE_GATE_FULL && !aligned16(a.dgate)) return false;
  return a.H % (16 / dtype_size(a.dtype)) == 0 && rows_aligned16(a.x, a.ld_x, a.dtype) &&
         rows_aligned16(a.o, a.ld_o, a.dtype) && rows_aligned16(a.dr, a.ld_dr, a.dtype) &&
         rows_aligned16(a.dh, a.ld_dh, a.dtype) &&
         (a.gate_kind != QMOE_GATE_FULL || rows_aligned16(a.gate, a.ld_gate, a.dtype));
}
// Elements of a thread's fragment.
inline int norm_frag(int dtype, bool vec) { return vec && dtype != QMOE_F32 ? 8 : 4; }
// Fragments a thread holds of a row.
inline int norm_vpt(int64_t H, int frag, int tpr) {
  int v = 1;
  while ((int64_t)v * frag * tpr < H) v *= 2;
  return v;
}

// Calls f(type, 16-byte accesses?, fragments of a thread).
template <int DT, bool VECTOR, typename F>
cudaError_t by_vpt(int vpt, F&& f) {
  using D = std::integral_constant<int, DT>;
  using V = std::integral_constant<bool, VECTOR>;
  switch (vpt) {
    case 1: return f(D{}, V{}, std::integral_constant<int, 1>{});
    case 2: return f(D{}, V{}, std::integral_constant<int, 2>{});
    case 4: return f(D{}, V{}, std::integral_constant<int, 4>{});
    default: break;
  }
  if constexpr (Frag<DT, VECTOR>::n == 4) {
    if (vpt == 8) return f(D{}, V{}, std::integral_constant<int, 8>{});
  }
  return cudaErrorInvalidValue;
}
template <typename F>
cudaError_t by_norm(int dtype, bool vec, int vpt, F&& f) {
  if (dtype == QMOE_F32) return vec ? by_vpt<QMOE_F32, true>(vpt, f) : by_vpt<QMOE_F32, false>(vpt, f);
  if (dtype == QMOE_F16) return vec ? by_vpt<QMOE_F16, true>(vpt, f) : by_vpt<QMOE_F16, false>(vpt, f);
  return vec ? by_vpt<QMOE_BF16, true>(vpt, f) : by_vpt<QMOE_BF16, false>(vpt, f);
}

}  // namespace qmoe
