// What the forward and the backward of the block norms share (qmoe_norm.cu,
// qmoe_norm_grad.cu): the sum of a row, the rows on their way, the vectors over
// the columns, and the choice of a kernel by type, alignment and row length.
#pragma once

#include <algorithm>

#include "qmoe_ops.cuh"

namespace qmoe {

// Two fp32 values in one instruction.  The norms issue some thirty
// instructions a value even so, close to what a multiprocessor can issue in the
// time the value's bytes take.
__device__ __forceinline__ uint64_t bits2(float2 a) { return *reinterpret_cast<uint64_t*>(&a); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// The pairs of a fragment.
template <int DT, bool VECTOR>
__device__ __forceinline__ void get2(const Frag<DT, VECTOR>& f, float2 (&v)[Frag<DT, VECTOR>::n / 2]) {
  constexpr int N = Frag<DT, VECTOR>::n;
  float e[N];
  f.get(e);
#pragma unroll
  for (int i = 0; i < N / 2; ++i) v[i] = make_float2(e[2 * i], e[2 * i + 1]);
}
template <int DT, bool VECTOR>
__device__ __forceinline__ void set2(Frag<DT, VECTOR>& f, const float2 (&v)[Frag<DT, VECTOR>::n / 2]) {
  constexpr int N = Frag<DT, VECTOR>::n;
  float e[N];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    e[2 * i] = v[i].x;
    e[2 * i + 1] = v[i].y;
  }
  f.set(e);
}

// Sum of v over the threads of a row (blockDim.x of them: 8, 16 or whole
// warps; every thread of the block calls it).  `red` holds 2 x 16 floats and
// `turn` alternates between its halves: a half is written again only after the
// barrier of the sum in between, which its readers have passed.
__device__ __forceinline__ float row_sum(float v, float* red, int& turn) {
  const int width = min((int)blockDim.x, 32);
  for (int o = width >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (blockDim.x <= 32) return v;
  const int tid = threadIdx.y * blockDim.x + threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nw = blockDim.x >> 5, w0 = threadIdx.y * nw;   // at most 16 warps
  float* half = red + turn * 16;
  turn ^= 1;
  if (lane == 0) half[warp] = v;
  __syncthreads();
  v = lane < nw ? half[w0 + lane] : 0.f;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return __shfl_sync(0xffffffffu, v, 0);
}

// What a thread needs to know of its place: the elements from its fragment p
// to the row's end (none: it has no such fragment), and where that fragment
// lies behind its first one, in memory and in a ring.
template <int DT, bool VECTOR>
struct Place {
  using F = Frag<DT, VECTOR>;
  int threads, left, step;
  uint32_t frag_bytes;   // the fragments p of all of a CTA's threads in a ring
  __device__ __forceinline__ explicit Place(int64_t H) {
    threads = blockDim.x;
    left = (int)H - F::first(threadIdx.x);
    step = F::step(threads);
    frag_bytes = blockDim.x * blockDim.y * 16;
  }
  __device__ __forceinline__ int left_of(int p) const { return left - p * step; }
  __device__ __forceinline__ bool has(int p) const { return left_of(p) > 0; }
};

// Whether rows can be copied ahead: 16 bytes at a time, or for 32-bit rows on
// any boundary 4 (cp.async knows no 2).
template <int DT, bool VECTOR>
constexpr bool kCopies = VECTOR || DT == QMOE_F32;

// The rows of one tensor as a thread sees them: its fragments of row after row
// of a CTA.  With a RING a thread copies its own fragments of the next rows into
// shared memory (cp.async) while it works on this one; nobody else reads them,
// so there is no barrier to wait at.  Otherwise they are loaded when they are
// used.
template <int DT, bool VECTOR, int VPT, bool RING>
struct Rows {
  using F = Frag<DT, VECTOR>;
  using T = typename ElemT<DT>::t;
  const T* next;      // this thread's first element of the row to be fetched next, without RING of the row in work
  int64_t step;       // elements from a CTA's row to its next
  uint32_t ring;      // shared address of this thread's first fragment in ring row 0
  bool there;

  // `slot` counts the tensors that are there: their fragments lie side by side
  // in a ring row.
  __device__ __forceinline__ Rows(const void* base, int64_t ld, int64_t row, int64_t rows, uint32_t ring0, int& slot,
                                  const Place<DT, VECTOR>& at) {
    there = base != nullptr;
    next = static_cast<const T*>(base) + row * ld + F::first(threadIdx.x);
    step = rows * ld;
    ring = ring0 + slot * VPT * at.frag_bytes + (threadIdx.y * blockDim.x + threadIdx.x) * 16;
    slot += there ? 1 : 0;
  }
  __device__ __forceinline__ void fetch(uint32_t row, const Place<DT, VECTOR>& at) const {   // `row`: offset of the ring row
    if (!there) return;
    if constexpr (VECTOR) {
#pragma unroll
      for (int p = 0; p < VPT; ++p)
        if (at.has(p))
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ring + row + p * at.frag_bytes), "l"(next + p * at.step)
                       : "memory");
    } else {
#pragma unroll
      for (int p = 0; p < VPT; ++p)
#pragma unroll
        for (int i = 0; i < F::n; ++i) {   // zeros past the row's end
          const bool in = i * at.threads < at.left_of(p);
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(ring + row + p * at.frag_bytes + 4 * i),
                       "l"(in ? next + p * at.step + i * at.threads : next), "r"(in ? 4 : 0)
                       : "memory");
        }
    }
  }
  __device__ __forceinline__ void advance() { next += step; }
  __device__ __forceinline__ void get(uint32_t row, int p, const Place<DT, VECTOR>& at, float2 (&v)[F::n / 2]) const {
    F f;
    if constexpr (RING && VECTOR) {
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(f.u.x), "=r"(f.u.y), "=r"(f.u.z), "=r"(f.u.w)
                   : "r"(ring + row + p * at.frag_bytes)
                   : "memory");
    } else if constexpr (RING) {
      asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(f.e[0]), "=f"(f.e[1]), "=f"(f.e[2]), "=f"(f.e[3])
                   : "r"(ring + row + p * at.frag_bytes)
                   : "memory");
    } else {
      f.load(next + p * at.step, at.left_of(p), at.threads);
    }
    get2(f, v);
  }
};
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A product of up to two vectors over the columns (weight, channel gate), ones
// where there are none.  It is the same for every row: a thread's only
// fragment stays in registers as fp32, two as they are in memory, more are
// loaded again (loaded for every row they came from the L2, time after time:
// the rings leave little of the L1).  SHARED: a thread keeps its fragments in
// shared memory, behind the ring, where the registers are needed otherwise.
template <int DT, bool VECTOR, int VPT, bool SHARED>
struct Columns {
  using F = Frag<DT, VECTOR>;
  using T = typename ElemT<DT>::t;
  static constexpr int N2 = F::n / 2;
  const T *a, *b;
  float2 held[VPT == 1 ? N2 : 1];
  F fa[VPT == 2 && !SHARED ? 2 : 1], fb[VPT == 2 && !SHARED ? 2 : 1];
  uint32_t place, part;   // SHARED: this thread's first fragment of `a`, bytes from there to the one of `b`
  __device__ __forceinline__ void compute(const F& x, const F& y, float2 (&v)[N2]) const {
    if (a) {
      get2(x, v);
    } else {
#pragma unroll
      for (int i = 0; i < N2; ++i) v[i] = both(1.f);
    }
    if (b) {
      float2 w[N2];
      get2(y, w);
#pragma unroll
      for (int i = 0; i < N2; ++i) v[i] = mul2(v[i], w[i]);
    }
  }
  // fragments of 16 bytes in shared memory, read by the thread that wrote them
  static __device__ __forceinline__ void keep(uint32_t to, const F& f) {
    static_assert(sizeof(F) == 16);
    const uint4 u = *reinterpret_cast<const uint4*>(&f);
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(u.x), "r"(u.y), "r"(u.z), "r"(u.w) : "memory");
  }
  static __device__ __forceinline__ void kept(uint32_t from, F& f) {
    uint4 u;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "r"(from)
                 : "memory");
    *reinterpret_cast<uint4*>(&f) = u;
  }
  // `shared`: where the fragments go if they are kept there, moved past them
  __device__ __forceinline__ Columns(const void* a_, const void* b_, const Place<DT, VECTOR>& at, uint32_t& shared) {
    place = shared + (threadIdx.y * blockDim.x + threadIdx.x) * 16;
    part = VPT * at.frag_bytes;
    a = a_ ? static_cast<const T*>(a_) + F::first(threadIdx.x) : nullptr;
    b = b_ ? static_cast<const T*>(b_) + F::first(threadIdx.x) : nullptr;
    if constexpr (SHARED) {
#pragma unroll
      for (int p = 0; p < VPT; ++p) {
        F x;
        if (a && at.has(p)) {
          x.load(a + p * at.step, at.left_of(p), at.threads);
          keep(place + p * at.frag_bytes, x);
        }
        if (b && at.has(p)) {
          x.load(b + p * at.step, at.left_of(p), at.threads);
          keep(place + part + p * at.frag_bytes, x);
        }
      }
      shared += part * (b ? 2 : 1);
    } else if constexpr (VPT <= 2) {
#pragma unroll
      for (int p = 0; p < VPT; ++p) {
        if (a && at.has(p)) fa[p].load(a + p * at.step, at.left_of(p), at.threads);
        if (b && at.has(p)) fb[p].load(b + p * at.step, at.left_of(p), at.threads);
      }
      if constexpr (VPT == 1) compute(fa[0], fb[0], held);
    }
  }
  __device__ __forceinline__ void get(int p, const Place<DT, VECTOR>& at, float2 (&v)[N2]) const {
    if constexpr (SHARED) {
      F x, y;
      if (a) kept(place + p * at.frag_bytes, x);
      if (b) kept(place + part + p * at.frag_bytes, y);
      compute(x, y, v);
    } else if constexpr (VPT == 1) {
#pragma unroll
      for (int i = 0; i < N2; ++i) v[i] = held[i];
    } else if constexpr (VPT == 2) {
      compute(fa[p], fb[p], v);
    } else {
      F x, y;
      if (a) x.load(a + p * at.step, at.left_of(p), at.threads);
      if (b) y.load(b + p * at.step, at.left_of(p), at.threads);
      compute(x, y, v);
    }
  }
};

// A thread's fragment p of an output row (`out`: the thread's first element).
template <int DT, bool VECTOR>
__device__ __forceinline__ void put(typename ElemT<DT>::t* out, int p, const Place<DT, VECTOR>& at,
                                    const float2 (&v)[Frag<DT, VECTOR>::n / 2]) {
  Frag<DT, VECTOR> f;
  set2(f, v);
  f.store(out + p * at.step, at.left_of(p), at.threads);
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
