// Operators around the expert layer: argument blocks and launchers shared by
// their entry points (qmoe_ops_api.cu) and their kernels (qmoe_choice.cu,
// qmoe_sort.cu, qmoe_mx4.cu, qmoe_mx4_gemm.cu, qmoe_fp8.cu, qmoe_fp8_gemm.cu,
// qmoe_wgrad.cu, qmoe_norm.cu).
#pragma once

#include <utility>

#include "qmoe_internal.cuh"

namespace qmoe {

// Multiprocessors of the one GPU these kernels are built for: persistent CTAs
// are counted in them.
constexpr int kSms = 152;

// Experts one sort handles (a warp's counters of all experts are held in
// shared memory, 32 warps of them).
constexpr int kSortMaxExperts = 1024;

struct SortArgs {
  const void* ids;          // int32 or int64 [T, k], rows ld_ids apart
  int id_bytes;
  int64_t ld_ids;
  int64_t R;                // T * k
  int k, E;
  int* perm;                // [R]
  int* pos;                 // [R]
  int* offsets;             // [E + 1]
};
cudaError_t launch_expert_sort(const SortArgs& a, cudaStream_t s);

// Row copies and sums between token order and expert order.
struct RowsArgs {
  const void* src;          // dispatch: x [T, H]; combine / gather: y [R, H]; combine_grad: dout [T, H]
  int64_t ld_src;
  const void* y;            // combine_grad: y [R, H]
  int64_t ld_y;
  const float* w;           // [T, k] or null (all ones)
  const int* pos;           // [T, k]
  const int* offsets;       // [E + 1] (rows from offsets[E] on are written as zeros), or null
  int64_t T, H;
  int k, E, dtype;
  void* dst;                // dispatch: xs [R, H]; combine: out [T, H]; combine_grad: dy [R, H] or null
  float* dw;                // combine_grad: [T, k] or null
};
cudaError_t launch_dispatch(const RowsArgs& a, cudaStream_t s);
cudaError_t launch_combine(const RowsArgs& a, cudaStream_t s);
cudaError_t launch_combine_grad(const RowsArgs& a, cudaStream_t s);

// Microscaled 4-bit rows.  Codes: [rows, 16 * nb] bytes, nb = ceil(cols / 32)
// blocks a row, element d in byte d / 2 (even d in the low half).  Scales:
// groups of `panel` rows, each [ceil(nb / 4), panel, 4] bytes.
__host__ __device__ inline size_t mx4_scale_offset(int64_t row, int64_t q, int64_t panel, int64_t nq) {
  const int64_t g = row / panel;
  return (size_t)(((g * nq + q) * panel + (row - g * panel)) * 4);
}

struct Mx4QuantArgs {
  const void* x;            // [rows, cols] (gated activation: [rows, 2 * cols], gate | up)
  int64_t ld_x;
  int64_t rows, cols;
  int dtype;
  ActParams act;            // act = -1: none
  const int* pos;           // [rows, k]: the output rows of a row, or null: row i to row i
  const int* offsets;       // with pos: rows from offsets[E] to rows * k are written as zeros
  int k, E;
  int64_t panel;            // rows of a scale panel of the output
  uint8_t* codes;
  uint8_t* scales;
};
cudaError_t launch_mx4_quantize(const Mx4QuantArgs& a, cudaStream_t s);

struct Mx4DequantArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t rows, cols, panel;
  int dtype;
  void* out;                // [rows, cols]
  int64_t ld_out;
};
cudaError_t launch_mx4_dequantize(const Mx4DequantArgs& a, cudaStream_t s);

struct Mx4MatmulArgs {
  const uint8_t* a_codes;   // [R, 16 * nb]
  const uint8_t* a_scales;  // one panel of R rows
  const uint8_t* w_codes;   // [E, N, 16 * nb]
  const uint8_t* w_scales;  // E panels of N rows
  const int* offsets;       // [E + 1], or null: one group of R rows
  int64_t R;
  int E, N, K;
  int out_dtype;
  void* out;                // [R, N]
  int64_t ld_out;
  WaitCfg wait;
};
cudaError_t launch_mx4_matmul(const Mx4MatmulArgs& a, int inject_stall, cudaStream_t s);

// The router.
struct ChoiceArgs {
  const void* logits;       // [T, E], rows ld apart
  int64_t ld;
  int dtype;
  const float* bias;        // [E] or null
  int64_t T;
  int E, k, scoring, groups, top_groups, best, renorm;
  float scale;
  int room;                 // values of a warp in shared memory (set by the launch,
  uint32_t group_magic;     // and so is this)
  int* ids;                 // [T, k]
  float* w;                 // [T, k]
  // gradient
  const float* dw;          // [T, k]
  void* dlogits;            // [T, E]
};
cudaError_t launch_choice(const ChoiceArgs& a, cudaStream_t s);
cudaError_t launch_choice_grad(const ChoiceArgs& a, cudaStream_t s);
constexpr int kChoiceMax = 32;   // slots, groups: a lane each

// 8-bit rows.  Codes: rows of fp8_pitch(cols) bytes.  Scales of rows: one panel
// [ceil(nb / 4), rows, 4] bytes a matrix, nb = ceil(cols / 128) (the layout of the
// 4-bit rows); of blocks: [ceil(rows / 128), nb] a matrix.
__host__ __device__ inline int64_t fp8_pitch(int64_t cols) { return (cols + 15) / 16 * 16; }

struct Fp8QuantArgs {
  const void* x;            // [rows, cols] (gated activation: [rows, 2 * cols], gate | up)
  int64_t ld_x;
  int64_t rows, cols;
  int dtype;
  ActParams act;            // act = -1: none
  const int* pos;           // as in Mx4QuantArgs
  const int* offsets;
  int k, E;
  int64_t panel;            // rows of a matrix
  int square;               // a scale per 128 x 128 block
  uint8_t* codes;
  uint8_t* scales;
};
cudaError_t launch_fp8_quantize(const Fp8QuantArgs& a, cudaStream_t s);

struct Fp8DequantArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t rows, cols, panel;
  int square, dtype;
  void* out;                // [rows, cols]
  int64_t ld_out;
};
cudaError_t launch_fp8_dequantize(const Fp8DequantArgs& a, cudaStream_t s);

struct Fp8MatmulArgs {
  const uint8_t* a_codes;   // [R, inner]
  const uint8_t* a_scales;  // one panel of R rows
  const uint8_t* w_codes;   // [E, N, K]
  const uint8_t* w_scales;  // blocks of each
  const int* offsets;       // [E + 1], or null: one group of R rows
  int64_t R;
  int E, N, K;
  int back;                 // 0: rows of K to rows of N; 1: rows of N to rows of K
  int out_dtype;
  void* out;                // [R, N or K]
  int64_t ld_out;
  WaitCfg wait;
};
cudaError_t launch_fp8_matmul(const Fp8MatmulArgs& a, int inject_stall, cudaStream_t s);

// Gradient of the experts' weights.
struct WgradArgs {
  const void* dy;           // [R, N]
  int64_t ld_dy;
  const void* x;            // [R, K]
  int64_t ld_x;
  const int* offsets;       // as above
  int64_t R;
  int E, N, K;
  int dtype, out_dtype;     // 16-bit; any
  void* dw;                 // [E, N, K]
  uint8_t* workspace;       // tensor maps, aligned copies of operands that TMA cannot read
  WaitCfg wait;
};
cudaError_t launch_weight_grad(const WgradArgs& a, int inject_stall, cudaStream_t s);
size_t weight_grad_workspace(const void* dy, int64_t ld_dy, const void* x, int64_t ld_x, int64_t R, int64_t E, int64_t N, int64_t K);

// Norms around a block.

struct NormArgs {
  const void* x;
  int64_t ld_x;
  const void* o;            // null: r = residual_scale * x
  int64_t ld_o;
  const void* gate;
  int gate_kind;
  int64_t ld_gate;          // QMOE_GATE_FULL
  const void* w_post;       // null: the branch is not normalised
  const void* w_pre;        // null: no h
  float residual_scale, eps;
  int64_t T, H;
  int dtype;
  // forward
  void* r;
  void* h;
  float* rstd_post;
  float* rstd_pre;
  // backward
  const void* dr;           // gradients of r and h (null: zero)
  int64_t ld_dr;
  const void* dh;
  int64_t ld_dh;
  void* dx;
  void* d_o;
  void* dgate;
  void* dw_post;
  void* dw_pre;
  float* partial;           // [CTAs, sums, H]
};
cudaError_t launch_block_norm(const NormArgs& a, cudaStream_t s);
cudaError_t launch_block_norm_grad(const NormArgs& a, cudaStream_t s);
// Longest row the norm kernels hold in registers.
constexpr int64_t kNormMaxWidth = 16384;
size_t block_norm_grad_workspace(int64_t T, int64_t H, int dtype);

inline int dtype_size(int dtype) { return dtype == QMOE_F32 ? 4 : 2; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
// Every row of a matrix starts on a 16-byte boundary.
inline bool rows_aligned16(const void* p, int64_t ld, int dtype) {
  return p == nullptr || (aligned16(p) && ld * dtype_size(dtype) % 16 == 0);
}

}  // namespace qmoe

#ifdef __CUDACC__
namespace qmoe {

// Launches with programmatic dependent launch: the kernel may start while the
// one before it on the stream ends, and waits (op_begin) before it touches
// memory.  Small calls follow one another at launch latency; this takes its
// greater part off.
template <typename... Params, typename... Args>
cudaError_t launch_op(void (*kern)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}
// Lets a kernel take more dynamic shared memory than a launch gets unasked (48 KB
// with the static part, at most 8 KB here).  The limit belongs to the kernel in
// the whole process: it is always set to the same value, the most that any call
// of this kernel needs, so that calls from several threads do not lower it under
// one another.
template <typename... Params>
cudaError_t allow_shared(void (*kern)(Params...), size_t bytes, int most) {
  if (bytes <= 40 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
}
// First thing in an operator's kernel: lets the next one start (once every CTA
// of this one has), and waits for the ones before.  What follows sees their
// memory, and as every operator waits, theirs before them too.  Tensors are read
// by plain loads only: they may still be written when this kernel starts, so
// the non-coherent path, which asks that memory is not written during the
// kernel's life (and whose loads may be moved ahead of the wait), is not open.
__device__ __forceinline__ void op_begin() {
  pdl_launch_dependents();
  pdl_wait();
}
// 16 bytes, loaded where the code has it (after the wait, which is volatile too).
__device__ __forceinline__ uint4 ld_here_v4(const void* p) {
  uint4 r;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}
// 16 bytes of a row that is read once: past the L1.
__device__ __forceinline__ uint4 ld_once_v4(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

template <int DT>
struct ElemT;
template <>
struct ElemT<QMOE_F32> {
  using t = float;
};
template <>
struct ElemT<QMOE_F16> {
  using t = __half;
};
template <>
struct ElemT<QMOE_BF16> {
  using t = __nv_bfloat16;
};

template <int DT>
__device__ __forceinline__ void unpack2(uint32_t u, float& a, float& b) {
  if constexpr (DT == QMOE_F16) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u));
    a = f.x;
    b = f.y;
  } else {
    a = __uint_as_float(u << 16);
    b = __uint_as_float(u & 0xffff0000u);
  }
}
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (DT == QMOE_F16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// VEC consecutive values as elements of type DT, in 16-byte accesses (VEC *
// size a multiple of 16).
template <int DT, int VEC>
__device__ __forceinline__ void store_vec(void* base, size_t i, const float (&v)[VEC]) {
  if constexpr (DT == QMOE_F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
#pragma unroll
    for (int q = 0; q < VEC / 4; ++q) p[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
  } else {
    uint4* p = reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + i);
#pragma unroll
    for (int q = 0; q < VEC / 8; ++q)
      p[q] = make_uint4(pack2<DT>(v[8 * q], v[8 * q + 1]), pack2<DT>(v[8 * q + 2], v[8 * q + 3]),
                        pack2<DT>(v[8 * q + 4], v[8 * q + 5]), pack2<DT>(v[8 * q + 6], v[8 * q + 7]));
  }
}

// A thread's share of a row per step, kept as it is in memory until it is
// used.  VECTOR: one aligned 16-byte access.  Otherwise, for rows that do not
// start on 16-byte boundaries, four elements a row's thread count apart, so
// that a warp's accesses stay side by side and four are in flight.
template <int DT, bool VECTOR>
struct Frag;

template <int DT>
struct Frag<DT, true> {
  static constexpr int n = DT == QMOE_F32 ? 4 : 8;   // elements
  uint4 u;
  // first element of a thread, elements of a step of all of a row's threads
  __device__ static __forceinline__ int first(int thread) { return thread * n; }
  __device__ static __forceinline__ int step(int threads) { return threads * n; }
  // from the thread's first element, `left` elements before the row's end
  __device__ __forceinline__ void load(const typename ElemT<DT>::t* p, int, int) {
    u = *reinterpret_cast<const uint4*>(p);
  }
  // the same for rows that are read once: they do not pass through the L1
  __device__ __forceinline__ void load_once(const typename ElemT<DT>::t* p, int, int) { u = ld_once_v4(p); }
  __device__ __forceinline__ void get(float (&v)[n]) const {
    if constexpr (DT == QMOE_F32) {
      v[0] = __uint_as_float(u.x);
      v[1] = __uint_as_float(u.y);
      v[2] = __uint_as_float(u.z);
      v[3] = __uint_as_float(u.w);
    } else {
      unpack2<DT>(u.x, v[0], v[1]);
      unpack2<DT>(u.y, v[2], v[3]);
      unpack2<DT>(u.z, v[4], v[5]);
      unpack2<DT>(u.w, v[6], v[7]);
    }
  }
  __device__ __forceinline__ void set(const float (&v)[n]) {
    if constexpr (DT == QMOE_F32)
      u = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    else
      u = make_uint4(pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7]));
  }
  __device__ __forceinline__ void store(typename ElemT<DT>::t* p, int, int) const { *reinterpret_cast<uint4*>(p) = u; }
};

template <int DT>
struct Frag<DT, false> {
  static constexpr int n = 4;
  using T = typename ElemT<DT>::t;
  T e[n];
  __device__ static __forceinline__ int first(int thread) { return thread; }
  __device__ static __forceinline__ int step(int threads) { return threads * n; }
  __device__ __forceinline__ void load(const T* p, int left, int threads) {
#pragma unroll
    for (int i = 0; i < n; ++i) e[i] = i * threads < left ? p[i * threads] : T(0.f);
  }
  __device__ __forceinline__ void load_once(const T* p, int left, int threads) { load(p, left, threads); }
  __device__ __forceinline__ void get(float (&v)[n]) const {
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = load_d<DT>(&e[i], 0);
  }
  __device__ __forceinline__ void set(const float (&v)[n]) {
#pragma unroll
    for (int i = 0; i < n; ++i) store_d<DT>(&e[i], 0, v[i]);
  }
  __device__ __forceinline__ void store(T* p, int left, int threads) const {
#pragma unroll
    for (int i = 0; i < n; ++i)
      if (i * threads < left) p[i * threads] = e[i];
  }
};

// Threads of a row whose elements they take `per` at a time: as few steps as
// 512 threads allow, whole warps (or 8 or 16 lanes for the shortest rows), so
// that few threads idle in the last step; several short rows share a CTA.
struct RowShape {
  int tpr, rpb;
};
inline RowShape row_shape(int64_t H, int per, int most = 512) {
  const int64_t n = (H + per - 1) / per, steps = (n + most - 1) / most, lanes = (n + steps - 1) / steps;
  RowShape r;
  r.tpr = lanes <= 8 ? 8 : lanes <= 16 ? 16 : (int)((lanes + 31) / 32 * 32);
  r.rpb = r.tpr <= 128 ? 128 / r.tpr : 1;
  return r;
}

}  // namespace qmoe
#endif
