// Microscaled 4-bit floating point rows: quantisation and its inverse.
//
// A row is cut into blocks of 32 values (OCP Microscaling Formats, MXFP4).  A
// block's scale is the power of two s = 2^clamp(floor(log2(amax)) - 2, -127,
// 127), stored as its exponent + 127 (E8M0); an element is x / s rounded to
// the nearest E2M1 value (0, 0.5, 1, 1.5, 2, 3, 4, 6; ties to the even code),
// saturated at 6.  x / s only moves the exponent, so the one rounding is the
// element's own and the result does not depend on how it is computed.  A
// block that holds a NaN or an infinity gets the NaN scale 255 (and codes 0):
// no E2M1 value stands for either.
//
// Memory-bound: a warp takes 256 values of a row, 8 a lane (one 16-byte load
// of 16-bit values), two shuffles find a block's maximum among its four lanes,
// and the lane writes four bytes of codes.  With a plan the row goes straight
// to its rows in expert order: read once, quantised once, written k times at
// 17/32 byte a value, instead of k 16-bit copies read again.  (bf16, rows of
// 4127 that start anywhere: 2880 of them in 12 us, read back in 10; 4096 rows of
// 1536 to eight places each 11 us.)
#include <algorithm>
#include <cstring>

#include "qmoe_ops.cuh"

namespace qmoe {

constexpr int kQuantSeg = 256;    // values of a warp
constexpr int kQuantWarps = 8;

// Two values to E2M1 codes in one byte (lo in the low half), round to nearest
// even, saturating.
__device__ __forceinline__ uint32_t e2m1_pair(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tcvt.u32.u8 %0, b;\n\t}" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}
// Both values of a byte of codes, as packed f16 (exact).
__device__ __forceinline__ float2 e2m1_values(uint32_t byte) {
  uint32_t h;
  asm("{\n\t.reg .b8 b;\n\tcvt.u8.u32 b, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(h) : "r"(byte));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Eight elements of a row a lane, c .. c + 7, loaded in two steps so that the
// next ones are on their way while these are worked on.  VEC: the rows start on
// 16-byte boundaries, and so do the lane's elements.  Otherwise the lane loads
// the aligned 16 bytes that hold the first of them (32-bit types: also the next
// 16), takes the following ones from the next lane, which starts 8 elements on,
// and shifts.  `size` is the number of elements of the tensor: aligned words
// that are not wholly inside it are read element by element.
// The loads of unaligned rows keep their place in the code (bf16, 2880 rows of
// 4127: 12.3 us, left to the compiler 12.6; aligned rows, 4096 of 4096: 11.8 / 10.7).
template <int DT, bool VEC>
struct Load8 {
  using T = typename ElemT<DT>::t;
  static constexpr int per = 16 / (int)sizeof(T);       // elements of 16 bytes
  static constexpr int words = DT == QMOE_F32 ? 8 : 4;  // 32-bit words of 8 elements
  uint32_t w[words], over[4];                           // over: lane 31's, what the next lane would have

  __device__ static __forceinline__ void aligned(const T* x, int64_t from, int64_t size, uint32_t* out) {
    if (from >= 0 && from + per <= size) {
      const uint4 u = VEC ? *reinterpret_cast<const uint4*>(x + from) : ld_here_v4(x + from);
      out[0] = u.x;
      out[1] = u.y;
      out[2] = u.z;
      out[3] = u.w;
    } else {
      T e[per];
#pragma unroll
      for (int i = 0; i < per; ++i) e[i] = from + i >= 0 && from + i < size ? x[from + i] : T(0.f);
      memcpy(out, e, 16);
    }
  }
  // Elements before the lane's first one in its aligned 16 bytes: the same for
  // every lane and step of a row.
  __device__ static __forceinline__ int early(const void* x, int64_t row0) {
    return VEC ? 0 : (int)((reinterpret_cast<uintptr_t>(static_cast<const T*>(x) + row0) & 15) / sizeof(T));
  }
  __device__ __forceinline__ void load(const void* base, int64_t at, int m, int64_t size) {
    const T* x = static_cast<const T*>(base);
#pragma unroll
    for (int q = 0; q < words / 4; ++q) aligned(x, at - m + q * per, size, w + 4 * q);
    if (!VEC && m && (threadIdx.x & 31) == 31) aligned(x, at - m + 8, size, over);
  }
  // The elements, past the row's last (left of them) 0.  Whole warp.
  __device__ __forceinline__ void get(int m, int left, float (&v)[8]) {
    if constexpr (!VEC) {
      uint32_t u[words + 4];
#pragma unroll
      for (int i = 0; i < words; ++i) u[i] = w[i];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t next = __shfl_down_sync(0xffffffffu, w[i], 1);
        u[words + i] = (threadIdx.x & 31) == 31 ? over[i] : next;
      }
      if constexpr (DT == QMOE_F32) {   // by m words
#pragma unroll
        for (int i = 0; i < 10; ++i) u[i] = (m & 2) ? u[i + 2] : u[i];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = (m & 1) ? u[i + 1] : u[i];
      } else {                          // by m halves of a word
#pragma unroll
        for (int i = 0; i < 6; ++i) u[i] = (m & 4) ? u[i + 2] : u[i];
#pragma unroll
        for (int i = 0; i < 5; ++i) u[i] = (m & 2) ? u[i + 1] : u[i];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = (m & 1) ? __funnelshift_r(u[i], u[i + 1], 16) : u[i];
      }
    }
    if constexpr (DT == QMOE_F32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) unpack2<DT>(w[i], v[2 * i], v[2 * i + 1]);
    }
    if (left < 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i >= left) v[i] = 0.f;
    }
  }
};

// A row takes blockDim.y warps, 256 values each per step; blockDim.z rows a CTA.
template <int DT, bool VEC, bool ACT>
__global__ void __launch_bounds__(32 * kQuantWarps) mx4_quantize_kernel(const Mx4QuantArgs a) {
  op_begin();
  const int64_t row = blockIdx.x * (int64_t)blockDim.z + threadIdx.z;
  if (row >= a.rows) return;
  const int lane = threadIdx.x;
  const int nb = (int)((a.cols + 31) / 32), nq = (nb + 3) / 4;
  const int64_t pitch = (int64_t)nb * 16;
  const int64_t row0 = row * a.ld_x;
  const int64_t hi = (a.rows - 1) * a.ld_x + (ACT ? 2 : 1) * a.cols;   // elements of x
  // the scale words of output row p start at its panel, 4 * panel bytes apart
  uint8_t* scales0 = nullptr;
  if (!a.pos) scales0 = a.scales + mx4_scale_offset(row, 0, a.panel, nq);
  const int64_t used = a.pos ? max(a.offsets[a.E], 0) : 0;
  // a routed row's output rows, a lane each, known before its values are
  const int first_rows = a.pos && lane < a.k ? a.pos[row * a.k + lane] : -1;
  const int cols = (int)a.cols, step = blockDim.y * kQuantSeg;
  const int m0 = Load8<DT, VEC>::early(a.x, row0), m1 = ACT ? Load8<DT, VEC>::early(a.x, row0 + a.cols) : 0;
  Load8<DT, VEC> next, next_up;
  auto fetch = [&](int c) {
    next.load(a.x, row0 + c, m0, hi);
    if (ACT) next_up.load(a.x, row0 + a.cols + c, m1, hi);
  };
  const int c0 = (int)threadIdx.y * kQuantSeg + lane * 8;   // four lanes a block
  fetch(c0);
  for (int c = c0; c - lane * 8 < cols; c += step) {
    const bool in = c < nb * 32;
    const int left = max(0, min(8, cols - c));
    Load8<DT, VEC> here = next, up = next_up;
    if (c - lane * 8 + step < cols) fetch(c + step);
    float v[8];
    here.get(m0, left, v);
    if (ACT) {
      float u[8];
      up.get(m1, left, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < left ? glu(a.act, v[i], u[i]) : 0.f;
    }
    // the largest magnitude of the block, as its bits (they order like the
    // values, NaN above infinity above every number)
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const bool bad = m >= 0x7f800000u;
    const int e = max((int)(m >> 23) - 2, 0);                       // biased exponent of the scale
    const float inv = __uint_as_float((uint32_t)(254 - e) << 23);   // 2^(127 - e): e <= 252
    uint32_t code = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) code |= e2m1_pair(v[2 * i] * inv, v[2 * i + 1] * inv) << (8 * i);
    uint32_t sc = in ? (bad ? 255u : (uint32_t)e) : 0u;
    if (bad) code = 0u;
    // four blocks' scale bytes in one word, held by the first lane of each 16
    sc |= __shfl_down_sync(0xffffffffu, sc, 4) << 8;
    sc |= __shfl_down_sync(0xffffffffu, sc, 8) << 16;
    const int q = c >> 7;
    const bool has_scale = (lane & 15) == 0 && q < nq;
    if (!a.pos) {
      if (in) *reinterpret_cast<uint32_t*>(a.codes + (size_t)(row * pitch + (c >> 1))) = code;
      if (has_scale) *reinterpret_cast<uint32_t*>(scales0 + (size_t)q * a.panel * 4) = sc;
    } else {   // one panel of rows * k rows
      uint8_t* codes = a.codes + (c >> 1);
      uint8_t* scales = a.scales + (size_t)q * a.panel * 4;
      auto put = [&](int64_t p, uint32_t code_word, uint32_t scale_word) {
        if (in) *reinterpret_cast<uint32_t*>(codes + (size_t)(p * pitch)) = code_word;
        if (has_scale) *reinterpret_cast<uint32_t*>(scales + (size_t)p * 4) = scale_word;
      };
      for (int j = 0; j < a.k; ++j) {
        const int p = j < 32 ? __shfl_sync(0xffffffffu, first_rows, j) : a.pos[row * a.k + j];
        if (p >= 0 && p < a.panel) put(p, code, sc);
      }
      for (int64_t p = used + row; p < a.panel; p += a.rows) put(p, 0u, 0u);   // rows without a route
    }
  }
}

// Warps of a row and rows of a CTA.  A warp that walks some steps of its row has
// the next one's loads in flight while it works, which one that ends after a
// step has not: up to `most` steps while every multiprocessor still gets 32
// warps, more where a row's kQuantWarps warps need them.  (Quantise and back,
// us, with 6 / with one: 8192 x 2048 f16 10.8 + 11.2 / 18.0 + 13.2, 20000 x 704
// bf16 11.1 + 10.6 / 21.7 + 21.7, 2880 x 4127 bf16 12.3 + 9.6 / 13.5 + 10.3;
// but 32-bit rows written, 2880 x 4128: 13.3 / 10.9 with 3.)
static dim3 mx4_block(int64_t segs, int64_t rows, int64_t most) {
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(most, rows * segs / (kSms * 32)));
  const int64_t at_most = std::min<int64_t>(kQuantWarps, (segs + want - 1) / want);
  const int64_t steps = (segs + at_most - 1) / at_most, warps = (segs + steps - 1) / steps;
  return dim3(32, (unsigned)warps, (unsigned)std::max<int64_t>(1, kQuantWarps / 2 / warps));
}

cudaError_t launch_mx4_quantize(const Mx4QuantArgs& a, cudaStream_t s) {
  const dim3 block = mx4_block((a.cols + kQuantSeg - 1) / kQuantSeg, a.rows, 6);
  const int64_t blocks = (a.rows + block.z - 1) / block.z;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const bool act = a.act.act >= 0;
  const bool vec = rows_aligned16(a.x, a.ld_x, a.dtype) && (!act || a.cols * dtype_size(a.dtype) % 16 == 0);
  auto run = [&](auto kern) {
    return launch_op(kern, dim3((unsigned)blocks), block, 0, s, a);
  };
  auto pick = [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    if (act) return vec ? run(mx4_quantize_kernel<DT, true, true>) : run(mx4_quantize_kernel<DT, false, true>);
    return vec ? run(mx4_quantize_kernel<DT, true, false>) : run(mx4_quantize_kernel<DT, false, false>);
  };
  if (a.dtype == QMOE_F32) return pick(std::integral_constant<int, QMOE_F32>{});
  if (a.dtype == QMOE_F16) return pick(std::integral_constant<int, QMOE_F16>{});
  return pick(std::integral_constant<int, QMOE_BF16>{});
}

// The values of the codes, rounded once to D.  A lane writes 8 of them, from a
// 16-byte boundary of the output on: where a row does not start on one, its
// lanes start m elements early, so a lane's values come from two words of
// codes and may belong to two blocks.
template <int DT>
__global__ void __launch_bounds__(32 * kQuantWarps) mx4_dequantize_kernel(const Mx4DequantArgs a) {
  op_begin();
  using T = typename ElemT<DT>::t;
  const int64_t row = blockIdx.x * (int64_t)blockDim.z + threadIdx.z;
  if (row >= a.rows) return;
  const int nb = (int)((a.cols + 31) / 32), nq = (nb + 3) / 4;
  const int64_t pitch = (int64_t)nb * 16;
  const size_t row0 = (size_t)(row * a.ld_out);
  const int m = (int)((reinterpret_cast<uintptr_t>(static_cast<const T*>(a.out) + row0) & 15) / sizeof(T));
  const uint32_t* words = reinterpret_cast<const uint32_t*>(a.codes + (size_t)row * pitch);
  const uint8_t* sc = a.scales + mx4_scale_offset(row, 0, a.panel, nq);
  const int cols = (int)a.cols;
  const size_t panel_bytes = 4 * (size_t)a.panel;
  auto scale_byte = [&](int x) -> uint32_t {   // of the block of element x
    const int blk = min(max(x, 0), cols - 1) >> 5;
    return sc[(size_t)(blk >> 2) * panel_bytes + (blk & 3)];
  };
  auto scale_of = [](uint32_t e) {   // 2^(e - 127); e = 0 is subnormal, 255 is NaN
    return __uint_as_float(e == 0 ? 0x00400000u : (e == 255 ? 0x7fc00000u : e << 23));
  };
  // codes and scale bytes of a step, loaded a step ahead
  uint32_t next_hi = 0, next_lo = 0, next_e0 = 0, next_e1 = 0;
  auto fetch = [&](int g) {
    next_hi = g < nb * 32 ? words[g >> 3] : 0u;
    next_lo = m && g > 0 ? words[(g >> 3) - 1] : 0u;
    next_e0 = scale_byte(g - m);
    next_e1 = m ? scale_byte(g - m + 7) : next_e0;
  };
  const int first = ((int)threadIdx.y * 32 + threadIdx.x) * 8, step = blockDim.y * kQuantSeg;
  if (first - m < cols) fetch(first);
  for (int g = first; g - m < cols; g += step) {
    const int c = g - m;   // g is on the codes' grid
    const uint32_t hi = next_hi, lo = next_lo;
    const uint32_t code = m ? __funnelshift_r(lo, hi, 32 - 4 * m) : hi;
    const float s0 = scale_of(next_e0), s1 = scale_of(next_e1);
    if (c + step < cols) fetch(g + step);
    const int change = m ? (int)((32 - (c & 31)) & 31) : 0;   // first element of the second block, if it is within 8
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = e2m1_values((code >> (8 * i)) & 0xffu);
      v[2 * i] = f.x * (change && 2 * i >= change ? s1 : s0);
      v[2 * i + 1] = f.y * (change && 2 * i + 1 >= change ? s1 : s0);
    }
    if (c >= 0 && c + 8 <= cols) {
      store_vec<DT, 8>(a.out, row0 + c, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i >= 0 && c + i < cols) store_d<DT>(a.out, row0 + c + i, v[i]);
    }
  }
}

cudaError_t launch_mx4_dequantize(const Mx4DequantArgs& a, cudaStream_t s) {
  // up to 7 elements early
  const dim3 block = mx4_block((a.cols + 7 + kQuantSeg - 1) / kQuantSeg, a.rows, a.dtype == QMOE_F32 ? 3 : 6);
  const int64_t blocks = (a.rows + block.z - 1) / block.z;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  auto run = [&](auto kern) {
    return launch_op(kern, dim3((unsigned)blocks), block, 0, s, a);
  };
  if (a.dtype == QMOE_F32) return run(mx4_dequantize_kernel<QMOE_F32>);
  if (a.dtype == QMOE_F16) return run(mx4_dequantize_kernel<QMOE_F16>);
  return run(mx4_dequantize_kernel<QMOE_BF16>);
}

}  // namespace qmoe
