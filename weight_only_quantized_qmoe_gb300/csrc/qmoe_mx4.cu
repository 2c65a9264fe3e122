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
// 17/32 byte a value, instead of k 16-bit copies read again.
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

// The eight elements from element `at` of x on, where `at` need not be on a
// 16-byte boundary: the lane loads the aligned 16 bytes that hold the first of
// them (32-bit types: also the next 16), takes the following ones from the
// next lane, which starts 8 elements on, and shifts.  Whole warp; the tensor has
// `hi` elements, and aligned words that are not wholly inside it are read
// element by element.  Elements past n (of the row) become 0.
template <int DT>
__device__ __forceinline__ void load8_shifted(const void* x, int64_t at, int64_t hi, int n, float (&v)[8]) {
  using T = typename ElemT<DT>::t;
  constexpr int per = 16 / (int)sizeof(T);       // elements of 16 bytes
  constexpr int words = DT == QMOE_F32 ? 8 : 4;  // 32-bit words a lane loads
  const T* p = static_cast<const T*>(x) + at;
  const int m = (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));   // the same for the whole warp
  uint32_t w[2 * words];
  auto aligned = [&](int64_t from, uint32_t* out) {   // 16 bytes from element `from` (aligned)
    if (from >= 0 && from + per <= hi) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(x) + from));
      out[0] = u.x;
      out[1] = u.y;
      out[2] = u.z;
      out[3] = u.w;
    } else {
      T e[per];
#pragma unroll
      for (int i = 0; i < per; ++i) e[i] = from + i >= 0 && from + i < hi ? static_cast<const T*>(x)[from + i] : T(0.f);
      memcpy(out, e, 16);
    }
  };
#pragma unroll
  for (int q = 0; q < words / 4; ++q) aligned(at - m + q * per, w + 4 * q);
#pragma unroll
  for (int i = 0; i < words; ++i) w[words + i] = __shfl_down_sync(0xffffffffu, w[i], 1);
  if ((threadIdx.x & 31) == 31 && m) aligned(at - m + 8, w + words);
  if constexpr (DT == QMOE_F32) {
    // shift by m words
#pragma unroll
    for (int i = 0; i < 10; ++i) w[i] = (m & 2) ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? __uint_as_float((m & 1) ? w[i + 1] : w[i]) : 0.f;
  } else {
    // shift by m halves of a word
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = (m & 4) ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = (m & 2) ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = (m & 1) ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
      unpack2<DT>(u, v[2 * i], v[2 * i + 1]);
      if (2 * i >= n) v[2 * i] = 0.f;
      if (2 * i + 1 >= n) v[2 * i + 1] = 0.f;
    }
  }
}

// Elements c .. c + 7 of the row that starts at element row0 and has n.
template <int DT, bool VEC>
__device__ __forceinline__ void load8(const void* x, int64_t row0, int64_t c, int64_t n, int64_t hi, float (&v)[8]) {
  const int left = (int)max((int64_t)0, min((int64_t)8, n - c));
  if constexpr (VEC) {
    if (left == 8) {
      load_vec<DT, 8>(x, (size_t)(row0 + c), v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < left ? load_d<DT>(x, (size_t)(row0 + c + i)) : 0.f;
    }
  } else {
    load8_shifted<DT>(x, row0 + c, hi, left, v);
  }
}

// A row takes blockDim.y warps, 256 values each per step; blockDim.z rows a CTA.
template <int DT, bool VEC, bool ACT>
__global__ void __launch_bounds__(32 * kQuantWarps) mx4_quantize_kernel(const Mx4QuantArgs a) {
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
  for (int64_t seg = threadIdx.y; seg * kQuantSeg < a.cols; seg += blockDim.y) {
    const int64_t c = seg * kQuantSeg + lane * 8;   // four lanes a block
    const bool in = c < (int64_t)nb * 32;
    float v[8];
    load8<DT, VEC>(a.x, row0, c, a.cols, hi, v);
    if (ACT) {
      float u[8];
      load8<DT, VEC>(a.x, row0 + a.cols, c, a.cols, hi, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = c + i < a.cols ? glu(a.act, v[i], u[i]) : 0.f;
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
    const int64_t q = c >> 7;
    const bool has_scale = (lane & 15) == 0 && q < nq;
    if (!a.pos) {
      if (in) *reinterpret_cast<uint32_t*>(a.codes + (size_t)(row * pitch + (c >> 1))) = code;
      if (has_scale) *reinterpret_cast<uint32_t*>(scales0 + (size_t)q * a.panel * 4) = sc;
    } else {   // one panel of rows * k rows
      uint8_t* codes = a.codes + (c >> 1);
      uint8_t* scales = a.scales + (size_t)q * a.panel * 4;
      for (int j = 0; j < a.k; ++j) {
        const int64_t p = a.pos[row * a.k + j];
        if (p < 0 || p >= a.panel) continue;
        if (in) *reinterpret_cast<uint32_t*>(codes + (size_t)(p * pitch)) = code;
        if (has_scale) *reinterpret_cast<uint32_t*>(scales + (size_t)p * 4) = sc;
      }
      for (int64_t p = used + row; p < a.panel; p += a.rows) {   // rows without a route
        if (in) *reinterpret_cast<uint32_t*>(codes + (size_t)(p * pitch)) = 0u;
        if (has_scale) *reinterpret_cast<uint32_t*>(scales + (size_t)p * 4) = 0u;
      }
    }
  }
}

// Warps of a row (the fewest steps eight warps allow) and rows of a CTA.
static dim3 mx4_block(int64_t segs) {
  const int64_t steps = (segs + kQuantWarps - 1) / kQuantWarps, warps = (segs + steps - 1) / steps;
  return dim3(32, (unsigned)warps, (unsigned)(kQuantWarps / warps));
}

cudaError_t launch_mx4_quantize(const Mx4QuantArgs& a, cudaStream_t s) {
  const dim3 block = mx4_block((a.cols + kQuantSeg - 1) / kQuantSeg);
  const int64_t blocks = (a.rows + block.z - 1) / block.z;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const bool act = a.act.act >= 0;
  const bool vec = rows_aligned16(a.x, a.ld_x, a.dtype) && (!act || a.cols * dtype_size(a.dtype) % 16 == 0);
  auto run = [&](auto kern) {
    kern<<<(unsigned)blocks, block, 0, s>>>(a);
    return cudaGetLastError();
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
  using T = typename ElemT<DT>::t;
  const int64_t row = blockIdx.x * (int64_t)blockDim.z + threadIdx.z;
  if (row >= a.rows) return;
  const int64_t nb = (a.cols + 31) / 32, nq = (nb + 3) / 4, pitch = nb * 16;
  const size_t row0 = (size_t)(row * a.ld_out);
  const int m = (int)((reinterpret_cast<uintptr_t>(static_cast<const T*>(a.out) + row0) & 15) / sizeof(T));
  const uint32_t* words = reinterpret_cast<const uint32_t*>(a.codes + (size_t)row * pitch);
  const uint8_t* sc = a.scales + mx4_scale_offset(row, 0, a.panel, nq);
  auto scale_of = [&](int64_t x) {   // of the block of element x; 2^(e - 127), e = 0 is subnormal, 255 is NaN
    const int64_t blk = min(max(x, (int64_t)0), a.cols - 1) >> 5;
    const uint32_t e = sc[(size_t)(blk >> 2) * a.panel * 4 + (blk & 3)];
    return __uint_as_float(e == 0 ? 0x00400000u : (e == 255 ? 0x7fc00000u : e << 23));
  };
  for (int64_t g = ((int64_t)threadIdx.y * 32 + threadIdx.x) * 8; g - m < a.cols; g += (int64_t)blockDim.y * kQuantSeg) {
    const int64_t c = g - m;   // g is on the codes' grid
    const uint32_t hi = g < nb * 32 ? words[g >> 3] : 0u, lo = m && g > 0 ? words[(g >> 3) - 1] : 0u;
    const uint32_t code = m ? __funnelshift_r(lo, hi, 32 - 4 * m) : hi;
    const float s0 = scale_of(c), s1 = m ? scale_of(c + 7) : s0;
    const int change = m ? (int)((32 - (c & 31)) & 31) : 0;   // first element of the second block, if it is within 8
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = e2m1_values((code >> (8 * i)) & 0xffu);
      v[2 * i] = f.x * (change && 2 * i >= change ? s1 : s0);
      v[2 * i + 1] = f.y * (change && 2 * i + 1 >= change ? s1 : s0);
    }
    if (c >= 0 && c + 8 <= a.cols) {
      store_vec<DT, 8>(a.out, row0 + c, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i >= 0 && c + i < a.cols) store_d<DT>(a.out, row0 + c + i, v[i]);
    }
  }
}

cudaError_t launch_mx4_dequantize(const Mx4DequantArgs& a, cudaStream_t s) {
  const dim3 block = mx4_block((a.cols + 7 + kQuantSeg - 1) / kQuantSeg);   // up to 7 elements early
  const int64_t blocks = (a.rows + block.z - 1) / block.z;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  auto run = [&](auto kern) {
    kern<<<(unsigned)blocks, block, 0, s>>>(a);
    return cudaGetLastError();
  };
  if (a.dtype == QMOE_F32) return run(mx4_dequantize_kernel<QMOE_F32>);
  if (a.dtype == QMOE_F16) return run(mx4_dequantize_kernel<QMOE_F16>);
  return run(mx4_dequantize_kernel<QMOE_BF16>);
}

}  // namespace qmoe
