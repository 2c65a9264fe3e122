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

// Values c .. c + 7 of row src (length n), past the end 0.
template <int DT, bool VEC>
__device__ __forceinline__ void load8(const void* src, size_t row0, int64_t c, int64_t n, float (&v)[8]) {
  if (VEC && c + 8 <= n) {
    load_vec<DT, 8>(src, row0 + c, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < n ? load_d<DT>(src, row0 + c + i) : 0.f;
  }
}

template <int DT, bool VEC, bool ACT>
__global__ void __launch_bounds__(32 * kQuantWarps) mx4_quantize_kernel(const Mx4QuantArgs a, int64_t nseg) {
  const int64_t wid = blockIdx.x * (int64_t)kQuantWarps + (threadIdx.x >> 5);
  const int64_t nb = (a.cols + 31) / 32, nq = (nb + 3) / 4, pitch = nb * 16;
  const int64_t row = wid / nseg;
  if (row >= a.rows) return;
  const int lane = threadIdx.x & 31;
  const int64_t c = (wid - row * nseg) * kQuantSeg + lane * 8;   // a multiple of 8; four lanes a block
  const bool in = c < nb * 32;
  float v[8];
  load8<DT, VEC>(a.x, (size_t)(row * a.ld_x), c, a.cols, v);
  if (ACT) {
    float u[8];
    load8<DT, VEC>(a.x, (size_t)(row * a.ld_x + a.cols), c, a.cols, u);
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
  auto put = [&](int64_t p, uint32_t codes, uint32_t scales) {
    if (in) *reinterpret_cast<uint32_t*>(a.codes + (size_t)p * pitch + (c >> 1)) = codes;
    if (has_scale) *reinterpret_cast<uint32_t*>(a.scales + mx4_scale_offset(p, q, a.panel, nq)) = scales;
  };
  if (!a.pos) {
    put(row, code, sc);
    return;
  }
  for (int j = 0; j < a.k; ++j) {
    const int p = a.pos[row * a.k + j];
    if (p >= 0 && p < a.rows * a.k) put(p, code, sc);
  }
  for (int64_t p = max(a.offsets[a.E], 0) + row; p < a.rows * a.k; p += a.rows) put(p, 0u, 0u);   // rows without a route
}

cudaError_t launch_mx4_quantize(const Mx4QuantArgs& a, cudaStream_t s) {
  const int64_t nseg = (a.cols + kQuantSeg - 1) / kQuantSeg;
  const int64_t blocks = (a.rows * nseg + kQuantWarps - 1) / kQuantWarps;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const bool act = a.act.act >= 0;
  const bool vec = rows_aligned16(a.x, a.ld_x, a.dtype) && (!act || a.cols * dtype_size(a.dtype) % 16 == 0);
  auto run = [&](auto kern) {
    kern<<<(unsigned)blocks, 32 * kQuantWarps, 0, s>>>(a, nseg);
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

// The values of the codes, rounded once to D: a lane takes 8 of them.
template <int DT, bool VEC>
__global__ void __launch_bounds__(32 * kQuantWarps) mx4_dequantize_kernel(const Mx4DequantArgs a, int64_t nseg) {
  const int64_t wid = blockIdx.x * (int64_t)kQuantWarps + (threadIdx.x >> 5);
  const int64_t nb = (a.cols + 31) / 32, nq = (nb + 3) / 4, pitch = nb * 16;
  const int64_t row = wid / nseg;
  if (row >= a.rows) return;
  const int64_t c = (wid - row * nseg) * kQuantSeg + (threadIdx.x & 31) * 8;
  if (c >= a.cols) return;
  const uint32_t code = *reinterpret_cast<const uint32_t*>(a.codes + (size_t)row * pitch + (c >> 1));
  const uint32_t e = a.scales[mx4_scale_offset(row, c >> 7, a.panel, nq) + ((c >> 5) & 3)];
  // 2^(e - 127); e = 0 is the subnormal 2^-127, 255 is NaN
  const float scale = __uint_as_float(e == 0 ? 0x00400000u : (e == 255 ? 0x7fc00000u : e << 23));
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = e2m1_values((code >> (8 * i)) & 0xffu);
    v[2 * i] = f.x * scale;
    v[2 * i + 1] = f.y * scale;
  }
  const size_t at = (size_t)(row * a.ld_out + c);
  if (VEC && c + 8 <= a.cols) {
    store_vec<DT, 8>(a.out, at, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < a.cols) store_d<DT>(a.out, at + i, v[i]);
  }
}

cudaError_t launch_mx4_dequantize(const Mx4DequantArgs& a, cudaStream_t s) {
  const int64_t nseg = (a.cols + kQuantSeg - 1) / kQuantSeg;
  const int64_t blocks = (a.rows * nseg + kQuantWarps - 1) / kQuantWarps;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const bool vec = rows_aligned16(a.out, a.ld_out, a.dtype);
  auto run = [&](auto kern) {
    kern<<<(unsigned)blocks, 32 * kQuantWarps, 0, s>>>(a, nseg);
    return cudaGetLastError();
  };
  if (a.dtype == QMOE_F32) return vec ? run(mx4_dequantize_kernel<QMOE_F32, true>) : run(mx4_dequantize_kernel<QMOE_F32, false>);
  if (a.dtype == QMOE_F16) return vec ? run(mx4_dequantize_kernel<QMOE_F16, true>) : run(mx4_dequantize_kernel<QMOE_F16, false>);
  return vec ? run(mx4_dequantize_kernel<QMOE_BF16, true>) : run(mx4_dequantize_kernel<QMOE_BF16, false>);
}

}  // namespace qmoe
