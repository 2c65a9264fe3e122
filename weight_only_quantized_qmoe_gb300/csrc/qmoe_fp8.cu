// 8-bit floating point rows and weights: quantisation and its inverse.
//
// Blocks of 128 values of a row, or of 128 x 128 of a weight, share a power-of-
// two scale s, the smallest that leaves their largest magnitude at most 448
// (the largest E4M3 value): with amax = m 2^p, 1 <= m < 2, s = 2^(p - 8) if m <=
// 1.75, else 2^(p - 7), at least 2^-127; it is stored as its exponent + 127
// (E8M0).  An element is x / s rounded to the nearest E4M3 value, ties to even;
// x / s only moves the exponent, so that is the one rounding and the codes do
// not depend on how they are computed.  Nothing saturates.  A block that holds a
// NaN or an infinity gets the NaN scale 255 and codes 0.
//
// Weights have square blocks so that their transpose has the same ones: one copy
// of a weight serves the product and the gradient of its rows.
//
// Memory-bound: a lane takes 16 values (one 16-byte store of codes), eight lanes
// a block, three shuffles for its largest.  Rows: a warp takes 512 values, the
// four scale bytes of one word (bf16, 16384 x 4096: 34.4 us, 5.9 TB/s; back 44.5, 4.5;
// 2880 rows of 4127, which start anywhere, 10.4, back 9.5; after a gated activation
// instructions bound it: 32768 x 1536 of gate | up 193 us, 1.3 TB/s).  Blocks: a CTA takes 128 x
// 128 values, which stay in registers (as they were loaded) until their largest is
// known (f32, 8 x 1537 x 2880: 32.3 us, 5.5 TB/s).
#include <algorithm>
#include <cstring>

#include "qmoe_ops.cuh"

namespace qmoe {

constexpr int kF8Seg = 512;      // values of a warp
constexpr int kF8Warps = 8;
constexpr int kF8Block = 128;

// Two values to E4M3 codes (lo in the low byte), to nearest even.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
  return r;
}
// Both values of a pair of codes (exact).
__device__ __forceinline__ float2 e4m3_values(uint32_t pair) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)pair));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ float e8m0_value(uint32_t e) {   // 2^(e - 127); e = 0 is subnormal, 255 is NaN
  return __uint_as_float(e == 0 ? 0x00400000u : (e == 255 ? 0x7fc00000u : e << 23));
}
// Scale byte of a block from the bits of its largest magnitude (they order like
// the values, NaN above infinity above every number).
__device__ __forceinline__ uint32_t fp8_scale_byte(uint32_t m) {
  const int e = (int)(m >> 23) - ((m & 0x7fffffu) <= 0x600000u ? 8 : 7);
  return m >= 0x7f800000u ? 255u : (uint32_t)max(e, 0);
}
// 16 codes of 16 values with a scale byte (255: zeros).
__device__ __forceinline__ uint4 fp8_codes(const float (&v)[16], uint32_t s) {
  const float inv = __uint_as_float((254u - min(s, 253u)) << 23);   // 2^(127 - s)
  uint32_t c[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    c[q] = e4m3_pair(v[4 * q] * inv, v[4 * q + 1] * inv) | e4m3_pair(v[4 * q + 2] * inv, v[4 * q + 3] * inv) << 16;
  return s == 255u ? make_uint4(0, 0, 0, 0) : make_uint4(c[0], c[1], c[2], c[3]);
}
__device__ __forceinline__ uint32_t largest(const float (&v)[16]) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  return m;
}

// Sixteen elements of a row a lane, c .. c + 15; consecutive lanes of a row hold
// consecutive ones, and `last` is set in the last such lane.  VEC: the rows start
// on 16-byte boundaries.  Otherwise the lane loads the aligned 16-byte words that
// hold the first of them, takes the following word from the next lane (the last
// one loads it) and shifts.  `size` is the number of elements of the tensor:
// words that are not wholly inside it are read element by element.
template <int DT, bool VEC>
struct Load16 {
  using T = typename ElemT<DT>::t;
  static constexpr int per = 16 / (int)sizeof(T);        // elements of 16 bytes
  static constexpr int words = DT == QMOE_F32 ? 16 : 8;  // 32-bit words of 16 elements
  uint32_t w[words], over[VEC ? 1 : 4];

  __device__ static __forceinline__ void aligned(const T* x, int64_t from, int64_t size, uint32_t* out) {
    if (from >= 0 && from + per <= size) {
      const uint4 u = ld_once_v4(x + from);
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
  __device__ __forceinline__ void load(const void* base, int64_t at, int m, int64_t size, bool last) {
    const T* x = static_cast<const T*>(base);
#pragma unroll
    for (int q = 0; q < words / 4; ++q) aligned(x, at - m + q * per, size, w + 4 * q);
    if constexpr (!VEC)
      if (m && last) aligned(x, at - m + 16, size, over);
  }
  // The elements, past the row's last (left of them) 0.  Whole warp.
  __device__ __forceinline__ void get(int m, int left, bool last, float (&v)[16]) const {
    uint32_t u[words + 4];
#pragma unroll
    for (int i = 0; i < words; ++i) u[i] = w[i];
    if constexpr (!VEC) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t next = __shfl_down_sync(0xffffffffu, w[i], 1);
        u[words + i] = last ? over[i] : next;
      }
      if constexpr (DT == QMOE_F32) {   // by m words
#pragma unroll
        for (int i = 0; i < words + 2; ++i) u[i] = (m & 2) ? u[i + 2] : u[i];
#pragma unroll
        for (int i = 0; i < words; ++i) u[i] = (m & 1) ? u[i + 1] : u[i];
      } else {                          // by m halves of a word
#pragma unroll
        for (int i = 0; i < words + 2; ++i) u[i] = (m & 4) ? u[i + 2] : u[i];
#pragma unroll
        for (int i = 0; i < words + 1; ++i) u[i] = (m & 2) ? u[i + 1] : u[i];
#pragma unroll
        for (int i = 0; i < words; ++i) u[i] = (m & 1) ? __funnelshift_r(u[i], u[i + 1], 16) : u[i];
      }
    }
    if constexpr (DT == QMOE_F32) {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(u[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) unpack2<DT>(u[i], v[2 * i], v[2 * i + 1]);
    }
    if (left < 16) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i >= left) v[i] = 0.f;
    }
  }
};

// Rows: blockDim.y warps a row, 512 values each per step; blockDim.z rows a CTA.
template <int DT, bool VEC, bool ACT>
__global__ void __launch_bounds__(32 * kF8Warps) fp8_quantize_kernel(const Fp8QuantArgs a) {
  op_begin();
  const int64_t row = blockIdx.x * (int64_t)blockDim.z + threadIdx.z;
  if (row >= a.rows) return;
  const int lane = threadIdx.x;
  const bool last = lane == 31;
  const int cols = (int)a.cols, nb = (cols + kF8Block - 1) / kF8Block, nq = (nb + 3) / 4;
  const int64_t pitch = fp8_pitch(a.cols);
  const int64_t row0 = row * a.ld_x;
  const int64_t size = (a.rows - 1) * a.ld_x + (ACT ? 2 : 1) * a.cols;   // elements of x
  const int64_t used = a.pos ? max(a.offsets[a.E], 0) : 0;
  // a routed row's output rows, a lane each, known before its values are
  const int first_rows = a.pos && lane < a.k ? a.pos[row * a.k + lane] : -1;
  const int step = blockDim.y * kF8Seg;
  const int m0 = Load16<DT, VEC>::early(a.x, row0), m1 = ACT ? Load16<DT, VEC>::early(a.x, row0 + a.cols) : 0;
  Load16<DT, VEC> next, next_up;
  auto fetch = [&](int c) {
    next.load(a.x, row0 + c, m0, size, last);
    if (ACT) next_up.load(a.x, row0 + a.cols + c, m1, size, last);
  };
  const int c0 = (int)threadIdx.y * kF8Seg + lane * 16;   // eight lanes a block
  fetch(c0);
  for (int c = c0; c - lane * 16 < cols; c += step) {
    const int left = max(0, min(16, cols - c));
    float v[16];
    next.get(m0, left, last, v);
    if (ACT) {
      float u[16];
      next_up.get(m1, left, last, u);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = i < left ? glu(a.act, v[i], u[i]) : 0.f;
    }
    if (c - lane * 16 + step < cols) fetch(c + step);
    uint32_t m = largest(v);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 4));
    const uint32_t s = fp8_scale_byte(m);
    const uint4 code = fp8_codes(v, s);
    // four blocks' scale bytes in one word (past the row's last: zeros)
    uint32_t word = c < cols ? s : 0u;
    word |= __shfl_down_sync(0xffffffffu, word, 8) << 8;
    word |= __shfl_down_sync(0xffffffffu, word, 16) << 16;
    const bool in = c < pitch, has_scale = lane == 0;
    const int q = c / kF8Seg;
    auto put = [&](uint8_t* codes, uint8_t* scales, const uint4& value, uint32_t scale_word) {
      if (in) *reinterpret_cast<uint4*>(codes + c) = value;
      if (has_scale) *reinterpret_cast<uint32_t*>(scales + (size_t)q * a.panel * 4) = scale_word;
    };
    if (!a.pos) {
      put(a.codes + (size_t)(row * pitch), a.scales + mx4_scale_offset(row, 0, a.panel, nq), code, word);
    } else {   // one panel of rows * k rows
      for (int j = 0; j < a.k; ++j) {
        const int p = j < 32 ? __shfl_sync(0xffffffffu, first_rows, j) : a.pos[row * a.k + j];
        if (p >= 0 && p < a.panel) put(a.codes + (size_t)(p * pitch), a.scales + (size_t)p * 4, code, word);
      }
      for (int64_t p = used + row; p < a.panel; p += a.rows)   // rows without a route
        put(a.codes + (size_t)(p * pitch), a.scales + (size_t)p * 4, make_uint4(0, 0, 0, 0), 0u);
    }
  }
}

// Blocks: a CTA takes 128 rows x 128 columns, 32 rows at a time, eight lanes a row.
// (bf16, 64 x 1536 x 4096: three CTAs a multiprocessor 199 us, 6.1 TB/s, two 246;
// 32-bit rows fill the registers of two.)
template <int DT, bool VEC>
__global__ void __launch_bounds__(256, DT == QMOE_F32 ? 2 : 3) fp8_quantize_blocks_kernel(const Fp8QuantArgs a, int row_blocks, int col_blocks) {
  op_begin();
  __shared__ uint32_t s_max[8];
  const int cb = blockIdx.x % col_blocks;
  const int64_t rest = blockIdx.x / col_blocks;
  const int rb = (int)(rest % row_blocks);
  const int64_t matrix = rest / row_blocks, first = matrix * a.panel + (int64_t)rb * kF8Block;
  const int rows = (int)min((int64_t)kF8Block, a.panel - (int64_t)rb * kF8Block);
  const int lane8 = threadIdx.x & 7, r0 = threadIdx.x >> 3, c = cb * kF8Block + lane8 * 16;
  const bool last = lane8 == 7;
  const int64_t pitch = fp8_pitch(a.cols), size = (a.rows - 1) * a.ld_x + a.cols;
  const int left = max(0, min(16, (int)a.cols - c));
  Load16<DT, VEC> raw[4];
  int early[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // a row past the last is read as the last one and left out
    const int64_t row0 = (first + min(r0 + 32 * i, rows - 1)) * a.ld_x;
    early[i] = Load16<DT, VEC>::early(a.x, row0);
    raw[i].load(a.x, row0 + c, early[i], size, last);
  }
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v[16];
    raw[i].get(early[i], left, last, v);
    m = max(m, largest(v));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, s_max[i]);
  const uint32_t s = fp8_scale_byte(m);
  if (threadIdx.x == 0) a.scales[(matrix * row_blocks + rb) * col_blocks + cb] = (uint8_t)s;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v[16];
    raw[i].get(early[i], left, last, v);
    const int r = r0 + 32 * i;
    if (r < rows && c < pitch) *reinterpret_cast<uint4*>(a.codes + (size_t)((first + r) * pitch) + c) = fp8_codes(v, s);
  }
}

// Warps of a row and rows of a CTA: a warp walks up to `most` steps of its row,
// the next one's loads in flight, while every multiprocessor still gets 32 warps.
static dim3 fp8_block(int64_t segs, int64_t rows, int64_t most) {
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(most, rows * segs / (kSms * 32)));
  const int64_t at_most = std::min<int64_t>(kF8Warps, (segs + want - 1) / want);
  const int64_t steps = (segs + at_most - 1) / at_most, warps = (segs + steps - 1) / steps;
  return dim3(32, (unsigned)warps, (unsigned)std::max<int64_t>(1, kF8Warps / 2 / warps));
}

cudaError_t launch_fp8_quantize(const Fp8QuantArgs& a, cudaStream_t s) {
  const bool act = a.act.act >= 0;
  const bool vec = rows_aligned16(a.x, a.ld_x, a.dtype) && (!act || a.cols * dtype_size(a.dtype) % 16 == 0);
  auto types = [&](auto&& f) {
    if (a.dtype == QMOE_F32) return f(std::integral_constant<int, QMOE_F32>{});
    if (a.dtype == QMOE_F16) return f(std::integral_constant<int, QMOE_F16>{});
    return f(std::integral_constant<int, QMOE_BF16>{});
  };
  if (a.square) {
    const int64_t rb = (a.panel + kF8Block - 1) / kF8Block, cb = (a.cols + kF8Block - 1) / kF8Block, matrices = a.rows / a.panel;
    if (rb > 0x7fffffff || matrices * rb > 0x7fffffff / cb) return cudaErrorInvalidValue;
    return types([&](auto dt) {
      constexpr int DT = decltype(dt)::value;
      return launch_op(vec ? fp8_quantize_blocks_kernel<DT, true> : fp8_quantize_blocks_kernel<DT, false>,
                       dim3((unsigned)(matrices * rb * cb)), dim3(256), 0, s, a, (int)rb, (int)cb);
    });
  }
  const dim3 block = fp8_block((a.cols + kF8Seg - 1) / kF8Seg, a.rows, 4);
  const int64_t blocks = (a.rows + block.z - 1) / block.z;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  return types([&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    auto run = [&](auto kern) { return launch_op(kern, dim3((unsigned)blocks), block, 0, s, a); };
    if (act) return vec ? run(fp8_quantize_kernel<DT, true, true>) : run(fp8_quantize_kernel<DT, false, true>);
    return vec ? run(fp8_quantize_kernel<DT, true, false>) : run(fp8_quantize_kernel<DT, false, false>);
  });
}

// The values of the codes, rounded once to D.  A lane writes 8 of them, from a
// 16-byte boundary of the output on: where a row does not start on one, its
// lanes start m elements early, so a lane's codes come from two 8-byte words and
// may belong to two blocks.
template <int DT>
__global__ void __launch_bounds__(32 * kF8Warps) fp8_dequantize_kernel(const Fp8DequantArgs a) {
  op_begin();
  using T = typename ElemT<DT>::t;
  const int64_t row = blockIdx.x * (int64_t)blockDim.z + threadIdx.z;
  if (row >= a.rows) return;
  const int cols = (int)a.cols, nb = (cols + kF8Block - 1) / kF8Block, nq = (nb + 3) / 4;
  const int pitch = (int)fp8_pitch(a.cols);
  const size_t row0 = (size_t)(row * a.ld_out);
  const int m = (int)((reinterpret_cast<uintptr_t>(static_cast<const T*>(a.out) + row0) & 15) / sizeof(T));
  const uint64_t* words = reinterpret_cast<const uint64_t*>(a.codes + (size_t)(row * pitch));
  const int64_t matrix = row / a.panel, r = row - matrix * a.panel, row_blocks = (a.panel + kF8Block - 1) / kF8Block;
  const uint8_t* sc = a.square ? a.scales + (matrix * row_blocks + r / kF8Block) * nb : a.scales + mx4_scale_offset(row, 0, a.panel, nq);
  const size_t panel_bytes = 4 * (size_t)a.panel;
  auto scale_byte = [&](int x) -> uint32_t {   // of the block of element x
    const int blk = min(max(x, 0), cols - 1) / kF8Block;
    return a.square ? sc[blk] : sc[(size_t)(blk >> 2) * panel_bytes + (blk & 3)];
  };
  // codes and scale bytes of a step, loaded a step ahead
  uint64_t next_hi = 0, next_lo = 0;
  uint32_t next_e0 = 0, next_e1 = 0;
  auto fetch = [&](int g) {
    next_hi = g < pitch ? words[g >> 3] : 0u;
    next_lo = m && g > 0 ? words[(g >> 3) - 1] : 0u;
    next_e0 = scale_byte(g - m);
    next_e1 = m ? scale_byte(g - m + 7) : next_e0;
  };
  const int first = ((int)threadIdx.y * 32 + threadIdx.x) * 8, step = blockDim.y * 256;
  if (first - m < cols) fetch(first);
  for (int g = first; g - m < cols; g += step) {
    const int c = g - m;   // g is on the codes' grid
    const uint64_t code = m ? next_lo >> (64 - 8 * m) | next_hi << (8 * m) : next_hi;
    const float s0 = e8m0_value(next_e0), s1 = e8m0_value(next_e1);
    if (c + step < cols) fetch(g + step);
    const int change = m ? (kF8Block - (c & (kF8Block - 1))) & (kF8Block - 1) : 0;   // first element of the second block, if within 8
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = e4m3_values((uint32_t)(code >> (16 * i)) & 0xffffu);
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

cudaError_t launch_fp8_dequantize(const Fp8DequantArgs& a, cudaStream_t s) {
  // up to 7 elements early
  const dim3 block = fp8_block((a.cols + 7 + 255) / 256, a.rows, a.dtype == QMOE_F32 ? 3 : 6);
  const int64_t blocks = (a.rows + block.z - 1) / block.z;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  auto run = [&](auto kern) { return launch_op(kern, dim3((unsigned)blocks), block, 0, s, a); };
  if (a.dtype == QMOE_F32) return run(fp8_dequantize_kernel<QMOE_F32>);
  if (a.dtype == QMOE_F16) return run(fp8_dequantize_kernel<QMOE_F16>);
  return run(fp8_dequantize_kernel<QMOE_BF16>);
}

}  // namespace qmoe
