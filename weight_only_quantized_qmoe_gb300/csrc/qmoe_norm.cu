// The norms before and after a block, fused with the gate of its output and
// the residual scale: forward.
//
//   oh = o * rstd_post, rstd_post = 1 / sqrt(mean(o^2) + eps)
//   n  = oh * w_post                        (w_post absent: n = o)
//   r  = residual_scale * x + gate * n      (gate absent: 1)
//   rh = r * rstd_pre,  rstd_pre = 1 / sqrt(mean(r^2) + eps)
//   h  = rh * w_pre
//
// Memory-bound: a row stays with its threads between the two sums, so x and o
// are read once and r and h written once.  The two sums of a row follow one
// another, so what decides is how many rows are on their way meanwhile: CTAs
// stay and walk the rows, a ring of rows ahead of themselves.  (bf16, 4096 rows
// of 4096: 29 us, 4.6 TB/s; rows loaded when they are used took 50.)
#include "qmoe_norm.cuh"

namespace qmoe {

// Rows in the ring of a CTA, the one in work among them, as its shared memory
// allows; 0: rows are loaded when they are used.
constexpr int norm_ahead(int vpt) { return vpt <= 2 ? 3 : vpt == 4 ? 2 : 0; }

// ALL: both norms and r are there, and no gate of its own for every value.
// Known when the kernel is compiled, the tests for each tensor leave the loop
// over the rows (bf16, with / without, 4096 rows of 4096: 29 / 33 us, 8192 of
// 2048: 36 / 45, 4096 of 8192: 52 / 58).
template <int DT, bool VECTOR, int VPT, bool ALL>
__global__ void __launch_bounds__(512) block_norm_kernel(const NormArgs a) {
  op_begin();
  using F = Frag<DT, VECTOR>;
  using T = typename ElemT<DT>::t;
  constexpr int N2 = F::n / 2, AHEAD = norm_ahead(VPT);
  constexpr bool RING = kCopies<DT, VECTOR> && AHEAD > 0;
  __shared__ float red[2 * 16];
  extern __shared__ __align__(16) uint8_t norm_ring[];
  const float inv_h = 1.f / (float)a.H;
  const bool full = !ALL && a.gate_kind == QMOE_GATE_FULL, branch = ALL || a.o;
  const int64_t stride = gridDim.x * (int64_t)blockDim.y;
  int64_t t = blockIdx.x * (int64_t)blockDim.y + threadIdx.y;
  int turn = 0, parts = 0;
  const uint32_t ring = smem_u32(norm_ring);
  const Place<DT, VECTOR> me(a.H);
  Rows<DT, VECTOR, VPT, RING> x(a.x, a.ld_x, t, stride, ring, parts, me), o(a.o, a.ld_o, t, stride, ring, parts, me),
      g(full ? a.gate : nullptr, a.ld_gate, t, stride, ring, parts, me);
  const uint32_t row_bytes = parts * VPT * me.frag_bytes;
  uint32_t cols = 0;   // none in shared memory
  const Columns<DT, VECTOR, VPT, false> post(a.w_post, a.gate_kind == QMOE_GATE_CHANNEL ? a.gate : nullptr, me, cols),
      pre(a.w_pre, nullptr, me, cols);
  const int64_t out_step = stride * a.H;
  T* out_r = static_cast<T*>(a.r) + t * a.H + F::first(threadIdx.x);
  T* out_h = static_cast<T*>(a.h) + t * a.H + F::first(threadIdx.x);
  int64_t ahead = t;   // the row fetched next
  auto fetch = [&](uint32_t at) {
    if constexpr (RING) {
      if (ahead < a.T) {
        x.fetch(at, me);
        o.fetch(at, me);
        g.fetch(at, me);
      }
      x.advance();
      o.advance();
      g.advance();
      ahead += stride;
      cp_async_commit();
    }
  };
#pragma unroll
  for (int s = 0; s + 1 < AHEAD; ++s) fetch(s * row_bytes);
  const uint32_t last = (RING ? AHEAD - 1 : 0) * row_bytes;
  uint32_t at = 0, to = last;
  float next_token = a.gate_kind == QMOE_GATE_TOKEN && t < a.T ? load_d<DT>(a.gate, (size_t)t) : 1.f;   // a row ahead
  // the rows of a block advance together (their sums share barriers)
  for (; t - threadIdx.y < a.T; t += stride, out_r += out_step, out_h += out_step) {
    const bool live = t < a.T;
    if constexpr (RING) {
      fetch(to);
      cp_async_wait<AHEAD - 1>();
    }
    float rstd1 = 1.f;
    if (ALL || (branch && a.w_post)) {
      float2 ss = both(0.f);
#pragma unroll
      for (int p = 0; p < VPT; ++p) {
        if (live && me.has(p)) {
          float2 v[N2];
          o.get(at, p, me, v);
#pragma unroll
          for (int i = 0; i < N2; ++i) ss = fma2(v[i], v[i], ss);
        }
      }
      rstd1 = rsqrtf(row_sum(ss.x + ss.y, red, turn) * inv_h + a.eps);
    }
    const float token = next_token;
    if (a.gate_kind == QMOE_GATE_TOKEN && t + stride < a.T) next_token = load_d<DT>(a.gate, (size_t)(t + stride));
    const float2 c1 = both(rstd1 * token), scale = both(a.residual_scale);
    float2 r[VPT][N2], ss = both(0.f);
#pragma unroll
    for (int p = 0; p < VPT; ++p) {
      if (live && me.has(p)) {
        x.get(at, p, me, r[p]);
#pragma unroll
        for (int i = 0; i < N2; ++i) r[p][i] = mul2(r[p][i], scale);
        if (branch) {
          float2 v[N2], w[N2];
          o.get(at, p, me, v);
          post.get(p, me, w);
          if (full) {
            float2 q[N2];
            g.get(at, p, me, q);
#pragma unroll
            for (int i = 0; i < N2; ++i) v[i] = mul2(v[i], q[i]);
          }
#pragma unroll
          for (int i = 0; i < N2; ++i) r[p][i] = fma2(mul2(v[i], c1), w[i], r[p][i]);
        }
        if (ALL || a.r) put<DT, VECTOR>(out_r, p, me, r[p]);
#pragma unroll
        for (int i = 0; i < N2; ++i) {
          if constexpr (!VECTOR) {   // past the row's end
            if (2 * i * me.threads >= me.left_of(p)) r[p][i].x = 0.f;
            if ((2 * i + 1) * me.threads >= me.left_of(p)) r[p][i].y = 0.f;
          }
          ss = fma2(r[p][i], r[p][i], ss);
        }
      }
    }
    if (a.rstd_post && live && threadIdx.x == 0) a.rstd_post[t] = rstd1;
    if (ALL || a.w_pre) {
      const float rstd2 = rsqrtf(row_sum(ss.x + ss.y, red, turn) * inv_h + a.eps);
      if (a.rstd_pre && live && threadIdx.x == 0) a.rstd_pre[t] = rstd2;
#pragma unroll
      for (int p = 0; p < VPT; ++p) {
        if (live && me.has(p)) {
          float2 w[N2];
          pre.get(p, me, w);
#pragma unroll
          for (int i = 0; i < N2; ++i) w[i] = mul2(mul2(r[p][i], both(rstd2)), w[i]);
          put<DT, VECTOR>(out_h, p, me, w);
        }
      }
    }
    if constexpr (RING) {
      to = at;   // this row's place is the next to be filled
      at = at == last ? 0 : at + row_bytes;
    } else {
      x.advance();
      o.advance();
      g.advance();
    }
  }
  if constexpr (RING) cp_async_wait<0>();
}

// Threads of a row at most.
constexpr int kNormThreads = 256;

// The most shared memory the ring of a kernel takes: x, o and a gate for every
// value, 512 threads.
constexpr int norm_ring_most(int vpt) { return norm_ahead(vpt) * 3 * vpt * 512 * 16; }

cudaError_t launch_block_norm(const NormArgs& a, cudaStream_t s) {
  const bool vec = norm_vec(a);
  const int frag = norm_frag(a.dtype, vec);
  const RowShape g = row_shape(a.H, frag, a.H > 2 * kNormThreads * frag ? 512 : kNormThreads);
  const int vpt = norm_vpt(a.H, frag, g.tpr);
  const int parts = 1 + (a.o ? 1 : 0) + (a.gate_kind == QMOE_GATE_FULL ? 1 : 0);
  const int threads = g.tpr * g.rpb;
  const bool all = a.o && a.w_post && a.w_pre && a.r && a.gate_kind != QMOE_GATE_FULL;
  const size_t ring = vec || a.dtype == QMOE_F32 ? (size_t)norm_ahead(vpt) * parts * vpt * threads * 16 : 0;
  return by_norm(a.dtype, vec, vpt, [&](auto dt, auto v, auto n) {
    auto kern = all ? block_norm_kernel<dt, v, n, true> : block_norm_kernel<dt, v, n, false>;
    const cudaError_t e = allow_shared(kern, ring, norm_ring_most(n));
    if (e != cudaSuccess) return e;
    int64_t blocks = (a.T + g.rpb - 1) / g.rpb;
    if (blocks > kSms) {   // as many as are resident at once
      int per = 0;
      const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kern, threads, ring);
      if (e != cudaSuccess) return e;
      blocks = std::min<int64_t>(blocks, (int64_t)kSms * std::max(1, per));
    }
    return launch_op(kern, dim3((unsigned)blocks), dim3(g.tpr, g.rpb), ring, s, a);
  });
}

}  // namespace qmoe
