// The norms before and after a block, fused with the gate of its output and
// the residual scale: forward.
//
//   oh = o * rstd_post, rstd_post = 1 / sqrt(mean(o^2) + eps)
//   n  = oh * w_post                        (w_post absent: n = o)
//   r  = residual_scale * x + gate * n      (gate absent: 1)
//   rh = r * rstd_pre,  rstd_pre = 1 / sqrt(mean(r^2) + eps)
//   h  = rh * w_pre
//
// Memory-bound: a row stays in its threads' registers between the two sums,
// so x and o are read once and r and h written once.  The two sums of a row
// follow one another, so what decides is how many rows are on their way
// meanwhile: CTAs stay and walk the rows, a ring of rows ahead of themselves.
#include "qmoe_norm.cuh"

namespace qmoe {

// Rows in the ring of a CTA, the one in work among them, as its shared memory
// allows; 0: rows are loaded when they are used.
constexpr int norm_ahead(int vpt) { return vpt <= 2 ? 3 : vpt == 4 ? 2 : 0; }

template <int DT, bool VECTOR, int VPT>
__global__ void __launch_bounds__(512) block_norm_kernel(const NormArgs a) {
  using F = Frag<DT, VECTOR>;
  constexpr int N = F::n, kNormAhead = norm_ahead(VPT);
  constexpr bool RING = VECTOR && kNormAhead > 0;
  __shared__ float red[2 * 16];
  extern __shared__ __align__(16) uint8_t norm_ring[];
  const int tid = threadIdx.y * blockDim.x + threadIdx.x, threads = blockDim.x * blockDim.y;
  const float inv_h = 1.f / (float)a.H;
  const bool full = a.gate_kind == QMOE_GATE_FULL;
  const int parts = 1 + (a.o ? 1 : 0) + (full ? 1 : 0);
  const int64_t stride = gridDim.x * (int64_t)blockDim.y;
  int turn = 0;
  // slot of vector p of part q (x, o, gate) in ring row s
  auto slot = [&](int s, int q, int p) { return norm_ring + (((size_t)s * parts + q) * VPT + p) * threads * 16 + tid * 16; };
  auto fetch = [&](int64_t t, int s) {
    if constexpr (RING) {
      if (t < a.T) {
        using T = typename ElemT<DT>::t;
#pragma unroll
        for (int p = 0; p < VPT; ++p) {
          const int64_t c = norm_column<DT, VECTOR>(p);
          if (c < a.H) {
            cp_async16(slot(s, 0, p), static_cast<const T*>(a.x) + t * a.ld_x + c);
            if (a.o) cp_async16(slot(s, 1, p), static_cast<const T*>(a.o) + t * a.ld_o + c);
            if (full) cp_async16(slot(s, 2, p), static_cast<const T*>(a.gate) + t * a.ld_gate + c);
          }
        }
      }
      cp_async_commit();
    }
  };
  auto part = [&](int s, int q, int p, const void* base, size_t row, int64_t c, float (&v)[N]) {
    F f;
    if constexpr (RING) f.u = *reinterpret_cast<const uint4*>(slot(s, q, p));
    else f.load(base, row, c, a.H, blockDim.x);
    f.get(v);
  };

  const int64_t first = blockIdx.x * (int64_t)blockDim.y + threadIdx.y;
#pragma unroll
  for (int s = 0; s + 1 < kNormAhead; ++s) fetch(first + s * stride, s);
  int s = 0;
  // the rows of a block advance together (their sums share barriers)
  for (int64_t t = first; t - threadIdx.y < a.T; t += stride) {
    const bool live = t < a.T;
    fetch(t + (kNormAhead - 1) * stride, s == 0 ? kNormAhead - 1 : s - 1);
    if constexpr (RING) cp_async_wait<kNormAhead - 1>();
    float r[VPT][N], n[VPT][N];
    float ss[1] = {0.f};
#pragma unroll
    for (int p = 0; p < VPT; ++p) {
      const int64_t c = norm_column<DT, VECTOR>(p);
      if (live && c < a.H) {
        part(s, 0, p, a.x, (size_t)(t * a.ld_x), c, r[p]);
        if (a.o) {
          part(s, 1, p, a.o, (size_t)(t * a.ld_o), c, n[p]);
#pragma unroll
          for (int i = 0; i < N; ++i) ss[0] = fmaf(n[p][i], n[p][i], ss[0]);
        }
      }
    }
    float rstd1 = 1.f;
    if (a.o && a.w_post) {
      row_sum<1>(ss, red, turn);
      rstd1 = rsqrtf(ss[0] * inv_h + a.eps);
    }
    const float token = live && a.gate_kind == QMOE_GATE_TOKEN ? load_d<DT>(a.gate, (size_t)t) : 1.f;
    ss[0] = 0.f;
#pragma unroll
    for (int p = 0; p < VPT; ++p) {
      const int64_t c = norm_column<DT, VECTOR>(p);
      if (live && c < a.H) {
        if (a.o) {
          float w[N], g[N];
          load_columns<DT, VECTOR>(a.w_post, c, a.H, w);
          if (full) {
            part(s, 2, p, a.gate, (size_t)(t * a.ld_gate), c, g);
          } else if (a.gate_kind == QMOE_GATE_CHANNEL) {
            load_columns<DT, VECTOR>(a.gate, c, a.H, g);
          } else {
#pragma unroll
            for (int i = 0; i < N; ++i) g[i] = token;
          }
#pragma unroll
          for (int i = 0; i < N; ++i) r[p][i] = fmaf(g[i], n[p][i] * rstd1 * w[i], a.residual_scale * r[p][i]);
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i) r[p][i] *= a.residual_scale;
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (VECTOR || c + (int64_t)i * blockDim.x < a.H) ss[0] = fmaf(r[p][i], r[p][i], ss[0]);
        if (a.r) {
          F f;
          f.set(r[p]);
          f.store(a.r, (size_t)(t * a.H), c, a.H, blockDim.x);
        }
      }
    }
    if (a.rstd_post && live && threadIdx.x == 0) a.rstd_post[t] = rstd1;
    if (a.w_pre) {
      row_sum<1>(ss, red, turn);
      const float rstd2 = rsqrtf(ss[0] * inv_h + a.eps);
      if (a.rstd_pre && live && threadIdx.x == 0) a.rstd_pre[t] = rstd2;
#pragma unroll
      for (int p = 0; p < VPT; ++p) {
        const int64_t c = norm_column<DT, VECTOR>(p);
        if (live && c < a.H) {
          float w[N];
          load_columns<DT, VECTOR>(a.w_pre, c, a.H, w);
#pragma unroll
          for (int i = 0; i < N; ++i) w[i] *= r[p][i] * rstd2;
          F f;
          f.set(w);
          f.store(a.h, (size_t)(t * a.H), c, a.H, blockDim.x);
        }
      }
    }
    if (++s == kNormAhead) s = 0;
  }
  if constexpr (RING) cp_async_wait<0>();
}

cudaError_t launch_block_norm(const NormArgs& a, cudaStream_t s) {
  const bool vec = norm_vec(a);
  const int frag = norm_frag(a.dtype, vec);
  // two fragments a thread up to 512 threads: enough rows at once, and few
  // enough registers for two CTAs a multiprocessor
  const RowShape g = row_shape(a.H, frag, a.H > 2 * 256 * frag ? 512 : 256);
  const int vpt = norm_vpt(a.H, frag, g.tpr);
  const int parts = 1 + (a.o ? 1 : 0) + (a.gate_kind == QMOE_GATE_FULL ? 1 : 0);
  const int threads = g.tpr * g.rpb;
  const size_t ring = vec ? (size_t)norm_ahead(vpt) * parts * vpt * threads * 16 : 0;
  return by_norm(a.dtype, vec, vpt, [&](auto dt, auto v, auto n) {
    auto kern = block_norm_kernel<dt, v, n>;
    if (ring > 40 * 1024) {   // beside the static sums: past the 48 KB a launch gets unasked
      const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ring);
      if (e != cudaSuccess) return e;
    }
    int64_t blocks = (a.T + g.rpb - 1) / g.rpb;
    if (blocks > kNormSms) {   // as many as are resident at once
      int per = 0;
      const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kern, threads, ring);
      if (e != cudaSuccess) return e;
      blocks = std::min<int64_t>(blocks, (int64_t)kNormSms * std::max(1, per));
    }
    kern<<<(unsigned)blocks, dim3(g.tpr, g.rpb), ring, s>>>(a);
    return cudaGetLastError();
  });
}

}  // namespace qmoe
