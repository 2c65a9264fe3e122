// The norms before and after a block: gradients.  With the forward's names
// (qmoe_norm.cu) and the incoming gradients dr, dh:
//
//   dr' = dr + rstd_pre * (dh w_pre - rh * mean(dh w_pre rh)),  dw_pre = sum_t dh rh
//   dx  = residual_scale * dr';  dn = dr' gate;  dgate = dr' n (summed to the gate's shape)
//   dw_post = sum_t dn oh;  do = rstd_post * (dn w_post - oh * mean(dn w_post oh))
//
// Memory-bound like the forward.  r is rebuilt in 32 bits from x and o (which
// are read anyway) instead of reading the rounded r.  The sums over the rows
// stay in the registers of the thread that owns the column while a CTA walks
// its rows, a ring of rows ahead of itself; the CTAs' sums go through a small
// fp32 workspace and a second launch adds them in order: no atomics, the
// same bits every run.
#include "qmoe_norm.cuh"

namespace qmoe {

// Rows in the ring of a CTA (see norm_ahead); up to five tensors a row here.
constexpr int norm_grad_ahead(int vpt) { return vpt == 1 ? 3 : vpt == 2 ? 2 : 0; }

// Sums over rows a CTA keeps, in this order in its slice of the workspace.
enum { SUM_PRE = 0, SUM_POST = 1, SUM_GATE = 2, SUM_KINDS = 3 };

// CHANNEL: a channel gate, whose gradient is a sum over the rows too.
template <int DT, bool VECTOR, int VPT, bool CHANNEL>
__global__ void __launch_bounds__(512) block_norm_grad_kernel(const NormArgs a) {
  using F = Frag<DT, VECTOR>;
  constexpr int N = F::n, kNormGradAhead = norm_grad_ahead(VPT);
  constexpr bool RING = VECTOR && kNormGradAhead > 0;
  __shared__ float red[2 * 16 * 2];
  extern __shared__ __align__(16) uint8_t norm_ring[];
  const int tid = threadIdx.y * blockDim.x + threadIdx.x, threads = blockDim.x * blockDim.y;
  const float inv_h = 1.f / (float)a.H;
  const bool full = !CHANNEL && a.gate_kind == QMOE_GATE_FULL;
  const int64_t stride = gridDim.x * (int64_t)blockDim.y;
  int turn = 0;
  // parts of a ring row: x, o, dr, dh, gate, as far as they are there
  const int q_o = 1, q_r = q_o + (a.o ? 1 : 0), q_h = q_r + (a.dr ? 1 : 0), q_g = q_h + (a.dh ? 1 : 0);
  const int parts = q_g + (full ? 1 : 0);
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
            if (a.o) cp_async16(slot(s, q_o, p), static_cast<const T*>(a.o) + t * a.ld_o + c);
            if (a.dr) cp_async16(slot(s, q_r, p), static_cast<const T*>(a.dr) + t * a.ld_dr + c);
            if (a.dh) cp_async16(slot(s, q_h, p), static_cast<const T*>(a.dh) + t * a.ld_dh + c);
            if (full) cp_async16(slot(s, q_g, p), static_cast<const T*>(a.gate) + t * a.ld_gate + c);
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

  float s_pre[VPT][N], s_post[VPT][N], s_gate[CHANNEL ? VPT : 1][N];
#pragma unroll
  for (int p = 0; p < VPT; ++p)
#pragma unroll
    for (int i = 0; i < N; ++i) s_pre[p][i] = s_post[p][i] = s_gate[CHANNEL ? p : 0][i] = 0.f;

  const int64_t first = blockIdx.x * (int64_t)blockDim.y + threadIdx.y;
#pragma unroll
  for (int s = 0; s + 1 < kNormGradAhead; ++s) fetch(first + s * stride, s);
  int s = 0;
  for (int64_t t = first; t - threadIdx.y < a.T; t += stride) {
    const bool live = t < a.T;
    fetch(t + (kNormGradAhead - 1) * stride, s == 0 ? kNormGradAhead - 1 : s - 1);
    const float rstd1 = live && a.o && a.w_post ? a.rstd_post[t] : 1.f;
    const float rstd2 = live && a.w_pre ? a.rstd_pre[t] : 0.f;
    const float token = live && a.gate_kind == QMOE_GATE_TOKEN ? load_d<DT>(a.gate, (size_t)t) : 1.f;
    auto gate = [&](int p, int64_t c, float (&g)[N]) {
      if (CHANNEL) {
        load_columns<DT, VECTOR>(a.gate, c, a.H, g);
      } else if (full) {
        part(s, q_g, p, a.gate, (size_t)(t * a.ld_gate), c, g);
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) g[i] = token;
      }
    };
    if constexpr (RING) cp_async_wait<kNormGradAhead - 1>();
    float oh[VPT][N], rh[VPT][N], d2[VPT][N];
    float sum[1] = {0.f};
#pragma unroll
    for (int p = 0; p < VPT; ++p) {
      const int64_t c = norm_column<DT, VECTOR>(p);
      if (live && c < a.H) {
        part(s, 0, p, a.x, (size_t)(t * a.ld_x), c, rh[p]);
#pragma unroll
        for (int i = 0; i < N; ++i) rh[p][i] *= a.residual_scale;
        if (a.o) {
          float w[N], g[N];
          part(s, q_o, p, a.o, (size_t)(t * a.ld_o), c, oh[p]);
          load_columns<DT, VECTOR>(a.w_post, c, a.H, w);
          gate(p, c, g);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            oh[p][i] *= rstd1;
            rh[p][i] = fmaf(g[i], oh[p][i] * w[i], rh[p][i]);
          }
        }
        if (a.dh) {
          float w[N];
          part(s, q_h, p, a.dh, (size_t)(t * a.ld_dh), c, d2[p]);
          load_columns<DT, VECTOR>(a.w_pre, c, a.H, w);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            rh[p][i] *= rstd2;
            s_pre[p][i] = fmaf(d2[p][i], rh[p][i], s_pre[p][i]);
            d2[p][i] *= w[i];
            sum[0] = fmaf(d2[p][i], rh[p][i], sum[0]);
          }
        }
      }
    }
    if (a.dh) row_sum<1>(sum, red, turn);
    const float m2 = sum[0] * inv_h;
    float sums[2] = {0.f, 0.f};   // of dn w_post oh, and of dr' n (the gate of a token)
#pragma unroll
    for (int p = 0; p < VPT; ++p) {
      const int64_t c = norm_column<DT, VECTOR>(p);
      if (live && c < a.H) {
        float d[N], out[N];
        if (a.dr) {
          part(s, q_r, p, a.dr, (size_t)(t * a.ld_dr), c, d);
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i) d[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (a.dh) d[i] += rstd2 * (d2[p][i] - rh[p][i] * m2);
          out[i] = a.residual_scale * d[i];
        }
        F f;
        if (a.dx) {
          f.set(out);
          f.store(a.dx, (size_t)(t * a.H), c, a.H, blockDim.x);
        }
        if (a.o) {
          float w[N], g[N], dg[N];
          load_columns<DT, VECTOR>(a.w_post, c, a.H, w);
          gate(p, c, g);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            // past the row's end every factor here is zero (o was loaded so)
            dg[i] = d[i] * (oh[p][i] * w[i]);
            const float dn = d[i] * g[i];
            s_post[p][i] = fmaf(dn, oh[p][i], s_post[p][i]);
            if (CHANNEL) s_gate[p][i] += dg[i];
            sums[1] += dg[i];
            d2[p][i] = dn * w[i];
            sums[0] = fmaf(d2[p][i], oh[p][i], sums[0]);
          }
          if (full && a.dgate) {
            f.set(dg);
            f.store(a.dgate, (size_t)(t * a.H), c, a.H, blockDim.x);
          }
        }
      }
    }
    if (a.o) {
      row_sum<2>(sums, red, turn);
      if (a.gate_kind == QMOE_GATE_TOKEN && a.dgate && live && threadIdx.x == 0) store_d<DT>(a.dgate, (size_t)t, sums[1]);
      const float m1 = a.w_post ? sums[0] * inv_h : 0.f;
      if (a.d_o) {
#pragma unroll
        for (int p = 0; p < VPT; ++p) {
          const int64_t c = norm_column<DT, VECTOR>(p);
          if (live && c < a.H) {
#pragma unroll
            for (int i = 0; i < N; ++i) d2[p][i] = rstd1 * (d2[p][i] - oh[p][i] * m1);
            F f;
            f.set(d2[p]);
            f.store(a.d_o, (size_t)(t * a.H), c, a.H, blockDim.x);
          }
        }
      }
    }
    if (++s == kNormGradAhead) s = 0;
  }
  if constexpr (RING) cp_async_wait<0>();
  // a slice of the workspace for each row of the block
  float* mine = a.partial + ((size_t)blockIdx.x * blockDim.y + threadIdx.y) * SUM_KINDS * (size_t)a.H;
#pragma unroll
  for (int p = 0; p < VPT; ++p) {
    const int64_t c = norm_column<DT, VECTOR>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t x = VECTOR ? c + i : c + (int64_t)i * blockDim.x;
      if (x >= a.H) continue;
      if (a.dw_pre) mine[SUM_PRE * a.H + x] = s_pre[p][i];
      if (a.dw_post) mine[SUM_POST * a.H + x] = s_post[p][i];
      if (CHANNEL && a.dgate) mine[SUM_GATE * a.H + x] = s_gate[CHANNEL ? p : 0][i];
    }
  }
}

// Adds the slices of the workspace: 32 columns a CTA, its 16 rows of threads
// take every 16th slice, then their sums in order.
constexpr int kSumRows = 16;
template <int DT>
__global__ void __launch_bounds__(32 * kSumRows) block_norm_sums_kernel(const NormArgs a, int slices) {
  __shared__ float part[kSumRows][33];
  const int kind = blockIdx.y;
  void* dst = kind == SUM_PRE ? a.dw_pre : kind == SUM_POST ? a.dw_post : (a.gate_kind == QMOE_GATE_CHANNEL ? a.dgate : nullptr);
  if (!dst) return;
  const int64_t c = blockIdx.x * (int64_t)32 + threadIdx.x;
  float s = 0.f;
  if (c < a.H) {
    const float* p = a.partial + kind * (size_t)a.H + c;
#pragma unroll 4
    for (int q = threadIdx.y; q < slices; q += kSumRows) s += p[(size_t)q * SUM_KINDS * a.H];
  }
  part[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && c < a.H) {
#pragma unroll
    for (int q = 1; q < kSumRows; ++q) s += part[q][threadIdx.x];
    store_d<DT>(dst, (size_t)c, s);
  }
}

namespace {

// CTAs: 512 threads a multiprocessor (their sums' workspace grows with them),
// no more than there are rows.
int64_t norm_grad_ctas(int64_t T, const RowShape& g) {
  return std::min<int64_t>((int64_t)kNormSms * std::max(1, 512 / (g.tpr * g.rpb)), (T + g.rpb - 1) / g.rpb);
}

}  // namespace

size_t block_norm_grad_workspace(int64_t T, int64_t H, int dtype) {
  // the larger of the two ways' needs (alignment decides which one runs)
  size_t most = 0;
  for (bool vec : {false, true}) {
    const RowShape s = row_shape(H, norm_frag(dtype, vec));
    most = std::max(most, (size_t)norm_grad_ctas(T, s) * s.rpb * SUM_KINDS * (size_t)H * sizeof(float));
  }
  return most;
}

cudaError_t launch_block_norm_grad(const NormArgs& a, cudaStream_t s) {
  const bool vec = norm_vec(a);
  const int frag = norm_frag(a.dtype, vec);
  const RowShape g = row_shape(a.H, frag);
  const int vpt = norm_vpt(a.H, frag, g.tpr);
  const int parts = 1 + (a.o ? 1 : 0) + (a.dr ? 1 : 0) + (a.dh ? 1 : 0) + (a.gate_kind == QMOE_GATE_FULL ? 1 : 0);
  const size_t ring = vec ? (size_t)norm_grad_ahead(vpt) * parts * vpt * g.tpr * g.rpb * 16 : 0;
  const int64_t ctas = norm_grad_ctas(a.T, g);
  if (ctas > 0) {   // without rows the sums are zeros
    const cudaError_t e = by_norm(a.dtype, vec, vpt, [&](auto dt, auto v, auto n) {
      auto run = [&](auto kern) {
        if (ring > 40 * 1024) {   // beside the static sums: past the 48 KB a launch gets unasked
          const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ring);
          if (err != cudaSuccess) return err;
        }
        kern<<<(unsigned)ctas, dim3(g.tpr, g.rpb), ring, s>>>(a);
        return cudaGetLastError();
      };
      return a.gate_kind == QMOE_GATE_CHANNEL ? run(block_norm_grad_kernel<dt, v, n, true>)
                                              : run(block_norm_grad_kernel<dt, v, n, false>);
    });
    if (e != cudaSuccess) return e;
  }
  const dim3 grid((unsigned)((a.H + 31) / 32), SUM_KINDS), block(32, kSumRows);
  const int slices = (int)(ctas * g.rpb);
  if (a.dtype == QMOE_F32) block_norm_sums_kernel<QMOE_F32><<<grid, block, 0, s>>>(a, slices);
  else if (a.dtype == QMOE_F16) block_norm_sums_kernel<QMOE_F16><<<grid, block, 0, s>>>(a, slices);
  else block_norm_sums_kernel<QMOE_BF16><<<grid, block, 0, s>>>(a, slices);
  return cudaGetLastError();
}

}  // namespace qmoe
