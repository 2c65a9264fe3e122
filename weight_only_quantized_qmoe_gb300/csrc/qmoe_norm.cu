// The norms before and after a block, fused with the gate of its output and
// the residual scale, and their gradients.
//
//   oh = o * rstd_post, rstd_post = 1 / sqrt(mean(o^2) + eps)
//   n  = oh * w_post                        (w_post absent: n = o)
//   r  = residual_scale * x + gate * n      (gate absent: 1)
//   rh = r * rstd_pre,  rstd_pre = 1 / sqrt(mean(r^2) + eps)
//   h  = rh * w_pre
// and with incoming gradients dr, dh:
//   dr' = dr + rstd_pre * (dh w_pre - rh * mean(dh w_pre rh)),  dw_pre = sum_t dh rh
//   dx  = residual_scale * dr';  dn = dr' gate;  dgate = dr' n (summed to the gate's shape)
//   dw_post = sum_t dn oh;  do = rstd_post * (dn w_post - oh * mean(dn w_post oh))
//
// Memory-bound: a row lives in the registers of its threads between its two
// reductions, so x and o are read once and r and h written once.  The backward
// rebuilds r in 32 bits from x and o (which it reads anyway) instead of
// reading the rounded r.  Its sums over the rows stay in the registers of the
// thread that owns the column while a CTA walks its rows; the CTAs' sums go
// through a small fp32 workspace and a second launch adds them in order: no
// atomics, the same bits every run.
#include <algorithm>

#include "qmoe_ops.cuh"

namespace qmoe {

// Sum of v over the threads of a row (blockDim.x of them, a power of two; all
// threads of the block call it).  `red` holds a float per warp, twice.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* red) {
  const int width = min((int)blockDim.x, 32);
#pragma unroll
  for (int i = 0; i < N; ++i)
    for (int o = width >> 1; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (blockDim.x <= 32) return;
  const int tid = threadIdx.y * blockDim.x + threadIdx.x, warp = tid >> 5;
  const int nw = blockDim.x >> 5, w0 = threadIdx.y * nw;
  __syncthreads();   // the last sum's readers are done
  if ((tid & 31) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) red[warp * N + i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float s = 0.f;
    for (int q = 0; q < nw; ++q) s += red[(w0 + q) * N + i];
    v[i] = s;
  }
}

template <int DT, int VEC>
__device__ __forceinline__ void load_or(const void* p, size_t i, float fallback, float (&v)[VEC]) {
  if (p) {
    load_vec<DT, VEC>(p, i, v);
  } else {
#pragma unroll
    for (int q = 0; q < VEC; ++q) v[q] = fallback;
  }
}

// The gate of row t, columns c ..
template <int DT, int VEC>
__device__ __forceinline__ void load_gate(const NormArgs& a, int64_t t, int64_t c, float (&g)[VEC]) {
  switch (a.gate_kind) {
    case QMOE_GATE_CHANNEL: load_vec<DT, VEC>(a.gate, (size_t)c, g); break;
    case QMOE_GATE_FULL: load_vec<DT, VEC>(a.gate, (size_t)(t * a.ld_gate + c), g); break;
    default: {
      const float s = a.gate_kind == QMOE_GATE_TOKEN ? load_d<DT>(a.gate, (size_t)t) : 1.f;
#pragma unroll
      for (int q = 0; q < VEC; ++q) g[q] = s;
    }
  }
}

// A thread holds VPT vectors of VEC columns: vector p at column
// (p * blockDim.x + threadIdx.x) * VEC.
template <int DT, int VEC, int VPT>
__global__ void __launch_bounds__(512) block_norm_kernel(const NormArgs a) {
  __shared__ float red[16];
  const int64_t t = blockIdx.x * (int64_t)blockDim.y + threadIdx.y;
  const bool live = t < a.T;
  const float inv_h = 1.f / (float)a.H;
  float r[VPT][VEC], n[VPT][VEC];
  float ss[1] = {0.f};
#pragma unroll
  for (int p = 0; p < VPT; ++p) {
    const int64_t c = ((int64_t)p * blockDim.x + threadIdx.x) * VEC;
    if (live && c < a.H) {
      load_vec<DT, VEC>(a.x, (size_t)(t * a.ld_x + c), r[p]);
      if (a.o) {
        load_vec<DT, VEC>(a.o, (size_t)(t * a.ld_o + c), n[p]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) ss[0] = fmaf(n[p][i], n[p][i], ss[0]);
      }
    }
  }
  float rstd1 = 1.f;
  if (a.o && a.w_post) {
    row_sum<1>(ss, red);
    rstd1 = rsqrtf(ss[0] * inv_h + a.eps);
  }
  ss[0] = 0.f;
#pragma unroll
  for (int p = 0; p < VPT; ++p) {
    const int64_t c = ((int64_t)p * blockDim.x + threadIdx.x) * VEC;
    if (live && c < a.H) {
      float w[VEC], g[VEC];
      if (a.o) {
        load_or<DT, VEC>(a.w_post, (size_t)c, 1.f, w);
        load_gate<DT, VEC>(a, t, c, g);
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        r[p][i] *= a.residual_scale;
        if (a.o) r[p][i] = fmaf(g[i], n[p][i] * rstd1 * w[i], r[p][i]);
        ss[0] = fmaf(r[p][i], r[p][i], ss[0]);
      }
      if (a.r) store_vec<DT, VEC>(a.r, (size_t)(t * a.H + c), r[p]);
    }
  }
  if (a.rstd_post && live && threadIdx.x == 0) a.rstd_post[t] = rstd1;
  if (!a.w_pre) return;
  row_sum<1>(ss, red);
  const float rstd2 = rsqrtf(ss[0] * inv_h + a.eps);
  if (a.rstd_pre && live && threadIdx.x == 0) a.rstd_pre[t] = rstd2;
#pragma unroll
  for (int p = 0; p < VPT; ++p) {
    const int64_t c = ((int64_t)p * blockDim.x + threadIdx.x) * VEC;
    if (live && c < a.H) {
      float w[VEC];
      load_vec<DT, VEC>(a.w_pre, (size_t)c, w);
#pragma unroll
      for (int i = 0; i < VEC; ++i) w[i] *= r[p][i] * rstd2;
      store_vec<DT, VEC>(a.h, (size_t)(t * a.H + c), w);
    }
  }
}

// Sums over rows a CTA keeps, in this order in its slice of the workspace.
enum { SUM_PRE = 0, SUM_POST = 1, SUM_GATE = 2, SUM_KINDS = 3 };

template <int DT, int VEC, int VPT>
__global__ void __launch_bounds__(512) block_norm_grad_kernel(const NormArgs a) {
  __shared__ float red[32];
  const float inv_h = 1.f / (float)a.H;
  float s_pre[VPT][VEC], s_post[VPT][VEC], s_gate[VPT][VEC];
#pragma unroll
  for (int p = 0; p < VPT; ++p)
#pragma unroll
    for (int i = 0; i < VEC; ++i) s_pre[p][i] = s_post[p][i] = s_gate[p][i] = 0.f;
  // the block's rows advance together (their sums are block-wide barriers)
  for (int64_t t0 = blockIdx.x * (int64_t)blockDim.y; t0 < a.T; t0 += gridDim.x * (int64_t)blockDim.y) {
    const int64_t t = t0 + threadIdx.y;
    const bool live = t < a.T;
    const float rstd1 = live && a.o && a.w_post ? a.rstd_post[t] : 1.f;
    const float rstd2 = live && a.w_pre ? a.rstd_pre[t] : 0.f;
    float oh[VPT][VEC], rh[VPT][VEC], d2[VPT][VEC];
    float sum[1] = {0.f};
#pragma unroll
    for (int p = 0; p < VPT; ++p) {
      const int64_t c = ((int64_t)p * blockDim.x + threadIdx.x) * VEC;
      if (live && c < a.H) {
        float w[VEC], g[VEC];
        load_vec<DT, VEC>(a.x, (size_t)(t * a.ld_x + c), rh[p]);
        if (a.o) {
          load_vec<DT, VEC>(a.o, (size_t)(t * a.ld_o + c), oh[p]);
          load_or<DT, VEC>(a.w_post, (size_t)c, 1.f, w);
          load_gate<DT, VEC>(a, t, c, g);
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          rh[p][i] *= a.residual_scale;
          if (a.o) {
            oh[p][i] *= rstd1;
            rh[p][i] = fmaf(g[i], oh[p][i] * w[i], rh[p][i]);
          }
          rh[p][i] *= rstd2;
        }
        if (a.dh) {
          load_vec<DT, VEC>(a.dh, (size_t)(t * a.ld_dh + c), d2[p]);
          load_vec<DT, VEC>(a.w_pre, (size_t)c, w);
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            s_pre[p][i] = fmaf(d2[p][i], rh[p][i], s_pre[p][i]);
            d2[p][i] *= w[i];
            sum[0] = fmaf(d2[p][i], rh[p][i], sum[0]);
          }
        }
      }
    }
    if (a.dh) row_sum<1>(sum, red);
    const float m2 = sum[0] * inv_h;
    float sums[2] = {0.f, 0.f};   // of d1 oh, and of dr' n (gate of a token)
#pragma unroll
    for (int p = 0; p < VPT; ++p) {
      const int64_t c = ((int64_t)p * blockDim.x + threadIdx.x) * VEC;
      if (live && c < a.H) {
        float d[VEC], out[VEC];
        load_or<DT, VEC>(a.dr, (size_t)(t * a.ld_dr + c), 0.f, d);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          if (a.dh) d[i] += rstd2 * (d2[p][i] - rh[p][i] * m2);
          out[i] = a.residual_scale * d[i];
        }
        if (a.dx) store_vec<DT, VEC>(a.dx, (size_t)(t * a.H + c), out);
        if (a.o) {
          float w[VEC], g[VEC], dg[VEC];
          load_or<DT, VEC>(a.w_post, (size_t)c, 1.f, w);
          load_gate<DT, VEC>(a, t, c, g);
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            dg[i] = d[i] * (oh[p][i] * w[i]);
            const float dn = d[i] * g[i];
            s_post[p][i] = fmaf(dn, oh[p][i], s_post[p][i]);
            if (a.gate_kind == QMOE_GATE_CHANNEL) s_gate[p][i] += dg[i];
            sums[1] += dg[i];
            d2[p][i] = dn * w[i];
            sums[0] = fmaf(d2[p][i], oh[p][i], sums[0]);
          }
          if (a.gate_kind == QMOE_GATE_FULL && a.dgate) store_vec<DT, VEC>(a.dgate, (size_t)(t * a.H + c), dg);
        }
      }
    }
    if (!a.o) continue;
    row_sum<2>(sums, red);
    if (a.gate_kind == QMOE_GATE_TOKEN && a.dgate && live && threadIdx.x == 0) store_d<DT>(a.dgate, (size_t)t, sums[1]);
    const float m1 = a.w_post ? sums[0] * inv_h : 0.f;
    if (a.d_o) {
#pragma unroll
      for (int p = 0; p < VPT; ++p) {
        const int64_t c = ((int64_t)p * blockDim.x + threadIdx.x) * VEC;
        if (live && c < a.H) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) d2[p][i] = rstd1 * (d2[p][i] - oh[p][i] * m1);
          store_vec<DT, VEC>(a.d_o, (size_t)(t * a.H + c), d2[p]);
        }
      }
    }
  }
  // one slice of the workspace per row of the block
  float* part = a.partial + ((size_t)blockIdx.x * blockDim.y + threadIdx.y) * SUM_KINDS * (size_t)a.H;
#pragma unroll
  for (int p = 0; p < VPT; ++p) {
    const int64_t c = ((int64_t)p * blockDim.x + threadIdx.x) * VEC;
    if (c < a.H) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        if (a.dw_pre) part[SUM_PRE * a.H + c + i] = s_pre[p][i];
        if (a.dw_post) part[SUM_POST * a.H + c + i] = s_post[p][i];
        if (a.dgate && a.gate_kind == QMOE_GATE_CHANNEL) part[SUM_GATE * a.H + c + i] = s_gate[p][i];
      }
    }
  }
}

// Adds the slices of the workspace: 32 columns and 8 slices at a time a CTA,
// then the 8 partial sums in order.
template <int DT>
__global__ void __launch_bounds__(256) block_norm_sums_kernel(const NormArgs a, int slices) {
  __shared__ float part[8][33];
  const int kind = blockIdx.y;
  void* dst = kind == SUM_PRE ? a.dw_pre : kind == SUM_POST ? a.dw_post : (a.gate_kind == QMOE_GATE_CHANNEL ? a.dgate : nullptr);
  if (!dst) return;
  const int64_t c = blockIdx.x * (int64_t)32 + threadIdx.x;
  float s = 0.f;
  if (c < a.H)
    for (int q = threadIdx.y; q < slices; q += 8) s += a.partial[((size_t)q * SUM_KINDS + kind) * (size_t)a.H + c];
  part[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && c < a.H) {
#pragma unroll
    for (int q = 1; q < 8; ++q) s += part[q][threadIdx.x];
    store_d<DT>(dst, (size_t)c, s);
  }
}

namespace {

struct NormShape {
  int tpr, rpb, vpt;
};
// Threads of a row: enough for one vector each up to 512, then more vectors.
NormShape norm_shape(int64_t H, int vec) {
  const int64_t n = (H + vec - 1) / vec;
  NormShape s;
  s.tpr = 8;
  while (s.tpr < 512 && s.tpr < n) s.tpr *= 2;
  s.rpb = s.tpr >= 128 ? 1 : 128 / s.tpr;
  const int64_t need = (n + s.tpr - 1) / s.tpr;
  s.vpt = 1;
  while (s.vpt < need) s.vpt *= 2;
  return s;
}

bool norm_vec(const NormArgs& a) {
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

// Calls f(type, elements of a vector, vectors of a thread).
template <int DT, int VEC, typename F>
cudaError_t by_vpt(int vpt, F&& f) {
  using D = std::integral_constant<int, DT>;
  using V = std::integral_constant<int, VEC>;
  switch (vpt) {
    case 1: return f(D{}, V{}, std::integral_constant<int, 1>{});
    case 2: return f(D{}, V{}, std::integral_constant<int, 2>{});
    case 4: return f(D{}, V{}, std::integral_constant<int, 4>{});
    case 8: return f(D{}, V{}, std::integral_constant<int, 8>{});
    default: break;
  }
  if constexpr (VEC == 1) {
    if (vpt == 16) return f(D{}, V{}, std::integral_constant<int, 16>{});
    if (vpt == 32) return f(D{}, V{}, std::integral_constant<int, 32>{});
  }
  return cudaErrorInvalidValue;
}
template <typename F>
cudaError_t by_norm(int dtype, bool vec, int vpt, F&& f) {
  if (dtype == QMOE_F32) return vec ? by_vpt<QMOE_F32, 4>(vpt, f) : by_vpt<QMOE_F32, 1>(vpt, f);
  if (dtype == QMOE_F16) return vec ? by_vpt<QMOE_F16, 8>(vpt, f) : by_vpt<QMOE_F16, 1>(vpt, f);
  return vec ? by_vpt<QMOE_BF16, 8>(vpt, f) : by_vpt<QMOE_BF16, 1>(vpt, f);
}

// CTAs of the backward: two a multiprocessor, no more than there are rows.
constexpr int64_t kNormGradCtas = 304;
int64_t norm_grad_ctas(int64_t T, int rpb) { return std::min<int64_t>(kNormGradCtas, (T + rpb - 1) / rpb); }

}  // namespace

size_t block_norm_grad_workspace(int64_t T, int64_t H, int dtype) {
  // the larger of the two vector widths' needs (which one runs depends on alignment)
  size_t most = 0;
  for (int vec : {1, 16 / dtype_size(dtype)}) {
    const NormShape s = norm_shape(H, vec);
    most = std::max(most, (size_t)norm_grad_ctas(T, s.rpb) * s.rpb * SUM_KINDS * (size_t)H * sizeof(float));
  }
  return most;
}

cudaError_t launch_block_norm(const NormArgs& a, cudaStream_t s) {
  const bool vec = norm_vec(a);
  const NormShape g = norm_shape(a.H, vec ? 16 / dtype_size(a.dtype) : 1);
  return by_norm(a.dtype, vec, g.vpt, [&](auto dt, auto v, auto vpt) {
    block_norm_kernel<dt, v, vpt><<<(unsigned)((a.T + g.rpb - 1) / g.rpb), dim3(g.tpr, g.rpb), 0, s>>>(a);
    return cudaGetLastError();
  });
}

cudaError_t launch_block_norm_grad(const NormArgs& a, cudaStream_t s) {
  const bool vec = norm_vec(a);
  const NormShape g = norm_shape(a.H, vec ? 16 / dtype_size(a.dtype) : 1);
  const int64_t ctas = norm_grad_ctas(a.T, g.rpb);
  if (ctas > 0) {   // without rows the sums are zeros
    const cudaError_t e = by_norm(a.dtype, vec, g.vpt, [&](auto dt, auto v, auto vpt) {
      block_norm_grad_kernel<dt, v, vpt><<<(unsigned)ctas, dim3(g.tpr, g.rpb), 0, s>>>(a);
      return cudaGetLastError();
    });
    if (e != cudaSuccess) return e;
  }
  const dim3 grid((unsigned)((a.H + 31) / 32), SUM_KINDS), block(32, 8);
  const int slices = (int)(ctas * g.rpb);
  if (a.dtype == QMOE_F32) block_norm_sums_kernel<QMOE_F32><<<grid, block, 0, s>>>(a, slices);
  else if (a.dtype == QMOE_F16) block_norm_sums_kernel<QMOE_F16><<<grid, block, 0, s>>>(a, slices);
  else block_norm_sums_kernel<QMOE_BF16><<<grid, block, 0, s>>>(a, slices);
  return cudaGetLastError();
}

}  // namespace qmoe
