// The norms before and after a block: gradients.  With the forward's names
// (qmoe_norm.cu) and the incoming gradients dr, dh:
//
//   d   = dr + rstd_pre * (dh w_pre - rh * mean(dh w_pre rh)),  dw_pre = sum_t dh rh
//   dx  = residual_scale * d;  dgate = d n (summed to the gate's shape)
//   dw_post = sum_t d gate oh;  do = rstd_post * (u - oh * mean(u oh)), u = d gate w_post
//
// With a gate that is the same for a whole row or a whole column these share
// their sums: a token's dgate is the row's sum of d w_post oh, gate times which
// is the sum in do; and S = sum_t d oh (times the token gate) gives dw_post =
// gate S and a channel's dgate = w_post S.
//
// Memory-bound like the forward, with nearly as many instructions as the bytes
// leave time for.  r is rebuilt in 32 bits from x and o (which are read anyway)
// instead of reading the rounded r.  The sums over the rows stay in the
// registers of the thread that owns the column while a CTA walks its rows, a
// ring of rows ahead of itself; the CTAs' sums go through a small fp32
// workspace and a second launch adds them in order: no atomics, the same bits
// every run.  (bf16, 4096 rows of 4096 with a channel gate: 49 us alone, 4.1 TB/s,
// half of the issue slots in use; one CTA a multiprocessor, as the sums and a
// row's values take 116 registers of 512 threads.)
#include "qmoe_norm.cuh"

namespace qmoe {

// Rows in the ring of a CTA (see norm_ahead); up to five tensors a row here.
constexpr int norm_grad_ahead(int vpt) { return vpt == 1 ? 3 : vpt == 2 ? 2 : 0; }

// Whether a thread's columns are in shared memory instead of its registers: with
// two fragments a thread, whose sums and values fill the registers (bf16, 4096
// rows of 8192: 113 us; when this was chosen 121, in registers 159), and where
// more would be loaded for every row element by element (f32, 2048 rows of 8191:
// 153 us, loaded 197; 16 bytes at a time, rows of 8192: 136, loaded 124).
constexpr bool columns_shared(int vpt, bool vector) { return vpt == 2 || (vpt > 2 && !vector); }

// Sums over rows a CTA keeps, in this order in its slice of the workspace.
enum { SUM_PRE = 0, SUM_POST = 1, SUM_KINDS = 2 };

// ALL: both norms and every row gradient are there, and no gate of its own for
// every value, as in a training step.  Known when the kernel is compiled, the
// tests for each tensor leave the loop over the rows (bf16, with / without,
// 4096 rows of 4096: 56 / 62 us, 8192 of 2048: 63 / 68; a gate for every value
// gained nothing by it: 66 / 66).
template <int DT, bool VECTOR, int VPT, bool ALL>
__global__ void __launch_bounds__(512) block_norm_grad_kernel(const NormArgs a) {
  op_begin();
  using F = Frag<DT, VECTOR>;
  using T = typename ElemT<DT>::t;
  constexpr int N2 = F::n / 2, AHEAD = norm_grad_ahead(VPT);
  constexpr bool RING = kCopies<DT, VECTOR> && AHEAD > 0;
  // rows that are loaded when they are used: a load does not pass a store that
  // the source has before it (f32, 2048 rows of 8192 / 8191: 124 / 153 us, after
  // it 135 / 183; 8191 with a gate for every value 292, after it 243)
  constexpr bool EARLY = ALL && !RING;
  __shared__ float red[2 * 16];
  extern __shared__ __align__(16) uint8_t norm_ring[];
  const float inv_h = 1.f / (float)a.H;
  const bool full = !ALL && a.gate_kind == QMOE_GATE_FULL;
  const bool branch = ALL || a.o, pre_norm = ALL || a.dh, post_norm = ALL || a.w_post;
  const int64_t stride = gridDim.x * (int64_t)blockDim.y;
  int64_t t = blockIdx.x * (int64_t)blockDim.y + threadIdx.y;
  int turn = 0, parts = 0;
  const uint32_t ring = smem_u32(norm_ring);
  const Place<DT, VECTOR> me(a.H);
  Rows<DT, VECTOR, VPT, RING> x(a.x, a.ld_x, t, stride, ring, parts, me), o(a.o, a.ld_o, t, stride, ring, parts, me),
      dr(a.dr, a.ld_dr, t, stride, ring, parts, me), dh(a.dh, a.ld_dh, t, stride, ring, parts, me),
      g(full ? a.gate : nullptr, a.ld_gate, t, stride, ring, parts, me);
  const uint32_t row_bytes = parts * VPT * me.frag_bytes;
  constexpr bool SHARED = columns_shared(VPT, VECTOR) && kCopies<DT, VECTOR>;
  uint32_t cols = ring + AHEAD * row_bytes;
  const Columns<DT, VECTOR, VPT, SHARED> post(a.w_post, a.gate_kind == QMOE_GATE_CHANNEL ? a.gate : nullptr, me, cols),
      pre(a.w_pre, nullptr, me, cols);
  const int64_t out_step = stride * a.H;
  int64_t out = t * a.H + F::first(threadIdx.x);
  int64_t ahead = t;
  auto fetch = [&](uint32_t at) {
    if constexpr (RING) {
      if (ahead < a.T) {
        x.fetch(at, me);
        o.fetch(at, me);
        dr.fetch(at, me);
        dh.fetch(at, me);
        g.fetch(at, me);
      }
      ahead += stride;
      cp_async_commit();
    }
    x.advance();
    o.advance();
    dr.advance();
    dh.advance();
    g.advance();
  };

  float2 s_pre[VPT][N2], s_post[VPT][N2];
#pragma unroll
  for (int p = 0; p < VPT; ++p)
#pragma unroll
    for (int i = 0; i < N2; ++i) s_pre[p][i] = s_post[p][i] = both(0.f);

  if constexpr (RING) {
#pragma unroll
    for (int s = 0; s + 1 < AHEAD; ++s) fetch(s * row_bytes);
  }
  const uint32_t last = (RING ? AHEAD - 1 : 0) * row_bytes;
  uint32_t at = 0, to = last;
  // a row's scalars, loaded a row ahead
  float next1 = 1.f, next2 = 1.f, next_token = 1.f;
  auto scalars = [&](int64_t row) {
    if (row >= a.T) return;
    if (branch && post_norm) next1 = a.rstd_post[row];
    if (pre_norm) next2 = a.rstd_pre[row];
    if (a.gate_kind == QMOE_GATE_TOKEN) next_token = load_d<DT>(a.gate, (size_t)row);
  };
  scalars(t);
  for (; t - threadIdx.y < a.T; t += stride, out += out_step) {
    const bool live = t < a.T;
    const float rstd1 = next1, rstd2 = next2, token = next_token;
    scalars(t + stride);
    if constexpr (RING) {
      fetch(to);
      cp_async_wait<AHEAD - 1>();
    }
    // rh and dh * w_pre, and the first sum
    float2 rh[VPT][N2], dn[VPT][N2], sum2 = both(0.f);
    if (pre_norm) {
      const float2 cx = both(a.residual_scale * rstd2), co = both(rstd1 * token * rstd2);
#pragma unroll
      for (int p = 0; p < VPT; ++p) {
        if (live && me.has(p)) {
          float2 v[N2], w[N2];
          x.get(at, p, me, rh[p]);
#pragma unroll
          for (int i = 0; i < N2; ++i) rh[p][i] = mul2(rh[p][i], cx);
          if (branch) {
            o.get(at, p, me, v);
            post.get(p, me, w);
            if (full) {
              float2 q[N2];
              g.get(at, p, me, q);
#pragma unroll
              for (int i = 0; i < N2; ++i) v[i] = mul2(v[i], q[i]);
            }
#pragma unroll
            for (int i = 0; i < N2; ++i) rh[p][i] = fma2(mul2(v[i], co), w[i], rh[p][i]);
          }
          dh.get(at, p, me, v);
          pre.get(p, me, w);
#pragma unroll
          for (int i = 0; i < N2; ++i) {
            s_pre[p][i] = fma2(v[i], rh[p][i], s_pre[p][i]);
            dn[p][i] = mul2(v[i], w[i]);
            sum2 = fma2(dn[p][i], rh[p][i], sum2);
          }
        }
      }
      sum2.x = row_sum(sum2.x + sum2.y, red, turn) * inv_h * -rstd2;
    }
    const float2 m2 = both(sum2.x), k2 = both(rstd2);
    // d and what follows from it: dx, u = d gate w_post (into dn), the second sum
    float2 sum1 = both(0.f);
#pragma unroll
    for (int p = 0; p < VPT; ++p) {
      if (live && me.has(p)) {
        float2 d[N2], v[N2], w[N2];
        if (ALL || a.dr) {
          dr.get(at, p, me, d);
        } else {
#pragma unroll
          for (int i = 0; i < N2; ++i) d[i] = both(0.f);
        }
        if (pre_norm) {
#pragma unroll
          for (int i = 0; i < N2; ++i) d[i] = fma2(rh[p][i], m2, fma2(dn[p][i], k2, d[i]));
        }
        if constexpr (EARLY) {
          o.get(at, p, me, v);
          post.get(p, me, w);
        }
        if (ALL || a.dx) {
          float2 e[N2];
#pragma unroll
          for (int i = 0; i < N2; ++i) e[i] = mul2(d[i], both(a.residual_scale));
          put<DT, VECTOR>(static_cast<T*>(a.dx) + out, p, me, e);
        }
        if (branch) {
          const float2 c1 = both(rstd1 * token);
          if constexpr (!EARLY) {
            o.get(at, p, me, v);
            post.get(p, me, w);
          }
#pragma unroll
          for (int i = 0; i < N2; ++i) dn[p][i] = mul2(d[i], w[i]);
          if (full) {
            float2 q[N2], e[N2];
            g.get(at, p, me, q);
#pragma unroll
            for (int i = 0; i < N2; ++i) {
              e[i] = mul2(mul2(dn[p][i], v[i]), both(rstd1));
              dn[p][i] = mul2(dn[p][i], q[i]);
              d[i] = mul2(d[i], q[i]);
            }
            if (a.dgate) put<DT, VECTOR>(static_cast<T*>(a.dgate) + out, p, me, e);
          }
#pragma unroll
          for (int i = 0; i < N2; ++i) {
            if constexpr (!VECTOR) {   // past the row's end (an infinite factor would make NaN of its zeros)
              if (2 * i * me.threads >= me.left_of(p)) dn[p][i].x = d[i].x = 0.f;
              if ((2 * i + 1) * me.threads >= me.left_of(p)) dn[p][i].y = d[i].y = 0.f;
            }
            s_post[p][i] = fma2(mul2(d[i], c1), v[i], s_post[p][i]);
            sum1 = fma2(dn[p][i], v[i], sum1);
          }
        }
      }
    }
    if (branch) {
      // without w_post the branch is not normalised: do = u
      float s1 = 0.f;
      if (post_norm || a.gate_kind == QMOE_GATE_TOKEN) s1 = row_sum(sum1.x + sum1.y, red, turn) * rstd1;
      if (a.gate_kind == QMOE_GATE_TOKEN && a.dgate && live && threadIdx.x == 0) store_d<DT>(a.dgate, (size_t)t, s1);
      if (ALL || a.d_o) {
        const float2 cu = both(rstd1 * token), co = both(post_norm ? -s1 * token * inv_h * rstd1 * rstd1 : 0.f);
#pragma unroll
        for (int p = 0; p < VPT; ++p) {
          if (live && me.has(p)) {
            float2 v[N2];
            o.get(at, p, me, v);
#pragma unroll
            for (int i = 0; i < N2; ++i) v[i] = post_norm ? fma2(v[i], co, mul2(dn[p][i], cu)) : mul2(dn[p][i], cu);
            put<DT, VECTOR>(static_cast<T*>(a.d_o) + out, p, me, v);
          }
        }
      }
    }
    if constexpr (RING) {
      to = at;
      at = at == last ? 0 : at + row_bytes;
    } else {
      fetch(0);   // only steps to the next row
    }
  }
  if constexpr (RING) cp_async_wait<0>();
  // a slice of the workspace for each row of the block
  float* mine = a.partial + ((size_t)blockIdx.x * blockDim.y + threadIdx.y) * SUM_KINDS * (size_t)a.H;
#pragma unroll
  for (int p = 0; p < VPT; ++p) {
#pragma unroll
    for (int i = 0; i < 2 * N2; ++i) {
      const int64_t col = F::first(threadIdx.x) + p * me.step + (VECTOR ? i : i * me.threads);
      if (col >= a.H) continue;
      if (a.dw_pre) mine[SUM_PRE * a.H + col] = i & 1 ? s_pre[p][i / 2].y : s_pre[p][i / 2].x;
      if (branch) mine[SUM_POST * a.H + col] = i & 1 ? s_post[p][i / 2].y : s_post[p][i / 2].x;
    }
  }
}

// Adds the slices of the workspace: 32 columns a CTA, its ROWS rows of threads
// take every ROWS-th slice, then their sums in order.  SUM_POST gives both
// dw_post and a channel gate's gradient.
template <int DT, int ROWS, int AHEAD>
__global__ void __launch_bounds__(32 * ROWS) block_norm_sums_kernel(const NormArgs a, int slices) {
  op_begin();
  __shared__ float part[ROWS][33];
  const int kind = blockIdx.y;
  const bool channel = a.gate_kind == QMOE_GATE_CHANNEL;
  if (kind == SUM_PRE ? !a.dw_pre : !a.dw_post && !(channel && a.dgate)) return;
  const int64_t c = blockIdx.x * (int64_t)32 + threadIdx.x;
  float s = 0.f;
  if (c < a.H) {
    const float* p = a.partial + kind * (size_t)a.H + c;
#pragma unroll AHEAD
    for (int q = threadIdx.y; q < slices; q += ROWS) s += p[(size_t)q * SUM_KINDS * a.H];
  }
  part[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y != 0 || c >= a.H) return;
#pragma unroll
  for (int q = 1; q < ROWS; ++q) s += part[q][threadIdx.x];
  if (kind == SUM_PRE) {
    store_d<DT>(a.dw_pre, (size_t)c, s);
    return;
  }
  if (a.dw_post) store_d<DT>(a.dw_post, (size_t)c, channel ? s * load_d<DT>(a.gate, (size_t)c) : s);
  if (channel && a.dgate) store_d<DT>(a.dgate, (size_t)c, a.w_post ? s * load_d<DT>(a.w_post, (size_t)c) : s);
}

namespace {

// CTAs: 512 threads a multiprocessor (their sums' workspace grows with them),
// no more than there are rows.
int64_t norm_grad_ctas(int64_t T, const RowShape& g) {
  return std::min<int64_t>((int64_t)kSms * std::max(1, 512 / (g.tpr * g.rpb)), (T + g.rpb - 1) / g.rpb);
}

// The most shared memory a kernel takes: rings of x, o, dr, dh and a gate for
// every value, and columns, 512 threads.
constexpr int norm_grad_shared_most(int vpt, bool vector) {
  return (norm_grad_ahead(vpt) * 5 + (columns_shared(vpt, vector) ? 3 : 0)) * vpt * 512 * 16;
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
  const int columns = columns_shared(vpt, vec) ? 3 : 0;   // kept in shared memory
  const size_t ring =
      vec || a.dtype == QMOE_F32 ? (size_t)(norm_grad_ahead(vpt) * parts + columns) * vpt * g.tpr * g.rpb * 16 : 0;
  const int64_t ctas = norm_grad_ctas(a.T, g);
  const bool all = a.o && a.w_post && a.dr && a.dh && a.dx && a.d_o && a.gate_kind != QMOE_GATE_FULL;
  if (ctas > 0) {   // without rows the sums are zeros
    const cudaError_t e = by_norm(a.dtype, vec, vpt, [&](auto dt, auto v, auto n) {
      auto kern = all ? block_norm_grad_kernel<dt, v, n, true> : block_norm_grad_kernel<dt, v, n, false>;
      const cudaError_t err = allow_shared(kern, ring, norm_grad_shared_most(n, v));
      if (err != cudaSuccess) return err;
      return launch_op(kern, dim3((unsigned)ctas), dim3(g.tpr, g.rpb), ring, s, a);
    });
    if (e != cudaSuccess) return e;
  }
  // (both launches, us, 16 rows of threads / 32: 64 slices 10.9 / 11.8, 152 of
  // 2048 columns 57.4 / 56.4, 304 of 1001 18.8 / 17.6, 1216 of 512 35.5 / 32.6)
  const int slices = (int)(ctas * g.rpb);
  const dim3 grid((unsigned)((a.H + 31) / 32), SUM_KINDS);
  auto sums = [&](auto dt) {
    return slices < 128 ? launch_op(block_norm_sums_kernel<dt, 16, 4>, grid, dim3(32, 16), 0, s, a, slices)
                        : launch_op(block_norm_sums_kernel<dt, 32, 8>, grid, dim3(32, 32), 0, s, a, slices);
  };
  if (a.dtype == QMOE_F32) return sums(std::integral_constant<int, QMOE_F32>{});
  if (a.dtype == QMOE_F16) return sums(std::integral_constant<int, QMOE_F16>{});
  return sums(std::integral_constant<int, QMOE_BF16>{});
}

}  // namespace qmoe
