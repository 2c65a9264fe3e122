// The router: experts chosen by their scores, and the gradient of the logits.
//
//   s_e = softmax(l)_e or sigmoid(l_e);  c_e = s_e + bias_e (without a bias the
//   order of the logits, the same but for rounding);  a group's score is the sum
//   of its one or two best c;  the k best c of the best groups are chosen, ties
//   to the lower index;  w_j = scale * s_j, or scale * s_j / (sum of the chosen s).
//
// The choice is that of scores in 64 bits.  It is made in 32 (FP64 runs at a
// 64th of the rate here): where two neighbours in the order are nearer than 32
// bits can tell, the warp repeats the token's choice in 64.  With keys that are
// the logits themselves nothing is rounded and nothing repeated.
//
// Bound: latency.  A warp takes a token: lane l holds the logits of experts l,
// l + 32, ..., a rank is one redux for the best key and one for the lowest index
// at it.  The logits are read once, two 4-byte words a token and rank written.
#include <algorithm>
#include <climits>

#include "qmoe_ops.cuh"
#include "qmoe_topk.cuh"

namespace qmoe {

constexpr int kChoiceWarps = 4;   // tokens of a CTA
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// Whether group g of `groups` is among the `top` best, as a bit per group.  c:
// the values of the experts, -infinity where one may not be chosen; a group's
// score is its best, or the sum of its two best (one where it has one).  32 lanes
// are shared among the groups.  unsure: set if the border between the last
// group kept and the first left out is nearer than tau + rel * their magnitude.
template <typename F>
__device__ __forceinline__ unsigned best_groups(const F* c, int E, int groups, int top, int best, F tau, F rel, bool* unsure) {
  const int lane = threadIdx.x & 31, n = E / groups;
  int per = 32;   // lanes of a group
  while (per * groups > 32) per >>= 1;
  const int g = lane / per, sub = lane % per;
  const F low = -static_cast<F>(INFINITY);
  F a1 = low, a2 = low;
  if (g < groups)
    for (int j = sub; j < n; j += per) {
      const F v = c[g * n + j];
      a2 = fmax(a2, fmin(a1, v));
      a1 = fmax(a1, v);
    }
  for (int o = per >> 1; o > 0; o >>= 1) {
    const F b1 = __shfl_xor_sync(kAll, a1, o), b2 = __shfl_xor_sync(kAll, a2, o);
    a2 = fmax(fmax(a2, b2), fmin(a1, b1));
    a1 = fmax(a1, b1);
  }
  const F score = best == 2 && a2 != low ? a1 + a2 : a1;
  int rank = 0;
  for (int h = 0; h < groups; ++h) {
    const F other = __shfl_sync(kAll, score, h * per);
    rank += other > score || (other == score && h < g) ? 1 : 0;
  }
  const bool one = sub == 0 && g < groups, kept = one && rank < top;
  const unsigned mask = __ballot_sync(kAll, kept);
  if (unsure) {
    // the last group kept and the first left out
    const unsigned last = __ballot_sync(kAll, one && rank == top - 1), next = __ballot_sync(kAll, one && rank == top);
    const F x = __shfl_sync(kAll, score, __ffs(last) - 1), y = __shfl_sync(kAll, score, __ffs(next) - 1);
    if (y != low && !(x - y > tau + rel * (fabs(x) + fabs(y)))) *unsure = true;
  }
  unsigned bits = 0;
  for (int h = 0; h < groups; ++h) bits |= (mask >> (h * per) & 1u) << h;
  return bits;
}

// The choice of a token in 64 bits, by a whole warp; c: room for E values.
// Lane j gets the expert of rank j, or -1.
template <int DT>
__device__ __noinline__ int choose64(const ChoiceArgs& a, const typename ElemT<DT>::t* row, double* c) {
  const int lane = threadIdx.x & 31, E = a.E;
  const double low = -static_cast<double>(INFINITY);
  double mx = low, sum = 0.0;
  if (a.scoring == QMOE_SCORE_SOFTMAX) {
    float m = -INFINITY;
    for (int e = lane; e < E; e += 32) m = fmaxf(m, load_d<DT>(row, e));
    mx = warp_max(m);
#pragma unroll 4
    for (int e = lane; e < E; e += 32) {
      const double l = load_d<DT>(row, e);
      sum += l == l ? exp(l - mx) : 0.0;
    }
    sum = warp_sum(sum);   // (unrolled loops: an exponential in 64 bits is some 3000 cycles of latency)
  }
  auto score = [&](double l) { return a.scoring == QMOE_SCORE_SOFTMAX ? exp(l - mx) / sum : 1.0 / (1.0 + exp(-l)); };
  const bool filter = a.top_groups < a.groups;
  // the keys of the groups: the scores themselves where there is no bias
#pragma unroll 4
  for (int e = lane; e < E; e += 32) {
    const double l = load_d<DT>(row, e);
    const double v = l > low ? score(l) + (a.bias ? (double)a.bias[e] : 0.0) : low;
    c[e] = v > low ? v : low;   // NaN too
  }
  __syncwarp();
  unsigned bits = kAll;
  if (filter) bits = best_groups<double>(c, E, a.groups, a.top_groups, a.best, 0.0, 0.0, nullptr);
  __syncwarp();
  const int n = E / a.groups;
  for (int e = lane; e < E; e += 32) {
    if (filter && !(bits >> (e / n) & 1u)) c[e] = low;
    else if (!a.bias && c[e] > low) c[e] = load_d<DT>(row, e);
  }
  __syncwarp();
  int mine = -1;
  for (int slot = 0; slot < a.k; ++slot) {
    double v = low;
    int at = INT_MAX;
    for (int e = lane; e < E; e += 32)
      if (c[e] > v) {
        v = c[e];
        at = e;
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double w = __shfl_xor_sync(kAll, v, o);
      const int b = __shfl_xor_sync(kAll, at, o);
      if (w > v || (w == v && b < at)) {
        v = w;
        at = b;
      }
    }
    if (at == INT_MAX) break;
    if (lane == slot) mine = at;
    if (lane == (at & 31)) c[at] = low;
    __syncwarp();
  }
  return mine;
}

// The same where only a few experts may be among the k best: lane i has one of n,
// `e` (-1: none).  list: room for 32.
template <int DT>
__device__ __noinline__ int choose64_of(const ChoiceArgs& a, const typename ElemT<DT>::t* row, int e, float mx, int* list) {
  const int lane = threadIdx.x & 31;
  double v = -static_cast<double>(INFINITY);
  if (a.scoring == QMOE_SCORE_SOFTMAX) {
    double sum = 0.0;
#pragma unroll 4
    for (int i = lane; i < a.E; i += 32) {
      const double l = load_d<DT>(row, i);
      sum += l == l ? exp(l - mx) : 0.0;
    }
    sum = warp_sum(sum);
    if (e >= 0) v = exp((double)load_d<DT>(row, e) - mx) / sum + (double)a.bias[e];
  } else if (e >= 0) {
    v = 1.0 / (1.0 + exp(-(double)load_d<DT>(row, e))) + (double)a.bias[e];
  }
  int rank = 0;
  for (int i = 0; i < 32; ++i) {
    const double w = __shfl_sync(kAll, v, i);
    const int f = __shfl_sync(kAll, e, i);
    rank += f >= 0 && (w > v || (w == v && f < e)) ? 1 : 0;
  }
  __syncwarp();
  list[lane] = -1;
  __syncwarp();
  if (e >= 0 && rank < a.k) list[rank] = e;
  __syncwarp();
  return list[lane];
}

template <int DT, int NPL>
__global__ void __launch_bounds__(32 * kChoiceWarps) choice_kernel(const ChoiceArgs a) {
  op_begin();
  extern __shared__ double choice_smem[];   // a.room a warp, where the choice may need them
  using T = typename ElemT<DT>::t;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.E, k = a.k;
  const int64_t t = blockIdx.x * (int64_t)kChoiceWarps + warp;
  if (t >= a.T) return;
  const T* row = static_cast<const T*>(a.logits) + (size_t)(t * a.ld);
  const bool softmax = a.scoring == QMOE_SCORE_SOFTMAX, filter = a.top_groups < a.groups;
  const bool by_score = a.bias || (filter && a.best == 2);   // keys that are rounded

  float l[NPL];
  bool nan = false;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = lane + 32 * i;
    l[i] = e < E ? load_d<DT>(row, e) : -INFINITY;
    if (isnan(l[i])) {   // never chosen
      nan = true;
      l[i] = -INFINITY;
    }
  }
  // softmax over all experts
  float mx = 0.f, sum = 1.f;
  if (softmax && (by_score || !a.renorm)) {
    float m = l[0];
#pragma unroll
    for (int i = 1; i < NPL; ++i) m = fmaxf(m, l[i]);
    mx = warp_max(m);
    sum = 0.f;
    if (mx > -INFINITY) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) sum += expf(l[i] - mx);
    }
    sum = warp_sum(sum);
  }

  int key[NPL];
  unsigned open = kAll;   // groups
  bool unsure = false;
  // how far two rounded keys may be off their difference: each by 2^-24 of its
  // score times 4 (sigmoid: an exponential, a sum, a division) or 42 (softmax:
  // with the sum of E terms, up to 32 of them one after the other in a lane),
  // taken as 8 and 64, and by its own rounding
  float tau = 0.f;
  {
    float c[NPL];
    if (by_score) {
      const float inv = 1.f / sum;
      tau = softmax ? inv * 0x1p-17f : 0x1p-20f;
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const int e = lane + 32 * i;
        float v = softmax ? expf(l[i] - mx) * inv : 1.f / (1.f + expf(-l[i]));
        if (a.bias && e < E) v += a.bias[e];
        if (isnan(v) && l[i] > -INFINITY) nan = true;
        c[i] = l[i] > -INFINITY && v > -INFINITY ? v : -INFINITY;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NPL; ++i) c[i] = l[i];
    }
    if (filter) {
      float* sm = reinterpret_cast<float*>(choice_smem + (size_t)warp * a.room);
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (lane + 32 * i < E) sm[lane + 32 * i] = c[i];
      __syncwarp();
      open = best_groups<float>(sm, E, a.groups, a.top_groups, a.best, tau + tau, 0x1p-21f, by_score ? &unsure : nullptr);
      __syncwarp();
    }
    const int n = E / a.groups;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = lane + 32 * i;
      const float v = a.bias ? c[i] : l[i];
      const bool may = c[i] > -INFINITY && (!filter || (open >> (e / n) & 1u));
      key[i] = may ? topk_order_key(v) : INT_MIN;
    }
  }
  const bool groups_unsure = __any_sync(kAll, unsure);
  int mine = -1, before = INT_MAX, kth = 0;
  for (int slot = 0; slot <= k; ++slot) {   // one more than asked for: the border of the last
    int best = key[0], at = lane;
#pragma unroll
    for (int i = 1; i < NPL; ++i)
      if (key[i] > best) {
        best = key[i];
        at = lane + 32 * i;
      }
    const int m = topk_redux_max(best);
    if (m == INT_MIN || (slot == k && !a.bias)) break;
    if (a.bias && slot > 0) {
      const float x = __int_as_float(before ^ ((before >> 31) & INT_MAX)), y = __int_as_float(m ^ ((m >> 31) & INT_MAX));
      if (!(x - y > tau + 0x1p-22f * (fabsf(x) + fabsf(y)))) unsure = true;
    }
    before = m;
    if (slot == k) break;
    kth = m;
    const int sel = topk_redux_min(best == m ? at : INT_MAX);
    if (lane == slot) mine = sel;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (sel == lane + 32 * i) key[i] = INT_MIN;
  }
  if (groups_unsure) {
    mine = choose64<DT>(a, row, choice_smem + (size_t)warp * a.room);
  } else if (unsure) {
    // those chosen, and those left that are as near to the last of them
    const float last = __int_as_float(kth ^ ((kth >> 31) & INT_MAX)), least = last - (tau + 0x1p-21f * fabsf(last));
    int* list = reinterpret_cast<int*>(choice_smem + (size_t)warp * a.room);
    int n = __popc(__ballot_sync(kAll, mine >= 0));
    __syncwarp();
    if (mine >= 0) list[lane] = mine;   // the lanes from 0 on
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const bool near = key[i] != INT_MIN && !(__int_as_float(key[i] ^ ((key[i] >> 31) & INT_MAX)) < least);
      const unsigned who = __ballot_sync(kAll, near);
      const int at = n + __popc(who & ((1u << lane) - 1u));
      if (near && at < 32) list[at] = lane + 32 * i;
      n += __popc(who);
    }
    __syncwarp();
    if (n <= 32) mine = choose64_of<DT>(a, row, lane < n ? list[lane] : -1, mx, list);
    else mine = choose64<DT>(a, row, choice_smem + (size_t)warp * a.room);
  }

  const float chosen = mine >= 0 ? load_d<DT>(row, mine) : -INFINITY;
  float w = 0.f;
  if (softmax && !a.renorm) {
    if (mine >= 0) w = expf(chosen - mx) / sum;
  } else if (!a.renorm) {
    if (mine >= 0) w = 1.f / (1.f + expf(-chosen));
  } else {
    // relative to the largest, so that scores too small for 32 bits keep their ratios
    const float m = warp_max(chosen);
    float p = 0.f;
    if (mine >= 0)
      p = softmax ? expf(chosen - m) : m > 0.f ? 1.f / (1.f + expf(-chosen)) : expf(chosen - m) / (1.f + expf(chosen));
    const float all = warp_sum(p);
    if (mine >= 0) w = p / all;
  }
  w *= a.scale;
  if (__any_sync(kAll, nan)) w = NAN;
  if (lane < k) {
    const size_t r = (size_t)t * k + lane;
    a.ids[r] = mine;
    a.w[r] = w;
  }
}

// dl = (dw / dl)^T dweights.  With g_j = scale * dweights_j and u_j the weights
// without their scale:
//   softmax             p_e ([e chosen] g_e - sum_j g_j u_j)
//   softmax, renormed   u_j (g_j - sum g u)          of the chosen, 0 of the others
//   sigmoid             s_j (1 - s_j) g_j
//   sigmoid, renormed   u_j (1 - s_j) (g_j - sum g u)
// An expert named twice gets the sum of its slots' terms, in their order.
template <int DT, int NPL>
__global__ void __launch_bounds__(32 * kChoiceWarps) choice_grad_kernel(const ChoiceArgs a) {
  op_begin();
  using T = typename ElemT<DT>::t;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.E, k = a.k;
  const int64_t t = blockIdx.x * (int64_t)kChoiceWarps + warp;
  if (t >= a.T) return;
  const T* row = static_cast<const T*>(a.logits) + (size_t)(t * a.ld);
  T* out = static_cast<T*>(a.dlogits) + (size_t)(t * E);
  const bool softmax = a.scoring == QMOE_SCORE_SOFTMAX;
  int id = lane < k ? a.ids[(size_t)t * k + lane] : -1;
  const bool has = id >= 0 && id < E;
  if (!has) id = -1;
  const float g = has ? a.scale * a.dw[(size_t)t * k + lane] : 0.f;
  const float chosen = has ? load_d<DT>(row, id) : -INFINITY;
  float mine;   // what this slot adds
  if (softmax && !a.renorm) {
    float l[NPL], m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = lane + 32 * i;
      l[i] = e < E ? load_d<DT>(row, e) : -INFINITY;
      m = fmaxf(m, l[i]);
    }
    m = warp_max(m);
    if (m == -INFINITY) m = 0.f;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      l[i] = expf(l[i] - m);
      sum += l[i];
    }
    sum = warp_sum(sum);
    const float inv = sum > 0.f || isnan(sum) ? 1.f / sum : 0.f;
    const float u = has ? expf(chosen - m) * inv : 0.f, all = warp_sum(g * u);
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = lane + 32 * i;
      if (e < E) store_d<DT>(out, e, -(l[i] * inv) * all);
    }
    mine = g * u;
    // the chosen ones' whole value replaces what was just written
    float total = 0.f;
    for (int j = 0; j < k; ++j) {
      const float v = __shfl_sync(kAll, mine, j);
      if (__shfl_sync(kAll, id, j) == id) total += v;
    }
    __syncwarp();
    if (has) store_d<DT>(out, id, total - u * all);
    return;
  }
  for (int e = lane; e < E; e += 32) store_d<DT>(out, e, 0.f);
  const float s = 1.f / (1.f + expf(-chosen)), rest = 1.f / (1.f + expf(chosen));   // sigmoid, 1 - sigmoid
  if (!a.renorm) {
    mine = has ? g * s * rest : 0.f;
  } else {
    const float m = warp_max(chosen);
    const float p = !has ? 0.f : softmax ? expf(chosen - m) : m > 0.f ? s : expf(chosen - m) / (1.f + expf(chosen));
    const float all = warp_sum(p), u = has ? p / all : 0.f, mean = warp_sum(g * u);
    mine = has ? u * (softmax ? 1.f : rest) * (g - mean) : 0.f;
  }
  float total = 0.f;
  for (int j = 0; j < k; ++j) {
    const float v = __shfl_sync(kAll, mine, j);
    if (__shfl_sync(kAll, id, j) == id) total += v;
  }
  __syncwarp();
  if (has) store_d<DT>(out, id, total);
}

namespace {

template <typename F>
cudaError_t with_types(const ChoiceArgs& a, F&& f) {
  auto pick = [&](auto dt) {
    const int npl = (a.E + 31) / 32;
    if (npl <= 2) return f(dt, std::integral_constant<int, 2>{});
    if (npl <= 4) return f(dt, std::integral_constant<int, 4>{});
    if (npl <= 8) return f(dt, std::integral_constant<int, 8>{});
    if (npl <= 16) return f(dt, std::integral_constant<int, 16>{});
    return f(dt, std::integral_constant<int, 32>{});
  };
  if (a.dtype == QMOE_F32) return pick(std::integral_constant<int, QMOE_F32>{});
  if (a.dtype == QMOE_F16) return pick(std::integral_constant<int, QMOE_F16>{});
  return pick(std::integral_constant<int, QMOE_BF16>{});
}

}  // namespace

cudaError_t launch_choice(const ChoiceArgs& a, cudaStream_t s) {
  const unsigned blocks = (unsigned)((a.T + kChoiceWarps - 1) / kChoiceWarps);
  ChoiceArgs args = a;
  args.room = a.bias || a.top_groups < a.groups ? std::max(a.E, 32) : 0;
  const size_t smem = sizeof(double) * kChoiceWarps * args.room;   // at most 32 KB
  return with_types(a, [&](auto dt, auto npl) {
    return launch_op(choice_kernel<decltype(dt)::value, decltype(npl)::value>, dim3(blocks), dim3(32 * kChoiceWarps), smem, s, args);
  });
}

cudaError_t launch_choice_grad(const ChoiceArgs& a, cudaStream_t s) {
  const unsigned blocks = (unsigned)((a.T + kChoiceWarps - 1) / kChoiceWarps);
  return with_types(a, [&](auto dt, auto npl) {
    return launch_op(choice_grad_kernel<decltype(dt)::value, decltype(npl)::value>, dim3(blocks), dim3(32 * kChoiceWarps), 0, s, a);
  });
}

}  // namespace qmoe
