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
// the logits themselves nothing is rounded and nothing repeated.  (A softmax over
// +infinity has no scores: that token's choice goes by its logits, its weights are NaN.)
//
// Bound: instructions and latency.  A warp takes a token: lane l holds the logits of
// experts l, l + 32, ..., sorted; a rank is one redux for the best key and one for
// the lowest index at it.  The logits are read once, two 4-byte words a token and
// rank written.  (8192 tokens, eight of 256 experts in f32, 8.4 MB: softmax 10.4 us,
// sigmoid with a random bias 15.6, with the four best of eight groups 17.3, softmax
// with a bias 22.5; the gradient 4.3.  Half of the issue slots are used.  Some ten of
// these tokens are repeated in 64 bits, and one that is takes as long as a third of
// the others together; more CTAs, fewer registers or a warp that loads its next
// token's logits early changed nothing.)  Equal neighbours are repeated too, and a bias
// of zeros makes many where logits are coarse or their scores near one: bf16 logits
// of spread 1.5 and 8 by sigmoid 23 and 39 us, by softmax 56 and 102; f32 logits of
// spread 5 and 8 by sigmoid 26 and 36.
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

// A score in 64 bits; mx and sum: of a softmax.
__device__ __forceinline__ double score64(int scoring, double l, double mx, double sum) {
  return scoring == QMOE_SCORE_SOFTMAX ? exp(l - mx) / sum : 1.0 / (1.0 + exp(-l));
}
// Sum of a softmax in 64 bits.  (Unrolled, here and below: an exponential in 64
// bits is some 3000 cycles of latency.)
template <int DT>
__device__ double softmax_sum64(const typename ElemT<DT>::t* row, int E, double mx) {
  double sum = 0.0;
#pragma unroll 4
  for (int e = threadIdx.x & 31; e < E; e += 32) {
    const double l = load_d<DT>(row, e);
    sum += l == l ? exp(l - mx) : 0.0;
  }
  return warp_sum(sum);
}

// The value of an order key (topk_order_key).
__device__ __forceinline__ float ordered_float(int key) { return __int_as_float(key ^ ((key >> 31) & INT_MAX)); }

// The two largest of a warp's values, in every lane (`lanes` of them that go together).
template <typename F>
__device__ __forceinline__ void two_best(F& a1, F& a2, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) {
    const F b1 = __shfl_xor_sync(kAll, a1, o), b2 = __shfl_xor_sync(kAll, a2, o);
    a2 = fmax(fmax(a2, b2), fmin(a1, b1));
    a1 = fmax(a1, b1);
  }
}
// How many groups come before this lane's own: larger, or equal with a lower index.
template <typename F>
__device__ __forceinline__ int group_rank(F score, unsigned among) {
  const int lane = threadIdx.x & 31;
  int rank = 0;
  for (unsigned m = among; m; m &= m - 1) {
    const int h = __ffs(m) - 1;
    const F other = __shfl_sync(kAll, score, h);
    rank += other > score || (other == score && h < lane) ? 1 : 0;
  }
  return rank;
}

// The r best of a few groups (bits of `among`) by scores in 64 bits.  c: the
// experts' values in 32, -infinity where one may not be chosen.
template <int DT>
__device__ __noinline__ unsigned best_groups64(const ChoiceArgs& a, const typename ElemT<DT>::t* row, const float* c, float mx,
                                               unsigned among, int r) {
  const int lane = threadIdx.x & 31, n = a.E / a.groups;
  const double low = -static_cast<double>(INFINITY);
  const double sum = a.scoring == QMOE_SCORE_SOFTMAX ? softmax_sum64<DT>(row, a.E, mx) : 1.0;
  double mine = low;
  for (unsigned m = among; m; m &= m - 1) {
    const int g = __ffs(m) - 1;
    double a1 = low, a2 = low;
#pragma unroll 4
    for (int j = lane; j < n; j += 32) {
      const int e = g * n + j;
      if (c[e] > -INFINITY) {
        const double v = score64(a.scoring, load_d<DT>(row, e), mx, sum) + (a.bias ? (double)a.bias[e] : 0.0);
        a2 = fmax(a2, fmin(a1, v));
        a1 = fmax(a1, v);
      }
    }
    two_best(a1, a2, 32);
    if (lane == g) mine = a.best == 2 && a2 != low ? a1 + a2 : a1;
  }
  const int rank = group_rank(mine, among);   // by every lane: it shuffles
  return __ballot_sync(kAll, (among >> lane & 1u) && rank < r);
}

// The top_groups best groups, a bit each.  c: as above, in shared memory.  A
// group's score is its best, or the sum of its two best (one where it has one; half of
// it here, which cannot overflow); the lanes are shared among the groups.  by_score: c
// is rounded, by tau / 2 of each value and 2^-24 of its own size, and of the terms of a
// sum that nearly cancel both show.  Groups whose bounds reach over the border go by
// their scores in 64 bits.
template <int DT>
__device__ __forceinline__ unsigned best_groups(const ChoiceArgs& a, const typename ElemT<DT>::t* row, const float* c, float mx,
                                                bool by_score, float tau) {
  const int lane = threadIdx.x & 31, n = a.E / a.groups;
  int per = 32;   // lanes of a group
  while (per * a.groups > 32) per >>= 1;
  const int g = lane / per;
  float a1 = -INFINITY, a2 = -INFINITY;
  if (g < a.groups)
    for (int j = lane % per; j < n; j += per) {
      const float v = c[g * n + j];
      a2 = fmaxf(a2, fminf(a1, v));
      a1 = fmaxf(a1, v);
    }
  two_best(a1, a2, per);
  float size = fabsf(a1);   // of its terms
  if (a.best == 2) {
    const float second = a2 == -INFINITY ? 0.f : 0.5f * a2;
    a1 = 0.5f * a1 + second;
    size = 0.5f * size + fabsf(second);
  }
  // group g's in lane g
  const float score = __shfl_sync(kAll, a1, (lane * per) & 31);
  const unsigned all = a.groups == 32 ? kAll : (1u << a.groups) - 1u;
  const bool one = lane < a.groups;
  const int rank = group_rank(score, all);
  const bool kept = rank < a.top_groups;
  const unsigned open = __ballot_sync(kAll, one && kept);
  if (!by_score) return open;
  // Bounds of the score, twice what the above comes to.  Infinite ones are exact.
  const float off = tau + 0x1p-22f * __shfl_sync(kAll, size, (lane * per) & 31);
  const float low = isinf(score) ? score : score - off, high = isinf(score) ? score : score + off;
  // the least bound of a group kept, the greatest of one left out
  const float in = ordered_float(topk_redux_min(one && kept ? topk_order_key(low) : INT_MAX));
  const float out = ordered_float(topk_redux_max(one && !kept ? topk_order_key(high) : INT_MIN));
  if (out == -INFINITY || in > out) return open;
  const unsigned sure = __ballot_sync(kAll, one && kept && low > out);
  const unsigned among = __ballot_sync(kAll, one && score > -INFINITY && (kept ? low <= out : high >= in));
  return sure | best_groups64<DT>(a, row, c, mx, among, a.top_groups - __popc(sure));
}

// The choice of a token in 64 bits from the open groups, by a whole warp; c: room
// for E values.  Lane j gets the expert of rank j, or -1.
template <int DT>
__device__ __noinline__ int choose64(const ChoiceArgs& a, const typename ElemT<DT>::t* row, float mx, unsigned open, double* c) {
  const int lane = threadIdx.x & 31, E = a.E, n = E / a.groups;
  const double low = -static_cast<double>(INFINITY);
  const double sum = a.scoring == QMOE_SCORE_SOFTMAX ? softmax_sum64<DT>(row, E, mx) : 1.0;
  __syncwarp();
#pragma unroll 4
  for (int e = lane; e < E; e += 32) {
    const double l = load_d<DT>(row, e);
    const double v = l > low && (open >> (e / n) & 1u) ? score64(a.scoring, l, mx, sum) + (double)a.bias[e] : low;
    c[e] = v > low ? v : low;   // NaN too
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
  const double sum = a.scoring == QMOE_SCORE_SOFTMAX ? softmax_sum64<DT>(row, a.E, mx) : 1.0;
  const double v = e >= 0 ? score64(a.scoring, load_d<DT>(row, e), mx, sum) + (double)a.bias[e] : -static_cast<double>(INFINITY);
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

// The choice of a token whose softmax is over +infinity, so that it has no scores: by
// the logits, and of the groups with the largest.  c: room for E values.
template <int DT>
__device__ __noinline__ int choose_by_logits(const ChoiceArgs& a, const typename ElemT<DT>::t* row, float* c) {
  const int lane = threadIdx.x & 31, E = a.E, n = E / a.groups;
  __syncwarp();
  for (int e = lane; e < E; e += 32) {
    const float l = load_d<DT>(row, e);
    c[e] = l > -INFINITY && (!a.bias || a.bias[e] > -INFINITY) ? l : -INFINITY;   // NaN closes too
  }
  __syncwarp();
  float group = -INFINITY;   // of lane g
  if (lane < a.groups)
    for (int j = 0; j < n; ++j) group = fmaxf(group, c[lane * n + j]);
  const int rank = group_rank(group, a.groups == 32 ? kAll : (1u << a.groups) - 1u);
  const unsigned open = __ballot_sync(kAll, lane < a.groups && rank < a.top_groups);
  int mine = -1;
  for (int slot = 0; slot < a.k; ++slot) {
    int v = INT_MIN, at = INT_MAX;
    for (int e = lane; e < E; e += 32)
      if (c[e] > -INFINITY && (open >> (e / n) & 1u) && topk_order_key(c[e]) > v) {
        v = topk_order_key(c[e]);
        at = e;
      }
    const int best = topk_redux_max(v);
    if (best == INT_MIN) break;
    at = topk_redux_min(v == best ? at : INT_MAX);
    if (lane == slot) mine = at;
    if (lane == (at & 31)) c[at] = -INFINITY;
    __syncwarp();
  }
  return mine;
}

// A lane's keys (INT_MIN: none) of experts lane, lane + 32, ...  Up to eight are
// sorted once, best first, and the head drops out as it is chosen; more are looked
// through for every rank.
template <int NPL>
struct LaneKeys {
  static constexpr bool sorted = NPL <= 8;
  int key[NPL], idx[sorted ? NPL : 1];
  __device__ __forceinline__ void sort() {
    if constexpr (sorted) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) idx[i] = (threadIdx.x & 31) + 32 * i;
      // neighbours change places only where the second is larger: equal keys keep their order
#pragma unroll
      for (int round = 0; round < NPL; ++round) {
#pragma unroll
        for (int i = round & 1; i + 1 < NPL; i += 2) {
          const bool swap = key[i + 1] > key[i];
          const int k = key[i], x = idx[i];
          key[i] = swap ? key[i + 1] : k;
          idx[i] = swap ? idx[i + 1] : x;
          key[i + 1] = swap ? k : key[i + 1];
          idx[i + 1] = swap ? x : idx[i + 1];
        }
      }
    }
  }
  __device__ __forceinline__ int index(int i) const {
    if constexpr (sorted) return idx[i];
    else return (threadIdx.x & 31) + 32 * i;
  }
  __device__ __forceinline__ void best(int& k, int& at) const {
    k = key[0];
    at = index(0);
    if constexpr (!sorted) {
#pragma unroll
      for (int i = 1; i < NPL; ++i)
        if (key[i] > k) {
          k = key[i];
          at = index(i);
        }
    }
  }
  __device__ __forceinline__ void drop(int sel) {
    if constexpr (sorted) {
      const bool pop = idx[0] == sel;
#pragma unroll
      for (int i = 0; i + 1 < NPL; ++i) {
        key[i] = pop ? key[i + 1] : key[i];
        idx[i] = pop ? idx[i + 1] : idx[i];
      }
      if (pop) key[NPL - 1] = INT_MIN;
    } else {
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (sel == index(i)) key[i] = INT_MIN;
    }
  }
};

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

  LaneKeys<NPL> keys;
  unsigned open = kAll;   // groups
  // how far two rounded keys may be off their difference: each by 2^-24 of its
  // score times 4 (sigmoid: the error of the exponential, 2 + 1.2 |l| steps, counts
  // s (1 - s) times; a sum and a division) or 42 (softmax: with the sum of E terms,
  // up to 32 of them one after the other in a lane), taken as 8 and 64, and by its
  // own rounding
  float tau = 0.f;
  {
    float c[NPL];
    if (by_score) {
      const float inv = 1.f / sum;
      tau = softmax ? inv * 0x1p-17f : 0x1p-20f;
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const int e = lane + 32 * i;
        float v = softmax ? __expf(l[i] - mx) * inv : __fdividef(1.f, 1.f + __expf(-l[i]));
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
      open = best_groups<DT>(a, row, sm, mx, by_score, tau);
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = lane + 32 * i;
      const float v = a.bias ? c[i] : l[i];
      const bool may = c[i] > -INFINITY && (!filter || (open >> ((uint32_t)e * a.group_magic >> 20) & 1u));
      keys.key[i] = may ? topk_order_key(v) : INT_MIN;
    }
  }
  keys.sort();
  bool unsure = false;
  int mine = -1, before = INT_MAX, kth = 0;
  for (int slot = 0; slot <= k; ++slot) {   // one more than asked for: the border of the last
    int best, at;
    keys.best(best, at);
    const int m = topk_redux_max(best);
    if (m == INT_MIN || (slot == k && !a.bias)) break;
    if (a.bias && slot > 0) {
      const float x = ordered_float(before), y = ordered_float(m);
      if (!(x - y > tau + 0x1p-22f * (fabsf(x) + fabsf(y)))) unsure = true;
    }
    before = m;
    if (slot == k) break;
    kth = m;
    const int sel = topk_redux_min(best == m ? at : INT_MAX);
    if (lane == slot) mine = sel;
    keys.drop(sel);
  }
  if (unsure) {   // (the same for the whole warp)
    // those chosen, and those left that are as near to the last of them
    const float last = ordered_float(kth), least = last - (tau + 0x1p-21f * fabsf(last));
    double* room = choice_smem + (size_t)warp * a.room;
    int* list = reinterpret_cast<int*>(room);
    int n = __popc(__ballot_sync(kAll, mine >= 0));
    __syncwarp();
    if (mine >= 0) list[lane] = mine;   // the lanes from 0 on
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int kv = keys.key[i];
      const bool near = kv != INT_MIN && !(ordered_float(kv) < least);
      const unsigned who = __ballot_sync(kAll, near);
      const int at = n + __popc(who & ((1u << lane) - 1u));
      if (near && at < 32) list[at] = keys.index(i);
      n += __popc(who);
    }
    __syncwarp();
    if (n <= 32) mine = choose64_of<DT>(a, row, lane < n ? list[lane] : -1, mx, list);
    else mine = choose64<DT>(a, row, mx, open, room);
  }

  // every score was NaN, so that nothing could be chosen
  if (softmax && by_score && mx == INFINITY) mine = choose_by_logits<DT>(a, row, reinterpret_cast<float*>(choice_smem + (size_t)warp * a.room));

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
  const int n = a.E / a.groups;   // e / n = (e * magic) >> 20, exactly, for e and n up to 1024
  args.group_magic = (uint32_t)(((1 << 20) + n - 1) / n);
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
