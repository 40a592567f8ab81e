// Experts and their weights from router scores.
//
// Scores are the softmax or the sigmoid of a token's logits.  Chosen are the k
// experts of the largest score + bias, of equal ones the lowest id, within the
// top_groups groups whose two best add up to most; weights are the scores, over
// their sum where renormalised, times a scale.  A logit that is not finite
// cannot be chosen.
//
// Which expert comes first is decided as in 64 bits.  Without bias and groups
// the logits' own order decides, exactly.  Otherwise values are made in fp32,
// whose error is at most kUlps half units of the score and of the sum; where
// two neighbours in the order (or the last group in and the first one out) lie
// nearer to one another than that, the warp makes the values that can matter
// again in 64 bits and chooses by those.
//
// A warp per token; lane L holds the experts L * kPer .. + kPer - 1, so a lower
// lane means a lower id.
#include "layer.cuh"
#include "typed.cuh"

namespace mmvq {

constexpr int kRouteWarps = 4;

// sigmoid(x) times exp(-c) where c = min(top, 0): the largest of several stays
// at a half or above however small they all are.
__device__ __forceinline__ float sigmoid_over(float x, float c) {
  return expf(fminf(x, 0.0f) - c) / (1.0f + expf(-fabsf(x)));
}

__device__ __forceinline__ double shfl_xor_f64(double v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }

template <typename T, int kPer>
struct RouteRow {
  const RouteTopk& a;
  const T* x;
  int lane, group_size;
  double* wide;  // [n_experts] of this warp
  float top, total;  // softmax: the largest logit and the sum of exp(x - top)

  __device__ __forceinline__ int expert(int i) const { return lane * kPer + i; }
  __device__ __forceinline__ bool finite(float v) const { return fabsf(v) < INFINITY; }
  __device__ __forceinline__ float score(float v) const {
    return a.sigmoid ? sigmoid_over(v, 0.0f) : expf(v - top) / total;
  }

  // In 64 bits: values of experts of kept groups that are at least `cut` in fp32 (all where cut is -inf), the
  // groups chosen again where `groups` says so; then the k best.  Lane j leaves with the id of choice j, or -1.
  __device__ __noinline__ int choose_wide(uint32_t keep, float cut, bool groups, const float (&v)[kPer]) {
    double z = 0.0;
    if (!a.sigmoid) {
      for (int i = 0; i < kPer; ++i) {
        const float l = expert(i) < a.n_experts ? to_f32(x[expert(i)]) : INFINITY;
        if (finite(l)) z += exp((double)l - (double)top);
      }
      for (int o = 16; o; o >>= 1) z += shfl_xor_f64(z, o);
    }
    const double minus = -(double)INFINITY;
#pragma unroll 1
    for (int i = 0; i < kPer; ++i) {
      const int e = expert(i);
      if (e >= a.n_experts) break;
      const float l = to_f32(x[e]);
      double d = minus;
      if (finite(l) && (groups || ((keep >> (e / group_size)) & 1)) && v[i] >= cut) {
        d = a.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - (double)top) / z;
        if (a.bias) d += (double)a.bias[e];
      }
      wide[e] = d;
    }
    __syncwarp();
    if (groups) {
      double two = minus;
      if (lane < a.n_groups) {
        double b1 = minus, b2 = minus;
        for (int e = lane * group_size; e < (lane + 1) * group_size; ++e) {
          const double d = wide[e];
          if (d > b1) { b2 = b1; b1 = d; } else if (d > b2) { b2 = d; }
        }
        two = b2 == minus ? b1 : b1 + b2;
      }
      int rank = 0;
      for (int g = 0; g < a.n_groups; ++g) {
        const double other = __shfl_sync(0xffffffffu, two, g);
        rank += other > two || (other == two && g < lane);
      }
      keep = __ballot_sync(0xffffffffu, lane < a.n_groups && rank < a.top_groups);
    }
    int mine = -1;
    for (int j = 0; j < a.k; ++j) {
      double b = minus;
      int id = 0x7fffffff;
      for (int i = 0; i < kPer; ++i) {
        const int e = expert(i);
        if (e < a.n_experts && ((keep >> (e / group_size)) & 1) && wide[e] > b) { b = wide[e]; id = e; }
      }
      for (int o = 16; o; o >>= 1) {
        const double ob = shfl_xor_f64(b, o);
        const int oi = __shfl_xor_sync(0xffffffffu, id, o);
        if (ob > b || (ob == b && oi < id)) { b = ob; id = oi; }
      }
      if (b == minus) break;
      if (lane == j) mine = id;
      if (id / kPer == lane) wide[id] = minus;
      __syncwarp();
    }
    return mine;
  }
};

template <typename T, int kPer>
__global__ void __launch_bounds__(32 * kRouteWarps) route_topk_kernel(const RouteTopk a) {
  extern __shared__ double wide_all[];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
  if (t >= a.n_tokens) return;
  RouteRow<T, kPer> r{a, static_cast<const T*>(a.logits) + t * a.ld, lane, a.n_experts / a.n_groups, wide_all + warp * a.n_experts, 0.0f, 1.0f};
  const bool grouped = a.top_groups < a.n_groups;
  const bool exact = !a.bias && !grouped;  // the logits' order is the scores'
  // half units that a value's fp32 error stays within: exp, sum, quotient and the sum with the bias
  constexpr float kUlps = (kPer + 24) * 0x1p-24f;

  float x[kPer], v[kPer];
  float top = -INFINITY;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    x[i] = -INFINITY;
    if (r.expert(i) < a.n_experts) x[i] = to_f32(r.x[r.expert(i)]);
    if (!(x[i] < INFINITY)) {  // NaN or +inf
      bad = true;
      x[i] = -INFINITY;
    }
    top = fmaxf(top, x[i]);
  }
  if (bad && a.status) *a.status = MMVQ_ERR_VALUE;
  top = warp_max(top);
  r.top = top == -INFINITY ? 0.0f : top;
  if (!a.sigmoid) {
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) z += expf(x[i] - r.top);
    r.total = warp_sum(z);
  }
  uint32_t keep = 0xffffffffu;
  bool groups_near = false;  // two groups are too near to tell
  if (exact) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = x[i];
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      v[i] = -INFINITY;
      if (x[i] > -INFINITY) v[i] = r.score(x[i]) + (a.bias ? a.bias[r.expert(i)] : 0.0f);
    }
  }
  if (grouped) {
    // lane g's group: its two best, one after another
    float two = -INFINITY, size = 0.0f;
    for (int g = 0; g < a.n_groups; ++g) {
      float b[2];
      int skip = -1;
      for (int n = 0; n < 2; ++n) {
        float m = -INFINITY;
        int id = -1;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int e = r.expert(i);
          if (e / r.group_size == g && e != skip && v[i] > m) { m = v[i]; id = e; }
        }
        b[n] = warp_max(m);
        const uint32_t who = __ballot_sync(0xffffffffu, m == b[n] && id >= 0);
        skip = who ? __shfl_sync(0xffffffffu, id, __ffs(who) - 1) : -1;
      }
      if (lane == g) {
        two = b[1] == -INFINITY ? b[0] : b[0] + b[1];
        // scores are at most 1 and the value less the bias: an error of both values and of their sum
        size = b[0] == -INFINITY ? 0.0f : 3.0f + fabsf(b[0]) + (b[1] == -INFINITY ? 0.0f : fabsf(b[1]));
      }
    }
    int rank = 0;
    float out = -INFINITY, in = INFINITY, most = 0.0f;
    for (int g = 0; g < a.n_groups; ++g) {
      const float other = __shfl_sync(0xffffffffu, two, g);
      rank += other > two || (other == two && g < lane);
    }
    const bool kept = lane < a.n_groups && rank < a.top_groups;
    keep = __ballot_sync(0xffffffffu, kept);
    if (kept) in = two;
    if (lane < a.n_groups && !kept) out = two;
    in = -warp_max(-in);
    out = warp_max(out);
    most = warp_max(size);
    groups_near = out > -INFINITY && in - out <= 2.0f * kUlps * most;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (r.expert(i) < a.n_experts && !((keep >> (r.expert(i) / r.group_size)) & 1)) v[i] = -INFINITY;
  }

  // k rounds of the best of all lanes; lane j keeps choice j, every lane the one after the last
  int mine = -1;
  float mv = -INFINITY, nv = -INFINITY;
  int next = -1;
  float left[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) left[i] = v[i];
  for (int j = 0; j <= a.k; ++j) {
    float m = -INFINITY;
    int at = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (left[i] > m) { m = left[i]; at = i; }
    const float b = warp_max(m);
    if (b == -INFINITY) break;
    const int who = __ffs(__ballot_sync(0xffffffffu, m == b)) - 1;
    const int id = __shfl_sync(0xffffffffu, r.expert(at), who);
    if (j == a.k) {
      nv = b;
      next = id;
      break;
    }
    if (lane == j) {
      mine = id;
      mv = b;
    }
    if (lane == who) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i == at) left[i] = -INFINITY;
    }
  }
  float mx = mine >= 0 ? to_f32(r.x[mine]) : -INFINITY;
  if (!exact) {
    const float fv = __shfl_down_sync(0xffffffffu, mv, 1);
    const int fi = __shfl_down_sync(0xffffffffu, mine, 1);
    const float v1 = lane == a.k - 1 ? nv : fv;
    const int i1 = lane == a.k - 1 ? next : fi;
    bool close = false;
    float slack = 0.0f;
    if (mine >= 0 && i1 >= 0) {
      const float x1 = to_f32(r.x[i1]), b0 = a.bias ? a.bias[mine] : 0.0f, b1 = a.bias ? a.bias[i1] : 0.0f;
      slack = kUlps * (r.score(mx) + fabsf(mv) + r.score(x1) + fabsf(v1)) + 0x1p-120f;
      close = mv - v1 <= slack && !(mx == x1 && b0 == b1);
    }
    if (__any_sync(0xffffffffu, close) || groups_near) {
      // what can still be among the k: everything within the errors of the last choice
      const float last = __shfl_sync(0xffffffffu, mine >= 0 ? mv : -INFINITY, a.k - 1);
      float cut = last - 2.0f * kUlps * (2.0f + 2.0f * fabsf(last));
      if (groups_near || !(cut < INFINITY)) cut = -INFINITY;  // also where a bias is infinite
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (groups_near && x[i] > -INFINITY) v[i] = 0.0f;  // all of them
      mine = r.choose_wide(keep, cut, groups_near, v);
      mx = mine >= 0 ? to_f32(r.x[mine]) : -INFINITY;
    }
  }

  float w = 0.0f;
  if (a.renormalize) {
    const float best = warp_max(mx);  // of the chosen
    if (mine >= 0) w = a.sigmoid ? sigmoid_over(mx, fminf(best, 0.0f)) : expf(mx - best);
    const float sum = warp_sum(w);
    if (mine >= 0) w = w / sum * a.scale;
  } else if (mine >= 0) {
    w = r.score(mx) * a.scale;
  }
  if (lane < a.k) {
    a.topk[t * a.k + lane] = mine;
    a.weights[t * a.k + lane] = w;
  }
}

int launch_route_topk(const RouteTopk& a, int dtype, cudaStream_t stream) {
  const dim3 grid((unsigned)((a.n_tokens + kRouteWarps - 1) / kRouteWarps));
  const size_t smem = a.bias || a.top_groups < a.n_groups ? sizeof(double) * kRouteWarps * a.n_experts : 0;
  return with_dtype(dtype, [&](auto v) {
    using T = decltype(v);
    auto kern = a.n_experts <= 32    ? route_topk_kernel<T, 1>
                : a.n_experts <= 64  ? route_topk_kernel<T, 2>
                : a.n_experts <= 128 ? route_topk_kernel<T, 4>
                : a.n_experts <= 256 ? route_topk_kernel<T, 8>
                : a.n_experts <= 512 ? route_topk_kernel<T, 16>
                                     : route_topk_kernel<T, 32>;
    return launch_pdl(kern, grid, dim3(32 * kRouteWarps), smem, stream, a);
  });
}

}  // namespace mmvq
