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
// whose error is at most kUlps of the score and of the sum, but for the rounding
// of a softmax's argument x - top, up to 64 half units where they are far apart.
// That one needs no room: without bias, as rounding keeps the order, two arguments are
// in the order of their logits or equal, and what is equal is too near to tell; with a
// bias, and for groups, errors count absolutely, and d exp(-d) stays below 0.37.
// Where two neighbours in the order, whose logits or biases differ (or the last group
// in and the first one out), lie nearer to one another than that, the warp makes the
// values that can matter again in 64 bits and chooses by those.
//
// A warp per token; lane L holds the experts L * kPer .. + kPer - 1, so a lower
// lane means a lower id.  Bound by instructions, not by the few bytes.  The lanes'
// best ones are sorted (values alone: a shuffle and a minimum or maximum a step); at
// least k experts reach the k-th of those, and the few that do, within their errors,
// are put one to a lane, which counts how many come before it.  Where more than 32
// do, the best is taken k times over first.  (8192 tokens, 8 of 256 in
// groups: 15.7 us; with every lane's experts sorted and the best taken k times 17.3.)
#include <cfloat>

#include "layer.cuh"
#include "typed.cuh"

namespace mmvq {

constexpr int kRouteWarps = 4;

// sigmoid(x)
__device__ __forceinline__ float sigmoid(float x) {
  const float t = expf(-fabsf(x)), r = __fdividef(1.0f, 1.0f + t);
  return x >= 0.0f ? r : t * r;
}
// sigmoid(x) over exp(c), c = min(top, 0): the largest of several stays at a half or
// above however small they all are.
__device__ __forceinline__ float sigmoid_over(float x, float c) {
  return expf(fminf(x, 0.0f) - c) / (1.0f + expf(-fabsf(x)));
}

// What choices in 64 bits need, for each warp: places for the experts' values and a list of ids.
struct WideScratch {
  double* value;   // [n_experts]
  uint16_t* list;  // [n_experts]
};
constexpr int kWideBytes = sizeof(double) + sizeof(uint16_t);  // an expert

// A token's logits and what its scores need.
struct RouteRow {
  const void* x;
  int lane, group_size;
  float top, total;  // softmax: the largest logit and the sum of exp(x - top)
};

// The value in 64 bits; z: the softmax's sum (any positive number where only the order counts).
template <typename T>
__device__ __forceinline__ double wide_value(const RouteTopk& a, const RouteRow& r, int e, double z) {
  const double l = (double)to_f32(static_cast<const T*>(r.x)[e]);
  const double d = a.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - (double)r.top) / z;
  return a.bias ? d + (double)a.bias[e] : d;
}

// The experts with may[i] >= cut[i] in w.list, in order, and their number.
template <int kPer>
__device__ __forceinline__ int list_wide(const float* may, const float* cut, int lane, WideScratch w) {
  int n = 0;
#pragma unroll 1
  for (int i = 0; i < kPer; ++i) n += __popc(__ballot_sync(0xffffffffu, may[i] > -INFINITY && may[i] >= cut[i]));
  // lane by lane: the ids before mine are those of lower lanes
  int mine = 0;
  for (int i = 0; i < kPer; ++i) mine += may[i] > -INFINITY && may[i] >= cut[i];
  int at = mine;
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, at, o);
    if (lane >= o) at += v;
  }
  at -= mine;
  for (int i = 0; i < kPer; ++i)
    if (may[i] > -INFINITY && may[i] >= cut[i]) w.list[at++] = (uint16_t)(lane * kPer + i);
  __syncwarp();
  return n;
}

// The softmax's sum in 64 bits, which the order depends on where there is a bias; else 1.
template <typename T, int kPer>
__device__ __forceinline__ double wide_total(const RouteTopk& a, const RouteRow& r) {
  if (a.sigmoid || !a.bias) return 1.0;
  double z = 0.0;
#pragma unroll 4
  for (int i = 0; i < kPer; ++i) {
    const int e = r.lane * kPer + i;
    const float l = e < a.n_experts ? to_f32(static_cast<const T*>(r.x)[e]) : INFINITY;
    if (fabsf(l) < INFINITY) z += exp((double)l - (double)r.top);
  }
  for (int o = 16; o; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  return z;
}

// The groups that stay, decided in 64 bits: bit g of the result.  Of each group only what can be
// among its two best is made again: what is at least cut (may: the values in fp32).
template <typename T, int kPer>
__device__ __noinline__ uint32_t groups_wide(const RouteTopk& a, const RouteRow r, const float* may, const float* cut, WideScratch w) {
  const double z = wide_total<T, kPer>(a, r), minus = -(double)INFINITY;
  const int n = list_wide<kPer>(may, cut, r.lane, w);
  for (int c = r.lane; c < n; c += 32) w.value[c] = wide_value<T>(a, r, w.list[c], z);
  __syncwarp();
  double two = minus;
  if (r.lane < a.n_groups) {
    double b1 = minus, b2 = minus;
    for (int c = 0; c < n; ++c) {
      if (w.list[c] / r.group_size != r.lane) continue;
      const double d = w.value[c];
      if (d > b1) { b2 = b1; b1 = d; } else if (d > b2) { b2 = d; }
    }
    two = b2 == minus ? b1 : b1 + b2;
  }
  __syncwarp();
  int rank = 0;
  for (int g = 0; g < a.n_groups; ++g) {
    const double other = __shfl_sync(0xffffffffu, two, g);
    rank += other > two || (other == two && g < r.lane);
  }
  return __ballot_sync(0xffffffffu, r.lane < a.n_groups && rank < a.top_groups);
}

// The choice in 64 bits among the experts with may[i] >= cut[i].  Lane j leaves with the id of
// choice j, or -1.
template <typename T, int kPer>
__device__ __noinline__ int choose_wide(const RouteTopk& a, const RouteRow r, const float* may, const float* cut, WideScratch w) {
  const double z = wide_total<T, kPer>(a, r), minus = -(double)INFINITY;
  const int lane = r.lane, n = list_wide<kPer>(may, cut, lane, w);
  if (n <= 32) {  // mostly: one a lane, ranked by comparing all with all
    const int id = lane < n ? w.list[lane] : 0x7fffffff;
    const double d = lane < n ? wide_value<T>(a, r, id, z) : 0.0;
    int rank = 0;
    for (int s = 0; s < n; ++s) {
      const double o = __shfl_sync(0xffffffffu, d, s);
      const int oi = __shfl_sync(0xffffffffu, id, s);
      rank += o > d || (o == d && oi < id);
    }
    __syncwarp();
    if (lane < n) w.list[rank] = (uint16_t)id;
    __syncwarp();
    return lane < min(n, a.k) ? w.list[lane] : -1;
  }
  for (int c = lane; c < n; c += 32) w.value[c] = wide_value<T>(a, r, w.list[c], z);
  __syncwarp();
  int mine = -1;
  for (int j = 0; j < a.k; ++j) {
    double b = minus;
    int at = 0x7fffffff;
    for (int c = lane; c < n; c += 32)
      if (w.value[c] > b) { b = w.value[c]; at = c; }
    for (int o = 16; o; o >>= 1) {
      const double ob = __shfl_xor_sync(0xffffffffu, b, o);
      const int oi = __shfl_xor_sync(0xffffffffu, at, o);
      if (ob > b || (ob == b && oi < at)) { b = ob; at = oi; }
    }
    if (b == minus) break;
    if (lane == j) mine = w.list[at];
    __syncwarp();
    if (lane == 0) w.value[at] = minus;
    __syncwarp();
  }
  return mine;
}

template <typename T, int kPer>
__global__ void __launch_bounds__(32 * kRouteWarps) route_topk_kernel(const __grid_constant__ RouteTopk a) {
  __shared__ int2 found[kRouteWarps][32];  // value and id
  extern __shared__ double wide_all[];  // WideScratch of each warp: all values, then all lists
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
  if (t >= a.n_tokens) return;
  const T* row = static_cast<const T*>(a.logits) + t * a.ld;
  const int group_size = a.n_experts / a.n_groups, first = lane * kPer;  // my first expert
  float softmax_top = 0.0f, total = 1.0f;
  auto score = [&](float l) { return a.sigmoid ? sigmoid(l) : __fdividef(expf(l - softmax_top), total); };
  const bool grouped = a.top_groups < a.n_groups;
  const bool exact = !a.bias && !grouped;  // the logits' order is the scores'
  // what a value's fp32 error stays within, its argument's rounding aside: exp (2 half units), the sum (kPer + 5
  // additions, its terms' own 2, their arguments' 7: the mean of d is at most log 1024), the quotient 4, the sum with
  // the bias 1, and what is left of the argument's own 1
  constexpr float kUlps = (kPer + 24) * 0x1p-24f;

  float x[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) x[i] = -INFINITY;
  constexpr int kBytes = kPer * (int)sizeof(T);
  if (kBytes >= 16 && (lane + 1) * kPer <= a.n_experts && reinterpret_cast<uintptr_t>(row) % 16 == 0) {
#pragma unroll
    for (int i = 0; i < kPer; i += kVec<T>) {
      if constexpr (kBytes >= 16) unpack16<T>(ldg_nc_v4(row + (first + i)), x + i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if ((first + i) < a.n_experts) x[i] = to_f32(row[(first + i)]);
  }
  float top = -INFINITY;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (!(x[i] < INFINITY)) {  // NaN or +inf
      bad = true;
      x[i] = -INFINITY;
    }
    top = fmaxf(top, x[i]);
  }
  if (bad && a.status) *a.status = MMVQ_ERR_VALUE;
  if (!a.sigmoid) {
    top = warp_max(top);
    softmax_top = top == -INFINITY ? 0.0f : top;
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) z += expf(x[i] - softmax_top);
    total = warp_sum(z);
  }
  float v[kPer];
  if (exact) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = x[i];
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      v[i] = -INFINITY;
      if (x[i] > -INFINITY) v[i] = score(x[i]) + (a.bias ? a.bias[(first + i)] : 0.0f);
      if (!(v[i] > -INFINITY)) v[i] = -INFINITY;  // a bias of NaN: fmaxf and fminf would lose it
    }
  }

  const WideScratch scratch{wide_all + warp * a.n_experts, reinterpret_cast<uint16_t*>(wide_all + kRouteWarps * a.n_experts) + warp * a.n_experts};
  if (grouped) {
    const int lanes = group_size / kPer;  // of a group, where it has whole ones
    const bool whole = lanes * kPer == group_size;
    // my lane's group (lane g's, where groups have no lanes of their own): its two best
    float b1 = -INFINITY, b2 = -INFINITY;
    int group = lane;
    if (whole) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        b2 = fmaxf(b2, fminf(b1, v[i]));
        b1 = fmaxf(b1, v[i]);
      }
      group = lane / lanes;
      const int begin = group * lanes;
      const float m1 = b1, m2 = b2;
      int from = lane;
      for (int s = 1; s < lanes; ++s) {
        from = from + 1 < begin + lanes ? from + 1 : begin;
        const float o1 = __shfl_sync(0xffffffffu, m1, from), o2 = __shfl_sync(0xffffffffu, m2, from);
        b2 = fmaxf(fmaxf(b2, o2), fminf(b1, o1));
        b1 = fmaxf(b1, o1);
      }
    } else {
      for (int g = 0; g < a.n_groups; ++g) {
        float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if ((uint32_t)(first + i - g * group_size) < (uint32_t)group_size) {
            m2 = fmaxf(m2, fminf(m1, v[i]));
            m1 = fmaxf(m1, v[i]);
          }
        const float best = warp_max(m1);
        // the best of one lane only: of what the others and its second have left
        const uint32_t who = __ballot_sync(0xffffffffu, m1 == best);
        const float second = warp_max(lane == __ffs(who) - 1 ? m2 : m1);
        if (lane == g) b1 = best, b2 = second;
      }
    }
    const bool real = group < a.n_groups;
    const float two = b2 == -INFINITY ? b1 : b1 + b2;
    // scores are at most 1: an error of both values and of their sum
    const float size = b1 == -INFINITY || !real ? 0.0f : 3.0f + fabsf(b1) + (b2 == -INFINITY ? 0.0f : fabsf(b2));
    int rank = 0;
    for (int g = 0; g < a.n_groups; ++g) {
      const float other = __shfl_sync(0xffffffffu, two, whole ? g * lanes : g);
      rank += other > two || (other == two && g < group);
    }
    const bool kept = real && rank < a.top_groups;
    const float in = -warp_max(kept ? -two : -INFINITY), out = warp_max(real && !kept ? two : -INFINITY);
    uint32_t keep = __ballot_sync(0xffffffffu, kept);  // bit of a group's lanes, or of the group
    // too near to tell, or a sum of two biases that fp32 does not hold
    const bool beyond = real && b1 > -INFINITY && !(fabsf(two) < INFINITY);
    if (__any_sync(0xffffffffu, beyond) || (out > -INFINITY && in - out <= 2.0f * kUlps * warp_max(size))) {
      float may[kPer], cut[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int e = first + i;
        const float second = __shfl_sync(0xffffffffu, b2, whole ? lane : min(e / group_size, 31));
        may[i] = v[i];
        cut[i] = second - 2.0f * kUlps * (2.0f + 2.0f * fabsf(second));
        if (!(cut[i] < INFINITY)) cut[i] = -INFINITY;  // fewer than two, or a bias that is infinite
      }
      keep = groups_wide<T, kPer>(a, RouteRow{row, lane, group_size, softmax_top, total}, may, cut, scratch);
      if (whole) keep = __ballot_sync(0xffffffffu, real && ((keep >> group) & 1));
    }
    if (whole) {
      const bool stays = (keep >> lane) & 1;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (!stays) v[i] = -INFINITY;
    } else {
      for (int i = 0, g = first / group_size, next_at = (g + 1) * group_size; i < kPer; ++i) {
        if (first + i == next_at) ++g, next_at += group_size;
        if (first + i < a.n_experts && !((keep >> g) & 1)) v[i] = -INFINITY;
      }
    }
  }

  // what a value's error stays within; with a bias an expert of any score, up to 1, can stand at a value
  auto error = [&](float value) { return kUlps * ((a.bias ? 1.0f : fabsf(value)) + fabsf(value)) + 0x1p-120f; };

  // As many lanes' best ones reach the k-th largest of them, and so do all that can be among the k, within their errors.
  float best = v[0];
#pragma unroll
  for (int i = 1; i < kPer; ++i) best = fmaxf(best, v[i]);
#pragma unroll
  for (int m = 2; m <= 32; m *= 2)
#pragma unroll
    for (int o = m / 2; o; o >>= 1) {
      const float other = __shfl_xor_sync(0xffffffffu, best, o);
      best = !(lane & o) == !(lane & m) ? fmaxf(best, other) : fminf(best, other);
    }
  float bound = __shfl_sync(0xffffffffu, best, a.k - 1);
  auto collect = [&]() {
    bound = fmaxf(bound, -FLT_MAX);
    if (!exact && bound < INFINITY) bound = fmaxf(bound - 3.0f * error(bound), -FLT_MAX);  // a bias can be infinite
    int n = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint32_t m = __ballot_sync(0xffffffffu, v[i] >= bound);
      const int at = n + __popc(m & ((1u << lane) - 1u));
      if (v[i] >= bound && at < 32) found[warp][at] = make_int2(__float_as_int(v[i]), first + i);
      n += __popc(m);
    }
    __syncwarp();
    return n;
  };
  int n = collect();

  int mine = -1;  // lane j's choice j
  if (n > 32) {
    // Fewer lanes than k have any, or many are equal: the best of all lanes, k times, for the k-th itself.
    float left[kPer], kth = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPer; ++i) left[i] = v[i];
#pragma unroll 1
    for (int j = 0; j < a.k; ++j) {
      float m = left[0];
      int at = 0;
#pragma unroll
      for (int i = 1; i < kPer; ++i)
        if (left[i] > m) m = left[i], at = i;
      kth = warp_max(m);
      if (kth == -INFINITY) break;
      const int who = __ffs(__ballot_sync(0xffffffffu, m == kth)) - 1;
      const int id = __shfl_sync(0xffffffffu, first + at, who);
      if (lane == j) mine = id;
      if (lane == who) {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (i == at) left[i] = -INFINITY;
      }
    }
    if (!exact) {
      __syncwarp();
      bound = kth;
      n = collect();
    }
  }
  bool close = n > 32 && !exact;  // two that are too near to tell
  if (n <= 32) {  // mostly: one a lane, which counts those before it
    const int2 e = found[warp][lane < n ? lane : 0];
    int rank = 0;
    for (int j = 0; j < n; ++j) {
      const int2 o = found[warp][j];
      const float ov = __int_as_float(o.x), ev = __int_as_float(e.x);
      rank += ov > ev || (ov == ev && o.y < e.y);
    }
    __syncwarp();
    if (lane < n) found[warp][rank] = e;
    __syncwarp();
    const int2 c = found[warp][lane < n ? lane : 0];
    mine = lane < min(n, a.k) ? c.y : -1;
    if (!exact) {
      // Neighbours in the order, down to the last that is within the errors of the last choice.  Equal logits
      // with equal biases are equal in 64 bits too; what comes after them is the last one's neighbour.
      const float cv = __int_as_float(c.x), next = __shfl_down_sync(0xffffffffu, cv, 1);
      const float last = __shfl_sync(0xffffffffu, cv, max(min(n, a.k) - 1, 0));
      const int id = __shfl_down_sync(0xffffffffu, c.y, 1);
      if (lane + 1 < n && cv - next <= error(cv) + error(next) && (lane < a.k || last - next <= error(last) + error(next)))
        close = to_f32(row[c.y]) != to_f32(row[id]) || (a.bias && a.bias[c.y] != a.bias[id]);
    }
  }
  if (__any_sync(0xffffffffu, close)) {
    float may[kPer], cut[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      may[i] = v[i];
      cut[i] = bound;
    }
    mine = choose_wide<T, kPer>(a, RouteRow{row, lane, group_size, softmax_top, total}, may, cut, scratch);
  }
  const float mx = mine >= 0 ? to_f32(row[mine]) : -INFINITY;

  float w = 0.0f;
  if (a.renormalize) {
    const float best = warp_max(mx);  // of the chosen
    if (mine >= 0) w = a.sigmoid ? sigmoid_over(mx, fminf(best, 0.0f)) : expf(mx - best);
    const float sum = warp_sum(w);
    if (mine >= 0) w = w / sum * a.scale;
  } else if (mine >= 0) {
    w = (a.sigmoid ? sigmoid_over(mx, 0.0f) : expf(mx - softmax_top) / total) * a.scale;
  }
  if (lane < a.k) {
    a.topk[t * a.k + lane] = mine;
    a.weights[t * a.k + lane] = w;
  }
}

int launch_route_topk(const RouteTopk& a, int dtype, cudaStream_t stream) {
  const dim3 grid((unsigned)((a.n_tokens + kRouteWarps - 1) / kRouteWarps));
  const size_t smem = a.bias || a.top_groups < a.n_groups ? (size_t)kWideBytes * kRouteWarps * a.n_experts : 0;
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
