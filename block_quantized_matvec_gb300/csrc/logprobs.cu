// Log probabilities of given tokens, entropy and the best alternatives of rows of logits.
//
// With m the largest of x = scale * logits and S, E the sums over all but one
// largest of exp(x - m) and exp(x - m) (x - m):
//   lse = m + log1p(S), log p(i) = (x_i - m) - log1p(S), H = log1p(S) - E / (1 + S);
// every difference is of terms of one sign, so that a row that is all but
// certain keeps its digits.
//
// A CTA per row: the maximum, the sums, then one pass for each alternative.
#include "layer.cuh"
#include "typed.cuh"

namespace mmvq {

constexpr int kRowThreads = 512;

// The larger value, of equal ones the lower place.
struct Best {
  float v;
  int i;
};
__device__ __forceinline__ Best better(Best a, Best b) {
  return b.v > a.v || (b.v == a.v && b.i < a.i) ? b : a;
}
__device__ __forceinline__ Best warp_best(Best b) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
    b = better(b, Best{__shfl_xor_sync(0xffffffffu, b.v, o), __shfl_xor_sync(0xffffffffu, b.i, o)});
  return b;
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads) logprobs_kernel(const TokenLogprobs a) {
  __shared__ Best part[kRowThreads / 32];
  __shared__ float sums[2][kRowThreads / 32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.logits) + row * a.ld;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto block_best = [&](Best b) {
    b = warp_best(b);
    if (lane == 0) part[warp] = b;
    __syncthreads();
    b = part[0];
    for (int w = 1; w < kRowThreads / 32; ++w) b = better(b, part[w]);
    __syncthreads();
    return b;
  };
  const Best none = {-INFINITY, 0x7fffffff};
  Best top = none;
  int bad = 0;
  for (int i = tid; i < a.vocab; i += kRowThreads) {
    const float v = to_f32(x[i]);
    bad |= !(v < INFINITY);
    if (v > -INFINITY) top = better(top, Best{v, i});
  }
  bad = __syncthreads_or(bad);
  top = block_best(top);
  const bool empty = top.v == -INFINITY;
  float s = 0.0f, e = 0.0f;
  for (int i = tid; i < a.vocab; i += kRowThreads) {
    const float d = (to_f32(x[i]) - top.v) * a.scale;
    if (i != top.i && d > -200.0f) {  // also not NaN: -inf less -inf
      const float p = expf(d);
      s += p;
      e = fmaf(p, d, e);
    }
  }
  s = warp_sum(s);
  e = warp_sum(e);
  if (lane == 0) {
    sums[0][warp] = s;
    sums[1][warp] = e;
  }
  __syncthreads();
  s = e = 0.0f;
  for (int w = 0; w < kRowThreads / 32; ++w) {
    s += sums[0][w];
    e += sums[1][w];
  }
  const float drop = log1pf(s);
  const float nan = __int_as_float(0x7fc00000);
  if (tid == 0) {
    if (bad && a.status) *a.status = MMVQ_ERR_VALUE;
    if (a.lse) a.lse[row] = bad ? nan : empty ? -INFINITY : fmaf(top.v, a.scale, drop);
    if (a.entropy) a.entropy[row] = bad ? nan : empty ? 0.0f : drop - e / (1.0f + s);
  }
  for (int j = tid; j < a.n_tokens; j += kRowThreads) {
    const int id = a.tokens[row * a.n_tokens + j];
    float p = nan;
    if (id < 0 || id >= a.vocab) {
      if (a.status) *a.status = MMVQ_ERR_ROUTING;
    } else if (!bad) {
      p = empty ? -INFINITY : (to_f32(x[id]) - top.v) * a.scale - drop;
    }
    a.logprobs[row * a.n_tokens + j] = p;
  }
  Best last = top;
  for (int j = 0; j < a.top; ++j) {
    if (tid == 0) {
      const bool no = bad || last.v == -INFINITY;
      a.top_ids[row * a.top + j] = no ? -1 : last.i;
      a.top_logprobs[row * a.top + j] = bad ? nan : no ? -INFINITY : (last.v - top.v) * a.scale - drop;
    }
    Best b = none;
    for (int i = tid; i < a.vocab; i += kRowThreads) {
      const float v = to_f32(x[i]);
      if (v > -INFINITY && (v < last.v || (v == last.v && i > last.i))) b = better(b, Best{v, i});
    }
    last = block_best(b);
  }
}

int launch_token_logprobs(const TokenLogprobs& a, int dtype, cudaStream_t stream) {
  return with_dtype(dtype, [&](auto v) {
    return launch_pdl(logprobs_kernel<decltype(v)>, dim3((unsigned)a.rows), dim3(kRowThreads), 0, stream, a);
  });
}

}  // namespace mmvq
