// The experts' rows weighted and added up for each token.
//
// out[t] = residual[t] + sigmoid(gate[t]) * shared[t] + sum_j weights[t][j] * y[p(t, j)]
// in fp32, j in order.  p is found in the experts' lists as route_groups makes
// them: slots t*k + j stand in rising order between the expert's offsets, so a
// search by halves gives the position without an inverse list.
//
// A CTA per token and 1024 columns; its first k threads look the positions up.
#include "layer.cuh"
#include "typed.cuh"

namespace mmvq {

constexpr int kCombineThreads = 128;
constexpr int kCombineCols = 1024;

// Position of `slot`, or -1.
__device__ __forceinline__ int find_slot(const CombineExperts& a, int slot) {
  const int e = a.topk[slot];
  if (e == -1) return -1;  // no expert
  int p = -1;
  if (e >= 0 && e < a.n_experts) {
    const int n = a.n_tokens * a.k;
    int lo = min(max(a.offsets[e], 0), n);
    const int end = min(max(a.offsets[e + 1], 0), n);
    int hi = end;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (a.slot_of[mid] < slot) lo = mid + 1; else hi = mid;
    }
    if (lo < end && a.slot_of[lo] == slot && lo < a.n_positions) p = lo;
  }
  if (p < 0 && a.status) *a.status = MMVQ_ERR_ROUTING;
  return p;
}

template <typename T>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const CombineExperts a, int chunks) {
  __shared__ int place[kCombineMaxTopk];
  __shared__ float weight[kCombineMaxTopk];
  grid_dependency_wait();
  grid_launch_dependents();
  const int t = blockIdx.x / chunks, chunk = blockIdx.x - t * chunks;
  for (int j = threadIdx.x; j < a.k; j += kCombineThreads) {
    place[j] = find_slot(a, t * a.k + j);
    weight[j] = a.weights[t * a.k + j];
  }
  __syncthreads();
  const int end = min(a.H, (chunk + 1) * kCombineCols);
  for (int c = chunk * kCombineCols + threadIdx.x; c < end; c += kCombineThreads) {
    float sum = a.residual ? to_f32(static_cast<const T*>(a.residual)[t * a.ldr + c]) : 0.0f;
    if (a.shared) {
      const float s = to_f32(static_cast<const T*>(a.shared)[t * a.lds + c]);
      sum += a.gate ? s / (1.0f + expf(-a.gate[t])) : s;
    }
    for (int j = 0; j < a.k; ++j)
      if (place[j] >= 0) sum = fmaf(weight[j], a.y[(int64_t)place[j] * a.H + c], sum);
    static_cast<T*>(a.out)[t * a.ldo + c] = from_f32<T>(sum);
  }
}

int launch_combine_experts(const CombineExperts& a, int dtype, cudaStream_t stream) {
  const int chunks = (a.H + kCombineCols - 1) / kCombineCols;
  return with_dtype(dtype, [&](auto v) {
    return launch_pdl(combine_kernel<decltype(v)>, dim3((unsigned)a.n_tokens * chunks), dim3(kCombineThreads), 0, stream, a, chunks);
  });
}

}  // namespace mmvq
