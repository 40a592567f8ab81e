// The experts' rows weighted and added up for each token.
//
// out[t] = residual[t] + sigmoid(gate[t]) * shared[t] + sum_j weights[t][j] * y[p(t, j)]
// in fp32, j in order.  p is found in the experts' lists as route_groups makes
// them: slots t*k + j stand in rising order between the expert's offsets, so a
// search gives the position without an inverse list.
//
// Bound by memory, each row read once: a CTA takes a token (few tokens: a share
// of its columns, so that the GPU is full), its warps look the slots' positions
// up, 32 places of the list at a time, and a thread then has the 16-byte pieces
// of eight rows in flight.  Rows that no four columns can be taken of at once
// (their number or an address) go column by column.
#include "layer.cuh"
#include "typed.cuh"

namespace mmvq {

constexpr int kCombineThreads = 128;
constexpr int kCombineRows = 8;  // rows in flight
constexpr int kCombineCtas = 2 * 152;

// Position of `slot`, or -1; by all lanes of a warp.
__device__ __forceinline__ int find_slot(const CombineExperts& a, int slot, int lane) {
  const int e = a.topk[slot];
  if (e == -1) return -1;  // no expert
  int p = -1;
  if (e >= 0 && e < a.n_experts) {
    const int n = a.n_tokens * a.k;
    int lo = min(max(a.offsets[e], 0), n), hi = min(max(a.offsets[e + 1], 0), n);
    while (hi - lo > 32) {  // down to a 32nd at every step
      const int step = (hi - lo + 31) / 32, i = lo + lane * step;
      const uint32_t m = __ballot_sync(0xffffffffu, i < hi && a.slot_of[i] <= slot);
      const int at = m ? 31 - __clz(m) : 0;
      lo += at * step;
      hi = min(lo + step, hi);
    }
    const uint32_t m = __ballot_sync(0xffffffffu, lo + lane < hi && a.slot_of[lo + lane] == slot);
    if (m) p = lo + __ffs(m) - 1;
    if (p >= a.n_positions) p = -1;
  }
  if (p < 0 && a.status) *a.status = MMVQ_ERR_ROUTING;
  return p;
}

template <typename T, int N>
__device__ __forceinline__ void load_cols(const T* p, float (&v)[N]) {
  if constexpr (N == 1) {
    v[0] = to_f32(*p);
  } else if constexpr (sizeof(T) == 4) {
    const float4 f = *reinterpret_cast<const float4*>(p);
    v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
  } else {
    const uint2 r = *reinterpret_cast<const uint2*>(p);
    const T* h = reinterpret_cast<const T*>(&r);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = to_f32(h[i]);
  }
}
template <typename T, int N>
__device__ __forceinline__ void store_cols(T* p, const float (&v)[N]) {
  if constexpr (N == 1) {
    *p = from_f32<T>(v[0]);
  } else if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2(T{}, v[0], v[1]), pack2(T{}, v[2], v[3]));
  }
}

template <typename T, int N>  // N columns of a thread at once: 4 or 1
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const CombineExperts a, int chunks) {
  __shared__ int place[kCombineMaxTopk];
  __shared__ float weight[kCombineMaxTopk];
  grid_dependency_wait();
  grid_launch_dependents();
  const int t = blockIdx.x / chunks, chunk = blockIdx.x - t * chunks;
  const int lane = threadIdx.x & 31;
  const T* residual = a.residual ? static_cast<const T*>(a.residual) + t * a.ldr : nullptr;
  const T* shared = a.shared ? static_cast<const T*>(a.shared) + t * a.lds : nullptr;
  T* out = static_cast<T*>(a.out) + t * a.ldo;
  const float gate = a.gate ? 1.0f / (1.0f + expf(-a.gate[t])) : 1.0f;
  const int pieces = a.H / N;
  const int begin = (int)((int64_t)pieces * chunk / chunks) + threadIdx.x, end = (int)((int64_t)pieces * (chunk + 1) / chunks);
  auto start = [&](int c, float (&sum)[N]) {  // what is there besides the experts' rows
#pragma unroll
    for (int i = 0; i < N; ++i) sum[i] = 0.0f;
    if (residual) load_cols(residual + (int64_t)c * N, sum);
    if (shared) {
      float s[N];
      load_cols(shared + (int64_t)c * N, s);
#pragma unroll
      for (int i = 0; i < N; ++i) sum[i] = fmaf(gate, s[i], sum[i]);
    }
  };
  float sum[N];
  if (begin < end) start(begin, sum);
  for (int j = threadIdx.x >> 5; j < a.k; j += kCombineThreads / 32) {
    const int p = find_slot(a, t * a.k + j, lane);
    if (lane == 0) {
      place[j] = p;
      weight[j] = a.weights[t * a.k + j];
    }
  }
  __syncthreads();
  for (int c = begin; c < end; c += kCombineThreads) {
    if (c != begin) start(c, sum);
    const float* y = a.y + (int64_t)c * N;
    for (int j = 0; j < a.k; j += kCombineRows) {
      float v[kCombineRows][N];
      int p[kCombineRows];
#pragma unroll
      for (int i = 0; i < kCombineRows; ++i) {
        p[i] = j + i < a.k ? place[j + i] : -1;
        if (p[i] >= 0) {
          if constexpr (N == 4) {
            const uint4 r = ldg_nc_v4(y + (int64_t)p[i] * a.H);
            unpack16<float>(r, v[i]);
          } else {
            v[i][0] = y[(int64_t)p[i] * a.H];
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kCombineRows; ++i)
        if (p[i] >= 0) {
#pragma unroll
          for (int n = 0; n < N; ++n) sum[n] = fmaf(weight[j + i], v[i][n], sum[n]);
        }
    }
    store_cols(out + (int64_t)c * N, sum);
  }
}

int launch_combine_experts(const CombineExperts& a, int dtype, cudaStream_t stream) {
  return with_dtype(dtype, [&](auto v) {
    using T = decltype(v);
    auto fits = [](const void* p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % (4 * sizeof(T)) == 0 && (!p || ld % 4 == 0); };
    const bool four = a.H % 4 == 0 && reinterpret_cast<uintptr_t>(a.y) % 16 == 0 && fits(a.residual, a.ldr) && fits(a.shared, a.lds) &&
                      fits(a.out, a.ldo);
    const int most = (a.H / (four ? 4 : 1) + kCombineThreads - 1) / kCombineThreads;
    const int chunks = min(most, (kCombineCtas + a.n_tokens - 1) / a.n_tokens);
    return launch_pdl(four ? combine_kernel<T, 4> : combine_kernel<T, 1>, dim3((unsigned)a.n_tokens * chunks), dim3(kCombineThreads), 0, stream, a,
                      chunks);
  });
}

}  // namespace mmvq
