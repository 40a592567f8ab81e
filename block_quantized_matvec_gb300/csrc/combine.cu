// The experts' rows weighted and added up for each token.
//
// out[t] = residual[t] + sigmoid(gate[t]) * shared[t] + sum_j weights[t][j] * y[p(t, j)]
// in fp32, j in order.  p is found in the experts' lists as route_groups makes
// them: slots t*k + j stand in rising order between the expert's offsets, so a
// search gives the position without an inverse list.
//
// Bound by memory, each row read once (4099 tokens of 8 x 2560, residual, shared
// expert, bf16: 67.7 us, 5.9 TB/s): a CTA takes a token (few tokens: a share
// of its columns, so that the GPU is full), its warps look the slots' positions
// up, 32 places of the list at a time, and a thread then has eight 16-byte pieces
// in flight, of as many rows, or of four or two rows at several places where a
// token has no more (1944 tokens of one row of 6564: 32.0 us with one piece at a
// time, 16.5 with four).  Rows that no four columns can be taken of at once (their number or an
// address) go by two or column by column (5772 tokens of 6 rows of 350: 22.0 us
// by one, 18.5 by two).
#include "layer.cuh"
#include "typed.cuh"

namespace mmvq {

constexpr int kCombineThreads = 128;
constexpr int kCombineLoads = 8;  // pieces of a thread in flight
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

// N columns side by side, from memory (values that are read once: kOnce) and to it.
template <int N, bool kOnce = false, typename T>
__device__ __forceinline__ void load_cols(const T* p, float (&v)[N]) {
  constexpr int kBytes = N * (int)sizeof(T);
  uint32_t w[(kBytes + 3) / 4];
  if constexpr (kBytes == 16) {
    const uint4 r = kOnce ? ldg_nc_v4(p) : *reinterpret_cast<const uint4*>(p);
    w[0] = r.x, w[1] = r.y, w[2] = r.z, w[3] = r.w;
  } else if constexpr (kBytes == 8) {
    const uint2 r = *reinterpret_cast<const uint2*>(p);
    w[0] = r.x, w[1] = r.y;
  } else if constexpr (kBytes == 4) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else {
    w[0] = *reinterpret_cast<const uint16_t*>(p);
  }
  T t[N];
  memcpy(t, w, kBytes);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = to_f32(t[i]);
}
template <int N, typename T>
__device__ __forceinline__ void store_cols(T* p, const float (&v)[N]) {
  constexpr int kBytes = N * (int)sizeof(T);
  T t[N];
#pragma unroll
  for (int i = 0; i < N; ++i) t[i] = from_f32<T>(v[i]);
  if constexpr (kBytes == 16) {
    uint4 r;
    memcpy(&r, t, 16);
    *reinterpret_cast<uint4*>(p) = r;
  } else if constexpr (kBytes == 8) {
    uint2 r;
    memcpy(&r, t, 8);
    *reinterpret_cast<uint2*>(p) = r;
  } else if constexpr (kBytes == 4) {
    uint32_t r;
    memcpy(&r, t, 4);
    *reinterpret_cast<uint32_t*>(p) = r;
  } else {
    *p = t[0];
  }
}

// N columns of a piece (4, 2 or 1); a thread has kPieces of them at once, of kCombineLoads / kPieces rows.
template <typename T, int N, int kPieces>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const __grid_constant__ CombineExperts a, int chunks) {
  constexpr int kRows = kCombineLoads / kPieces;
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
  float sum[kPieces][N];
  auto start = [&](int c) {  // what is there besides the experts' rows
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
#pragma unroll
      for (int i = 0; i < N; ++i) sum[u][i] = 0.0f;
      const int64_t at = (int64_t)(c + u * kCombineThreads) * N;
      if (residual && c + u * kCombineThreads < end) load_cols<N>(residual + at, sum[u]);
    }
    if (shared) {
#pragma unroll
      for (int u = 0; u < kPieces; ++u)
        if (c + u * kCombineThreads < end) {
          float s[N];
          load_cols<N>(shared + (int64_t)(c + u * kCombineThreads) * N, s);
#pragma unroll
          for (int i = 0; i < N; ++i) sum[u][i] = fmaf(gate, s[i], sum[u][i]);
        }
    }
  };
  start(begin);
  for (int j = threadIdx.x >> 5; j < a.k; j += kCombineThreads / 32) {
    const int p = find_slot(a, t * a.k + j, lane);
    if (lane == 0) {
      place[j] = p;
      weight[j] = a.weights[t * a.k + j];
    }
  }
  __syncthreads();
  for (int c = begin; c < end; c += kPieces * kCombineThreads) {
    if (c != begin) start(c);
    for (int j = 0; j < a.k; j += kRows) {
      float v[kRows][kPieces][N];
      int p[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        p[i] = j + i < a.k ? place[j + i] : -1;
#pragma unroll
        for (int u = 0; u < kPieces; ++u)
          if (p[i] >= 0 && c + u * kCombineThreads < end)
            load_cols<N, true>(a.y + (int64_t)p[i] * a.H + (int64_t)(c + u * kCombineThreads) * N, v[i][u]);
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i)
        if (p[i] >= 0) {
#pragma unroll
          for (int u = 0; u < kPieces; ++u)
#pragma unroll
            for (int n = 0; n < N; ++n) sum[u][n] = fmaf(weight[j + i], v[i][u][n], sum[u][n]);
        }
    }
#pragma unroll
    for (int u = 0; u < kPieces; ++u)
      if (c + u * kCombineThreads < end) store_cols<N>(out + (int64_t)(c + u * kCombineThreads) * N, sum[u]);
  }
}

template <typename T, int N>
static int launch_columns(const CombineExperts& a, cudaStream_t stream) {
  // few tokens: shares of at least one round of a CTA's threads
  const int most = (a.H / N + kCombineThreads - 1) / kCombineThreads;
  const int chunks = min(most, (kCombineCtas + a.n_tokens - 1) / a.n_tokens);
  const int per_thread = (most + chunks - 1) / chunks;
  auto kern = a.k <= 2 && per_thread > 2 ? combine_kernel<T, N, 4> : a.k <= 4 && per_thread > 1 ? combine_kernel<T, N, 2> : combine_kernel<T, N, 1>;
  return launch_pdl(kern, dim3((unsigned)a.n_tokens * chunks), dim3(kCombineThreads), 0, stream, a, chunks);
}

int launch_combine_experts(const CombineExperts& a, int dtype, cudaStream_t stream) {
  return with_dtype(dtype, [&](auto v) {
    using T = decltype(v);
    auto by = [&](int n) {
      auto fits = [n](const void* p, int64_t ld, size_t size) { return reinterpret_cast<uintptr_t>(p) % (n * size) == 0 && (!p || ld % n == 0); };
      return a.H % n == 0 && fits(a.y, a.H, 4) && fits(a.residual, a.ldr, sizeof(T)) && fits(a.shared, a.lds, sizeof(T)) &&
             fits(a.out, a.ldo, sizeof(T));
    };
    return by(4) ? launch_columns<T, 4>(a, stream) : by(2) ? launch_columns<T, 2>(a, stream) : launch_columns<T, 1>(a, stream);
  });
}

}  // namespace mmvq
