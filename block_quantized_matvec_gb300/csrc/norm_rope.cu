// RMS norm of every query and key head and the rotation by its token's position.
//
// z = x * rsqrt(mean(x^2) + eps) * w over a head's D values; of the first `rot`,
// pair i (i and i + rot/2, or 2i and 2i + 1) turns by position[axis(i)] times a
// frequency.  Angles are kept in turns as 64-bit fixed point: a position times
// the table's step wraps as the angle does, so a position of 2^31 loses 2^-34
// turns, and sin and cos are taken of a remainder within an eighth of a turn.
//
// A warp per row; a lane holds pairs lane, lane + 32, ..., those past rot / 2
// made of neighbours that do not turn.
#include "layer.cuh"
#include "typed.cuh"

namespace mmvq {

// cos and sin of 2 pi * phase / 2^64.
__device__ __forceinline__ float2 turn(uint64_t phase) {
  const uint32_t quarter = (uint32_t)((phase + (1ull << 61)) >> 62);
  const int64_t rest = (int64_t)(phase - ((uint64_t)quarter << 62));  // within an eighth of a turn
  float s, c;
  sincospif((float)(int32_t)(rest >> 30) * 0x1p-33f, &s, &c);
  const float x = quarter & 1 ? -s : c, y = quarter & 1 ? c : s;
  return quarter & 2 ? make_float2(-x, -y) : make_float2(x, y);
}

template <typename T, int D>
__global__ void __launch_bounds__(128) norm_rope_kernel(const NormRope a) {
  grid_dependency_wait();
  grid_launch_dependents();
  constexpr int kPairs = D / 64;
  const int lane = threadIdx.x & 31, heads = a.q.heads + a.k.heads, half = a.rot / 2;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int64_t t = row / heads;
  if (t >= a.n_tokens) return;
  const int h = (int)(row - t * heads);
  const bool is_q = h < a.q.heads;
  const RopeHeads& r = is_q ? a.q : a.k;
  const int hh = is_q ? h : h - a.q.heads;
  const T* x = static_cast<const T*>(r.x) + t * r.ldx + hh * r.hx;
  T* y = static_cast<T*>(r.y) + t * r.ldy + hh * r.hy;
  float v[kPairs][2], sum = 0.0f;
  int at[kPairs][2];
#pragma unroll
  for (int j = 0; j < kPairs; ++j) {
    const int i = lane + 32 * j;
    const bool halves = i < half && !a.interleaved;
    at[j][0] = halves ? i : 2 * i;
    at[j][1] = halves ? i + half : 2 * i + 1;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      v[j][e] = to_f32(x[at[j][e]]);
      sum = fmaf(v[j][e], v[j][e], sum);
    }
  }
  if (a.norm) {
    const float scale = rsqrtf(warp_sum(sum) * (1.0f / D) + a.eps);
#pragma unroll
    for (int j = 0; j < kPairs; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) v[j][e] *= scale * (r.weight ? r.weight[at[j][e]] : 1.0f);
  }
#pragma unroll
  for (int j = 0; j < kPairs; ++j) {
    const int i = lane + 32 * j;
    if (i < half) {
      const int64_t axis = a.table[half + i];
      if (axis >= 0 && axis < a.n_axes) {
        const int64_t pos = a.positions[axis * a.ld_positions + t];
        const float2 w = turn((uint64_t)a.table[i] * (uint64_t)pos);
        const float p = v[j][0] * w.x - v[j][1] * w.y, q = v[j][0] * w.y + v[j][1] * w.x;
        v[j][0] = p;
        v[j][1] = q;
      } else if (a.status) {
        *a.status = MMVQ_ERR_SHAPE;
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) y[at[j][e]] = from_f32<T>(v[j][e]);
  }
}

int launch_norm_rope(const NormRope& a, int dtype, int head_dim, cudaStream_t stream) {
  const int64_t rows = (int64_t)a.n_tokens * (a.q.heads + a.k.heads);
  const dim3 grid((unsigned)((rows + 3) / 4));
  return with_dtype(dtype, [&](auto v) {
    using T = decltype(v);
    auto kern = head_dim == 64 ? norm_rope_kernel<T, 64> : head_dim == 128 ? norm_rope_kernel<T, 128> : norm_rope_kernel<T, 256>;
    return launch_pdl(kern, grid, dim3(128), 0, stream, a);
  });
}

}  // namespace mmvq
