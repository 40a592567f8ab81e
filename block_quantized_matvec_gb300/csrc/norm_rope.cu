// RMS norm of every query and key head and the rotation by its token's position.
//
// z = x * rsqrt(mean(x^2) + eps) * w over a head's D values; of the first `rot`,
// pair i (i and i + rot/2, or 2i and 2i + 1) turns by position[axis(i)] times a
// frequency.  Angles are kept in turns as 64-bit fixed point: a position times
// the table's step wraps as the angle does, so a position of 2^31 loses 2^-34
// turns, and sin and cos are taken of a remainder within an eighth of a turn.
//
// Rows are read and written once and little is computed, so memory bounds the
// kernel where there are many (16385 tokens of 40 x 128 bf16, in a replayed graph: 53.4 us,
// 6.3 TB/s; neighbours 52.7; fp32 103.5 and 103.2).
// norm_rope_vec_kernel: a lane holds two 16-byte vectors of a row, where i turns with
// i + rot/2 two that are rot/2 apart, so that D / (2 * 16 bytes) lanes share a row and
// only the mean square crosses lanes.  A warp stays with a token: its lanes share out
// the sines and cosines, then every lane keeps the weights times those of its own
// pairs for all heads, four numbers a pair; rows come through a ring of asynchronous
// copies (80.7 us with one row's loads ahead).
// Halves that are no multiple of a vector and rows off 16 bytes take
// norm_rope_any_kernel: a warp per row, two values at a time, its token's angles made
// for every head anew, so instructions bound it (the same prompt with 84 values turning
// 226 us).  Few tokens cost it nothing (64 of them 2.5 us, by vectors 2.9).
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

// What stands in the place of a cosine where a pair does not turn.
constexpr float kNoTurn = 2.0f;

// cos and sin of pair i's angle at token t; kNoTurn where its axis is none.
__device__ __forceinline__ float2 pair_turn(const NormRope& a, int i, int64_t t) {
  const int64_t axis = a.table[a.rot / 2 + i];
  if (axis < 0 || axis >= a.n_axes) {
    if (a.status) *a.status = MMVQ_ERR_SHAPE;
    return make_float2(kNoTurn, 0.0f);
  }
  return turn((uint64_t)a.table[i] * (uint64_t)(int64_t)a.positions[axis * a.ld_positions + t]);
}

template <typename T, int D>
__global__ void __launch_bounds__(128) norm_rope_any_kernel(const NormRope a) {
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
      const float2 w = pair_turn(a, i, t);
      if (w.x != kNoTurn) {
        const float p = v[j][0] * w.x - v[j][1] * w.y, q = v[j][0] * w.y + v[j][1] * w.x;
        v[j][0] = p;
        v[j][1] = q;
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) y[at[j][e]] = from_f32<T>(v[j][e]);
  }
}

constexpr int kRopeWarps = 8;
constexpr int kRopeWarpsAtOnce = 152 * 24;
constexpr int kRopeStages = 4;  // steps of a warp's ring of rows

template <typename T, int D, bool kInterleaved>
__global__ void __launch_bounds__(32 * kRopeWarps, 3) norm_rope_vec_kernel(const __grid_constant__ NormRope a, int splits) {
  constexpr int V = kVec<T>, kLanes = D / (2 * V), kRows = 32 / kLanes;  // lanes of a row, rows of a warp
  __shared__ float2 turns[kRopeWarps][D / 2];
  __shared__ uint4 ring[kRopeWarps][kRopeStages][2][32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t unit = blockIdx.x * kRopeWarps + warp;
  const uint32_t t32 = unit / splits;
  if (t32 >= (uint32_t)a.n_tokens) return;
  const int64_t t = t32;
  // the token's rows, kRows at a time: queries, then keys; this warp's share of those steps
  const int q_steps = (a.q.heads + kRows - 1) / kRows, steps = q_steps + (a.k.heads + kRows - 1) / kRows;
  const int part = unit - t32 * splits;
  const int lo = (int)((int64_t)steps * part / splits), hi = (int)((int64_t)steps * (part + 1) / splits);

  const int u = lane % kLanes, mine = lane / kLanes, half = a.rot / 2;
  const int turning = half / V;  // vectors of a half
  // neighbouring lanes have neighbouring vectors, so that no 32-byte sector is fetched twice
  const int v0 = V * (kInterleaved || u < turning ? u : u + turning), v1 = V * (!kInterleaved && u < turning ? u + turning : u + kLanes);
  auto fetch = [&](int step) {
    if (step < hi) {
      const RopeHeads& r = step < q_steps ? a.q : a.k;
      const int h = (step < q_steps ? step : step - q_steps) * kRows + mine;
      if (h < r.heads) {
        const T* x = static_cast<const T*>(r.x) + t * r.ldx + h * r.hx;
        uint4* to = &ring[warp][(step - lo) % kRopeStages][0][lane];
        copy16(to, x + v0);
        copy16(to + 32, x + v1);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int s = 0; s < kRopeStages - 1; ++s) fetch(lo + s);
  for (int i = lane; i < half; i += 32) turns[warp][i] = pair_turn(a, i, t);
  __syncwarp();

  // weights of values i of v0 and v1, and with them the turn of their pair:
  // out0 = x0 * aa - x1 * ab, out1 = x0 * ba + x1 * bb.  A value that does not turn takes nothing of its
  // neighbour, not even 0 times what is infinite or no number (7596 tokens of 26 x 256 bf16, 64 of them
  // turning, 35.7 -> 36.5 us; a branch by lanes in place of the selection 37.0).
  float aa[V], ab[V], ba[V], bb[V];
  uint32_t turned = 0;    // bit i: pair i turns
  bool all_turn = false;  // all pairs of the warp's lanes do
  auto weigh = [&](const float* weight) {
    float w[2 * V];
#pragma unroll
    for (int i = 0; i < 2 * V; ++i) w[i] = 1.0f;
    if (a.norm && weight) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const float4 f = *reinterpret_cast<const float4*>(weight + v0 + i), g = *reinterpret_cast<const float4*>(weight + v1 + i);
        w[i] = f.x, w[i + 1] = f.y, w[i + 2] = f.z, w[i + 3] = f.w;
        w[V + i] = g.x, w[V + i + 1] = g.y, w[V + i + 2] = g.z, w[V + i + 3] = g.w;
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int pair = !kInterleaved ? u * V + i : i < V / 2 ? v0 / 2 + i : v1 / 2 + i - V / 2;
      float2 c = pair < half ? turns[warp][pair] : make_float2(kNoTurn, 0.0f);
      if (c.x != kNoTurn) turned |= 1u << i; else c.x = 1.0f;
      const float w0 = kInterleaved ? w[2 * i] : w[i], w1 = kInterleaved ? w[2 * i + 1] : w[V + i];
      aa[i] = w0 * c.x;
      ab[i] = w1 * c.y;
      ba[i] = w0 * c.y;
      bb[i] = w1 * c.x;
    }
    all_turn = __all_sync(0xffffffffu, turned == (1u << V) - 1u);
  };

#pragma unroll 1
  for (int step = lo; step < hi; ++step) {
    if (step == lo || step == q_steps) weigh(step < q_steps ? a.q.weight : a.k.weight);
    fetch(step + kRopeStages - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(kRopeStages - 1) : "memory");
    const uint4* from = &ring[warp][(step - lo) % kRopeStages][0][lane];
    float v[2 * V];
    unpack16<T>(from[0], v);
    unpack16<T>(from[32], v + V);
    float scale = 1.0f;
    if (a.norm) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 2 * V; ++i) sum = fmaf(v[i], v[i], sum);
#pragma unroll
      for (int o = kLanes / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      scale = rsqrtf(sum * (1.0f / D) + a.eps);
    }
    float out[2 * V];
    auto rotate = [&](auto whole) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int i0 = kInterleaved ? 2 * i : i, i1 = kInterleaved ? 2 * i + 1 : V + i;
        const bool with = whole.value || ((turned >> i) & 1);
        out[i0] = scale * (with ? v[i0] * aa[i] - v[i1] * ab[i] : v[i0] * aa[i]);
        out[i1] = scale * (with ? v[i0] * ba[i] + v[i1] * bb[i] : v[i1] * bb[i]);
      }
    };
    if (all_turn) rotate(std::true_type{}); else rotate(std::false_type{});
    const RopeHeads& r = step < q_steps ? a.q : a.k;
    const int h = (step < q_steps ? step : step - q_steps) * kRows + mine;
    if (h < r.heads) {
      T* y = static_cast<T*>(r.y) + t * r.ldy + h * r.hy;
      *reinterpret_cast<uint4*>(y + v0) = pack16<T>(out);
      *reinterpret_cast<uint4*>(y + v1) = pack16<T>(out + V);
    }
  }
}

// Whether 16-byte accesses reach every vector of these heads.
static bool rope_vectors(const RopeHeads& r, int size) {
  const int V = 16 / size;
  return reinterpret_cast<uintptr_t>(r.x) % 16 == 0 && reinterpret_cast<uintptr_t>(r.y) % 16 == 0 &&
         reinterpret_cast<uintptr_t>(r.weight) % 16 == 0 && r.ldx % V == 0 && r.hx % V == 0 && r.ldy % V == 0 && r.hy % V == 0;
}

int launch_norm_rope(const NormRope& a, int dtype, int head_dim, cudaStream_t stream) {
  return with_dtype(dtype, [&](auto v) {
    using T = decltype(v);
    const int size = (int)sizeof(T), V = kVec<T>;
    if (rope_vectors(a.q, size) && (!a.k.heads || rope_vectors(a.k, size)) && (a.interleaved || a.rot / 2 % V == 0)) {
      // A token's heads are shared out to several warps: where tokens are few, to as many as fill the GPU, up to one
      // step each; else in shares of four steps or more, for four rounds of warps, so that the last round costs
      // little (7596 tokens of 36 x 256: 64.7 us with a warp a token, 59.3 so, 61.1 in eight rounds).
      const int rows = 64 * V / head_dim;
      const int steps = (a.q.heads + rows - 1) / rows + (a.k.heads + rows - 1) / rows;
      const bool few = (int64_t)steps * a.n_tokens <= kRopeWarpsAtOnce;
      const int splits = few ? steps : (int)min((int64_t)max(1, steps / 4), (4 * (int64_t)kRopeWarpsAtOnce + a.n_tokens - 1) / a.n_tokens);
      const int64_t units = (int64_t)a.n_tokens * splits;
      auto kern = a.interleaved ? (head_dim == 64    ? norm_rope_vec_kernel<T, 64, true>
                                   : head_dim == 128 ? norm_rope_vec_kernel<T, 128, true>
                                                     : norm_rope_vec_kernel<T, 256, true>)
                                : (head_dim == 64    ? norm_rope_vec_kernel<T, 64, false>
                                   : head_dim == 128 ? norm_rope_vec_kernel<T, 128, false>
                                                     : norm_rope_vec_kernel<T, 256, false>);
      return launch_pdl(kern, dim3((unsigned)((units + kRopeWarps - 1) / kRopeWarps)), dim3(32 * kRopeWarps), 0, stream, a, splits);
    }
    const int64_t rows = (int64_t)a.n_tokens * (a.q.heads + a.k.heads);
    auto kern = head_dim == 64 ? norm_rope_any_kernel<T, 64> : head_dim == 128 ? norm_rope_any_kernel<T, 128> : norm_rope_any_kernel<T, 256>;
    return launch_pdl(kern, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, stream, a);
  });
}

}  // namespace mmvq
