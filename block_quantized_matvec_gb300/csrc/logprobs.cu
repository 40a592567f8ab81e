// Log probabilities of given tokens, entropy and the best alternatives of rows of logits.
//
// With m the largest of x = scale * logits and S, E the sums over all but one
// largest of exp(x - m) and exp(x - m) (x - m):
//   lse = m + log1p(S), log p(i) = (x_i - m) - log1p(S), H = log1p(S) - E / (1 + S);
// every difference is of terms of one sign, so that a row that is all but
// certain keeps its digits.
//
// One pass.  Each warp keeps its best `live` logits (those asked for, at least
// eight) in order, one a lane, and the sums over all others, of 2^y and 2^y y with
// y = (x - C) log2(e) - R: R is near the list's last, so that terms are summed at
// their own size also where the first stands far above, and C is 0 but where
// x log2(e) is so large that R would be a unit off; there C is the list's last and R 0.
// A logit that enters the list is taken out of the sums, one that leaves it is added to
// them, also where lists are merged at the end; what remains besides the sums is the
// list, whose first is m.
//
// What it spends: about 42 instructions for 8 logits of 16 bits (a maximum in
// pairs, conversions, two packed fp32 operations and an ex2 each), so the row comes
// through a ring of asynchronous copies, each thread's own, and CTAs are small: six
// rows an SM, which wait for one another at no barrier.  Lists are entered rarely:
// from its first batch of vectors, and again from 3, 9, 33, ... of them, each CTA finds
// a bound that `live` values reach, by counting its threads' largest ones
// in 64 bins; a warp looks closer only where the largest of a batch reaches the bound
// or its list's last, and then at a lane's vectors one value a lane.  (Code for that
// unrolled over the batch's values took 688 us for 2048 rows of 151936 in place of
// 192: the warps waited for instructions.)
//
// A row is shared out to the CTAs of a cluster where rows are few; the first one
// reads the others' lists and sums from their shared memory.
//
// Measured with 20 alternatives: 2048 x 151936 bf16 117 us (5.3 TB/s; instructions
// bound it, 58% of the issue slots), 1 x 151936 fp32 9 us (latency).  With five tokens
// above a finite mask of -1e9 in place of -inf 308 us: the mask is the list's last, and
// all of a CTA's first values are compared with it.
#include <cfloat>

#include <cooperative_groups.h>

#include "layer.cuh"
#include "typed.cuh"

namespace mmvq {

namespace cg = cooperative_groups;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// How far above R the list's last may stand, in powers of two, before R follows:
// the entropy's sum cancels by that much at most.
constexpr float kSlack = 3.0f;
// |x log2(e)| from which on C is taken off first: R, rounded, is off by half its unit, 1 from here on, which the
// entropy's sum cancels by; 128 of them, from 2^31 on, are an exponent that fp32 does not hold.
constexpr float kFar = 0x1p24f;
constexpr int kStages = 2;   // batches of the ring
constexpr int kBins = 64;    // of the bound's count
constexpr int kLeast = 8;    // a list's entries, however few are asked for
constexpr int kAgain = 4;    // the bound is found in batch 0, 2, and each time that many times as far on

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Four 32-bit words of -inf of the type.
template <typename T>
__device__ __forceinline__ uint4 minus_infinity() {
  const uint32_t w = sizeof(T) == 4 ? 0xff800000u : std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u;
  return make_uint4(w, w, w, w);
}

template <typename T>
using Pair = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;

// The largest of the values of n vectors, NaN where one is.
template <typename T, int n>
__device__ __forceinline__ float vectors_max(const uint4* r) {
  if constexpr (sizeof(T) == 4) {
    float m = __uint_as_float(r[0].x);
#pragma unroll
    for (int i = 0; i < n; ++i) {
      m = max_nan(m, max_nan(__uint_as_float(r[i].x), __uint_as_float(r[i].y)));
      m = max_nan(m, max_nan(__uint_as_float(r[i].z), __uint_as_float(r[i].w)));
    }
    return m;
  } else {
    auto pair = [](uint32_t w) { return *reinterpret_cast<const Pair<T>*>(&w); };
    Pair<T> m = pair(r[0].x);
#pragma unroll
    for (int i = 0; i < n; ++i) {
      m = __hmax2_nan(m, __hmax2_nan(pair(r[i].x), pair(r[i].y)));
      m = __hmax2_nan(m, __hmax2_nan(pair(r[i].z), pair(r[i].w)));
    }
    return max_nan(to_f32(m.x), to_f32(m.y));
  }
}

// A vector that is partly outside the row: value by value.
template <typename T>
__device__ __noinline__ uint4 load_edge(const T* x, int first, int vocab) {
  uint4 r = minus_infinity<T>();
  T v[kVec<T>];
#pragma unroll
  for (int i = 0; i < kVec<T>; ++i) {
    v[i] = from_f32<T>(-INFINITY);
    if (first + i >= 0 && first + i < vocab) v[i] = x[first + i];
  }
  memcpy(&r, v, sizeof(r));
  return r;
}

// What a CTA, or a row, has seen: its list in order, and the sums over all others.
struct RowPart {
  float v[32];
  int id[32];
  float s, t, C, R;
  int bad;
};

// A warp's list (one entry a lane, lanes from `live` on empty) and sums (a lane's share).
struct RowState {
  float v;
  int id;
  float2 s2, t2;  // shares of the sums of 2^y and 2^y y
  float C, R;     // reference; R = -inf: nothing seen yet
  bool bad;       // a NaN or +inf was

  __device__ __forceinline__ void add(float x, float L) {
    const float y = fmaxf(fmaf(x - C, L, -R), -200.0f), e = exp2_approx(y);
    s2.x += e;
    t2.x = fmaf(e, y, t2.x);
  }
  // The sums stated for another reference, which is not below this one.
  __device__ __forceinline__ void refer(float to_c, float to_r, float L) {
    if (R > -INFINITY) {
      const float d = fmaxf(fmaf(C - to_c, L, R - to_r), -1000.0f), f = exp2_approx(d);
      t2.x = f * fmaf(d, s2.x, t2.x);
      t2.y = f * fmaf(d, s2.y, t2.y);
      s2.x *= f;
      s2.y *= f;
    }
    C = to_c;
    R = to_r;
  }
  // The value m as the reference.
  __device__ __forceinline__ void refer(float m, float L) {
    const bool far = !(fabsf(m * L) < kFar);
    refer(far ? m : 0.0f, far ? 0.0f : m * L, L);
  }
};

__device__ __forceinline__ bool before(float v, int i, float w, int j) { return v > w || (v == w && i < j); }

// One step of a sort: of this lane's entry and that of lane ^ o, the better one where `keep`.
__device__ __forceinline__ void exchange(float& v, int& id, int o, bool keep) {
  const float ov = __shfl_xor_sync(0xffffffffu, v, o);
  const int oi = __shfl_xor_sync(0xffffffffu, id, o);
  if (before(ov, oi, v, id) == keep) v = ov, id = oi;
}
// The warp's 32 entries in falling order (a bitonic sort).
__device__ __forceinline__ void sort(float& v, int& id, int lane) {
#pragma unroll
  for (int n = 2; n <= 32; n *= 2)
#pragma unroll
    for (int o = n / 2; o; o >>= 1) exchange(v, id, o, !(lane & o) == !(lane & n));
}

// The entries (v, id), in falling order, into a's list: of 32 + 32 the lane's and the
// opposite one of the others; the better of the two are the best 32.  What leaves the
// list goes into the sums.
__device__ __forceinline__ void absorb(RowState& a, float v, int id, int live, int lane, float L) {
  float w = __shfl_sync(0xffffffffu, v, 31 - lane);
  const int j = __shfl_sync(0xffffffffu, id, 31 - lane);
  if (before(w, j, a.v, a.id)) {
    const float x = a.v;
    a.v = w, a.id = j;
    w = x;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) exchange(a.v, a.id, o, !(lane & o));
  const float more = lane >= live ? a.v : -INFINITY;
  if (lane >= live) a.v = -INFINITY, a.id = 0x7fffffff;
  const float out = warp_max(fmaxf(w, more));  // the best of those that leave
  if (out > -INFINITY) {
    if (fmaf(out - a.C, L, -a.R) > kSlack) a.refer(out, L);
    if (w > -INFINITY) a.add(w, L);
    if (more > -INFINITY) a.add(more, L);
  }
}

// Where a CTA's warps bring their lists together.
template <int kWarps>
struct Meeting {
  int2 entry[64 * kWarps];  // value and id; before, 64 of each warp that wait to be sorted
  RowPart row;
  int count[kWarps], bad[kWarps];
  float s[kWarps], t[kWarps];
};

// A bound that at least `live` of the threads' values reach and few more, -inf where that many are not
// finite: the values are counted in bins from the least to the largest.
template <int kWarps>
__device__ __forceinline__ float bound_of(float value, int live, float2 (&ends)[kWarps], int (&count)[kBins], int warp, int lane) {
  constexpr int kThreads = 32 * kWarps;
  const int tid = 32 * warp + lane;
  const float up = warp_max(value), down = -warp_max(value > -INFINITY ? -value : -INFINITY);
  __syncthreads();
  if (lane == 0) ends[warp] = make_float2(down, up);
  if (tid < kBins) count[tid] = 0;
  if (kBins > kThreads && tid + kThreads < kBins) count[tid + kThreads] = 0;
  if (__syncthreads_count(value > -INFINITY) < live) return -INFINITY;
  float l = INFINITY, h = -INFINITY;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    l = fminf(l, ends[w].x);
    h = fmaxf(h, ends[w].y);
  }
  const float per = h - l < INFINITY && h - l > 1e-30f ? (kBins - 0.5f) / (h - l) : 0.0f;  // bins a unit
  if (value > -INFINITY) atomicAdd(&count[min((int)((value - l) * per), kBins - 1)], 1);
  __syncthreads();
  // the highest bin that `live` stand in or above; its lower end less a hundredth of it, for the roundings
  const int c1 = count[2 * lane + 1], c0 = count[2 * lane];
  int above = c0 + c1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_down_sync(0xffffffffu, above, o);
    if (lane + o < 32) above += n;
  }
  const int pair = 31 - __clz(__ballot_sync(0xffffffffu, above >= live));
  const int bin = 2 * pair + __shfl_sync(0xffffffffu, above - c0 >= live, pair);
  return bin > 0 && per > 0.0f ? fmaxf(l, fmaf((float)bin - 0.01f, 1.0f / per, l)) : l;
}

// The warps' lists (each its list and the entries waiting) and sums as one, in warp 0's state.  At
// least `live` entries reach `least`, so what does not goes into the sums; of the others, a handful,
// each thread takes one and counts those before it.
template <int kWarps>
__device__ __forceinline__ void join(Meeting<kWarps>& m, RowState& st, float wait_v, int wait_id, float least, int live, int warp, int lane, float L) {
  const int tid = 32 * warp + lane;
  if (least > -INFINITY) {
    if (fmaf(least - st.C, L, -st.R) > 0.0f) st.refer(least, L);
    if (wait_v > -INFINITY && wait_v < least) st.add(wait_v, L);
    if (st.v > -INFINITY && st.v < least) st.add(st.v, L);
  }
  const uint32_t waits = __ballot_sync(0xffffffffu, wait_v > -INFINITY && wait_v >= least);
  const uint32_t lists = __ballot_sync(0xffffffffu, st.v > -INFINITY && st.v >= least);
  const uint32_t below = (1u << lane) - 1u;
  const int waiting = __popc(waits);
  if (lane == 0) m.count[warp] = waiting + __popc(lists);
  if (warp == 0) {
    m.row.v[lane] = -INFINITY;
    m.row.id[lane] = 0x7fffffff;
  }
  __syncthreads();
  const int c = lane < kWarps ? m.count[lane] : 0;
  const int n = __reduce_add_sync(0xffffffffu, c), base = __reduce_add_sync(0xffffffffu, lane < warp ? c : 0);
  if ((waits >> lane) & 1) m.entry[base + __popc(waits & below)] = make_int2(__float_as_int(wait_v), wait_id);
  if ((lists >> lane) & 1) m.entry[base + waiting + __popc(lists & below)] = make_int2(__float_as_int(st.v), st.id);
  __syncthreads();
  for (int i = tid; i < n; i += 32 * kWarps) {
    const float v = __int_as_float(m.entry[i].x);
    const int id = m.entry[i].y;
    int at = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
      const int2 o = m.entry[j];
      at += before(__int_as_float(o.x), o.y, v, id);
    }
    if (at < live) {
      m.row.v[at] = v;
      m.row.id[at] = id;
    }
  }
  __syncthreads();
  const float last = m.row.v[live - 1];
  if (last > -INFINITY) {  // a full list: what comes after it goes into the sums
    const int last_id = m.row.id[live - 1];
    st.refer(last, L);
    for (int i = tid; i < n; i += 32 * kWarps) {
      const float v = __int_as_float(m.entry[i].x);
      if (before(last, last_id, v, m.entry[i].y)) st.add(v, L);
    }
  }
  const float s = warp_sum(st.s2.x + st.s2.y), t = warp_sum(st.t2.x + st.t2.y);
  const bool bad = __any_sync(0xffffffffu, st.bad);
  if (lane == 0) {
    m.s[warp] = s;
    m.t[warp] = t;
    m.bad[warp] = bad;
  }
  __syncthreads();
  if (warp == 0) {
    const float ss = warp_sum(lane < kWarps ? m.s[lane] : 0.0f), tt = warp_sum(lane < kWarps ? m.t[lane] : 0.0f);
    st.s2 = make_float2(lane == 0 ? ss : 0.0f, 0.0f);
    st.t2 = make_float2(lane == 0 ? tt : 0.0f, 0.0f);
    st.bad = __any_sync(0xffffffffu, lane < kWarps && m.bad[lane]);
    st.v = m.row.v[lane];
    st.id = m.row.id[lane];
  }
}

template <typename T, int kWarps, int kUnroll>  // kUnroll: 16-byte vectors of a thread in a batch
__global__ void __launch_bounds__(32 * kWarps, kWarps == 16 ? 2 : kWarps == 4 ? 7 : 1) logprobs_kernel(const TokenLogprobs a, int cluster) {
  constexpr int V = kVec<T>, kThreads = 32 * kWarps;
  // a lane's values are looked at 32 at a time, or all at once where they are fewer
  static_assert(kUnroll * V % 32 == 0 || kUnroll * V < 32);
  __shared__ Meeting<kWarps> meeting;
  __shared__ float2 ends[kWarps];
  __shared__ float said[2];
  __shared__ int count[kBins];
  extern __shared__ uint4 ring[];  // [kStages][kUnroll][kThreads]
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t row = blockIdx.x / cluster;
  const int rank = blockIdx.x - (int)row * cluster;
  const T* x = static_cast<const T*>(a.logits) + row * a.ld;
  const float L = a.scale * kLog2e;
  const int live = max(kLeast, a.top);

  // the row's vectors by address: the first and the last may be partly outside
  const int ahead = (int)(reinterpret_cast<uintptr_t>(x) % 16 / sizeof(T));
  const int vectors = (a.vocab + ahead + V - 1) / V, share = (vectors + cluster - 1) / cluster;
  const int lo = rank * share, hi = min(vectors, lo + share);
  const int whole = (a.vocab + ahead) / V;  // vectors from here on are not
  RowState st;
  st.v = -INFINITY;
  st.id = 0x7fffffff;
  st.s2 = st.t2 = make_float2(0.0f, 0.0f);
  st.C = 0.0f;
  st.R = -INFINITY;
  st.bad = false;
  // values from last_v on may enter the list, in batches to come those from `look` on
  float last_v = -FLT_MAX, look = -FLT_MAX, largest = -INFINITY, bound = -INFINITY;
  int next = 0;
  const float one_over_L = 1.0f / L;
  const float2 L2 = make_float2(L, L);
  // entries that are still to be sorted into the list, this warp's part of the meeting's
  int2* const wait = meeting.entry + 64 * warp;
  int waiting = 0;  // below 32 but while a lane is looked at
  auto settle = [&]() {
    __syncwarp();
    waiting -= 32;
    const int2 e = wait[waiting + lane];
    float v = __int_as_float(e.x);
    int id = e.y;
    __syncwarp();
    sort(v, id, lane);
    absorb(st, v, id, live, lane, L);
    const float lv = __shfl_sync(0xffffffffu, st.v, live - 1);
    if (lv >= last_v) {
      last_v = lv;
      // the ids of later batches are higher, so equal values come too late
      look = lv == 0.0f ? __uint_as_float(1u) : __uint_as_float(__float_as_uint(lv) + (lv > 0.0f ? 1 : -1));
      if (fmaf(lv - st.C, L, -st.R) > kSlack) st.refer(lv, L);
    }
  };

  const int batches = (hi - lo + kThreads * kUnroll - 1) / (kThreads * kUnroll);
  const int inside = min(hi, whole) - kThreads * kUnroll;  // batches that begin behind it are not all whole vectors
  // this thread's vectors of a stage, kThreads apart
  auto stage = [&](int b) { return ring + (b % kStages) * kUnroll * kThreads + tid; };
  auto fetch = [&](int b) {
    const int begin = lo + b * kThreads * kUnroll, first = begin + tid;
    uint4* to = stage(b);
    const T* from = x + ((int64_t)first * V - ahead);
    if (begin > 0 && begin <= inside) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) copy16(to + u * kThreads, from + u * kThreads * V);
    } else if (b < batches) {
#pragma unroll 1
      for (int u = 0; u < kUnroll; ++u) {
        const int j = first + u * kThreads;
        if (j >= hi) to[u * kThreads] = minus_infinity<T>();
        else if ((j > 0 || ahead == 0) && j < whole) copy16(to + u * kThreads, from + u * kThreads * V);
        else to[u * kThreads] = load_edge(x, j * V - ahead, a.vocab);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int b = 0; b < kStages - 1; ++b) fetch(b);
  // the first given token of this thread, under way with the first batch
  float given = 0.0f;
  bool is_token = false;
  if (rank == 0 && tid < a.n_tokens) {
    const int id = a.tokens[row * a.n_tokens + tid];
    is_token = id >= 0 && id < a.vocab;
    if (is_token) given = to_f32(x[id]);
  }

#pragma unroll 1
  for (int b = 0; b < batches; ++b) {
    fetch(b + kStages - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    uint4* const mine = stage(b);
    float most;
    {
      uint4 raw[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) raw[u] = mine[u * kThreads];
      most = vectors_max<T, kUnroll>(raw);
    }
    if (most < INFINITY) largest = fmaxf(largest, most); else st.bad = true;

    if (b == next) {  // 0, 2, 8, 32, ...
      next = max(2, kAgain * next);
      // at least `live` of the threads' largest reach it
      const float l = bound_of<kWarps>(largest, live, ends, count, warp, lane);
      if (l > -INFINITY) {
        bound = l;
        if (l > last_v) {
          last_v = look = l;
          if (fmaf(l - st.C, L, -st.R) > kSlack) st.refer(l, L);
        }
      }
    }

    uint32_t lanes = __ballot_sync(0xffffffffu, most >= look);
    if (lanes) {
      __syncwarp();  // the lanes' copies
      // a lane's vectors, 32 of their values one a lane
      T* const near = reinterpret_cast<T*>(mine - lane + lane / V * kThreads) + lane % V;
      const int id0 = (lo + b * kThreads * kUnroll + warp * 32 + lane / V * kThreads) * V - ahead + lane % V;
#pragma unroll 1
      do {
        const int src = __ffs(lanes) - 1;
        lanes &= lanes - 1;
#pragma unroll
        for (int g = 0; g < kUnroll * V; g += 32) {
          T* const p = near + src * V + g * kThreads;
          const float v = kUnroll * V >= 32 || lane < kUnroll * V ? to_f32(*p) : -INFINITY;
          const uint32_t who = __ballot_sync(0xffffffffu, v >= last_v);
          if (who) {
            if (v >= last_v) {
              wait[waiting + __popc(who & ((1u << lane) - 1u))] = make_int2(__float_as_int(v), id0 + src * V + g * kThreads);
              *p = from_f32<T>(-INFINITY);
            }
            waiting += __popc(who);
            if (waiting >= 32) settle();
          }
        }
      } while (lanes);
      __syncwarp();
    }

    if (st.R == -INFINITY) continue;  // all there was is in the list
    // what is so small that it adds nothing, and -inf, enter as one finite value of that kind; far from 0 a 128th below C is
    const bool far = st.C != 0.0f;
    const float2 R2 = make_float2(-st.R, -st.R), C2 = make_float2(-st.C, -st.C);
    const T least = from_f32<T>(fmaxf(far ? st.C - fabsf(st.C) * 0x1p-7f : (st.R - 160.0f) * one_over_L,
                                      std::is_same<T, __half>::value ? -65504.0f : -3.0e38f));
    // a batch's sums by themselves: however long the row, few additions follow one another
    auto stream = [&](auto is_far) {
      float2 s2 = make_float2(0.0f, 0.0f), t2 = s2;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const uint4 raw = mine[u * kThreads];
        float v[V];
        if constexpr (sizeof(T) == 4) {
          unpack16<T>(raw, v);
#pragma unroll
          for (int i = 0; i < V; ++i) v[i] = fmaxf(v[i], least);
        } else {
          Pair<T> both;
          both.x = both.y = least;
          uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const Pair<T> p = __hmax2(*reinterpret_cast<Pair<T>*>(&w[i]), both);
            w[i] = *reinterpret_cast<const uint32_t*>(&p);
          }
          unpack16<T>(make_uint4(w[0], w[1], w[2], w[3]), v);
        }
#pragma unroll
        for (int i = 0; i < V; i += 2) {
          const float2 x2 = make_float2(v[i], v[i + 1]);
          const float2 y = is_far.value ? __fmul2_rn(__fadd2_rn(x2, C2), L2) : __ffma2_rn(x2, L2, R2);
          const float2 e = make_float2(exp2_approx(y.x), exp2_approx(y.y));
          s2 = __fadd2_rn(s2, e);
          t2 = __ffma2_rn(e, y, t2);
        }
      }
      st.s2 = __fadd2_rn(st.s2, s2);
      st.t2 = __fadd2_rn(st.t2, t2);
    };
    const float least_y = fmaf(to_f32(least) - st.C, L, -st.R);
    if (least_y <= -150.0f && least_y > -INFINITY) {
      if (far) stream(std::true_type{}); else stream(std::false_type{});
    } else {
      // Logits so large, or a scale so small, that the type has no such value, or a scale so large that it is infinitely
      // far off: for fp16 scales below about 0.0016
      // (2048 x 151936 at 0.0015: 247 us, at 1: 113; 301 x 50021: 20.9 and 15.7).
#pragma unroll 1
      for (int u = 0; u < kUnroll; ++u)
#pragma unroll 1
        for (int i = 0; i < V; ++i) st.add(to_f32(reinterpret_cast<const T*>(mine + u * kThreads)[i]), L);
    }
  }

  __syncwarp();
  float wait_v = -INFINITY;
  int wait_id = 0x7fffffff;
  if (lane < waiting) {
    wait_v = __int_as_float(wait[lane].x);
    wait_id = wait[lane].y;
  }
  join(meeting, st, wait_v, wait_id, bound, live, warp, lane, L);
  if (cluster > 1) {
    if (tid == 0) {
      meeting.row.s = st.s2.x;
      meeting.row.t = st.t2.x;
      meeting.row.C = st.C;
      meeting.row.R = st.R;
    }
    if (warp == 0) meeting.row.bad = st.bad;
    cg::this_cluster().sync();
    st.s2 = st.t2 = make_float2(0.0f, 0.0f);
    st.C = 0.0f;
    st.R = -INFINITY;
    st.bad = false;
    wait_v = -INFINITY;
    if (rank == 0 && warp < cluster) {  // a CTA's to each warp
      const RowPart& from = *cg::this_cluster().map_shared_rank(&meeting.row, warp);
      wait_v = from.v[lane];
      wait_id = from.id[lane];
      if (lane == 0) {
        st.s2.x = from.s;
        st.t2.x = from.t;
      }
      st.C = from.C;
      st.R = from.R;
      st.bad = from.bad;
    }
    cg::this_cluster().sync();  // all are read: the others may leave
    if (rank != 0) return;
    st.v = -INFINITY;
    // what cannot be among the row's best: one row of 151936 with 32 alternatives 14.4 us with all lists compared, 9.4 so
    const float least = bound_of<kWarps>(wait_v, live, ends, count, warp, lane);
    join(meeting, st, wait_v, wait_id, least, live, warp, lane, L);
  }

  const float nan = __int_as_float(0x7fc00000);
  if (warp == 0) {
    const bool bad = __any_sync(0xffffffffu, st.bad);
    const float m = __shfl_sync(0xffffffffu, st.v, 0);
    const bool empty = m == -INFINITY;
    // x - m, at most 0, and what its two roundings left
    const float diff = st.v - m, back = diff - st.v, d = diff * a.scale;
    float e = 0.0f, ed = 0.0f;
    if (lane > 0 && d > -200.0f) {
      const float rest = fmaf(diff, a.scale, -d) + ((st.v - (diff - back)) - (m + back)) * a.scale;
      e = fmaf(expf(d), rest, expf(d));
      ed = e * d;
    }
    const float s = warp_sum(st.s2.x + st.s2.y), t = warp_sum(st.t2.x + st.t2.y);
    if (lane == 0 && st.R > -INFINITY && s > 0.0f) {
      // From the reference to m, and what L's rounding makes of the mean x: both exponents
      // can be large where the sums are small, hence in 64 bits.
      const double exact = (double)a.scale * 1.4426950408889634074;
      const double Y = fmax(-400.0, (double)st.R + ((double)st.C - (double)m) * exact + (double)((t / s + st.R) / L) * (exact - (double)L));
      const double near = rint(Y);
      const float f = ldexpf(exp2f((float)(Y - near)), (int)near);
      e = f * s;
      ed = f * kLn2 * fmaf((float)Y, s, t);
    }
    const float S = warp_sum(e), E = warp_sum(ed);
    const float drop = log1pf(S);
    if (lane == 0) {
      if (bad && a.status) *a.status = MMVQ_ERR_VALUE;
      if (a.lse) a.lse[row] = bad ? nan : empty ? -INFINITY : fmaf(m, a.scale, drop);
      if (a.entropy) a.entropy[row] = bad ? nan : empty ? 0.0f : drop - E / (1.0f + S);
      said[0] = bad ? nan : m;
      said[1] = drop;
    }
    if (lane < a.top) {
      const bool no = bad || st.v == -INFINITY;
      a.top_ids[row * a.top + lane] = no ? -1 : st.id;
      a.top_logprobs[row * a.top + lane] = bad ? nan : no ? -INFINITY : d - drop;
    }
  }
  if (a.n_tokens == 0) return;
  __syncthreads();
  const float m = said[0], drop = said[1];
  for (int j = tid; j < a.n_tokens; j += kThreads) {
    if (j != tid) {
      const int id = a.tokens[row * a.n_tokens + j];
      is_token = id >= 0 && id < a.vocab;
      if (is_token) given = to_f32(x[id]);
    }
    if (!is_token && a.status) *a.status = MMVQ_ERR_ROUTING;
    a.logprobs[row * a.n_tokens + j] = !is_token || m != m ? nan : m == -INFINITY ? m : (given - m) * a.scale - drop;
  }
}

template <typename T, int kWarps, int kUnroll>
static int launch_rows(const TokenLogprobs& a, int cluster, cudaStream_t stream) {
  auto kern = logprobs_kernel<T, kWarps, kUnroll>;
  const int smem = kStages * kUnroll * 32 * kWarps * 16;
  static int per_device[64];  // whether the kernel has its attributes there
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return MMVQ_ERR_CUDA;
  if (!__atomic_load_n(&per_device[dev], __ATOMIC_ACQUIRE)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
        cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
      return MMVQ_ERR_CUDA;
    __atomic_store_n(&per_device[dev], 1, __ATOMIC_RELEASE);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.rows * cluster);
  cfg.blockDim = dim3(32 * kWarps);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, a, cluster) == cudaSuccess ? MMVQ_OK : MMVQ_ERR_CUDA;
}

int launch_token_logprobs(const TokenLogprobs& a, int dtype, cudaStream_t stream) {
  return with_dtype(dtype, [&](auto v) {
    using T = decltype(v);
    constexpr int kSms = 152;
    const int vectors = (a.vocab + 2 * kVec<T> - 1) / kVec<T>;
    // Many short rows: a warp each (2048 x 1000 bf16 13.6 us, by CTAs of 4 warps 21.5; 16 x 1000 9.3 and 7.0).
    if (vectors <= 160 && a.rows > 4 * kSms) return launch_rows<T, 1, 4>(a, 1, stream);
    // CTAs of 4 warps, six an SM, spend less on a row than those of 16, two an SM, but need more rows to fill the
    // GPU.  (bf16, 4 and 16 warps: 600 rows of 152000 54.6 and 47.9 us, of 50000 28.2 and 26.8; 1000 rows 75.5 and
    // 78.8, 39.7 and 45.5; 152 and 300 rows of 4000 7.6 and 6.6, 7.6 and 8.1.  fp32, 1000 rows of 152000: 125 and 104.)
    if (a.rows > (vectors <= 1024 ? 1 : vectors <= 32768 ? 4 : 8) * kSms) return launch_rows<T, 4, 8>(a, 1, stream);
    // Few rows: a cluster's CTAs share one, as far as each has a batch and the GPU has places.  (bf16, by 1, 2, 4, 8,
    // 16 CTAs: one row of 152000 15.1, 13.2, 11.4, 9.9, 9.1 us, 15 rows 15.3, 13.4, 11.6, 11.1, 15.3, 64 rows 15.7, 14.1, 15.6;
    // one row of 50000 9.9, 10.6, 9.2, 9.1, 8.9, of 16000 6.4, 8.9, 8.3.)
    int cluster = 1;
    if (vectors > 4096)
      while (cluster < 16 && vectors > 2000 * cluster && (int64_t)a.rows * 2 * cluster <= (cluster == 8 ? 64 : 128)) cluster *= 2;
    return launch_rows<T, 16, 4>(a, cluster, stream);
  });
}

}  // namespace mmvq
