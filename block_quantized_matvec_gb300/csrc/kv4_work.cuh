// The division of an attention batch's work among the CTAs, and the joining of
// items that were split.  An item's fixed cost counts as 32 tiles and a CTA takes
// 16 units at least: 64 bf16 sequences of 128 .. 8192 tokens take 80.4 us with 16
// units an item, 76.3 with 24, 76.7 with 32 and 82.1 with 64; 32 fp16 windows of 4096
// 50.8, 50.2, 50.7 and 54.9.  Joins of over 24 parts go in two steps of about their
// square root, since one CTA reads them all.
#pragma once
#include "kv4_attention.cuh"

namespace mmvq {

constexpr float kKv4Lazy = 2.0f;    // slack of the softmax reference, log2 units
constexpr float kKv4Boost = 12.0f;  // p is at most 2^(kKv4Lazy + kKv4Boost) = 2^14, below fp16's largest
constexpr int kKv4Join = 32;        // parts that are joined at a time: at least sqrt(kKv4MaxCtas)
constexpr int kKv4JoinAtOnce = 24;  // more are joined in two steps

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ __half2 h2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
__device__ __forceinline__ uint32_t u32(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  return u32(__hmul2_rn(h2(a), h2(b)));
}
__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
  return u32(__hfma2(h2(a), h2(b), h2(c)));
}
__device__ __forceinline__ uint32_t add2(uint32_t a, uint32_t b) {
  return u32(__hadd2_rn(h2(a), h2(b)));
}

// 2^e, -126 <= e <= 127, and the exponent of a positive normal x.
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }
__device__ __forceinline__ int exponent(float x) { return (__float_as_int(x) >> 23) - 127; }

// a / b of unsigned numbers: most fit 32 bits, whose division is several times shorter.
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// The division of `total` units among n CTAs: the first `more` have share + 1.
struct Shares {
  int64_t share, more;
  __device__ __forceinline__ Shares(int64_t total, int n) : share(divide(total, n)), more(total - share * n) {}
  __device__ __forceinline__ int64_t begin(int i) const { return i * share + min((int64_t)i, more); }
  __device__ __forceinline__ int cta_of(int64_t unit) const {
    const int64_t large = more * (share + 1);
    return (int)(unit < large ? divide(unit, share + 1) : more + divide(unit - large, share));
  }
};

// N values from src in fp32; `vector`: src is 16-byte aligned.
template <int N, typename T>
__device__ __forceinline__ void kv4_load_values(const T* src, bool vector, float (&q)[N]) {
  constexpr int kEach = 16 / sizeof(T);
  if constexpr (N % kEach == 0) {
    if (vector) {
#pragma unroll
      for (int k = 0; k < N / kEach; ++k) {
        const uint4 v = reinterpret_cast<const uint4*>(src)[k];
        const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
        for (int i = 0; i < kEach; ++i) q[kEach * k + i] = kv4_load(e + i);
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) q[i] = kv4_load(src + i);
}

// The units of a batch before each thread's sequences, in shared memory, and where each thread has one, the sequences.
template <int kThreads>
struct Kv4Plan {
  int64_t before[kThreads];
  int64_t warp_units[kThreads / 32];
  Kv4Seq seq[kThreads];
};

// Fills the plan (by all threads of the CTA); the batch's units.
template <int kThreads>
__device__ __forceinline__ int64_t kv4_plan(const Kv4Batch& a, const Kv4Attention& p, int rows_block,
                                            Kv4Plan<kThreads>& plan, int tid) {
  const int lane = tid & 31, warp = tid >> 5;
  const int chunk = (a.n_seqs + kThreads - 1) / kThreads;
  int error = 0;
  int64_t mine = 0;
  for (int b = tid * chunk; b < min(a.n_seqs, (tid + 1) * chunk); ++b) {
    const Kv4Seq s = kv4_seq(a, p, rows_block, b, &error);
    if (chunk == 1) plan.seq[tid] = s;
    mine += (int64_t)a.n_kv_heads * s.blocks * s.item_units();
  }
  if (error && blockIdx.x == 0) kv4_set_status(a.status, error);
  int64_t up_to = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, up_to, o);
    if (lane >= o) up_to += x;
  }
  if (lane == 31) plan.warp_units[warp] = up_to;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) up_to += plan.warp_units[w];
    total += plan.warp_units[w];
  }
  plan.before[tid] = up_to - mine;
  __syncthreads();
  return total;
}

// CTAs that take part.
__device__ __forceinline__ int kv4_ctas(int64_t total) {
  return (int)min((int64_t)gridDim.x, (total + kKv4MinUnits - 1) / kKv4MinUnits);
}

// An item, and the part of its tiles that is this CTA's.
struct Kv4Item {
  Kv4Seq s;
  int b, head, row0, n_rows;  // of the sequence's rows of the kv head: row0 .. row0 + n_rows - 1
  int tile0, tile1;
  int64_t begin;              // its first unit
  int first, last;            // the CTAs that have tiles of it
};

// The item of `unit`, which is moved past this CTA's part of it.  False where that part holds none of its tiles.
template <int kThreads>
__device__ __forceinline__ bool kv4_next(const Kv4Batch& a, const Kv4Attention& p, int rows_block,
                                         const Kv4Plan<kThreads>& plan, const Shares& shares, int cta,
                                         int64_t& unit, Kv4Item& it) {
  const int64_t lo = shares.begin(cta), hi = shares.begin(cta + 1);
  const int chunk = (a.n_seqs + kThreads - 1) / kThreads;
  int th = 0, error = 0;
#pragma unroll
  for (int o = 256; o > 0; o >>= 1)
    if (th + o < kThreads && plan.before[th + o] <= unit) th += o;
  it.b = th * chunk;
  int64_t at = plan.before[th];
  it.s = chunk == 1 ? plan.seq[th] : kv4_seq(a, p, rows_block, it.b, &error);
  for (;;) {
    const int64_t units = (int64_t)a.n_kv_heads * it.s.blocks * it.s.item_units();
    if (at + units > unit) break;
    at += units;
    it.s = kv4_seq(a, p, rows_block, ++it.b, &error);
  }
  const int item = (int)divide(unit - at, it.s.item_units());
  it.begin = at + (int64_t)item * it.s.item_units();
  const int64_t end = it.begin + it.s.item_units(), tiles = it.begin + kKv4ItemUnits;  // units from there on: tiles
  it.tile0 = (int)max(unit - tiles, (int64_t)0);
  it.tile1 = (int)(min(hi, end) - tiles);
  unit = min(hi, end);
  if (it.tile1 <= it.tile0) return false;
  it.head = item / it.s.blocks;
  it.row0 = (item - it.head * it.s.blocks) * rows_block;
  it.n_rows = min(rows_block, it.s.n_new * (p.n_heads / a.n_kv_heads) - it.row0);
  it.first = lo <= tiles ? cta : shares.cta_of(tiles);
  it.last = hi >= end ? cta : shares.cta_of(end - 1);
  return true;
}

// Partial results of a row are unnormalised values, ref and sum: the values and the sum are in units of 2^ref.  A part
// without a finite score has ref -inf and sum 0 (or NaN, which must stay).
template <int kRows>
struct Kv4JoinSmem {
  float ref[kKv4Join][kRows], sum[kKv4Join][kRows], factor[kKv4Join][kRows];  // of a row's parts
  float row_ref[kRows], row_sum[kRows];
  int last;

  // A row's parts 0 .. n - 1: the row's ref and sum, and the factor of each part.
  __device__ __forceinline__ void weigh(int row, int n) {
    float top = -INFINITY, total = 0.0f;
#pragma unroll 8
    for (int k = 0; k < n; ++k) top = fmaxf(top, ref[k][row]);
#pragma unroll 8
    for (int k = 0; k < n; ++k) {
      const float r = ref[k][row], u = sum[k][row];
      const float f = r == -INFINITY ? (u == 0.0f ? 0.0f : 1.0f) : ex2(r - top);
      factor[k][row] = f;
      total = fmaf(f, u, total);
    }
    row_ref[row] = top;
    row_sum[row] = total;
  }
};

// Where the parts of an item lie: CTA i's in the second of its slots where CTA i has earlier items, else in the first.
template <int kRows, int D>
__device__ __forceinline__ float* kv4_slot(const Kv4Attention& p, const Shares& shares, const Kv4Item& it, int i) {
  float* slots = reinterpret_cast<float*>(static_cast<uint8_t*>(p.workspace) + kKv4CounterBytes);
  return slots + (2 * (int64_t)i + (shares.begin(i) < it.begin ? 1 : 0)) * kv4_slot_floats(kRows, D);
}

// Four values of a row to the outputs.
template <typename T>
__device__ __forceinline__ void kv4_store_row(const Kv4Batch& a, const Kv4Attention& p, const Kv4Item& it, int D,
                                              int row, int d4, float4 v, float ref, float sum) {
  const int group = p.n_heads / a.n_kv_heads, r = it.row0 + row, t = r / group;
  const int64_t out = (int64_t)(it.s.first + t) * p.n_heads + it.head * group + (r - t * group);
  const float inv = sum == 0.0f ? 0.0f : __fdividef(1.0f, sum);
  kv4_store4(static_cast<T*>(p.y) + out * D + 4 * d4, v.x * inv, v.y * inv, v.z * inv, v.w * inv);
  if (p.lse && d4 == 0) p.lse[out] = sum == 0.0f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
}

// Joins the parts of a split item, this CTA's being in its slot: in groups by the last CTA of a group to arrive, then
// the groups by the last group's; always added in the order of the CTAs.  By all threads of the CTA.
template <int kThreads, int kRows, int D, typename T>
__device__ __forceinline__ void kv4_join(const Kv4Batch& a, const Kv4Attention& p, const Shares& shares,
                                         const Kv4Item& it, int cta, Kv4JoinSmem<kRows>& sm, int tid) {
  uint32_t* counters = static_cast<uint32_t*>(p.workspace);
  auto slot_of = [&](int i) { return kv4_slot<kRows, D>(p, shares, it, i); };
  auto arrive = [&](uint32_t* counter, int n) {
    __threadfence();
    __syncthreads();
    if (tid == 0) {
      const bool is_last = atomicAdd(counter, 1u) == (uint32_t)n - 1u;
      if (is_last) *counter = 0u;
      sm.last = is_last;
    }
    __syncthreads();
    __threadfence();
    return sm.last != 0;
  };
  // parts of CTAs from, from + step, ...: n of them, at most kKv4Join
  auto join = [&](int from, int step, int n, bool final) {
    const float* base = slot_of(from);
    const float* rest = slot_of(from + step);  // the others lie at equal distances: their first slots
    const int64_t stride = 2 * (int64_t)step * kv4_slot_floats(kRows, D);
    for (int idx = tid; idx < n * kRows; idx += kThreads) {
      const int k = idx / kRows, row = idx % kRows;
      if (row < it.n_rows) {
        const float2 rs = __ldcg(reinterpret_cast<const float2*>((k ? rest + (k - 1) * stride : base) + kRows * D) + row);
        sm.ref[k][row] = rs.x;
        sm.sum[k][row] = rs.y;
      }
    }
    __syncthreads();
    if (tid < it.n_rows) sm.weigh(tid, n);
    __syncthreads();
    // a few vectors a thread at a time, four parts of each in flight
    constexpr int kEach = kRows * D / 4 >= 4 * kThreads ? 4 : (kRows * D / 4 + kThreads - 1) / kThreads;
    const int total = it.n_rows * (D / 4);
    for (int at = tid; at < total; at += kEach * kThreads) {
      float4 v[kEach];
#pragma unroll
      for (int e = 0; e < kEach; ++e) v[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
      for (int k = 0; k < n; ++k) {
        const float* part = k ? rest + (k - 1) * stride : base;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          const int idx = at + e * kThreads;
          if (idx < total) {
            const float4 x = __ldcg(reinterpret_cast<const float4*>(part) + idx);
            const float f = sm.factor[k][idx / (D / 4)];
            v[e].x = fmaf(f, x.x, v[e].x);
            v[e].y = fmaf(f, x.y, v[e].y);
            v[e].z = fmaf(f, x.z, v[e].z);
            v[e].w = fmaf(f, x.w, v[e].w);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        const int idx = at + e * kThreads, row = idx / (D / 4);
        if (idx < total) {
          if (final) kv4_store_row<T>(a, p, it, D, row, idx % (D / 4), v[e], sm.row_ref[row], sm.row_sum[row]);
          else reinterpret_cast<float4*>(slot_of(from))[idx] = v[e];
        }
      }
    }
    if (!final && tid < it.n_rows)
      *reinterpret_cast<float2*>(slot_of(from) + kRows * D + 2 * tid) = make_float2(sm.row_ref[tid], sm.row_sum[tid]);
  };
  const int parts = it.last - it.first + 1;
  int per = parts;
  if (parts > kKv4JoinAtOnce) {
    per = 1;
    while (per * per < parts) ++per;
  }
  const int grp = (cta - it.first) / per, from = it.first + grp * per, n = min(per, it.last + 1 - from);
  const int n_groups = (parts + per - 1) / per;
  if (arrive(counters + 2 * from + (grp == 0 ? 1 : 0), n)) {
    join(from, 1, n, n_groups == 1);
    if (n_groups > 1 && arrive(counters + 2 * kKv4MaxCtas + it.first, n_groups)) join(it.first, per, n_groups, true);
  }
}

}  // namespace mmvq
