// Keys and values quantised into the 4-bit cache, and read back from it.
//
// Where sequences have 16 new rows or more on average, a warp takes a tile's
// rows of one kv head.  Lanes own what the tile layout gives them: key words
// are 8 consecutive values of a token, so a block's extremes meet in 2
// shuffles and its codes leave in 16-byte stores; value words, 4 consecutive
// values of two tokens, are put together from those by 2 shuffles (both
// tokens present: 16-byte stores, one: 2-byte ones).  Whole tiles move as
// 512-byte rows of the layout on the cache's side and 64- or 128-byte runs on
// the plain side, nothing is staged in shared memory.  With fewer rows a warp
// takes one row, so that a decode step's rows spread over the GPU.
//
// Measured on GB300 (6768 GB/s copied).  Append of 24575 fp32 tokens, 2 heads of
// 256 (116 MB): 23.7 us, 4.9 TB/s; of 24 bf16 prompts of 50 .. 1201 tokens behind 37
// cached ones, 8 heads of 128 (81 MB): 38.4 us, 2.1 TB/s.  Both are bound by
// instructions and the latency of a warp's few loads (55 to 66% of the issue
// slots; 21 and 24 instructions a value).  CTAs of 2 warps: a warp that finds
// nothing to do, or two segments, holds up no others (8 warps: 24.5 and 43 us).
// Read of 65536 bf16 tokens, 8 heads of 128 (352 MB): 55 us, 6.4 TB/s, DRAM: 20
// warps an SM with all of a tile's words in flight (24: 56 us, 32: 63, 40: 75).
// One row a warp: 4.4 us for one token, launch and three loads in a row.
#include "kv4.cuh"

namespace mmvq {
namespace {

constexpr int kCtaWarps = 2;  // of the kernels that take tiles

struct Kv4Src {
  const void* k;
  const void* v;
  int64_t ldk, hk, ldv, hv;  // strides of a token and of a head, in elements
  bool vector;               // all rows lie on 16-byte boundaries
};

// N consecutive values in fp32; `vector`: 16-byte boundaries (of 16 bytes or less: of that size).
template <int N, typename T>
__device__ __forceinline__ void load_run(const T* src, bool vector, float (&x)[N]) {
  if (vector) {
    if constexpr (N * sizeof(T) >= 16) {
#pragma unroll
      for (int k = 0; k < (int)(N * sizeof(T) / 16); ++k) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4*>(src) + k);
        const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
        for (int i = 0; i < (int)(16 / sizeof(T)); ++i) x[k * (16 / sizeof(T)) + i] = kv4_load(e + i);
      }
    } else {
      const uint2 v = __ldcs(reinterpret_cast<const uint2*>(src));
      const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = kv4_load(e + i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = kv4_load(src + i);
  }
}

// Eight consecutive values of a 2-byte type as they lie in memory.
template <typename T>
__device__ __forceinline__ uint4 load_raw(const T* src, bool vector) {
  if (vector) return __ldcs(reinterpret_cast<const uint4*>(src));
  const uint16_t* p = reinterpret_cast<const uint16_t*>(src);
  return make_uint4(p[0] | p[1] << 16, p[2] | p[3] << 16, p[4] | p[5] << 16, p[6] | p[7] << 16);
}

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// x / 15 correctly rounded (where it does not underflow): a quotient by the rounded reciprocal, corrected once by its
// exact remainder.  Checked for every significand against the division; the power of two does not matter.
__device__ __forceinline__ float divide15(float x) {
  const float c = 1.0f / 15.0f, q = __fmul_rn(x, c);
  return fmaf(fmaf(-15.0f, q, x), c, q);
}

// W blocks of 32 values, N of each in every one of 32 / N neighbouring lanes: the codes of this lane's values (value i
// of block w in bits 4 i of codes[w]), and d (low half) and z as fp16 of block (this lane's place in the blocks) % W,
// whose numbers this lane works out for all of them.
//
// Beyond fp16's range (and for NaN) the values are clamped first (NaN to 0); odd: whether one was not finite.
//
// The quotient (x - z) / d is correctly rounded without a division each: Markstein's correction of x * r by
// its exact remainder, r the correctly rounded reciprocal of d.
template <int W, int N>
__device__ __forceinline__ void quantize_blocks(float (&x)[W][N], uint32_t (&codes)[W], uint32_t& dz, bool& odd) {
  constexpr int kLanes = 32 / N;
  static_assert(W <= kLanes, "a lane for each block");
  const int lane = threadIdx.x & 31, own = lane % W, from = lane & ~(kLanes - 1);
  float hi[W], lo[W];
  auto extremes = [&]() {
#pragma unroll
    for (int w = 0; w < W; ++w) {
      hi[w] = lo[w] = x[w][0];
#pragma unroll
      for (int i = 1; i < N; ++i) hi[w] = max_nan(hi[w], x[w][i]), lo[w] = min_nan(lo[w], x[w][i]);
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) {
        hi[w] = max_nan(hi[w], __shfl_xor_sync(0xffffffffu, hi[w], o));
        lo[w] = min_nan(lo[w], __shfl_xor_sync(0xffffffffu, lo[w], o));
      }
    }
  };
  extremes();
  float top = fmaxf(hi[0], -lo[0]);
  bool nan = hi[0] != hi[0];
#pragma unroll
  for (int w = 1; w < W; ++w) top = fmaxf(top, fmaxf(hi[w], -lo[w])), nan |= hi[w] != hi[w];
  if (__any_sync(0xffffffffu, top > kFp16Max || nan)) {
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        odd |= !(fabsf(x[w][i]) < INFINITY);
        x[w][i] = x[w][i] != x[w][i] ? 0.0f : fminf(fmaxf(x[w][i], -kFp16Max), kFp16Max);
      }
    extremes();
  }
  float top_own = hi[0], low_own = lo[0];
#pragma unroll
  for (int w = 1; w < W; ++w)
    if (own == w) top_own = hi[w], low_own = lo[w];
  const __half dh = __float2half_rn(divide15(__fsub_rn(top_own, low_own)));
  const __half zh = __float2half_rn(__fmul_rn(__fadd_rn(top_own, low_own), 0.5f));
  dz = (uint32_t)__half_as_ushort(dh) | (uint32_t)__half_as_ushort(zh) << 16;
  const float d_own = __half2float(dh), z_own = __half2float(zh);
  const float r_own = d_own > 0.0f ? __frcp_rn(d_own) : 0.0f;  // without a step every quotient, and code, is 0
  auto quotient = [](float v, float d, float z, float r) {
    const float e = __fsub_rn(v, z), q = __fmul_rn(e, r);
    return fmaf(fmaf(-d, q, e), r, q);
  };
  // a z or d that was rounded by much against d: codes beyond 0 and 15.  The rounded sum decides: 7.5 and the largest
  // number below 8 are 15.5, which rounds to 16.
  const bool outside = !(__fadd_rn(quotient(top_own, d_own, z_own, r_own), 7.5f) < 15.5f &&
                         quotient(low_own, d_own, z_own, r_own) >= -8.0f);
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const float d = __shfl_sync(0xffffffffu, d_own, from + w), z = __shfl_sync(0xffffffffu, z_own, from + w);
    const float r = __shfl_sync(0xffffffffu, r_own, from + w), mid = r > 0.0f ? 7.5f : 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) x[w][i] = __fadd_rn(quotient(x[w][i], d, z, r), mid);
  }
  if (__any_sync(0xffffffffu, outside)) {
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
      for (int i = 0; i < N; ++i) x[w][i] = fminf(fmaxf(x[w][i], 0.0f), 15.0f);
  }
#pragma unroll
  for (int w = 0; w < W; ++w) {
    // 1.5 * 2^23 added, the bits are that number's plus the value rounded to even: the former's share is taken off
    codes[w] = 0;
    uint32_t share = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      codes[w] += __float_as_uint(__fadd_rn(x[w][i], 12582912.0f)) << (4 * i);
      share += 0x4b400000u << (4 * i);
    }
    codes[w] -= share;
  }
}

// Rows of sequence b in its tile number `tile`.
struct Segment {
  int b, tile;
  int t0, t1;      // tokens of the tile
  int64_t row0;    // the row of token 0 (may lie outside the sequence)
};

// The tile, of head 0, or NULL and *status set.
template <int D>
__device__ __forceinline__ uint8_t* segment_tile(const Kv4Batch& a, const Segment& s, int lane) {
  uint8_t* tile = kv4_tile(a, kv4_tile_bytes(D), s.b, s.tile);
  if (!tile && lane == 0) kv4_set_status(a.status, MMVQ_ERR_ROUTING);
  return tile;
}

// Calls f(segment) for the segments that begin in rows [r, r + chunk): a segment is the rows of a sequence that
// lie in one tile, or with a chunk of 1 a row.  Rows in no sequence are skipped, and those before a sequence's
// beginning (for which before(row) is called).
template <typename F, typename B>
__device__ __forceinline__ void for_segments(const Kv4Batch& a, int r, int chunk, int lane, F f, B before) {
  const int r0 = r, end = (int)min((int64_t)a.n_tokens, (int64_t)r + chunk);
  Kv4Place q = {0, 0, r, 0};  // the sequence of row r: none yet
#pragma unroll 1
  while (r < end) {
    if (r >= q.end && !kv4_place(a, r, lane, q)) {
      q.end = ++r;
      continue;
    }
    const int pos = q.len - (q.end - r);
    int n = 1;
    if (pos < 0) {
      before(r);
    } else {
      Segment s = {q.b, pos / kKv4Tile, pos % kKv4Tile, 0, 0};
      n = chunk == 1 ? 1 : min(kKv4Tile - s.t0, min(a.n_tokens, q.end) - r);
      s.t1 = s.t0 + n;
      s.row0 = (int64_t)r - s.t0;
      if (chunk == 1 || max(q.first, r - s.t0) >= r0) f(s);  // else it began in an earlier chunk
    }
    r += n;
  }
}

// One row of one head a warp: an octet of lanes a block, of the keys' blocks and then the values'.
template <int D, typename T>
__global__ void __launch_bounds__(256) kv4_append_rows_kernel(Kv4Batch a, Kv4Src src) {
  constexpr int nb = D / 32, kTurns = nb / 2;
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, g = lane & 7;
  const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t r = item / a.n_kv_heads;
  const int head = (int)(item % a.n_kv_heads);
  if (r >= a.n_tokens) return;
  const T* k = static_cast<const T*>(src.k) + r * src.ldk + head * src.hk;
  const T* v = static_cast<const T*>(src.v) + r * src.ldv + head * src.hv;
  float x[kTurns][4];
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int q = 4 * i + (lane >> 3);
    load_run((q < nb ? k : v) + 32 * (q % nb) + 4 * g, src.vector, x[i]);
  }
  Kv4Place q;
  if (!kv4_place(a, (int)r, lane, q)) return;
  const int pos = q.len - (q.end - (int)r);
  if (pos < 0) return;
  uint8_t* tile = kv4_tile(a, kv4_tile_bytes(D), q.b, pos / kKv4Tile);
  if (!tile) {
    if (lane == 0) kv4_set_status(a.status, MMVQ_ERR_ROUTING);
    return;
  }
  tile += head * kv4_head_stride(a, kv4_tile_bytes(D));
  const int t = pos % kKv4Tile;
  bool odd = false;
  uint32_t codes[kTurns], dz;
  quantize_blocks(x, codes, dz, odd);
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int q = 4 * i + (lane >> 3), blk = q % nb, j = nb * (t >> 3) + blk;
    const bool key = q < nb;
    const int at = key ? kv4_word(j, 4 * (t & 7) + (g >> 1)) + 2 * (g & 1)
                       : 8 * D + kv4_word(j, 4 * g + ((t & 7) >> 1)) + 2 * (t & 1);
    *reinterpret_cast<uint16_t*>(tile + at) = (uint16_t)codes[i];
  }
  if (g < kTurns) {
    const int q = 4 * g + (lane >> 3), blk = q % nb;
    const int sc = q < nb ? kv4_key_scale(D, t, blk) : kv4_value_scale(D, t, blk);
    *reinterpret_cast<uint16_t*>(tile + sc) = (uint16_t)dz;
    *reinterpret_cast<uint16_t*>(tile + sc + D) = (uint16_t)(dz >> 16);
  }
  if (odd) kv4_set_status(a.status, MMVQ_ERR_VALUE);
}

// A chunk of one head a warp, either its keys or its values, and of heads of 256 one half of the blocks; half a
// tile's tokens at a time.  The rows are requested before the page is looked up.
template <int D, typename T>
__global__ void __launch_bounds__(32 * kCtaWarps, (sizeof(T) == 2 ? 20 : 32) / kCtaWarps) kv4_append_kernel(Kv4Batch a, Kv4Src src, int chunk) {
  constexpr int nb = D / 32, kN = nb < 4 ? nb : 4, kGroups = nb / kN;  // blocks of a warp
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int64_t item = (int64_t)blockIdx.x * kCtaWarps + (threadIdx.x >> 5);
  const int part = (int)(item % (2 * kGroups)), b0 = part % kGroups * kN;
  const bool keys = part < kGroups;
  const int64_t unit = item / (2 * kGroups);
  const int head = (int)(unit % a.n_kv_heads);
  if (unit / a.n_kv_heads * chunk >= a.n_tokens) return;
  const int r0 = (int)(unit / a.n_kv_heads) * chunk;
  const T* base = static_cast<const T*>(keys ? src.k : src.v) + head * (keys ? src.hk : src.hv) + 32 * b0 + 8 * c;
  const int64_t ld = keys ? src.ldk : src.ldv;
  bool odd = false;
  for_segments(a, r0, chunk, lane, [&](const Segment& s) {
    uint8_t* tile = nullptr;
    // this lane: values 8 c .. + 7 of every block of tokens g and 8 + g; of 2-byte types the second half's are
    // requested with the first's (fp32 would need twice the registers for it)
    constexpr bool kBoth = sizeof(T) == 2;
    uint4 ahead[kN];
    auto on_of = [&](int h) { return 8 * h + g >= s.t0 && 8 * h + g < s.t1; };
    auto row_of = [&](int h) { return base + (s.row0 + 8 * h + g) * ld; };
    if constexpr (kBoth) {
#pragma unroll
      for (int w = 0; w < kN; ++w) {
        ahead[w] = make_uint4(0u, 0u, 0u, 0u);
        if (on_of(1)) ahead[w] = load_raw(row_of(1) + 32 * w, src.vector);
      }
    }
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      const int t = 8 * h + g;
      const bool on = on_of(h);
      float x[kN][8];
#pragma unroll
      for (int w = 0; w < kN; ++w) {
        if constexpr (kBoth) {
          uint4 v = ahead[w];
          if (h == 0) v = on ? load_raw(row_of(0) + 32 * w, src.vector) : make_uint4(0u, 0u, 0u, 0u);
          const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[w][i] = kv4_load(e + i);
        } else if (on) {
          load_run(row_of(h) + 32 * w, src.vector, x[w]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[w][i] = 0.0f;
        }
      }
      if (h == 0) {
        tile = segment_tile<D>(a, s, lane);
        if (!tile) return;
        tile += head * kv4_head_stride(a, kv4_tile_bytes(D));
      }
      uint32_t words[kN], dz;
      quantize_blocks(x, words, dz, odd);
      if (on && c < kN) {
        const int sc = keys ? kv4_key_scale(D, t, b0 + c) : kv4_value_scale(D, t, b0 + c);
        *reinterpret_cast<uint16_t*>(tile + sc) = (uint16_t)dz;
        *reinterpret_cast<uint16_t*>(tile + sc + D) = (uint16_t)(dz >> 16);
      }
      if (keys) {
        if (on) {
          uint8_t* at = tile + kv4_word(nb * h + b0, lane);
          if constexpr (kN == 4) *reinterpret_cast<uint4*>(at) = make_uint4(words[0], words[1], words[2], words[3]);
          else *reinterpret_cast<uint2*>(at) = make_uint2(words[0], words[1]);
        }
      } else {
        // the layout's word of this lane: values 4 g .. + 3 of tokens 2 c and 2 c + 1 of the half, which lanes
        // (2 c, g / 2) and (2 c + 1, g / 2) hold, in the half word g % 2
        const int from = 8 * c + (g >> 1), u = 8 * h + 2 * c;
        const bool on0 = u >= s.t0 && u < s.t1, on1 = u + 1 >= s.t0 && u + 1 < s.t1;
#pragma unroll
        for (int w = 0; w < kN; ++w) {
          const uint32_t w0 = __shfl_sync(0xffffffffu, words[w], from), w1 = __shfl_sync(0xffffffffu, words[w], from + 4);
          words[w] = __byte_perm(w0, w1, g & 1 ? 0x7632 : 0x5410);
        }
        uint8_t* at = tile + 8 * D + kv4_word(nb * h + b0, lane);
        if (on0 && on1) {
          if constexpr (kN == 4) *reinterpret_cast<uint4*>(at) = make_uint4(words[0], words[1], words[2], words[3]);
          else *reinterpret_cast<uint2*>(at) = make_uint2(words[0], words[1]);
        } else if (on0 || on1) {
          const int e = on1 ? 1 : 0;
#pragma unroll
          for (int w = 0; w < kN; ++w)
            *reinterpret_cast<uint16_t*>(at + 4 * w + 2 * e) = (uint16_t)(words[w] >> (16 * e));
        }
      }
    }
  }, [](int) {});
  if (odd) kv4_set_status(a.status, MMVQ_ERR_VALUE);
}

// N 32-bit words at p, aligned to their size (to 16 bytes at most).
template <int N>
__device__ __forceinline__ void load_words_global(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    static_assert(N == 1, "one, two or four");
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// Eight or four values from their codes to p.
template <typename T>
__device__ __forceinline__ void store_codes(T* p, uint32_t codes, float d, float z) {
  kv4_store4(p, kv4_value(codes & 15u, d, z), kv4_value(codes >> 4 & 15u, d, z), kv4_value(codes >> 8 & 15u, d, z),
             kv4_value(codes >> 12 & 15u, d, z));
}
template <typename T>
__device__ __forceinline__ void store_codes8(T* p, uint32_t codes, float d, float z) {
  if constexpr (sizeof(T) == 4) {
    store_codes(p, codes, d, z);
    store_codes(p + 4, codes >> 16, d, z);
  } else {
    T v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) kv4_store(v + i, kv4_value(codes >> (4 * i) & 15u, d, z));
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(v);
  }
}

// A chunk of one head a warp, of heads of 256 one half of the blocks.
template <int D, typename T>
__global__ void __launch_bounds__(32 * kCtaWarps, 20 / kCtaWarps) kv4_read_kernel(Kv4Batch a, T* __restrict__ k_out, T* __restrict__ v_out,
                                                          int chunk) {
  constexpr int nb = D / 32, kN = nb < 4 ? nb : 4, kGroups = nb / kN;
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int64_t item = (int64_t)blockIdx.x * kCtaWarps + (threadIdx.x >> 5);
  const int b0 = (int)(item % kGroups) * kN;
  const int64_t unit = item / kGroups;
  const int head = (int)(unit % a.n_kv_heads);
  if (unit / a.n_kv_heads * chunk >= a.n_tokens) return;
  const int r0 = (int)(unit / a.n_kv_heads) * chunk;
  const int64_t ld = (int64_t)a.n_kv_heads * D;
  T* k = k_out + head * D + 32 * b0;
  T* v = v_out + head * D + 32 * b0;
  auto zero_row = [&](int64_t r) {
    if (lane < 8 * kN) {
      kv4_store4(k + r * ld + 4 * lane, 0.0f, 0.0f, 0.0f, 0.0f);
      kv4_store4(v + r * ld + 4 * lane, 0.0f, 0.0f, 0.0f, 0.0f);
    }
  };
  for_segments(a, r0, chunk, lane, [&](const Segment& s) {
    const uint8_t* tile = segment_tile<D>(a, s, lane);
    if (!tile) {
      for (int t = s.t0; t < s.t1; ++t) zero_row(s.row0 + t);
      return;
    }
    tile += head * kv4_head_stride(a, kv4_tile_bytes(D));
    auto on = [&](int t) { return t >= s.t0 && t < s.t1; };
    // the words of this lane's tokens and their steps and midpoints, all requested before the first is used
    uint32_t kw[2][kN], kd[2][kN / 2], kz[2][kN / 2], vw[2][kN], vd[2][kN], vz[2][kN];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (on(8 * h + g)) {
        const uint8_t* sc = tile + kv4_key_scale(D, 8 * h + g, b0);
        load_words_global(tile + kv4_word(nb * h + b0, lane), kw[h]);
        load_words_global(sc, kd[h]);
        load_words_global(sc + D, kz[h]);
      }
      if (on(8 * h + 2 * c) || on(8 * h + 2 * c + 1)) {
        const uint8_t* sc = tile + kv4_value_scale(D, 8 * h + 2 * c, b0);
        load_words_global(tile + 8 * D + kv4_word(nb * h + b0, lane), vw[h]);
        load_words_global(sc, vd[h]);
        load_words_global(sc + D, vz[h]);
      }
    }
    auto half_at = [](uint32_t pair, int i) { return half_bits_to_float((uint16_t)(pair >> (16 * i))); };
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (on(8 * h + g)) {
        T* row = k + (s.row0 + 8 * h + g) * ld + 8 * c;
#pragma unroll
        for (int w = 0; w < kN; ++w)
          store_codes8(row + 32 * w, kw[h][w], half_at(kd[h][w / 2], w & 1), half_at(kz[h][w / 2], w & 1));
      }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (on(8 * h + 2 * c + e)) {
          T* row = v + (s.row0 + 8 * h + 2 * c + e) * ld + 4 * g;
#pragma unroll
          for (int w = 0; w < kN; ++w)
            store_codes(row + 32 * w, vw[h][w] >> (16 * e), half_at(vd[h][w], e), half_at(vz[h][w], e));
        }
  }, zero_row);
}

// Rows of a warp: a tile's where sequences have that many new rows, else one (a decode step's rows then
// spread over the GPU instead of following one another in a warp).
int chunk_of(const Kv4Batch& a) { return a.n_tokens >= kKv4Tile * a.n_seqs ? kKv4Tile : 1; }

// A warp per chunk, head and part.
template <typename K, typename... Args>
int launch_chunks(K kern, const Kv4Batch& a, int parts, cudaStream_t stream, Args... args) {
  const int chunk = chunk_of(a);
  const int64_t items = ((int64_t)a.n_tokens + chunk - 1) / chunk * a.n_kv_heads * parts;
  const int64_t ctas = (items + kCtaWarps - 1) / kCtaWarps;
  if (ctas > 0x7fffffffLL) return MMVQ_ERR_SHAPE;
  return launch_pdl(kern, dim3((unsigned)ctas), dim3(32 * kCtaWarps), 0, stream, a, args..., chunk);
}

template <int D, typename T>
int append_dim(const Kv4Batch& a, const Kv4Src& s, cudaStream_t stream) {
  if (chunk_of(a) > 1) return launch_chunks(kv4_append_kernel<D, T>, a, D == 256 ? 4 : 2, stream, s);
  const int64_t items = (int64_t)a.n_tokens * a.n_kv_heads;
  if ((items + 7) / 8 > 0x7fffffffLL) return MMVQ_ERR_SHAPE;
  return launch_pdl(kv4_append_rows_kernel<D, T>, dim3((unsigned)((items + 7) / 8)), dim3(256), 0, stream, a, s);
}

template <typename T>
int append_typed(const Kv4Batch& a, const Kv4Src& s, int D, cudaStream_t stream) {
  if (D == 64) return append_dim<64, T>(a, s, stream);
  if (D == 128) return append_dim<128, T>(a, s, stream);
  return append_dim<256, T>(a, s, stream);
}

template <typename T>
int read_typed(const Kv4Batch& a, int D, void* k, void* v, cudaStream_t stream) {
  T* ko = static_cast<T*>(k);
  T* vo = static_cast<T*>(v);
  if (D == 64) return launch_chunks(kv4_read_kernel<64, T>, a, 1, stream, ko, vo);
  if (D == 128) return launch_chunks(kv4_read_kernel<128, T>, a, 1, stream, ko, vo);
  return launch_chunks(kv4_read_kernel<256, T>, a, 2, stream, ko, vo);
}

}  // namespace

int launch_kv4_append(const Kv4Batch& a, int D, int dtype, const void* k, const void* v,
                      const int64_t (&strides)[4], cudaStream_t stream) {
  Kv4Src s = {k, v, strides[0], strides[1], strides[2], strides[3], false};
  uintptr_t bits = reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v);
  for (int64_t x : strides) bits |= (uintptr_t)(x * (dtype == MMVQ_F32 ? 4 : 2));
  s.vector = (bits & 15) == 0;
  if (dtype == MMVQ_F32) return append_typed<float>(a, s, D, stream);
  if (dtype == MMVQ_F16) return append_typed<__half>(a, s, D, stream);
  return append_typed<__nv_bfloat16>(a, s, D, stream);
}

int launch_kv4_read(const Kv4Batch& a, int D, int dtype, void* k, void* v, cudaStream_t stream) {
  if (dtype == MMVQ_F32) return read_typed<float>(a, D, k, v, stream);
  if (dtype == MMVQ_F16) return read_typed<__half>(a, D, k, v, stream);
  return read_typed<__nv_bfloat16>(a, D, k, v, stream);
}

}  // namespace mmvq
