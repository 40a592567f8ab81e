// Keys and values quantised into the 4-bit cache, and read back from it.
//
// Where sequences have 16 new rows or more on average, a warp takes a tile's
// rows of one kv head.  Lanes own what the tile layout gives them: key words
// are 8 consecutive values of a token, so a block's extremes meet in 2
// shuffles and its codes leave in 16-byte stores; value words, 4 consecutive
// values of two tokens, are put together from those by 2 shuffles (both
// tokens present: 16-byte stores, one: 2-byte ones).  Whole tiles move as
// 512-byte rows of the layout on the cache's side and 64- or 128-byte runs on
// the plain side, nothing is staged in shared memory.  With fewer rows a warp takes one row, so that a
// decode step's rows spread over the GPU.
#include "kv4.cuh"

namespace mmvq {
namespace {

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
// of block w in bits 4 i of codes[w]), and the blocks' d (low half) and z as fp16.
//
// Beyond fp16's range (and for NaN) the values are clamped first (NaN to 0); odd: whether one was not finite.
//
// The quotient (x - z) / d is correctly rounded without a division each: Markstein's correction of x * r by
// its exact remainder, r the correctly rounded reciprocal of d.
template <int W, int N>
__device__ __forceinline__ void quantize_blocks(float (&x)[W][N], uint32_t (&codes)[W], uint32_t (&dz)[W], bool& odd) {
  float hi[W], lo[W];
  auto extremes = [&]() {
#pragma unroll
    for (int w = 0; w < W; ++w) {
      hi[w] = lo[w] = x[w][0];
#pragma unroll
      for (int i = 1; i < N; ++i) hi[w] = max_nan(hi[w], x[w][i]), lo[w] = min_nan(lo[w], x[w][i]);
#pragma unroll
      for (int o = 1; o < 32 / N; o <<= 1) {
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
  bool outside = false;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const __half dh = __float2half_rn(divide15(__fsub_rn(hi[w], lo[w])));
    const __half zh = __float2half_rn(__fmul_rn(__fadd_rn(hi[w], lo[w]), 0.5f));
    dz[w] = (uint32_t)__half_as_ushort(dh) | (uint32_t)__half_as_ushort(zh) << 16;
    const float d = __half2float(dh), z = __half2float(zh);
    const float r = d > 0.0f ? __frcp_rn(d) : 0.0f;  // without a step every quotient is 0: set to 0 below
    auto quotient = [&](float v) {
      const float e = __fsub_rn(v, z), q = __fmul_rn(e, r);
      return fmaf(fmaf(-d, q, e), r, q);
    };
    // a z that was rounded by much against d: codes beyond 0 and 15
    outside |= !(quotient(hi[w]) < 8.0f && quotient(lo[w]) >= -8.0f);
#pragma unroll
    for (int i = 0; i < N; ++i) x[w][i] = __fadd_rn(quotient(x[w][i]), d > 0.0f ? 7.5f : 0.0f);
  }
  if (__any_sync(0xffffffffu, outside)) {
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
      for (int i = 0; i < N; ++i) x[w][i] = fminf(fmaxf(x[w][i], 0.0f), 15.0f);
  }
#pragma unroll
  for (int w = 0; w < W; ++w) {
    codes[w] = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)  // 1.5 * 2^23 added: the sum's last bits are the number rounded to even
      codes[w] |= (__float_as_uint(__fadd_rn(x[w][i], 12582912.0f)) & 15u) << (4 * i);
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
  int b = 0, pos = 0, first = 0, last = r;  // the sequence of row r, its rows: none yet
#pragma unroll 1
  while (r < end) {
    if (r >= last) {
      if (!kv4_place(a, r, lane, b, pos)) {
        last = ++r;
        continue;
      }
      first = a.offsets[b];
      last = min(a.n_tokens, a.offsets[b + 1]);
    }
    int n = 1;
    if (pos < 0) {
      before(r);
    } else {
      Segment s = {b, pos / kKv4Tile, pos % kKv4Tile, 0, 0};
      n = chunk == 1 ? 1 : min(kKv4Tile - s.t0, last - r);
      s.t1 = s.t0 + n;
      s.row0 = (int64_t)r - s.t0;
      if (chunk == 1 || max(first, r - s.t0) >= r0) f(s);  // else it began in an earlier chunk
    }
    r += n;
    pos += n;
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
  int b, pos;
  if (!kv4_place(a, (int)r, lane, b, pos) || pos < 0) return;
  uint8_t* tile = kv4_tile(a, kv4_tile_bytes(D), b, pos / kKv4Tile);
  if (!tile) {
    if (lane == 0) kv4_set_status(a.status, MMVQ_ERR_ROUTING);
    return;
  }
  tile += head * kv4_head_stride(a, kv4_tile_bytes(D));
  const int t = pos % kKv4Tile;
  bool odd = false;
  uint32_t codes[kTurns], dz[kTurns];
  quantize_blocks(x, codes, dz, odd);
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int q = 4 * i + (lane >> 3), blk = q % nb, j = nb * (t >> 3) + blk;
    const bool key = q < nb;
    const int at = key ? kv4_word(j, 4 * (t & 7) + (g >> 1)) + 2 * (g & 1)
                       : 8 * D + kv4_word(j, 4 * g + ((t & 7) >> 1)) + 2 * (t & 1);
    *reinterpret_cast<uint16_t*>(tile + at) = (uint16_t)codes[i];
    if (g < 2) {
      const int sc = key ? kv4_key_scale(D, t, blk) : kv4_value_scale(D, t, blk);
      *reinterpret_cast<uint16_t*>(tile + sc + g * D) = (uint16_t)(dz[i] >> (16 * g));
    }
  }
  if (odd) kv4_set_status(a.status, MMVQ_ERR_VALUE);
}

// A chunk of one head a warp, either its keys or its values, and of heads of 256 one half of the blocks; half a
// tile's tokens at a time.  The rows are requested before the page is looked up.
template <int D, typename T>
__global__ void __launch_bounds__(256, 4) kv4_append_kernel(Kv4Batch a, Kv4Src src, int chunk) {
  constexpr int nb = D / 32, kN = nb < 4 ? nb : 4, kGroups = nb / kN;  // blocks of a warp
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
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
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      // this lane: values 8 c .. + 7 of every block of token 8 h + g
      const int t = 8 * h + g;
      const bool on = t >= s.t0 && t < s.t1;
      float x[kN][8];
#pragma unroll
      for (int w = 0; w < kN; ++w) {
        if (on) {
          load_run(base + (s.row0 + t) * ld + 32 * w, src.vector, x[w]);
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
      uint32_t words[kN], dz[kN];
      quantize_blocks(x, words, dz, odd);
      if (keys) {
        if (on) {
          uint8_t* at = tile + kv4_word(nb * h + b0, lane);
          uint8_t* sc = tile + kv4_key_scale(D, t, b0) + c * D;  // lanes 0 and 1 of a token store its d, its z
          uint32_t two[2];
#pragma unroll
          for (int w = 0; w < kN; w += 2) two[w / 2] = __byte_perm(dz[w], dz[w + 1], c ? 0x7632 : 0x5410);
          if constexpr (kN == 4) {
            *reinterpret_cast<uint4*>(at) = make_uint4(words[0], words[1], words[2], words[3]);
            if (c < 2) *reinterpret_cast<uint2*>(sc) = make_uint2(two[0], two[1]);
          } else {
            *reinterpret_cast<uint2*>(at) = make_uint2(words[0], words[1]);
            if (c < 2) *reinterpret_cast<uint32_t*>(sc) = two[0];
          }
        }
      } else {
        // the layout's word of this lane: values 4 g .. + 3 of tokens 2 c and 2 c + 1 of the half, which lanes
        // (2 c, g / 2) and (2 c + 1, g / 2) hold, in the half word g % 2; tokens 2 c, 2 c + 1: their d and z too
        const int from = 8 * c + (g >> 1), u = 8 * h + 2 * c;
        const bool on0 = u >= s.t0 && u < s.t1, on1 = u + 1 >= s.t0 && u + 1 < s.t1;
        uint32_t two[kN];
#pragma unroll
        for (int w = 0; w < kN; ++w) {
          const uint32_t w0 = __shfl_sync(0xffffffffu, words[w], from), w1 = __shfl_sync(0xffffffffu, words[w], from + 4);
          const uint32_t s0 = __shfl_sync(0xffffffffu, dz[w], from), s1 = __shfl_sync(0xffffffffu, dz[w], from + 4);
          words[w] = __byte_perm(w0, w1, g & 1 ? 0x7632 : 0x5410);
          two[w] = __byte_perm(s0, s1, g & 1 ? 0x7632 : 0x5410);  // g = 0: both d; g = 1: both z
        }
        uint8_t* at = tile + 8 * D + kv4_word(nb * h + b0, lane);
        uint8_t* sc = tile + kv4_value_scale(D, u, b0) + (g & 1) * D;
        if (on0 && on1) {
          if constexpr (kN == 4) {
            *reinterpret_cast<uint4*>(at) = make_uint4(words[0], words[1], words[2], words[3]);
            if (g < 2) *reinterpret_cast<uint4*>(sc) = make_uint4(two[0], two[1], two[2], two[3]);
          } else {
            *reinterpret_cast<uint2*>(at) = make_uint2(words[0], words[1]);
            if (g < 2) *reinterpret_cast<uint2*>(sc) = make_uint2(two[0], two[1]);
          }
        } else if (on0 || on1) {
          const int e = on1 ? 1 : 0;
#pragma unroll
          for (int w = 0; w < kN; ++w) {
            *reinterpret_cast<uint16_t*>(at + 4 * w + 2 * e) = (uint16_t)(words[w] >> (16 * e));
            if (g < 2) *reinterpret_cast<uint16_t*>(sc + 4 * w + 2 * e) = (uint16_t)(two[w] >> (16 * e));
          }
        }
      }
    }
  }, [](int) {});
  if (odd) kv4_set_status(a.status, MMVQ_ERR_VALUE);
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

template <int D, typename T>
__global__ void __launch_bounds__(256) kv4_read_kernel(Kv4Batch a, T* __restrict__ k_out, T* __restrict__ v_out,
                                                       int chunk) {
  constexpr int nb = D / 32;
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int r0 = (int)(item / a.n_kv_heads) * chunk, head = (int)(item % a.n_kv_heads);
  if (item / a.n_kv_heads * chunk >= a.n_tokens) return;
  const int64_t ld = (int64_t)a.n_kv_heads * D;
  T* k = k_out + head * D;
  T* v = v_out + head * D;
  auto zero_row = [&](int64_t r) {
    for (int i = lane; i < D / 4; i += 32) {
      kv4_store4(k + r * ld + 4 * i, 0.0f, 0.0f, 0.0f, 0.0f);
      kv4_store4(v + r * ld + 4 * i, 0.0f, 0.0f, 0.0f, 0.0f);
    }
  };
  for_segments(a, r0, chunk, lane, [&](const Segment& s) {
    const uint8_t* tile = segment_tile<D>(a, s, lane);
    if (!tile) {
      for (int t = s.t0; t < s.t1; ++t) zero_row(s.row0 + t);
      return;
    }
    tile += head * kv4_head_stride(a, kv4_tile_bytes(D));
    // the tile's words of this lane's tokens, all requested before the first is used
    uint4 kw[nb / 2], vw[nb / 2];
    bool kon[2], von[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      kon[h] = 8 * h + g >= s.t0 && 8 * h + g < s.t1;
#pragma unroll
      for (int e = 0; e < 2; ++e) von[h][e] = 8 * h + 2 * c + e >= s.t0 && 8 * h + 2 * c + e < s.t1;
    }
#pragma unroll
    for (int q = 0; q < nb / 2; ++q) {
      const int h0 = 4 * q / nb, h1 = (4 * q + 3) / nb;
      kw[q] = vw[q] = make_uint4(0, 0, 0, 0);
      if (kon[h0] || kon[h1]) kw[q] = *reinterpret_cast<const uint4*>(tile + 512 * q + 16 * lane);
      if (von[h0][0] || von[h0][1] || von[h1][0] || von[h1][1])
        vw[q] = *reinterpret_cast<const uint4*>(tile + 8 * D + 512 * q + 16 * lane);
    }
#pragma unroll
    for (int j = 0; j < 2 * nb; ++j) {
      const int h = j / nb, b = j % nb, t = 8 * h + g;
      const uint32_t w = j % 4 == 0 ? kw[j / 4].x : j % 4 == 1 ? kw[j / 4].y : j % 4 == 2 ? kw[j / 4].z : kw[j / 4].w;
      if (kon[h]) {
        const uint16_t* sc = reinterpret_cast<const uint16_t*>(tile + kv4_key_scale(D, t, b));
        store_codes8(k + (s.row0 + t) * ld + 32 * b + 8 * c, w, half_bits_to_float(sc[0]),
                     half_bits_to_float(sc[D / 2]));
      }
    }
#pragma unroll
    for (int j = 0; j < 2 * nb; ++j) {
      const int h = j / nb, b = j % nb, t = 8 * h + 2 * c;
      const uint32_t w = j % 4 == 0 ? vw[j / 4].x : j % 4 == 1 ? vw[j / 4].y : j % 4 == 2 ? vw[j / 4].z : vw[j / 4].w;
      if (von[h][0] || von[h][1]) {
        const uint32_t* sc = reinterpret_cast<const uint32_t*>(tile + kv4_value_scale(D, t, b));
        const uint32_t d = sc[0], z = sc[D / 4];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (von[h][e])
            store_codes(v + (s.row0 + t + e) * ld + 32 * b + 4 * g, w >> (16 * e),
                        half_bits_to_float((uint16_t)(d >> (16 * e))), half_bits_to_float((uint16_t)(z >> (16 * e))));
      }
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
  if ((items + 7) / 8 > 0x7fffffffLL) return MMVQ_ERR_SHAPE;
  return launch_pdl(kern, dim3((unsigned)((items + 7) / 8)), dim3(256), 0, stream, a, args..., chunk);
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
  return launch_chunks(kv4_read_kernel<256, T>, a, 1, stream, ko, vo);
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
