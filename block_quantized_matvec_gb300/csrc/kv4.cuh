// The 4-bit key/value cache: block format, tile layout and the arguments that
// every kernel of the cache takes.
//
// Format.  32 consecutive values of a head's key (or value) vector share a
// step d = fp16((max - min) / 15) and a midpoint z = fp16((max + min) / 2);
// a code c in 0..15 stands for z + d * (c - 7.5), and a value x gets
// c = rint((x - z) / d + 7.5) clamped to 0..15 (0 where d is 0), every
// operation in fp32 and correctly rounded.  The midpoint form keeps the codes'
// part of a sum centred: sums over many tokens lose no bits to an offset.
//
// Layout.  A tile holds 16 tokens of one kv head in 20 * D bytes, in the order
// in which the warp-level matrix instructions of the attention take it, so
// that each lane fetches its share with 16-byte loads.  With nb = D / 32,
// token t of the tile and word(j, lane) = 512 * (j / 4) + 16 * lane + 4 * (j % 4):
//   [0, 8D)      key codes: word(nb * (t / 8) + b, 4 * (t % 8) + u) = values
//                32 b + 8 u .. + 7 of token t, value i in bits 4 i .. 4 i + 3
//   [8D, 16D)    value codes: word(nb * (t / 8) + b, 4 * g + (t % 8) / 2) =
//                values 32 b + 4 g .. + 3 of token t (t even: low half, odd:
//                high half), value i in bits 4 i .. 4 i + 3 of the half
//   [16D, 17D)   key d, fp16 [t][b];      [17D, 18D)  key z, the same
//   [18D, 19D)   value d, fp16 [(t % 8) / 2][t / 8][b][t % 2]
//   [19D, 20D)   value z, the same
// No two tokens share a byte, so tokens are written without reading.
#pragma once
#include <cuda_bf16.h>

#include "common.cuh"

namespace mmvq {

constexpr int kKv4Tile = 16;        // tokens of a tile
constexpr int kKv4MaxNew = 8;       // query tokens of a sequence
constexpr int kKv4MaxSeqs = 4096;
constexpr float kFp16Max = 65504.0f;

__host__ __device__ constexpr int kv4_tile_bytes(int D) { return 20 * D; }
__host__ __device__ constexpr int kv4_word(int j, int lane) {
  return 512 * (j >> 2) + 16 * lane + 4 * (j & 3);
}
// Byte offsets in a tile of token t's d; z lies D bytes further.
__host__ __device__ constexpr int kv4_key_scale(int D, int t, int b) {
  return 16 * D + 2 * (t * (D / 32) + b);
}
__host__ __device__ constexpr int kv4_value_scale(int D, int t, int b) {
  return 18 * D + 2 * ((((t & 7) >> 1) * 2 + (t >> 3)) * (D / 32) * 2 + 2 * b + (t & 1));
}

// A paged cache and the batch of sequences in it.
struct Kv4Batch {
  uint8_t* cache;             // [n_pages][n_kv_heads][page_tokens / 16] tiles
  int64_t n_pages;
  int page_tokens;
  int n_kv_heads;
  const int32_t* page_table;  // [n_seqs][ld_table]
  int64_t ld_table;
  const int32_t* offsets;     // [n_seqs + 1]: rows of sequence b
  const int32_t* lens;        // [n_seqs]: tokens of sequence b, the new ones included
  int n_seqs;
  int n_tokens;               // rows
  int32_t* status;
};

__device__ __forceinline__ void kv4_set_status(int32_t* status, int code) {
  if (status) *status = code;
}

// A sequence: its number, rows first .. end - 1, and length.
struct Kv4Place {
  int b, first, end, len;
};

// Row r's sequence, by a search over the offsets, 32 at a time, by all lanes of the warp; false where r lies in none.
// The last step's lanes hold the sequence's numbers already.
__device__ __forceinline__ bool kv4_place(const Kv4Batch& a, int r, int lane, Kv4Place& s) {
  int lo = 0, n = a.n_seqs;  // the sequence lies in [lo, lo + n)
  while (n > 32) {
    const int step = (n + 31) / 32;
    const bool starts = lane * step < n && a.offsets[lo + lane * step] <= r;
    const uint32_t m = __ballot_sync(0xffffffffu, starts);
    const int last = m ? 31 - __clz(m) : 0;
    n = min(step, n - last * step);
    lo += last * step;
  }
  const int i = lo + min(lane, n - 1);
  const int first = a.offsets[i], end = a.offsets[i + 1], len = max(0, a.lens[i]);  // positions stay in range
  const uint32_t m = __ballot_sync(0xffffffffu, lane < n && first <= r);
  const int at = m ? 31 - __clz(m) : 0;
  s.b = lo + at;
  s.first = __shfl_sync(0xffffffffu, first, at);
  s.end = __shfl_sync(0xffffffffu, end, at);
  s.len = __shfl_sync(0xffffffffu, len, at);
  return r >= s.first && r < s.end;
}

// The tile of position pos of sequence b (head 0), or NULL where the table
// has no such page.
__device__ __forceinline__ uint8_t* kv4_tile(const Kv4Batch& a, int tile_bytes, int b, int tile) {
  const int per_page = a.page_tokens / kKv4Tile;
  const int pi = tile / per_page;
  if (pi >= a.ld_table) return nullptr;
  const int64_t page = a.page_table[(int64_t)b * a.ld_table + pi];
  if (page < 0 || page >= a.n_pages) return nullptr;
  return a.cache + (page * a.n_kv_heads * per_page + (tile - pi * per_page)) * tile_bytes;
}
// Bytes from a tile of head h to that of head h + 1.
__device__ __forceinline__ int64_t kv4_head_stride(const Kv4Batch& a, int tile_bytes) {
  return (int64_t)(a.page_tokens / kKv4Tile) * tile_bytes;
}

__device__ __forceinline__ float kv4_load(const float* p) { return *p; }
__device__ __forceinline__ float kv4_load(const __half* p) { return __half2float(*p); }
__device__ __forceinline__ float kv4_load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void kv4_store(float* p, float v) { *p = v; }
__device__ __forceinline__ void kv4_store(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void kv4_store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Four values to p, aligned to four elements.
__device__ __forceinline__ void kv4_store4(float* p, float x, float y, float z, float w) {
  *reinterpret_cast<float4*>(p) = make_float4(x, y, z, w);
}
__device__ __forceinline__ void kv4_store4(__half* p, float x, float y, float z, float w) {
  __half2 v[2] = {__floats2half2_rn(x, y), __floats2half2_rn(z, w)};
  *reinterpret_cast<uint2*>(p) = *reinterpret_cast<uint2*>(v);
}
__device__ __forceinline__ void kv4_store4(__nv_bfloat16* p, float x, float y, float z, float w) {
  __nv_bfloat162 v[2] = {__floats2bfloat162_rn(x, y), __floats2bfloat162_rn(z, w)};
  *reinterpret_cast<uint2*>(p) = *reinterpret_cast<uint2*>(v);
}

// The value a code stands for: (c - 7.5) * d is exact in fp32.
__device__ __forceinline__ float kv4_value(uint32_t c, float d, float z) {
  return fmaf((float)c - 7.5f, d, z);
}

}  // namespace mmvq
