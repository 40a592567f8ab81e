// Arguments of the attention over the 4-bit cache, and how its work is divided.
//
// The rows of a sequence's query tokens that share a kv head (tokens x heads
// of the group, token-major) are taken in blocks of 8 * NT; such a block and
// its kv head are an item.  Its work is its 16-token tiles that any of its
// rows may see, and kKv4ItemUnits tiles' time for beginning and ending it.
// The units of the batch's items, in order of (sequence, kv head, row block,
// tile), are divided evenly over the grid's CTAs: whatever the lengths, every
// CTA gets the same work, and the host needs to know no length.  A CTA's
// share covers whole items and up to two parts of items; parts are joined by
// the CTA that finishes last.
#pragma once
#include "kv4.cuh"

namespace mmvq {

struct Kv4Attention {
  const void* q;    // [n_tokens][n_heads][D]: strides ldq (token), hq (head), in elements
  int64_t ldq, hq;
  int n_heads;
  float scale;
  int window;       // 0: none
  int sinks;
  void* y;          // [n_tokens][n_heads][D]
  float* lse;       // [n_tokens][n_heads], may be NULL
  void* workspace;
  bool q_vector;    // the rows of q lie on 16-byte boundaries
  uint64_t page_mul;  // tile / (tiles per page) = tile * page_mul >> page_shift
  int page_shift;
};

constexpr int kKv4MaxSms = 160, kKv4MaxCtasSm = 4;  // of a launch
constexpr int kKv4MaxCtas = kKv4MaxSms * kKv4MaxCtasSm;
constexpr int kKv4ItemUnits = 32;     // what an item costs besides its tiles
constexpr int kKv4MinUnits = 16;      // of a CTA: below, fewer CTAs take part

// Workspace: join counters (two per CTA for the groups of a split item, one for
// the groups' results), then two partial results per CTA.  An SM's CTAs have at
// most 4096 / D rows between them.
constexpr int kKv4CounterBytes = kKv4MaxCtas * 3 * 4;
__host__ __device__ constexpr int kv4_rows_sm(int D) { return 4096 / D; }
__host__ __device__ constexpr int64_t kv4_slot_floats(int rows, int D) { return (int64_t)rows * (D + 2); }

// What a sequence asks for.
struct Kv4Seq {
  int first;   // its first row
  int n_new;   // rows (0: nothing to do)
  int len;     // cached tokens (some may lie past the page table)
  int sink_tiles, skip, tiles;  // tile i of `tiles` is i + (i >= sink_tiles ? skip : 0)
  int blocks;  // row blocks
  __device__ __forceinline__ int item_units() const { return tiles + kKv4ItemUnits; }
};

// A sequence without visible tokens still counts a tile, so that its zeros get written.
// Errors only ever set *error.
__device__ __forceinline__ Kv4Seq kv4_seq(const Kv4Batch& a, const Kv4Attention& p, int rows_block,
                                          int b, int* error) {
  Kv4Seq s;
  s.first = a.offsets[b];
  const int end = a.offsets[b + 1];
  s.n_new = end - s.first;
  s.len = max(0, a.lens[b]);
  if (s.n_new < 0 || s.n_new > kKv4MaxNew || s.first < 0 || end > a.n_tokens) {
    *error = s.n_new > kKv4MaxNew && s.first >= 0 && end <= a.n_tokens ? MMVQ_ERR_NCOLS
                                                                        : MMVQ_ERR_ROUTING;
    s.n_new = 0;
  }
  // tiles past the page table are no work: a length that is wrong by much would otherwise be hours of it
  const int64_t in_table = a.ld_table * (a.page_tokens / kKv4Tile);
  int end_tile = (int)(((int64_t)s.len + kKv4Tile - 1) / kKv4Tile);
  if (end_tile > in_table) {
    end_tile = (int)in_table;
    if (s.n_new > 0) *error = MMVQ_ERR_ROUTING;
  }
  s.sink_tiles = s.skip = 0;
  if (p.window > 0) {
    const int64_t from = max((int64_t)0, (int64_t)s.len - s.n_new - p.window + 1);
    s.sink_tiles = (int)(((int64_t)min(p.sinks, s.len) + kKv4Tile - 1) / kKv4Tile);
    s.skip = max(0, min((int)(from / kKv4Tile), end_tile) - s.sink_tiles);
  }
  s.tiles = max(1, end_tile - s.skip);
  const int group = p.n_heads / a.n_kv_heads;
  s.blocks = (s.n_new * group + rows_block - 1) / rows_block;
  return s;
}

}  // namespace mmvq
