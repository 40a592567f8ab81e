// Attention of 1-8 query tokens a sequence over the 4-bit cache.
//
// Mathematics.  A warp takes tiles of 16 cached tokens.  Scores come as
// S^T[tokens x rows] = K Q^T from m16n8k16 f16 products whose A operand is the
// tile's codes: masked out of its word a code c stands, as the bits of an
// fp16, for c * 2^-24 (low nibble of a byte) or c * 2^-20 (high nibble), so a
// key costs no conversion; for fp32 queries it becomes c - 8, in values c - 8 or
// c - 7 (centred() below).
// The rows of Q are scaled by a power of two each, and by 16 more where they
// meet low nibbles.  Per block of 32 the sum is multiplied by the block's d in
// fp32; sum(z sum(q)) and sum(d sum(q)) (the codes' offset) over the blocks
// are one more product, sum(q) in two fp16 parts.  Probabilities
// p = 2^(s - m + 12) use a reference m that is only moved when a score exceeds
// it by 2 (in log2 units): the result does not depend on m, and most tiles skip
// the maximum across lanes and the rescaling.  O^T[values x rows] += V^T P':
// A = c - 8 (even tokens) or c - 7 (odd), B = p d per block of 32; sum(p z) and
// sum(+-p d) one more product.
//
// Precision.  fp32 q enters as two fp16 parts (22 bits), and for fp32 and fp16
// the products p d do too.  bf16 keeps 11 bits of p and of p d, finer than its
// own 8: outputs next to the middle of two bf16 numbers then round to the other
// one (2e-4 off an fp32 form in 2-norm, while both are 1.7e-3 off 64 bits); two
// parts cost 15 to 18% (64 sequences 83 -> 98 us).  For fp16 and bf16 the keys'
// codes are subnormal, and a sum of 16 products keeps about 17 bits of the
// largest: the log-sum-exp is 1e-7 to 6e-7 off, with c - 8 there too 3e-8 to
// 1.5e-7 at 3 to 7% of the time.
// Sums over tokens: a tile's products start from zero and are added in fp32, rounded to nearest.  The tensor core
// cuts its sum off towards zero at every product, which is of no account within a tile, but where it keeps the sum
// of all tiles is 1.3e-7 a tile that the sum falls short (fp32, 131072 tokens a sequence, one-signed midpoints:
// 1.4e-5 off after 108 tiles of a warp, 1.5e-4 after 1700; with the additions 1.2e-7 and 2.3e-7).  They cost 2 to 5% of
// the time (131071 fp32 tokens 53 -> 55 us).
//
// Why warp-level products.  Each 32-block of a key has its own factor on the
// sum, and each block of a value its own on the probability, so a product
// reaches over 32 values only, and the accumulators are needed in registers
// between them.  (Decoded to fp16 for tcgen05 instead, keys keep 11 bits: with
// 96 rows of bf16 an attempt took 124 us against 144, with the log-sum-exp 2e-4
// off, inside 2^-18 of the products' magnitudes.  Keys in two parts fit shared
// memory next to 128 rows of Q in steps of 32 tokens; that has not been built.)
//
// What bounds it, measured on GB300 (6768 GB/s copied):
//  - one row tile, D = 128 (64 bf16 sequences of 128 .. 8192 tokens, 32 / 8
//    heads, 337 MB): 77 us, 4.4 TB/s.  The instructions: 59% of the issue slots,
//    44% of the ALU pipe (masking codes out of words), tensor pipe 22%.
//    Three CTAs of 4 warps an SM at 168 registers: 77 us; four at 128: 81; one of
//    12 at 168, which begins and ends its items alone: 114.
//  - two row tiles, D = 256: the latency of 8 warps an SM at 255 registers (128 of
//    them accumulators).  131071 fp32 tokens, 24 / 2 heads, 84 MB: 55 us, of which
//    about 31 tiles and 10 joining 76 parts a head; tensor pipe 32%, issue 35%.
//    8 x 8 query tokens over 16389, bf16: 147 us, tensor pipe 33%, issue 47%.
//    Without the additions (52 and 144 us), splitting the values between two warps
//    (175 for the latter), 32 rows a warp (159) and two CTAs of 4 warps (142; but 59
//    instead of 52 for the former) were no better.
//  - short batches, 14 us for 77 tokens: work division, first tile and queries, the
//    tile (its code is fetched for the first time) and results follow one another.
#include "kv4.cuh"
#include "kv4_work.cuh"

namespace mmvq {
namespace {

constexpr int kStages = 4;

__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                      uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same from zero.
__device__ __forceinline__ void mma16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ void mma8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(b0));
}

// c += a, rounded to nearest, two numbers an instruction.
__device__ __forceinline__ void add4(float (&c)[4], const float (&a)[4]) {
#pragma unroll
  for (int e = 0; e < 4; e += 2) {
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\tadd.rn.f32x2 x, x, y;\n\t"
        "mov.b64 {%0, %1}, x;\n\t}"
        : "+f"(c[e]), "+f"(c[e + 1])
        : "f"(a[e]), "f"(a[e + 1]));
  }
}

// Transposes an 8 x 8 matrix of fp16 held two of a row a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The codes of two words, low nibbles in a0 and a1, high ones in a2 and a3: as they are, or less a centre of 8 (in the
// halves' second one kOdd, 8 or 7) as c - 8 and 16 (c - 8), exactly: set below 1024 as the mantissa's last bits, from
// which 1024 and the centre are taken off.  The tensor core aligns a subnormal by its nominal exponent and cuts off
// what lies far below it (sums then keep about 17 bits); these are normal numbers.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {  // one instruction
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
template <int kOdd>
__device__ __forceinline__ void centred(uint32_t w0, uint32_t w1, uint32_t& a0, uint32_t& a1, uint32_t& a2,
                                        uint32_t& a3) {
  constexpr uint32_t low = 0xe400e408u + (kOdd << 16), high = 0xe400e480u + (kOdd << 20);  // - 1032, - 1152
  a0 = add2(and_or(w0, 0x000f000fu, 0x64006400u), low);
  a1 = add2(and_or(w1, 0x000f000fu, 0x64006400u), low);
  a2 = add2(and_or(w0, 0x00f000f0u, 0x64006400u), high);
  a3 = add2(and_or(w1, 0x00f000f0u, 0x64006400u), high);
}
__device__ __forceinline__ void plain(uint32_t w0, uint32_t w1, uint32_t& a0, uint32_t& a1, uint32_t& a2,
                                      uint32_t& a3) {
  a0 = w0 & 0x000f000fu, a1 = w1 & 0x000f000fu;
  a2 = w0 & 0x00f000f0u, a3 = w1 & 0x00f000f0u;
}

// a b - c, rounded once: what a product c = a b lost in rounding, exactly.
__device__ __forceinline__ uint32_t residue2(uint32_t a, uint32_t b, uint32_t c) {
  return u32(__hfma2(h2(a), h2(b), __hneg2(h2(c))));
}

// A kernel's instance: heads of D values, NT tiles of 8 rows, QS: fp32 queries in two parts.
template <int D_, int NT_, bool QS_>
struct Shape {
  static constexpr int D = D_, NT = NT_;
  static constexpr bool QS = QS_;
  static constexpr int nb = D / 32, kGroups = nb > 4 ? nb / 4 : 1, kOfGroup = nb / kGroups;  // blocks
  static constexpr int kRows = 8 * NT;
  // The accumulators, 4 registers per 16 values and row tile, and the ring, 80 D bytes a warp, decide.  32 accumulators
  // at most: four CTAs of 4 warps and 128 registers a thread; of these D = 128, whose loads and masks spill at that
  // (64 bf16 sequences 81 us), three and 168 (77).  64 of D = 128: one CTA of 12 warps and 168.  D = 256: 8 warps and
  // 255, with 128 accumulators for want of registers, with 64 because the rings of 12 do not fit.
  static constexpr int kWarps = D * NT <= 128 ? 4 : D == 128 ? 12 : 8;
  static constexpr int kCtas = D * NT <= 128 ? (D == 128 ? 3 : 4) : 1;
  static constexpr int kThreads = 32 * kWarps;
  static_assert(kCtas <= kKv4MaxCtasSm && kCtas * kRows <= kv4_rows_sm(D), "the workspace");
  static constexpr int kBytes = kv4_tile_bytes(D);
};

template <typename S>
struct Smem {
  static constexpr int kRing = kStages * S::kBytes;  // of a warp
  uint8_t ring[S::kWarps][kRing];   // tiles; afterwards the warps' results [row][D]
  // [block][part][row tile][lane]: the B operands of a block's two products
  uint8_t q[S::nb * (S::QS ? 2 : 1) * S::NT * 32 * 16];
  __half q_sum[S::kRows][S::kGroups][4][S::kOfGroup];  // sum(q) of a block, and its multiple for d, in two parts each
  float row_factor[S::kRows];
  int row_pos[S::kRows];
  Kv4JoinSmem<S::kRows> join;       // of the warps' results, then of an item's parts
  Kv4Plan<S::kThreads> plan;
  static_assert(kRing >= S::kRows * S::D * 4, "a warp's results fit its ring");
};

// The query rows of a block into q, q_sum, row_factor and row_pos, by 8 warps at most.
template <typename S, typename T>
__device__ __forceinline__ void load_queries(const Kv4Batch& a, const Kv4Attention& p, Smem<S>& sm,
                                             const Kv4Seq& s, int head, int row0, int tid) {
  constexpr int D = S::D, NT = S::NT;
  constexpr bool QS = S::QS;
  constexpr int kUsed = S::kThreads < 256 ? S::kThreads : 256;
  constexpr int kPer = kUsed / S::kRows, kOwn = D / kPer;  // threads a row, values a thread
  if (tid >= kUsed) return;
  const int row = tid / kPer, sub = tid % kPer;
  const int group = p.n_heads / a.n_kv_heads;
  const int r = row0 + row;
  const bool on = r < s.n_new * group;
  const int t = on ? r / group : 0;
  float q[kOwn], top = 0.0f;
  if (on) {
    kv4_load_values(static_cast<const T*>(p.q) + (int64_t)(s.first + t) * p.ldq +
                    (int64_t)(head * group + r - t * group) * p.hq + sub * kOwn,
                p.q_vector, q);
  } else {
#pragma unroll
    for (int i = 0; i < kOwn; ++i) q[i] = 0.0f;
  }
#pragma unroll
  for (int i = 0; i < kOwn; ++i) top = fmaxf(top, fabsf(q[i]));
#pragma unroll
  for (int o = 1; o < kPer; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  // largest |q| into [2^6, 2^7), or [2^4, 2^5) in two parts: 16 q and 7.5 times, or 16 times, a sum of 32 stay
  // below fp16's largest
  const int e = top > 0.0f && top < INFINITY ? min((QS ? 4 : 6) - exponent(top), 126) : 0;
  const float f = p.scale < 0.0f ? -pow2(e) : pow2(e);  // the factor of the scores is not negative
#pragma unroll
  for (int i = 0; i < kOwn; ++i) q[i] *= f;
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const int d = sub * kOwn + i, b = d / 32, u = d % 32 / 8, n = d % 8;
    const float x = (n & 1) ? q[i] : 16.0f * q[i];
    const __half hi = __float2half_rn(x);
    uint8_t* at = sm.q + (size_t)((b * (QS ? 2 : 1) * NT + row / 8) * 32 + (row % 8) * 4 + u) * 16 +
                  ((n & 3) / 2) * 8 + (n & 1) * 4 + (n >> 2) * 2;
    *reinterpret_cast<__half*>(at) = hi;
    if (QS) *reinterpret_cast<__half*>(at + NT * 32 * 16) = __float2half_rn(x - __half2float(hi));
  }
  constexpr int kBlk = 32 / kOwn;  // threads a block
  static_assert(kOwn <= 32, "a block is of one thread or more");
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kOwn; ++i) sum += q[i];
#pragma unroll
  for (int o = 1; o < kBlk; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (sub % kBlk == 0) {
    const int b = sub / kBlk;
    constexpr float kOff = QS ? 0.5f : -7.5f;  // the codes enter less 8, or as they are
    if (QS) sum *= 16.0f;  // as the products do
    const __half hi = __float2half_rn(sum), mid = __float2half_rn(kOff * sum);
    auto& out = sm.q_sum[row][b / S::kOfGroup];
    out[0][b % S::kOfGroup] = hi;
    out[1][b % S::kOfGroup] = __float2half_rn(sum - __half2float(hi));
    out[2][b % S::kOfGroup] = mid;
    out[3][b % S::kOfGroup] = __float2half_rn(fmaf(kOff, sum, -__half2float(mid)));
  }
  if (sub == 0) {
    // a power of two in two steps: it can pass fp32's range where the product does not
    constexpr int kUnit = QS ? -4 : 20;
    const int f2 = kUnit - e;
    const float factor = fabsf(p.scale) * 1.4426950408889634f * pow2(f2 / 2) * pow2(f2 - f2 / 2);
    sm.row_factor[row] = fminf(fmaxf(factor, 1e-37f), 1e37f);  // not 0: masked scores are -inf
    sm.row_pos[row] = on ? max(-1, s.len - s.n_new + t) : -1;  // less a window of up to 2^31 - 1: in range
  }
}

// Of N 32-bit words in shared memory, by the widest loads that their alignment allows.
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int k = 0; k < N / 4; ++k) {
      const uint4 v = *reinterpret_cast<const uint4*>(p + 16 * k);
      w[4 * k] = v.x, w[4 * k + 1] = v.y, w[4 * k + 2] = v.z, w[4 * k + 3] = v.w;
    }
  } else if constexpr (N % 2 == 0) {
#pragma unroll
    for (int k = 0; k < N / 2; ++k) {
      const uint2 v = *reinterpret_cast<const uint2*>(p + 8 * k);
      w[2 * k] = v.x, w[2 * k + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) w[k] = *reinterpret_cast<const uint32_t*>(p + 4 * k);
  }
}

__device__ __forceinline__ float half_of(uint32_t pair, int i) {
  return __half2float(i ? __high2half(h2(pair)) : __low2half(h2(pair)));
}

template <typename S, bool PS, typename T>
__global__ void __launch_bounds__(S::kThreads, S::kCtas)
    kv4_attention_kernel(const Kv4Batch a, const Kv4Attention p) {
  constexpr int D = S::D, NT = S::NT, nb = S::nb, kRows = S::kRows, kBytes = S::kBytes;
  constexpr int kThreads = S::kThreads, kWarps = S::kWarps, kGroups = S::kGroups;
  constexpr bool QS = S::QS;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Smem<S>& sm = *reinterpret_cast<Smem<S>*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  grid_dependency_wait();
  // The next kernel may be launched now: whatever it is, it waits for this one's results
  grid_launch_dependents();

  const int64_t total = kv4_plan(a, p, kRows, sm.plan, tid);
  const int n_ctas = kv4_ctas(total), cta = blockIdx.x;
  if (cta >= n_ctas) return;
  const Shares shares(total, n_ctas);
  const int per_page = a.page_tokens / kKv4Tile;
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(sm.ring[warp]) + lane * 16;

  for (int64_t unit = shares.begin(cta); unit < shares.begin(cta + 1);) {
    Kv4Item it;
    if (!kv4_next(a, p, kRows, sm.plan, shares, cta, unit, it)) continue;
    const Kv4Seq& s = it.s;
    const int tile0 = it.tile0, tile1 = it.tile1, n_rows = it.n_rows;

    __syncthreads();  // the item before is done with the shared memory

    // ---- the warp's share of the tiles, one after the other through its ring; the page after a tile's is looked
    // up with it, and the last bits of `present` say which of the fetched tiles are there
    const int begin = tile0 + (tile1 - tile0) * warp / kWarps, end = tile0 + (tile1 - tile0) * (warp + 1) / kWarps;
    const uint8_t* head_base = a.cache + (int64_t)it.head * per_page * kv4_tile_bytes(D) + lane * 16;
    const int64_t page_bytes = (int64_t)a.n_kv_heads * per_page * kv4_tile_bytes(D);
    const int32_t* table = a.page_table + (int64_t)it.b * a.ld_table;
    const int pos_lo = max(0, s.len - s.n_new);  // of the sequence's rows that see anything
    auto tile_of = [&](int i) { return i + (i >= s.sink_tiles ? s.skip : 0); };
    const int gap = s.skip > 0 ? s.sink_tiles : -1;  // the tile before which some are skipped
    uint32_t present = 0;
    int next = begin, pi = 0, in_page = 0, page_after = -1;
    bool there = false;
    const uint8_t* src = head_base;
    auto page_at = [&](int i) { return i < a.ld_table && s.len > 0 ? table[i] : -1; };
    auto enter = [&](int page) {  // page pi of the table
      there = page >= 0 && page < a.n_pages;
      src = head_base + page * page_bytes + in_page * kv4_tile_bytes(D);
      page_after = page_at(pi + 1);
    };
    auto find = [&]() {  // where tile `next` lies
      const int tile = tile_of(next);
      pi = (int)(((uint64_t)(uint32_t)tile * p.page_mul) >> p.page_shift);
      in_page = tile - pi * per_page;
      enter(page_at(pi));
    };
    auto fetch = [&](int stage) {
      const bool on = next < end && there;
      present = present << 1 | (on ? 1u : 0u);
      if (on) {
        const uint32_t dst = ring + stage * kBytes;
#pragma unroll
        for (int k = 0; k < (kBytes + 511) / 512; ++k)
          if ((k + 1) * 512 <= kBytes || k * 512 + lane * 16 < kBytes) cp_async16(dst + k * 512, src + k * 512);
      }
      cp_async_commit();
      if (++next == gap) {
        find();
      } else if (++in_page == per_page) {
        in_page = 0;
        ++pi;
        enter(page_after);
      } else {
        src += kv4_tile_bytes(D);
      }
    };
    if (begin < end) find();
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) fetch(k);

    load_queries<S, T>(a, p, sm, s, it.head, it.row0, tid);
    __syncthreads();

    // ---- what a lane keeps of the queries: columns 2c, 2c + 1 of each row tile
    float fac[NT][2];
    uint32_t qz[NT][kGroups][2];  // B operands of the products with midpoints and steps
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        fac[n][e] = sm.row_factor[8 * n + 2 * c + e];
      }
      // k positions: of 4 blocks, both parts of sum(q), then both of -7.5 sum(q); of 2, all four at once
#pragma unroll
      for (int k = 0; k < kGroups; ++k) {
        const uint32_t* qs = reinterpret_cast<const uint32_t*>(sm.q_sum[8 * n + g][k]);
        qz[n][k][0] = qs[c];
        qz[n][k][1] = nb == 2 ? 0u : qs[4 + c];
      }
    }
    float o[NT][2 * nb][4], oz[NT][4], bar[NT][2], ref[NT][2], l[NT][2];  // bar: a score above it moves ref
    int E = 0;  // p is smaller by 2^E where steps reach 2^(E + 1): p d stays in fp16's range
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < 2 * nb; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][i][e] = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) oz[n][e] = 0.0f;
      bar[n][0] = bar[n][1] = -INFINITY;
      ref[n][0] = ref[n][1] = 0.0f;
      l[n][0] = l[n][1] = 0.0f;
    }

    int stage = 0;
    for (int i = begin; i < end; ++i) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      const bool on = present >> (kStages - 2) & 1;
      fetch((stage + kStages - 1) % kStages);
      const uint8_t* tp = sm.ring[warp] + stage * kBytes;
      stage = (stage + 1) % kStages;
      const int key0 = tile_of(i) * kKv4Tile;
      if (!on) {
        if (lane == 0 && key0 < s.len) kv4_set_status(a.status, MMVQ_ERR_ROUTING);
        continue;
      }

      // ---- scores
      uint32_t kw[2 * nb], kd[2][nb / 2];
#pragma unroll
      for (int k = 0; k < nb / 2; ++k) {
        const uint4 v = *reinterpret_cast<const uint4*>(tp + 512 * k + 16 * lane);
        kw[4 * k] = v.x, kw[4 * k + 1] = v.y, kw[4 * k + 2] = v.z, kw[4 * k + 3] = v.w;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) load_words(tp + kv4_key_scale(D, g + 8 * h, 0), kd[h]);
      float x[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) x[n][0] = x[n][1] = x[n][2] = x[n][3] = 0.0f;
#pragma unroll
      for (int k = 0; k < kGroups; ++k) {  // midpoints and steps of this lane's k positions
        uint32_t az[2], ad[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint8_t* at = tp + kv4_key_scale(D, g + 8 * h, 4 * k);
          az[h] = *reinterpret_cast<const uint32_t*>(at + (nb == 2 ? (c < 2 ? D : 0) : D + 4 * (c & 1)));
          ad[h] = nb == 2 ? 0u : *reinterpret_cast<const uint32_t*>(at + 4 * (c & 1));
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if constexpr (nb == 2) mma8(x[n], az[0], az[1], qz[n][k][0]);
          else if (k == 0) mma16_first(x[n], az[0], az[1], ad[0], ad[1], qz[n][k][0], qz[n][k][1]);
          else mma16(x[n], az[0], az[1], ad[0], ad[1], qz[n][k][0], qz[n][k][1]);
        }
      }
      if constexpr (!QS) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[n][e] *= 0x1p-20f;
      }
#pragma unroll
      for (int b2 = 0; b2 < nb; ++b2) {
        float acc[NT][4];
        uint32_t ka[2][4];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const uint32_t w0 = kw[b2] >> (8 * hh), w1 = kw[nb + b2] >> (8 * hh);
          if constexpr (QS) centred<8>(w0, w1, ka[hh][0], ka[hh][1], ka[hh][2], ka[hh][3]);
          else plain(w0, w1, ka[hh][0], ka[hh][1], ka[hh][2], ka[hh][3]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint8_t* qp = sm.q + (size_t)((b2 * (QS ? 2 : 1) * NT + n) * 32 + lane) * 16;
          if constexpr (QS) {
            const uint4 q = *reinterpret_cast<const uint4*>(qp + NT * 32 * 16);
            mma16_first(acc[n], ka[0][0], ka[0][1], ka[0][2], ka[0][3], q.x, q.y);
            mma16(acc[n], ka[1][0], ka[1][1], ka[1][2], ka[1][3], q.z, q.w);
          }
          const uint4 q = *reinterpret_cast<const uint4*>(qp);
          if constexpr (QS) mma16(acc[n], ka[0][0], ka[0][1], ka[0][2], ka[0][3], q.x, q.y);
          else mma16_first(acc[n], ka[0][0], ka[0][1], ka[0][2], ka[0][3], q.x, q.y);
          mma16(acc[n], ka[1][0], ka[1][1], ka[1][2], ka[1][3], q.z, q.w);
        }
        const float d0 = half_of(kd[0][b2 / 2], b2 & 1), d1 = half_of(kd[1][b2 / 2], b2 & 1);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          x[n][0] = fmaf(d0, acc[n][0], x[n][0]);
          x[n][1] = fmaf(d0, acc[n][1], x[n][1]);
          x[n][2] = fmaf(d1, acc[n][2], x[n][2]);
          x[n][3] = fmaf(d1, acc[n][3], x[n][3]);
        }
      }

      // ---- values: steps of the lane's token pairs (2c, 2c + 1) + 8 h, midpoints of block g
      constexpr uint32_t kOddSign = 0x80000000u;  // of the high half, the odd token
      uint32_t ds[2 * nb], vz[2], vs[2] = {0u, 0u};  // and the steps of block g, less for the odd tokens
      load_words(tp + 18 * D + 8 * nb * c, ds);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint8_t* at = tp + 18 * D + 8 * nb * c + 4 * (h * nb + g);
        vs[h] = g < nb ? *reinterpret_cast<const uint32_t*>(at) ^ kOddSign : 0u;
        vz[h] = g < nb ? *reinterpret_cast<const uint32_t*>(at + D) : 0u;
      }

      // ---- masks: a tile that every row sees in full needs none
      const bool all = key0 + kKv4Tile - 1 <= pos_lo &&
                       (p.window == 0 || key0 > s.len - 1 - p.window || key0 + kKv4Tile <= p.sinks);
      if (!all) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = key0 + g + 8 * (e >> 1), q = sm.row_pos[8 * n + 2 * c + (e & 1)];
            const bool see = key <= q && (p.window == 0 || key > q - p.window || key < p.sinks);
            if (!see) x[n][e] = -INFINITY;
          }
        // values that no row sees may be anything: their steps and midpoints become zero
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t keep = 0;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int key = key0 + 8 * h + 2 * c + e;
            if (key < s.len && (p.window == 0 || key > pos_lo - p.window || key < p.sinks))
              keep |= 0xffffu << (16 * e);
          }
#pragma unroll
          for (int k = 0; k < nb; ++k) ds[h * nb + k] &= keep;
          vz[h] &= keep;
          vs[h] &= keep;
        }
      }
      bool move = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) move |= fmaxf(x[n][e], x[n][e + 2]) > bar[n][e];
      // or a step of 2 or more, also one that E covers: then every tile comes here (64 bf16 sequences 77 us, 81 with
      // steps up to 2.8, 88 with steps up to 11)
      if (__any_sync(0xffffffffu, move || ((vs[0] | vs[1]) & 0x40004000u))) {
        uint32_t top = max(max(vs[0] & 0x7fffu, vs[0] >> 16 & 0x7fffu), max(vs[1] & 0x7fffu, vs[1] >> 16 & 0x7fffu));
        top = __reduce_max_sync(0xffffffffu, top);
        const int E2 = max(E, (int)(top >> 10) - 15);  // its exponent
        const int E1 = E;
        E = E2;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float fr[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float t = fmaxf(x[n][e], x[n][e + 2]);
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
            // ref = (largest score) * fac - kKv4Boost + E, from none (bar -inf, ref 0) or the last one on
            const bool none = bar[n][e] == -INFINITY, some = t > -INFINITY;
            float r = t * fac[n][e] - kKv4Boost;
            if (!none) r = fmaxf(r, ref[n][e] - E1);
            if (none && !some) r = -E;
            r += E;
            fr[e] = none ? 0.0f : ex2(ref[n][e] - r);
            ref[n][e] = r;
            bar[n][e] = fmaxf(bar[n][e], t + kKv4Lazy / fac[n][e]);
            l[n][e] *= fr[e];
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            oz[n][e] *= fr[e & 1];
#pragma unroll
            for (int k = 0; k < 2 * nb; ++k) o[n][k][e] *= fr[e & 1];
          }
        }
      }

      // ---- probabilities, turned into the B operand; their products with the midpoints (rows 0 to 7) and the
      // steps (rows 8 to 15)
      uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float pr[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) pr[e] = ex2(fmaf(x[n][e], fac[n][e & 1], -ref[n][e & 1]));
        l[n][0] += pr[0] + pr[2];
        l[n][1] += pr[1] + pr[3];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const __half2 hi2 = __floats2half2_rn(pr[2 * h], pr[2 * h + 1]);
          ph[n][h] = transpose8(u32(hi2));
          if constexpr (PS) {
            const float2 back = __half22float2(hi2);
            pl[n][h] = transpose8(u32(__floats2half2_rn(pr[2 * h] - back.x, pr[2 * h + 1] - back.y)));
          }
        }
        float acc[4];
        mma16_first(acc, vz[0], vs[0], vz[1], vs[1], ph[n][0], ph[n][1]);
        if constexpr (PS) mma16(acc, vz[0], vs[0], vz[1], vs[1], pl[n][0], pl[n][1]);
        add4(oz[n], acc);
      }
      // ---- weighted values
      uint32_t vw[2 * nb];
#pragma unroll
      for (int k = 0; k < nb / 2; ++k) {
        const uint4 v = *reinterpret_cast<const uint4*>(tp + 8 * D + 512 * k + 16 * lane);
        vw[4 * k] = v.x, vw[4 * k + 1] = v.y, vw[4 * k + 2] = v.z, vw[4 * k + 3] = v.w;
      }
#pragma unroll
      for (int b2 = 0; b2 < nb; ++b2) {
        uint32_t bh[NT][2], bl[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t d = ds[h * nb + b2];
            bh[n][h] = mul2(ph[n][h], d);
            if constexpr (PS) bl[n][h] = fma2(pl[n][h], d, residue2(ph[n][h], d, bh[n][h]));
          }
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const uint32_t w0 = vw[b2] >> (8 * hh), w1 = vw[nb + b2] >> (8 * hh);
          uint32_t a0, a1, a2, a3;
          // c - 8 for even tokens and c - 7 for odd ones here, and at the end half of sum(p d) over the even less that
          // over the odd: neither sum drifts off with the tokens.  (c - 8 for all leaves a sum of half a step a token,
          // whose rounding is what remains where values cancel: fp32, 131072 tokens and even probabilities, 8.7e-6 off
          // after 1700 tiles of a warp, 6.2e-7 so.)  Codes as they are, with -7.5 sum(p d), cost 3% less for
          // fp16, but put the output 2.5 of its own roundings off there.  2 c - 15, which needs no sum(p d), takes a
          // shift more a word: 64 bf16 sequences 82 us.
          centred<7>(w0, w1, a0, a2, a1, a3);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float acc[4];
            mma16_first(acc, a0, a1, a2, a3, bh[n][0], bh[n][1]);
            if constexpr (PS) mma16(acc, a0, a1, a2, a3, bl[n][0], bl[n][1]);
            add4(o[n][2 * b2 + hh], acc);
          }
        }
      }
    }
    cp_async_wait<0>();
    __syncwarp();

    // ---- the warp's result, in its ring: [row][D], in units of 2^(ref)
    float* res = reinterpret_cast<float*>(sm.ring[warp]);
    // low nibbles entered as c - 8 or c - 7, high ones as 16 times that
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float t = l[n][e];
        t += __shfl_xor_sync(0xffffffffu, t, 4);
        t += __shfl_xor_sync(0xffffffffu, t, 8);
        t += __shfl_xor_sync(0xffffffffu, t, 16);
        const int row = 8 * n + 2 * c + e;
        if (g == 0) {
          sm.join.ref[warp][row] = bar[n][e] == -INFINITY ? -INFINITY : ref[n][e];
          sm.join.sum[warp][row] = t;
        }
        const float z0 = fmaf(0.5f, oz[n][e + 2], oz[n][e]);
#pragma unroll
        for (int b2 = 0; b2 < nb; ++b2) {
          const float z = __shfl_sync(0xffffffffu, z0, 4 * b2 + c);
          float4 v;
          v.x = o[n][2 * b2][e] + z;
          v.y = fmaf(o[n][2 * b2][e + 2], 0x1p-4f, z);
          v.z = o[n][2 * b2 + 1][e] + z;
          v.w = fmaf(o[n][2 * b2 + 1][e + 2], 0x1p-4f, z);
          *reinterpret_cast<float4*>(res + row * D + 32 * b2 + 4 * g) = v;
        }
      }
    }
    __syncthreads();

    // ---- the CTA's result: to the outputs, or to a slot of the workspace
    if (tid < n_rows) sm.join.weigh(tid, kWarps);
    __syncthreads();
    float* slot = it.last > it.first ? kv4_slot<kRows, D>(p, shares, it, cta) : nullptr;
    for (int idx = tid; idx < n_rows * (D / 4); idx += kThreads) {
      const int row = idx / (D / 4), d4 = idx - row * (D / 4);
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = sm.join.factor[w][row];
        const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(sm.ring[w]) + row * D + 4 * d4);
        v.x = fmaf(f, x.x, v.x);
        v.y = fmaf(f, x.y, v.y);
        v.z = fmaf(f, x.z, v.z);
        v.w = fmaf(f, x.w, v.w);
      }
      if (!slot) {
        kv4_store_row<T>(a, p, it, D, row, d4, v, sm.join.row_ref[row], sm.join.row_sum[row]);
      } else {
        *reinterpret_cast<float4*>(slot + row * D + 4 * d4) = v;
        if (d4 == 0)
          *reinterpret_cast<float2*>(slot + kRows * D + 2 * row) =
              make_float2(sm.join.row_ref[row], sm.join.row_sum[row]);
      }
    }
    if (slot) kv4_join<kThreads, kRows, D, T>(a, p, shares, it, cta, sm.join, tid);
  }
}

template <int D, int NT, bool QS, bool PS, typename T>
int launch(const Kv4Batch& a, const Kv4Attention& p, cudaStream_t stream) {
  using S = Shape<D, NT, QS>;
  auto kern = kv4_attention_kernel<S, PS, T>;
  constexpr int kSmem = (int)sizeof(Smem<S>);
  static int per_device[64];  // CTAs of a full launch, by device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return MMVQ_ERR_CUDA;
  int ctas = __atomic_load_n(&per_device[dev], __ATOMIC_ACQUIRE);
  if (ctas == 0) {
    int sms = 0, per_sm = 0;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, S::kThreads, kSmem) != cudaSuccess ||
        per_sm < 1)
      return MMVQ_ERR_CUDA;
    ctas = min(sms, kKv4MaxSms) * min(per_sm, S::kCtas);
    __atomic_store_n(&per_device[dev], ctas, __ATOMIC_RELEASE);
  }
  // no more CTAs than the longest sequences that the table can hold would use
  const int rows = p.n_heads / a.n_kv_heads * kKv4MaxNew;
  const int64_t units = (int64_t)a.n_seqs * a.n_kv_heads * ((rows + 8 * NT - 1) / (8 * NT)) *
                        (a.ld_table * (a.page_tokens / kKv4Tile) + kKv4ItemUnits);
  const int64_t most = (units + kKv4MinUnits - 1) / kKv4MinUnits;
  const int grid = (int)(most < ctas ? most : ctas);
  return launch_pdl(kern, dim3(grid), dim3(S::kThreads), kSmem, stream, a, p);
}

template <int D, bool QS, bool PS, typename T>
int launch_rows(const Kv4Batch& a, const Kv4Attention& p, cudaStream_t stream) {
  // rows that share a kv head, if the sequences have equally many new tokens
  const int rows = p.n_heads / a.n_kv_heads * ((a.n_tokens + a.n_seqs - 1) / a.n_seqs);
  if (rows <= 8) return launch<D, 1, QS, PS, T>(a, p, stream);
  return launch<D, 2, QS, PS, T>(a, p, stream);
}

template <bool QS, bool PS, typename T>
int launch_typed(const Kv4Batch& a, const Kv4Attention& p, int D, cudaStream_t stream) {
  if (D == 64) return launch_rows<64, QS, PS, T>(a, p, stream);
  if (D == 128) return launch_rows<128, QS, PS, T>(a, p, stream);
  return launch_rows<256, QS, PS, T>(a, p, stream);
}

}  // namespace

int launch_kv4_attention(const Kv4Batch& a, const Kv4Attention& args, int D, int dtype,
                         cudaStream_t stream) {
  Kv4Attention p = args;
  // tiles are below 2^27: with the shift, the rounded-up reciprocal gives the exact quotient
  const uint64_t per_page = (uint64_t)(a.page_tokens / kKv4Tile);
  p.page_shift = per_page < 16 ? 36 : 40;
  p.page_mul = ((1ull << p.page_shift) + per_page - 1) / per_page;
  const int64_t size = dtype == MMVQ_F32 ? 4 : 2;
  p.q_vector = ((reinterpret_cast<uintptr_t>(p.q) | (uintptr_t)(p.ldq * size) | (uintptr_t)(p.hq * size)) & 15) == 0;
  if (dtype == MMVQ_F32) return launch_typed<true, true, float>(a, p, D, stream);
  if (dtype == MMVQ_F16) return launch_typed<false, true, __half>(a, p, D, stream);
  return launch_typed<false, false, __nv_bfloat16>(a, p, D, stream);
}

int64_t kv4_attention_workspace_bytes(int D) {
  return kKv4CounterBytes + 2 * kKv4MaxSms * kv4_slot_floats(kv4_rows_sm(D), D) * 4;
}

}  // namespace mmvq
