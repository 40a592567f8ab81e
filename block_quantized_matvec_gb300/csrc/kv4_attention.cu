// Attention of 1-8 query tokens a sequence over the 4-bit cache: a CTA per
// query row, a warp per cached token, running maximum and sum in fp32.
#include "kv4.cuh"
#include "kv4_attention.cuh"

namespace mmvq {
namespace {

template <int D, typename T>
__global__ void __launch_bounds__(128) kv4_attention_kernel(Kv4Batch a, Kv4Attention p) {
  constexpr int nb = D / 32, kOwn = D / 32;  // values of a lane: lane + 32 i
  __shared__ float acc_s[4][D], max_s[4], sum_s[4];
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = blockIdx.x, hq = blockIdx.y;
  const int h = hq / (p.n_heads / a.n_kv_heads);
  int b, pos;
  if (!kv4_place(a, r, lane, b, pos)) return;
  const int first = __ldg(a.offsets + b), end = __ldg(a.offsets + b + 1);
  if (end - first > kKv4MaxNew) {
    if (threadIdx.x == 0) kv4_set_status(a.status, MMVQ_ERR_NCOLS);
    return;
  }
  float q[kOwn], o[kOwn], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    q[i] = kv4_load(static_cast<const T*>(p.q) + r * p.ldq + hq * p.hq + lane + 32 * i);
    o[i] = 0.0f;
  }
  const int64_t hs = kv4_head_stride(a, kv4_tile_bytes(D));
  for (int64_t key = warp; key <= pos; key += 4) {
    if (p.window > 0 && key <= (int64_t)pos - p.window && key >= p.sinks) continue;
    const uint8_t* tile = kv4_tile(a, kv4_tile_bytes(D), b, (int)(key / kKv4Tile));
    if (!tile) {
      if (lane == 0) kv4_set_status(a.status, MMVQ_ERR_ROUTING);
      continue;
    }
    tile += h * hs;
    const int t = (int)(key % kKv4Tile);
    float s = 0.0f, v[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int j = nb * (t >> 3) + i;
      const uint8_t kc = tile[kv4_word(j, 4 * (t & 7) + lane / 8) + (lane % 8) / 2];
      const uint8_t vc = tile[8 * D + kv4_word(j, 4 * (lane / 4) + (t & 7) / 2) + 2 * (t & 1) + lane % 4 / 2];
      const uint16_t* ks = reinterpret_cast<const uint16_t*>(tile + kv4_key_scale(D, t, i));
      const uint16_t* vs = reinterpret_cast<const uint16_t*>(tile + kv4_value_scale(D, t, i));
      const int sh = 4 * (lane & 1);
      s = fmaf(q[i], kv4_value((kc >> sh) & 15u, half_bits_to_float(ks[0]), half_bits_to_float(ks[D / 2])), s);
      v[i] = kv4_value((vc >> sh) & 15u, half_bits_to_float(vs[0]), half_bits_to_float(vs[D / 2]));
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= p.scale;
    const float m2 = fmaxf(m, s);
    const float f = m == -INFINITY ? 0.0f : expf(m - m2), e = s == -INFINITY ? 0.0f : expf(s - m2);
    l = l * f + e;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) o[i] = o[i] * f + e * v[i];
    m = m2;
  }
#pragma unroll
  for (int i = 0; i < kOwn; ++i) acc_s[warp][lane + 32 * i] = o[i];
  if (lane == 0) max_s[warp] = m, sum_s[warp] = l;
  __syncthreads();
  float top = -INFINITY, total = 0.0f;
  for (int w = 0; w < 4; ++w) top = fmaxf(top, max_s[w]);
  float f[4];
  for (int w = 0; w < 4; ++w) {
    f[w] = max_s[w] == -INFINITY ? 0.0f : expf(max_s[w] - top);
    total += f[w] * sum_s[w];
  }
  for (int d = threadIdx.x; d < D; d += 128) {
    float y = 0.0f;
    for (int w = 0; w < 4; ++w) y += f[w] * acc_s[w][d];
    kv4_store(static_cast<T*>(p.y) + ((int64_t)r * p.n_heads + hq) * D + d,
              total == 0.0f ? 0.0f : y / total);
  }
  if (p.lse && threadIdx.x == 0)
    p.lse[(int64_t)r * p.n_heads + hq] = total == 0.0f ? -INFINITY : top + logf(total);
}

template <typename T>
int attention_typed(const Kv4Batch& a, const Kv4Attention& p, int D, cudaStream_t stream) {
  const dim3 grid(a.n_tokens, p.n_heads), block(128);
  if (D == 64) return launch_pdl(kv4_attention_kernel<64, T>, grid, block, 0, stream, a, p);
  if (D == 128) return launch_pdl(kv4_attention_kernel<128, T>, grid, block, 0, stream, a, p);
  return launch_pdl(kv4_attention_kernel<256, T>, grid, block, 0, stream, a, p);
}

}  // namespace

int launch_kv4_attention(const Kv4Batch& a, const Kv4Attention& p, int D, int dtype,
                         cudaStream_t stream) {
  if (dtype == MMVQ_F32) return attention_typed<float>(a, p, D, stream);
  if (dtype == MMVQ_F16) return attention_typed<__half>(a, p, D, stream);
  return attention_typed<__nv_bfloat16>(a, p, D, stream);
}

int64_t kv4_attention_workspace_bytes(int) { return 256; }

}  // namespace mmvq
