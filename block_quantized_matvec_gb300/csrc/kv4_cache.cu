// Keys and values quantised into the 4-bit cache, and read back from it: a
// warp per token and kv head, four consecutive values a lane (kv4.cuh).
#include "kv4.cuh"

namespace mmvq {
namespace {

struct Kv4Src {
  const void* k;
  const void* v;
  int64_t ldk, hk, ldv, hv;  // strides of a token and of a head, in elements
};

// Quantises the block whose values lane .. lane + 7 (an aligned octet) hold,
// four each: the lane's codes (value i in bits 4 i), d (low half) and z.
__device__ __forceinline__ uint32_t kv4_quantize(float (&x)[4], uint32_t& dz, bool& odd) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (!(fabsf(x[i]) <= kFp16Max)) {
      odd |= !(fabsf(x[i]) < INFINITY);
      x[i] = x[i] != x[i] ? 0.0f : copysignf(kFp16Max, x[i]);
    }
  }
  float hi = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
  float lo = fminf(fminf(x[0], x[1]), fminf(x[2], x[3]));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
  }
  const __half dh = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.0f));
  const __half zh = __float2half_rn(__fmul_rn(__fadd_rn(hi, lo), 0.5f));
  const float d = __half2float(dh), z = __half2float(zh);
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float c = rintf(__fadd_rn(__fdiv_rn(__fsub_rn(x[i], z), d), 7.5f));
    codes |= (d > 0.0f ? (uint32_t)fminf(fmaxf(c, 0.0f), 15.0f) : 0u) << (4 * i);
  }
  dz = (uint32_t)__half_as_ushort(dh) | ((uint32_t)__half_as_ushort(zh) << 16);
  return codes;
}

// Blocks q (of 2 nb: the keys' then the values') are taken four at a time, a
// block per octet of lanes.
template <int D, typename T>
__global__ void __launch_bounds__(256) kv4_append_kernel(Kv4Batch a, Kv4Src s) {
  constexpr int nb = D / 32;
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (item >= (int64_t)a.n_tokens * a.n_kv_heads) return;
  const int r = (int)(item / a.n_kv_heads), h = (int)(item - (int64_t)r * a.n_kv_heads);
  int b, pos;
  if (!kv4_place(a, r, lane, b, pos) || pos < 0) return;
  uint8_t* tile = kv4_tile(a, kv4_tile_bytes(D), b, pos / kKv4Tile);
  if (!tile) {
    if (lane == 0) kv4_set_status(a.status, MMVQ_ERR_ROUTING);
    return;
  }
  tile += h * kv4_head_stride(a, kv4_tile_bytes(D));
  const int t = pos % kKv4Tile;
  const T* k = static_cast<const T*>(s.k) + r * s.ldk + h * s.hk;
  const T* v = static_cast<const T*>(s.v) + r * s.ldv + h * s.hv;
  bool odd = false;
#pragma unroll
  for (int q0 = 0; q0 < 2 * nb; q0 += 4) {
    const int q = q0 + (lane >> 3), g = lane & 7;  // this octet's block, the lane in it
    const int blk = q % nb;
    const bool key = q < nb;
    const T* src = (key ? k : v) + 32 * blk + 4 * g;
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = kv4_load(src + i);
    uint32_t dz;
    const uint32_t codes = kv4_quantize(x, dz, odd);
    const int j = nb * (t >> 3) + blk;
    const int at = key ? kv4_word(j, 4 * (t & 7) + (g >> 1)) + 2 * (g & 1)
                       : 8 * D + kv4_word(j, 4 * g + ((t & 7) >> 1)) + 2 * (t & 1);
    *reinterpret_cast<uint16_t*>(tile + at) = (uint16_t)codes;
    if (g < 2) {
      const int sc = key ? kv4_key_scale(D, t, blk) : kv4_value_scale(D, t, blk);
      *reinterpret_cast<uint16_t*>(tile + sc + g * D) = (uint16_t)(g ? dz >> 16 : dz & 0xffffu);
    }
  }
  if (odd) kv4_set_status(a.status, MMVQ_ERR_VALUE);
}

template <int D, typename T>
__global__ void __launch_bounds__(256) kv4_read_kernel(Kv4Batch a, T* __restrict__ k_out,
                                                       T* __restrict__ v_out) {
  constexpr int nb = D / 32;
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (item >= (int64_t)a.n_tokens * a.n_kv_heads) return;
  const int r = (int)(item / a.n_kv_heads), h = (int)(item - (int64_t)r * a.n_kv_heads);
  int b, pos;
  if (!kv4_place(a, r, lane, b, pos)) return;
  const uint8_t* tile = nullptr;
  if (pos >= 0) {
    tile = kv4_tile(a, kv4_tile_bytes(D), b, pos / kKv4Tile);
    if (tile) tile += h * kv4_head_stride(a, kv4_tile_bytes(D));
    else if (lane == 0) kv4_set_status(a.status, MMVQ_ERR_ROUTING);
  }
  const int t = pos & (kKv4Tile - 1);
#pragma unroll
  for (int q0 = 0; q0 < 2 * nb; q0 += 4) {
    const int q = q0 + (lane >> 3), g = lane & 7;
    const int blk = q % nb;
    const bool key = q < nb;
    float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (tile) {
      const int j = nb * (t >> 3) + blk;
      const int at = key ? kv4_word(j, 4 * (t & 7) + (g >> 1)) + 2 * (g & 1)
                         : 8 * D + kv4_word(j, 4 * g + ((t & 7) >> 1)) + 2 * (t & 1);
      const int sc = key ? kv4_key_scale(D, t, blk) : kv4_value_scale(D, t, blk);
      const uint32_t codes = *reinterpret_cast<const uint16_t*>(tile + at);
      const float d = half_bits_to_float(*reinterpret_cast<const uint16_t*>(tile + sc));
      const float z = half_bits_to_float(*reinterpret_cast<const uint16_t*>(tile + sc + D));
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = kv4_value((codes >> (4 * i)) & 15u, d, z);
    }
    T* out = (key ? k_out : v_out) + item * D + 32 * blk + 4 * g;
#pragma unroll
    for (int i = 0; i < 4; ++i) kv4_store(out + i, x[i]);
  }
}

template <typename T>
int append_typed(const Kv4Batch& a, const Kv4Src& s, int D, cudaStream_t stream) {
  const int64_t items = (int64_t)a.n_tokens * a.n_kv_heads;
  const dim3 grid((unsigned)((items + 7) / 8)), block(256);
  if (D == 64) return launch_pdl(kv4_append_kernel<64, T>, grid, block, 0, stream, a, s);
  if (D == 128) return launch_pdl(kv4_append_kernel<128, T>, grid, block, 0, stream, a, s);
  return launch_pdl(kv4_append_kernel<256, T>, grid, block, 0, stream, a, s);
}

template <typename T>
int read_typed(const Kv4Batch& a, int D, void* k, void* v, cudaStream_t stream) {
  const int64_t items = (int64_t)a.n_tokens * a.n_kv_heads;
  const dim3 grid((unsigned)((items + 7) / 8)), block(256);
  T* ko = static_cast<T*>(k);
  T* vo = static_cast<T*>(v);
  if (D == 64) return launch_pdl(kv4_read_kernel<64, T>, grid, block, 0, stream, a, ko, vo);
  if (D == 128) return launch_pdl(kv4_read_kernel<128, T>, grid, block, 0, stream, a, ko, vo);
  return launch_pdl(kv4_read_kernel<256, T>, grid, block, 0, stream, a, ko, vo);
}

}  // namespace

int launch_kv4_append(const Kv4Batch& a, int D, int dtype, const void* k, const void* v,
                      const int64_t (&strides)[4], cudaStream_t stream) {
  const Kv4Src s = {k, v, strides[0], strides[1], strides[2], strides[3]};
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
