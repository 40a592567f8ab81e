// Arguments of the layer's steps between the products, as the entry points
// (api.cu) pass them on once checked.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace mmvq {

constexpr int kRopeMaxAxes = 4;
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxTopk = 32;
constexpr int kRouteMaxGroups = 32;
constexpr int kCombineMaxTopk = 256;
constexpr int kLogprobsMaxTop = 32;

// One tensor of heads [n_tokens][heads][head_dim], read at x and written at y.
struct RopeHeads {
  const void* x;
  int64_t ldx, hx;  // elements from token to token, from head to head
  void* y;
  int64_t ldy, hy;
  const float* weight;  // [head_dim] or NULL: ones
  int heads;
};

struct NormRope {
  RopeHeads q, k;
  const int32_t* positions;  // [n_axes][ld_positions]
  int64_t ld_positions;
  int n_axes;
  const int64_t* table;  // [2][rot / 2]: turn per position in 2^-64 turns; axis
  int rot;
  float eps;
  bool norm, interleaved;
  int n_tokens;
  int32_t* status;
};

struct RouteTopk {
  const void* logits;
  int64_t ld;
  int n_tokens, n_experts, k;
  bool sigmoid, renormalize;
  const float* bias;
  int n_groups, top_groups;
  float scale;
  int32_t* topk;
  float* weights;
  int32_t* status;
};

struct CombineExperts {
  const float* y;
  int64_t n_positions;
  int H;
  const int32_t* topk;
  const float* weights;
  int n_tokens, k;
  const int32_t* offsets;
  int n_experts;
  const int32_t* slot_of;
  const void* residual;
  int64_t ldr;
  const void* shared;
  int64_t lds;
  const float* gate;
  void* out;
  int64_t ldo;
  int32_t* status;
};

struct TokenLogprobs {
  const void* logits;
  int64_t ld;
  int rows, vocab;
  float scale;
  const int32_t* tokens;
  int n_tokens, top;
  float* lse;
  float* entropy;
  float* logprobs;
  int32_t* top_ids;
  float* top_logprobs;
  int32_t* status;
};

int launch_norm_rope(const NormRope& a, int dtype, int head_dim, cudaStream_t stream);
int launch_route_topk(const RouteTopk& a, int dtype, cudaStream_t stream);
int launch_combine_experts(const CombineExperts& a, int dtype, cudaStream_t stream);
int launch_token_logprobs(const TokenLogprobs& a, int dtype, cudaStream_t stream);

}  // namespace mmvq
