// Arguments of the attention over the 4-bit cache.
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
};

}  // namespace mmvq
