// Problem descriptions of the operators between a layer's linears (rotary positions, expert
// routing, dispatch and combine, shared-prefix attention); shared by their kernels and the C ABI.
#pragma once

#include "awq_internal.cuh"

namespace awq {

// A paged key/value cache: [num_pages, page_size, heads, head_dim] of 16-bit elements, strides in
// elements, the head's elements contiguous; keys and values with the same strides.
struct PagedKV {
  uint16_t* k;
  uint16_t* v;
  int num_pages, page_size, heads, head_dim;
  int64_t page_stride, token_stride, head_stride;
};

struct RopeTableProblem {
  float* table;  // [max_position, rot]: rot / 2 cosines, then rot / 2 sines
  int64_t max_position;
  int rot;
  double base;
  int scaling;  // awq_rope_scaling_t
  double factor;
  double original;  // positions the frequencies were trained on
  double p0, p1;    // yarn: turns of the fast and slow ends; banded: low and high factor
  double attention_factor;
  cudaStream_t stream;
};

struct RopeProblem {
  const uint16_t *q, *k, *v;  // v: append only
  const int* positions;       // [T]
  const float* table;
  int64_t T;
  int Hq, Hkv, D, rot, max_position;
  int64_t q_st, q_sh, k_st, k_sh, v_st, v_sh;  // token and head strides, elements
  uint16_t* q_out;
  uint16_t* k_out;  // plain form
  int64_t qo_st, qo_sh, ko_st, ko_sh;
  const int* slots;  // append: cache cell of each token, [T]
  PagedKV kv;
  bool append, interleaved, bf16;
  cudaStream_t stream;
};

struct RouteProblem {
  const void* logits;  // [T, E], row stride ld
  int64_t T, ld;
  int E, k;
  int dtype;  // awq_dtype_t
  bool sigmoid;
  const float* bias;  // [E] or nullptr
  int groups, topk_groups, group_best;
  bool renormalize;
  float scale;
  float* weights;  // [T, k]
  int* experts;    // [T, k]
  cudaStream_t stream;
};

struct DispatchProblem {
  const uint16_t* x;  // [T, W], row stride ld
  int64_t T, ld;
  int W;
  const int* experts;  // [T, k]
  int k, E;
  uint16_t* routed;  // [T k, W]
  int* offsets;      // [E + 1]
  int* rows;         // [T, k]
  void* workspace;
  cudaStream_t stream;
};

struct CombineProblem {
  const uint16_t* y;  // [R, W]
  int64_t R;
  int W;
  const float* weights;  // [T, k]
  const int* rows;       // [T, k]
  int64_t T;
  int k;
  const uint16_t* base;  // [T, W] or nullptr
  uint16_t* out;         // [T, W]
  bool bf16;
  cudaStream_t stream;
};

struct AttentionProblem {
  const uint16_t* q;  // [B, n, Hq, D], strides in elements
  int64_t q_sb, q_sn, q_sh;
  int B, n, Hq;
  PagedKV kv;
  const int* prefix_pages;
  int64_t prefix_len;
  const int* pages;  // [B, W], row stride pages_ld
  int64_t pages_ld;
  int W;
  const int* lens;  // [B]
  int64_t max_len;
  float scale;
  uint16_t* out;  // [B, n, Hq, D]
  bool bf16;
  bool give_up;  // self test: the kernels' bounded waits give up at once
  void* workspace;
  cudaStream_t stream;
};

cudaError_t launch_rope_table(const RopeTableProblem& p);
cudaError_t launch_rope(const RopeProblem& p);
cudaError_t launch_route(const RouteProblem& p);

// Experts and places a routing call can have (a warp holds a token's scores in registers).
constexpr int kRouteMaxE = 1024;
constexpr int kRouteMaxK = 32;
constexpr int kDispatchMaxE = 4096;

size_t dispatch_workspace_bytes(int64_t R, int E);
cudaError_t launch_dispatch(const DispatchProblem& p);
cudaError_t launch_combine(const CombineProblem& p);

bool attention_head_dim_supported(int64_t D);
// Workspace of an attention call (partial sums); a function of the host-side sizes only.
size_t attention_workspace_bytes(const AttentionProblem& p, int sms);
cudaError_t launch_attention(const AttentionProblem& p, int sms);

}  // namespace awq
