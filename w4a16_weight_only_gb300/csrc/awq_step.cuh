// Problem descriptions of the operators around a 4-bit key/value cache (append, read, attention), of
// the norms around a residual sum and of the mixture-of-experts layer of a few tokens; shared by
// their kernels and the C ABI.
#pragma once

#include "awq_internal.cuh"

namespace awq {

// A paged cache of 4-bit keys and values: [num_pages][heads] runs of page_size / 16 tiles, a tile holding
// 16 tokens of one head as
//   16 D / 2 bytes: codes of the keys       (Kv4::key_byte)
//   16 D / 2 bytes: codes of the values     (Kv4::value_byte)
//   64 G bytes: keys' (scale, minimum) pairs of 16-bit elements, [token][group], G = D / group
//   64 G bytes: the values'
// A code c stands for c * scale + minimum; the low nibble of a byte is the even element's.
struct Kv4Cache {
  uint8_t* data;
  int num_pages, page_size, heads, head_dim, group;
  int64_t page_stride, head_stride;  // bytes

  __host__ __device__ int groups() const { return head_dim / group; }
  __host__ __device__ int tile_bytes() const { return 16 * (head_dim + 8 * (head_dim / group)); }
};

struct Kv4 {
  // Byte of a tile's key codes that holds elements 2 i, 2 i + 1 of token r: words of eight elements, four
  // lanes' words side by side.  A panel of 128 elements (or the whole head below that) has 4 W words, of
  // which lane t of a quad needs words t, 4 + t, ..: they stand together, one vector load.
  __host__ __device__ static int key_byte(int D, int r, int i) {
    const int W = (D < 128 ? D : 128) / 32, panel = i / 64, word = i % 64 / 4;
    return panel * 1024 + r * 16 * W + (word % 4 * W + word / 4) * 4 + i % 4;
  }
  // The same of the values (offset from the first value byte).  A word holds elements 4 x .. 4 x + 3 of
  // tokens 2 t + 8 h and 2 t + 8 h + 1: the two tokens of a 32-bit fragment register.
  __host__ __device__ static int value_byte(int D, int r, int i) {
    const int u = i / 16, g = i / 2 % 8, e = i % 2, lane = 4 * g + r / 2 % 4, in = r / 8 * 4 + r % 2 * 2 + e;
    return u < D / 64 * 2 ? u / 2 * 512 + lane * 16 + u % 2 * 8 + in : D / 64 * 512 + lane * 8 + in;
  }
};

struct AppendKv4Problem {
  const uint16_t *q, *k, *v;
  const int* positions;  // [T]
  const float* table;    // nullptr: no rotation
  int64_t T;
  int Hq, Hkv, D, rot, max_position;
  int64_t q_st, q_sh, k_st, k_sh, v_st, v_sh;  // token and head strides, elements
  uint16_t* q_out;
  int64_t qo_st, qo_sh;
  const int* slots;  // [T]
  Kv4Cache cache;
  bool interleaved, bf16;
  cudaStream_t stream;
};

struct ReadKv4Problem {
  Kv4Cache cache;
  const int* slots;  // [T]
  int64_t T;
  uint16_t *k, *v;  // [T, heads, D]
  bool bf16;
  cudaStream_t stream;
};

struct AttentionKv4Problem {
  const uint16_t* q;  // [B, n, Hq, D], strides in elements
  int64_t q_sb, q_sn, q_sh;
  int B, n, Hq;
  Kv4Cache cache;
  const int* pages;  // [B, W], row stride pages_ld
  int64_t pages_ld;
  int W;
  const int* lens;  // [B]
  int window, sinks;  // window 0: none
  float scale;
  uint16_t* out;  // [B, n, Hq, D]
  bool bf16;
  bool give_up;  // self test: the kernel's bounded waits give up at once
  void* workspace;
  cudaStream_t stream;
};

struct ResidualNormProblem {
  const uint16_t *x, *residual, *gate;  // gate, residual: may be nullptr
  int64_t x_st, r_st, g_st;             // row strides, elements; g_st 0: one row
  const uint16_t *post_weight, *post_bias, *weight, *bias;  // [W] or nullptr
  float scale, eps;
  int64_t T;
  int W;
  bool layer;  // mean subtracted
  uint16_t *h, *y;  // [T, W]; y: nullptr without weight
  bool bf16;
  cudaStream_t stream;
};

// A stacked 4-bit linear [E, K, N], groups of G rows.
struct Stacked {
  const uint32_t *qw, *qz;
  const uint16_t* sc;
};

struct MoeLayerProblem {
  const uint16_t* x;  // [T, H], row stride x_st
  int64_t x_st;
  int T, H, I, E, k, G;
  const int* experts;    // [T, k]
  const float* weights;  // [T, k]
  Stacked up, down;      // [E, H, 2 I] (gate columns, then up columns), [E, I, H]
  const uint16_t* base;  // [T, H] or nullptr
  uint16_t* out;         // [T, H]
  bool bf16;
  bool give_up;  // self test: the kernels' bounded waits give up at once
  void* workspace;
  cudaStream_t stream;
};

constexpr int kMoeLayerMaxT = 16;

bool kv4_shape_supported(int64_t D, int64_t group);
cudaError_t launch_append_kv4(const AppendKv4Problem& p, int sms);
cudaError_t launch_read_kv4(const ReadKv4Problem& p);
size_t attention_kv4_workspace_bytes(const AttentionKv4Problem& p, int sms);
cudaError_t launch_attention_kv4(const AttentionKv4Problem& p, int sms);
cudaError_t launch_residual_norm(const ResidualNormProblem& p, int sms);
size_t moe_layer_workspace_bytes(int T, int k, int H, int I);
cudaError_t launch_moe_layer(const MoeLayerProblem& p, int sms);

}  // namespace awq
