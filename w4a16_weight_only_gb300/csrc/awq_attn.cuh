// Shared by the kernels of awq_attention_shared: how a call is cut into parts, and small helpers.
#pragma once

#include "awq_layer.cuh"
#include "awq_ptx.cuh"

namespace awq {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two values rounded once to the element type, lo in the low half.
template <bool kBF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (kBF) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  const int bytes = valid ? 16 : 0;  // 0: the 16 bytes are zero-filled, nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// How a call is cut.  Row r = (b n + i) Hq + h of the output; part s of row r is at
// part_o[(r parts + s) D], part_ml[r parts + s]; parts [0, prefix_parts) are the prefix's, then one
// per started `chunk` of the sequence's own keys.
struct Plan {
  int group;  // query heads per key/value head
  // prefix, streaming kernel: row tiles per key/value head, keys per part
  int prefix_tiles, prefix_chunk;
  // prefix, tensor-core kernel (tc): tiles of kTcRows rows per key/value head, kTcKeys-key steps per
  // tile; all steps of all tiles form one sequence of which block c takes [c per, (c + 1) per)
  bool tc;
  int tc_tiles, tc_steps, tc_per, tc_blocks;
  int prefix_parts;   // most parts a row's prefix has
  int chunk;          // private keys per part
  int private_parts;  // parts of the longest sequence
  int private_tiles;  // row tiles of one sequence
  int parts;          // prefix_parts + private_parts
  int mt;             // 16-row tiles per block of the streaming kernel
};

constexpr int kTcRows = 256;  // two 128-row tensor-core tiles
constexpr int kTcKeys = 128;

// First and last block of tile t's steps.
__host__ __device__ inline int tc_first_block(const Plan& pl, int t) {
  return static_cast<int>(static_cast<int64_t>(t) * pl.tc_steps / pl.tc_per);
}
__host__ __device__ inline int tc_last_block(const Plan& pl, int t) {
  return static_cast<int>((static_cast<int64_t>(t + 1) * pl.tc_steps - 1) / pl.tc_per);
}

struct AttnArgs {
  AttentionProblem p;
  Plan plan;
  float* part_o;
  float2* part_ml;
  unsigned int* status;
};

bool tc_head_dim_supported(int D);
cudaError_t launch_prefix_tc(const AttnArgs& a);

}  // namespace attn
}  // namespace awq
