// Shared by the kernels of awq_attention_shared: how a call is cut into parts, and small helpers.
#pragma once

#include "awq_layer.cuh"
#include "awq_ptx.cuh"

namespace awq {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f;

// A probability is kept as p = 2^(z - m + kLift), z the logit (base 2) and m the row's running maximum,
// raised only when a logit exceeds it by kRaise.  Largest p: 2^15, in fp16's range; fp16 numbers with
// their full 11 bits reach down to 2^-21 of the maximum (2^-14 without the lift).  The sum l and the
// sums of values carry the same factor; a part's maximum is written as m - kLift.
constexpr float kRaise = 8.f, kLift = 7.f;

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

// Copies a 64-element wide box of tokens.
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(ptx::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(ptx::smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

// Bounded waits give up after this long, set the bit in the status word and leave.
constexpr uint64_t kWaitLimitNs = 200ull * 1000 * 1000;
constexpr unsigned int kStatusAttnTimeout = 0x8u;

// How a call is cut.  Row r = (b n + i) Hq + h of the output; part s of row r is at
// part_o[(r parts + s) D], part_ml[r parts + s]; slots [0, prefix_parts) are the prefix's, the others
// the sequence's own.
//
// Tensor-core kernel (tc, the prefix's keys): row tiles of kTcRows rows per key/value head, steps of
// kTcKeys keys.  The row tiles of a head go side by side, one block each (tc_lanes blocks, a group), so
// that they read the same keys at the same time and HBM is read once; the steps of all heads form one
// sequence of which group g takes [g per, (g + 1) per), per being found on the device.  (More row tiles
// than SMs: a group is one block, and the steps of all heads' tiles form the sequence.)
//
// Streaming kernel (the sequences' own keys, and the prefix's without tc): units are (sequence, row
// tile), the prefix being a sequence of its own in front; a unit of L keys has ceil(L / kStreamKeys)
// steps; all steps of all units form one sequence of which share i takes [i per, (i + 1) per), per =
// max(per_min, total / shares) being found on the device, where the lengths are.  Every key/value head
// has a warp for each share: neighbouring warps read neighbouring heads of the same tokens at the
// same time.  The warp that ends a unit writes the unit's number of parts.
struct Plan {
  int group;  // query heads per key/value head
  int own_rows;  // rows of one sequence that share a key/value head
  bool tc;
  int sms;
  int tc_tiles, tc_steps, tc_lanes;
  int tc_per, tc_groups;             // least steps of a group, most groups
  int tile;                          // rows of a streaming unit
  int prefix_tiles, private_tiles;   // row tiles per key/value head of the streaming units
  int per_min, shares, blocks;       // streaming kernel
  int prefix_parts, private_parts;   // most parts of a row
  int parts;                         // their sum
};

constexpr int kStreamKeys = 16;
constexpr int kStreamWarps = 4;

constexpr int kTcRows = 256;  // two 128-row tensor-core tiles
constexpr int kTcKeys = 128;

// Unit (of the sequence of steps) of a head's row tile; first and last group of a unit's steps, of which a
// group takes `per`.
__host__ __device__ inline int tc_unit(const Plan& pl, int hk, int tile) { return pl.tc_lanes > 1 ? hk : hk * pl.tc_tiles + tile; }
__host__ __device__ inline int tc_first_group(const Plan& pl, int u, int per) { return u * pl.tc_steps / per; }
// First of the steps of a group, `total` for a group beyond the last.  Blocks are launched for the least
// steps a group can have; where the split leaves few groups, `per` is up to total (below 2^30) and the
// product passes 32 bits for the groups beyond the last.
__host__ __device__ inline int tc_first_step(int group, int per, int total) {
  const int64_t first = static_cast<int64_t>(group) * per;
  return first < total ? static_cast<int>(first) : total;
}
__host__ __device__ inline int tc_last_group(const Plan& pl, int u, int per) { return ((u + 1) * pl.tc_steps - 1) / per; }

// The two kernels of a call with tc run side by side, the tensor-core kernel on as many SMs as its share of
// the work, the streaming kernel on the others.  The lengths decide, so the device does.  A block's step of
// the one takes some 1.66 us of an SM and its start and end as long as three more, a step of a head of the
// other 0.11 us and a unit's start and end as long as two (heads of 128; fewer elements, less of both).  A
// streaming kernel that would get fewer than a twelfth of the SMs comes after, on all (128 sequences of
// up to 64 own keys over 32768: 109 us, 131 with 4 SMs).  Blocks of the tensor-core kernel beyond its
// share leave at once; the streaming kernel's blocks are one wave on the SMs left, or, where whole groups
// leave it much less than its share, as many as all SMs hold.  128 sequences of 1024 own keys over 32768
// shared ones, 8 heads: some 100 SMs and 50, 151 us of kernels with the join; one after the other on all
// SMs 192 us; 64 of 512 over 8197: 48 and 65 us.
//
// The costs were fitted to heads of 128, eight query rows per head and full row tiles.  With 0.35 to 2.8 times
// the streaming step's cost, the constants here are within 2 % of the best for heads of 64 and 96, 16-row
// units, row tiles filled to an eighth or a half, and one query head per key/value head; 14 % above it for
// pages of 20 tokens (212 us, 186 at 0.71 times the cost: 128 sequences over 16384) and 65 % for 32-row units
// (64 sequences of four new tokens: 350 us, 212 at 2.8 times the cost).
constexpr int64_t kTcStepNs = 1660, kTcFixedSteps = 3, kStreamStepNs = 108, kStreamFixedSteps = 2;

constexpr int kLeastShare = 12;

struct Split {
  int per;    // steps that a group of the tensor-core kernel takes
  int left;   // SMs on which the streaming kernel's blocks are one wave; 0: all
};

// `own`: steps of the sequences' own keys, per head; `units`: sequences times their row tiles.
__device__ inline Split split_sms(const Plan& pl, int heads, int64_t own, int64_t units) {
  const int total = heads * (pl.tc_tiles / pl.tc_lanes) * pl.tc_steps;
  const int64_t tc = (total + kTcFixedSteps * pl.tc_groups) * (pl.tc_lanes * kTcStepNs);
  const int64_t rest = min(own + kStreamFixedSteps * units, int64_t{1} << 32) * heads * kStreamStepNs;
  int share = static_cast<int>(pl.sms * tc / (tc + rest));  // SMs
  if ((pl.sms - share) * kLeastShare < pl.sms) share = pl.sms;
  const int groups = max(1, min(pl.tc_groups, (share + pl.tc_lanes / 2) / pl.tc_lanes));
  Split s;
  s.per = max(pl.tc_per, (total + groups - 1) / groups);
  s.left = pl.sms - (total + s.per - 1) / s.per * pl.tc_lanes;
  if (share == pl.sms || 4 * s.left < 3 * (pl.sms - share)) s.left = 0;
  return s;
}

// A number of parts as the join uses it.  A streaming warp that gave up a wait has written none, and the
// workspace may hold anything: whatever stands there, the join stays within the row's slots.
__host__ __device__ inline int parts_within(int count, int most) { return count < 0 ? 0 : count < most ? count : most; }

struct AttnArgs {
  AttentionProblem p;
  Plan plan;
  float* part_o;
  float2* part_ml;
  int* tc_per;  // steps of a tensor-core group
  int* counts;  // parts of each streaming unit, per head: [prefix_tiles][heads], then [B][private_tiles][heads]
  unsigned int* status;
};

__device__ __forceinline__ int own_length(const AttentionProblem& p, int b) {
  return min(max(__ldg(p.lens + b), 0), static_cast<int>(p.max_len));
}
__device__ __forceinline__ int stream_steps(int len) { return len / kStreamKeys + (len % kStreamKeys != 0); }

// The keys or values of the cache as [page][head][token][element] for boxes of 64 elements of `box`
// tokens, 128-byte swizzle.  False: the strides do not allow it.
bool make_cache_map(CUtensorMap* map, const void* base, const AttentionProblem& p, int box);
bool tc_head_dim_supported(int D);
cudaError_t launch_prefix_tc(const AttnArgs& a);

}  // namespace attn
}  // namespace awq
