// Around the grouped (mixture-of-experts) linears: routing of tokens to experts, the sort of the
// routed rows by expert (dispatch) and the weighted sum of a token's rows (combine).
#include "awq_layer.cuh"
#include "awq_ptx.cuh"

namespace awq {
namespace {

using namespace ptx;

constexpr unsigned kAll = 0xffffffffu;

// -------------------------------------------------------------------------------- routing ----

// An fp32 key as an unsigned whose order is the key's (-0 counts as +0).  0 is below every key and
// stands for "no expert".
__device__ __forceinline__ uint32_t ordered(float key) {
  const uint32_t u = __float_as_uint(key + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}

template <int DT>  // awq_dtype_t
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  if constexpr (DT == 1) return __ldg(static_cast<const float*>(p) + i);
  else return elem_to_float<DT == 2>(__ldg(static_cast<const uint16_t*>(p) + i));
}

// Good to one unit in the last place: for the keys, of which every expert has one (rounded reciprocals: 19.0
// against 18.3 us for 16381 tokens of 256 experts).  The k weights take the rounded one.
__device__ __forceinline__ float reciprocal(float x) {
  float y;
  asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One warp per token.  Lane l holds experts [l V, l V + V), V = ceil(E / 32) <= VT, so that the
// lowest lane and the lowest register of the equal keys is the lowest expert.  kVec: V == VT and rows
// allow 16-byte loads.  Bound by instructions;
// every maximum over the warp is one redux on the keys as ordered integers.
template <int DT, int VT, bool kVec>
__global__ void __launch_bounds__(128) route_kernel(const RouteProblem p) {
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const int V = kVec ? VT : (p.E + 31) / 32;
  const int e0 = lane * V;
  const int64_t row = t * p.ld;
  float x[VT];
  if constexpr (kVec) {
    constexpr int PER = DT == 1 ? 4 : 8;
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.logits) + (row + e0) * (DT == 1 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < VT / PER; ++i) {
      const uint4 v = __ldg(src + i);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (DT == 1) {
          x[i * 4 + j] = __uint_as_float(w[j]);
        } else {
          const float2 f = pair_to_float2<DT == 2>(w[j]);
          x[i * 8 + 2 * j] = f.x;
          x[i * 8 + 2 * j + 1] = f.y;
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < VT; ++i) x[i] = i < V && e0 + i < p.E ? load_logit<DT>(p.logits, row + e0 + i) : -INFINITY;
  }

  // scores; an expert whose logit is -inf is out
  float top = -INFINITY, inv = 0.f;
  const auto score_of = [&](float v) { return p.sigmoid ? __frcp_rn(1.f + expf(-v)) : expf(v - top) * inv; };
  float score[VT];
  if (p.sigmoid) {
#pragma unroll
    for (int i = 0; i < VT; ++i) score[i] = reciprocal(1.f + expf(-x[i]));
  } else {
#pragma unroll
    for (int i = 0; i < VT; ++i) top = fmaxf(top, x[i]);
    top = from_ordered(__reduce_max_sync(kAll, ordered(top)));
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < VT; ++i) {
      score[i] = x[i] == -INFINITY ? 0.f : expf(x[i] - top);
      sum += score[i];
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
    inv = __fdiv_rn(1.f, sum);
#pragma unroll
    for (int i = 0; i < VT; ++i) score[i] *= inv;
  }
  bool bad = false;
  uint32_t key[VT];
#pragma unroll
  for (int i = 0; i < VT; ++i) {
    const bool in = x[i] != -INFINITY;  // true for NaN
    bad |= in && isnan(score[i]);
    const float b = p.bias && in ? __ldg(p.bias + e0 + i) : 0.f;
    key[i] = in ? ordered(score[i] + b) : 0u;
  }
  bad = __any_sync(kAll, bad);

  if (p.groups > 1 && !bad) {
    const int per = p.E / p.groups;
    const bool even = p.E == 32 * V && 32 % p.groups == 0;  // a group is the experts of 32 / groups whole lanes
    uint32_t mine = 0u;  // a group's score: in all its lanes (even), or in lane g
    if (even) {
      uint32_t first = 0u, second = 0u;  // this lane's two best, then its group's
#pragma unroll
      for (int i = 0; i < VT; ++i) {
        second = max(second, min(first, key[i]));
        first = max(first, key[i]);
      }
      for (int d = 1; d < 32 / p.groups; d <<= 1) {
        const uint32_t of = __shfl_xor_sync(kAll, first, d), os = __shfl_xor_sync(kAll, second, d);
        second = max(max(second, os), min(first, of));
        first = max(first, of);
      }
      mine = p.group_best == 2 && second ? ordered(from_ordered(first) + from_ordered(second)) : first;
    } else {
      for (int g = 0; g < p.groups; ++g) {
        uint32_t first = 0u, second = 0u;  // this lane's two best of the group
#pragma unroll
        for (int i = 0; i < VT; ++i) {
          const int e = e0 + i;
          const uint32_t u = i < V && e >= g * per && e < (g + 1) * per ? key[i] : 0u;
          second = max(second, min(first, u));
          first = max(first, u);
        }
        const uint32_t best = __reduce_max_sync(kAll, first);
        uint32_t sum = best;
        if (p.group_best == 2 && best) {
          const int owner = __ffs(__ballot_sync(kAll, first == best)) - 1;
          const uint32_t next = __reduce_max_sync(kAll, lane == owner ? second : first);
          if (next) sum = ordered(from_ordered(best) + from_ordered(next));
        }
        if (lane == g) mine = sum;
      }
    }
    // a group is kept if fewer than topk_groups are better (ties: the lower index)
    const int width = even ? 32 / p.groups : 1, group = lane / width;
    int better = 0;
    for (int g = 0; g < p.groups; ++g) {
      const uint32_t other = __shfl_sync(kAll, mine, g * width);
      better += other > mine || (other == mine && g < group);
    }
    const bool keep = mine && better < p.topk_groups;
    if (even) {
      if (!keep) {
#pragma unroll
        for (int i = 0; i < VT; ++i) key[i] = 0u;
      }
    } else {
      const uint32_t kept = __ballot_sync(kAll, keep && lane < p.groups);
#pragma unroll
      for (int i = 0; i < VT; ++i) {
        const int e = e0 + i;
        if (i < V && e < p.E && !((kept >> (e / per)) & 1u)) key[i] = 0u;
      }
    }
  }

  int chosen = -1;  // lane j: place j
  float weight = 0.f;
  if (bad) {
    chosen = lane;
    weight = __int_as_float(0x7fffffff);
  } else {
    if constexpr (VT <= 8) {
      // Each lane sorts its keys once (a rank by comparing pairs, then a sorting network), so that a
      // place costs the maximum over the lanes' first keys and one shift (16381 tokens, 8 of 256 experts
      // in 8 groups: 18.5 us; 23.1 us when every place searches the lane's keys).
      uint32_t order = 0u;  // the lane's registers by falling key, four bits each
      int rank[VT];
#pragma unroll
      for (int i = 0; i < VT; ++i) rank[i] = 0;
#pragma unroll
      for (int i = 0; i < VT; ++i)
#pragma unroll
        for (int j = i + 1; j < VT; ++j) {
          const bool later = key[j] > key[i];  // equal keys: the lower register first
          rank[i] += later;
          rank[j] += !later;
        }
#pragma unroll
      for (int i = 0; i < VT; ++i) order |= static_cast<uint32_t>(i) << (4 * rank[i]);
#pragma unroll
      for (int n = 1; n < VT; n <<= 1)  // odd-even merge sort (Batcher), falling
#pragma unroll
        for (int d = n; d; d >>= 1)
#pragma unroll
          for (int i = d % n; i + d < VT; i += 2 * d)
#pragma unroll
            for (int j = 0; j < d; ++j)
              if (i + j + d < VT && (i + j) / (2 * n) == (i + j + d) / (2 * n)) {
                const uint32_t hi = max(key[i + j], key[i + j + d]);
                key[i + j + d] = min(key[i + j], key[i + j + d]);
                key[i + j] = hi;
              }
      for (int j = 0; j < p.k; ++j) {
        const uint32_t best = __reduce_max_sync(kAll, key[0]);
        if (!best) break;  // no expert left: the other places stay empty
        const int owner = __ffs(__ballot_sync(kAll, key[0] == best)) - 1;
        const int at = __shfl_sync(kAll, e0 + static_cast<int>(order & 15u), owner);
        if (lane == owner) {
          order >>= 4;
#pragma unroll
          for (int i = 0; i + 1 < VT; ++i) key[i] = key[i + 1];
          key[VT - 1] = 0u;
        }
        if (lane == j) chosen = at;
      }
    } else {
      uint32_t first = 0u;
#pragma unroll
      for (int i = 0; i < VT; ++i) first = max(first, key[i]);
      for (int j = 0; j < p.k; ++j) {
        const uint32_t best = __reduce_max_sync(kAll, first);
        if (!best) break;
        const int owner = __ffs(__ballot_sync(kAll, first == best)) - 1;
        int at = 0;
        if (lane == owner) {  // its first key of that value goes
          bool found = false;
          first = 0u;
#pragma unroll
          for (int i = 0; i < VT; ++i) {
            const bool hit = !found && key[i] == best;
            if (hit) {
              at = e0 + i;
              key[i] = 0u;
            }
            found |= hit;
            first = max(first, key[i]);
          }
        }
        at = __shfl_sync(kAll, at, owner);
        if (lane == j) chosen = at;
      }
    }
    if (chosen >= 0) weight = score_of(load_logit<DT>(p.logits, row + chosen));
    if (p.renormalize) {
      float sum = weight;
#pragma unroll
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
      weight = sum > 0.f ? __fdiv_rn(weight, sum) : 0.f;
    }
    weight *= p.scale;
  }
  if (lane < p.k) {
    p.weights[t * p.k + lane] = weight;
    p.experts[t * p.k + lane] = chosen;
  }
}

template <int DT, int VT>
cudaError_t launch_route_v(const RouteProblem& p) {
  const unsigned grid = static_cast<unsigned>((p.T + 3) / 4);
  constexpr int PER = DT == 1 ? 4 : 8;  // logits of 16 bytes
  if constexpr (VT % PER == 0) {
    if (p.E == 32 * VT && p.ld % PER == 0 && aligned(p.logits, 16)) {
      route_kernel<DT, VT, true><<<grid, 128, 0, p.stream>>>(p);
      return cudaGetLastError();
    }
  }
  route_kernel<DT, VT, false><<<grid, 128, 0, p.stream>>>(p);
  return cudaGetLastError();
}

template <int DT>
cudaError_t launch_route_dt(const RouteProblem& p) {
  const int V = (p.E + 31) / 32;
  if (V <= 1) return launch_route_v<DT, 1>(p);
  if (V <= 2) return launch_route_v<DT, 2>(p);
  if (V <= 4) return launch_route_v<DT, 4>(p);
  if (V <= 8) return launch_route_v<DT, 8>(p);
  if (V <= 16) return launch_route_v<DT, 16>(p);
  return launch_route_v<DT, 32>(p);
}

// ------------------------------------------------------------------------------- dispatch ----

// Every place (t, j) of the flat list of T k places gets one row: places sorted by expert, equal
// experts in flat order (a stable counting sort, so the rows do not depend on timing).  Places
// without an expert (an id outside [0, E)) sort behind all experts as bin E; their rows are zero.
constexpr int kSortThreads = 256;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortMinChunk = 1024;  // places per block
constexpr int kSortMaxBlocks = 128;

__host__ __device__ inline int64_t sort_chunk(int64_t R) {
  const int64_t c = (R + kSortMaxBlocks - 1) / kSortMaxBlocks;
  return c < kSortMinChunk ? kSortMinChunk : (c + kSortThreads - 1) / kSortThreads * kSortThreads;
}
inline int sort_blocks(int64_t R) { return static_cast<int>((R + sort_chunk(R) - 1) / sort_chunk(R)); }

__device__ __forceinline__ int bin_of(int id, int E) { return id >= 0 && id < E ? id : E; }

// Counts of a block's places per bin: hist[block][bin].
__global__ void __launch_bounds__(kSortThreads) dispatch_count_kernel(const DispatchProblem p, int* hist) {
  extern __shared__ int cnt[];
  const int64_t R = p.T * p.k, chunk = sort_chunk(R);
  const int64_t i0 = blockIdx.x * chunk, i1 = min(R, i0 + chunk);
  launch_dependents();
  for (int e = threadIdx.x; e <= p.E; e += kSortThreads) cnt[e] = 0;
  __syncthreads();
  for (int64_t i = i0 + threadIdx.x; i < i1; i += kSortThreads) atomicAdd(cnt + bin_of(__ldg(p.experts + i), p.E), 1);
  __syncthreads();
  int* mine = hist + static_cast<int64_t>(blockIdx.x) * (p.E + 1);
  for (int e = threadIdx.x; e <= p.E; e += kSortThreads) mine[e] = cnt[e];
}

// Rows of a block's places.  Warp w owns the w-th part of the block's places; cnt[w][bin] becomes
// the row of that warp's first place of the bin, and the warp hands rows out in flat order.
__global__ void __launch_bounds__(kSortThreads) dispatch_place_kernel(const DispatchProblem p, const int* hist, int blocks,
                                                                      int* dest) {
  extern __shared__ int cnt[];  // [kSortWarps][E + 1], then [E + 1] totals and [E + 1] of earlier blocks
  const int bins = p.E + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int* total = cnt + kSortWarps * bins;
  int* base = total + bins;
  const int64_t R = p.T * p.k, chunk = sort_chunk(R), part = chunk / kSortWarps;
  const int64_t w0 = blockIdx.x * chunk + warp * part, w1 = min(R, w0 + part);
  for (int e = threadIdx.x; e < (kSortWarps + 2) * bins; e += kSortThreads) cnt[e] = 0;
  __syncthreads();
  launch_dependents();
  for (int64_t i = w0 + lane; i < w1; i += 32) atomicAdd(cnt + warp * bins + bin_of(__ldg(p.experts + i), p.E), 1);
  __syncthreads();
  grid_dependency_wait();  // the counts of all blocks
  // each warp adds up every kSortWarps-th block's counts, 256 bins at a time in registers, so that some
  // thirty loads are in flight
  constexpr int kBins = 8;
  for (int e0 = 0; e0 < bins; e0 += 32 * kBins) {
    int before[kBins], all[kBins];  // a bin's places of earlier blocks, of all blocks
#pragma unroll
    for (int i = 0; i < kBins; ++i) before[i] = all[i] = 0;
#pragma unroll 4
    for (int b = warp; b < blocks; b += kSortWarps) {
      const int* counts = hist + static_cast<int64_t>(b) * bins + e0 + lane;
#pragma unroll
      for (int i = 0; i < kBins; ++i) {
        const int c = e0 + 32 * i + lane < bins ? __ldcg(counts + 32 * i) : 0;
        before[i] += b < static_cast<int>(blockIdx.x) ? c : 0;
        all[i] += c;
      }
    }
#pragma unroll
    for (int i = 0; i < kBins; ++i) {
      const int e = e0 + 32 * i + lane;
      if (e < bins) {
        if (before[i]) atomicAdd(base + e, before[i]);
        if (all[i]) atomicAdd(total + e, all[i]);
      }
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < bins; e += kSortThreads) {
    int before = base[e];
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = cnt[w * bins + e];
      cnt[w * bins + e] = before;
      before += c;
    }
  }
  __syncthreads();
  if (warp == 0) {  // exclusive sum of the totals: the experts' first rows
    int run = 0;
    for (int e0 = 0; e0 < bins; e0 += 32) {
      const int e = e0 + lane, c = e < bins ? total[e] : 0;
      int s = c;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(kAll, s, d);
        if (lane >= d) s += o;
      }
      if (e < bins) total[e] = run + s - c;
      run += __shfl_sync(kAll, s, 31);
    }
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int e = threadIdx.x; e < bins; e += kSortThreads) p.offsets[e] = total[e];
  }
  for (int64_t i0 = w0; i0 < w1; i0 += 32) {
    const int64_t i = i0 + lane;
    const bool in = i < w1;
    const int bin = in ? bin_of(__ldg(p.experts + i), p.E) : -1;
    const unsigned same = __match_any_sync(kAll, bin);
    if (in) {
      const int row = total[bin] + cnt[warp * bins + bin] + __popc(same & ((1u << lane) - 1u));
      dest[i] = bin < p.E ? row : ~row;  // complement: no expert, the row is zeroed
      p.rows[i] = bin < p.E ? row : -1;
    }
    __syncwarp();
    if (in && lane == __ffs(same) - 1) cnt[warp * bins + bin] += __popc(same);
    __syncwarp();
  }
}

// Copies a token's row to the rows of its places (zeros where a place has no expert); a token is read
// once.  Block (t, y): the y-th run of the row's vectors.  HBM-bound by the k rows written: 8192 tokens
// of 8 KB to 8 places each, 604 MB in 94 us (6.4 TB/s).
constexpr int kRowThreads = 128;

template <typename Vec>
__device__ __forceinline__ void copy_row(const DispatchProblem& p, int64_t t, const int* dest, int n) {
  for (uint32_t c = blockIdx.y * kRowThreads + threadIdx.x; c < static_cast<uint32_t>(n); c += gridDim.y * kRowThreads) {
    const Vec v = __ldg(reinterpret_cast<const Vec*>(p.x + t * p.ld) + c);
#pragma unroll 4
    for (int j = 0; j < p.k; ++j) {
      const int d = dest[j];
      // a place without an expert is marked by the complement of its row
      reinterpret_cast<Vec*>(p.routed + static_cast<int64_t>(d < 0 ? ~d : d) * p.W)[c] = d < 0 ? Vec{} : v;
    }
  }
}

template <typename Vec>
__global__ void __launch_bounds__(kRowThreads) dispatch_copy_kernel(const DispatchProblem p, const int* dest) {
  grid_dependency_wait();
  copy_row<Vec>(p, blockIdx.x, dest + static_cast<int64_t>(blockIdx.x) * p.k, p.W / static_cast<int>(sizeof(Vec) / 2));
}

// Few places: every block finds its token's rows by itself, by counting the places that sort before
// each of its own (lower bin, or the same bin earlier), and copies at once; the first block also
// writes the offsets.  One launch, no workspace.  T k compares per place, so for few places only: 3.2,
// 10.1 and 30.4 us for 256, 2048 and 4096 places of 8192-byte rows, against 12.0, 13.4 and 16.2 us for
// the sort's three launches.
constexpr int kFewPlaces = 2048;
constexpr int kFewK = 32;

template <typename Vec>
__global__ void __launch_bounds__(kRowThreads) dispatch_few_kernel(const DispatchProblem p) {
  __shared__ int place[kFewK];
  extern __shared__ int hist[];  // [E + 1], first block
  const int64_t t = blockIdx.x;
  const int R = static_cast<int>(p.T) * p.k, i0 = static_cast<int>(t) * p.k, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool writes_offsets = blockIdx.x == 0 && blockIdx.y == 0;
  // a warp takes every fourth place of the token
  for (int j = warp; j < p.k; j += kRowThreads / 32) {
    const int mine = bin_of(__ldg(p.experts + i0 + j), p.E);
    int before = 0;
    for (int i = lane; i < R; i += 32) {
      const int b = bin_of(__ldg(p.experts + i), p.E);
      before += b < mine || (b == mine && i < i0 + j);
    }
    before = __reduce_add_sync(kAll, before);
    if (lane == 0) place[j] = mine < p.E ? before : ~before;
    if (lane == 0 && blockIdx.y == 0) p.rows[i0 + j] = mine < p.E ? before : -1;
  }
  if (writes_offsets) {
    for (int e = threadIdx.x; e <= p.E; e += kRowThreads) hist[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < R; i += kRowThreads) atomicAdd(hist + bin_of(__ldg(p.experts + i), p.E), 1);
  }
  __syncthreads();
  copy_row<Vec>(p, t, place, p.W / static_cast<int>(sizeof(Vec) / 2));
  if (writes_offsets && warp == 0) {
    int run = 0;
    for (int e0 = 0; e0 <= p.E; e0 += 32) {
      const int e = e0 + lane, c = e <= p.E ? hist[e] : 0;
      int s = c;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(kAll, s, d);
        if (lane >= d) s += o;
      }
      if (e <= p.E) p.offsets[e] = run + s - c;
      run += __shfl_sync(kAll, s, 31);
    }
  }
}

// -------------------------------------------------------------------------------- combine ----

// Block (t, y): the y-th run of token t's columns.  A thread owns one vector of eight (kVec) columns
// or one column and has up to eight rows' loads in flight; sums run in the order of the places.
// HBM-bound by the rows read: 8192 tokens of 8 places each, rows of 8 KB, 578 MB in 86 us (6.7 TB/s).
template <bool kBF, bool kVec>
__global__ void __launch_bounds__(kRowThreads) combine_kernel(const CombineProblem p) {
  constexpr int PER = kVec ? 8 : 1, BATCH = 8;
  const int64_t t = blockIdx.x;
  for (uint32_t c = (blockIdx.y * kRowThreads + threadIdx.x) * PER; c < static_cast<uint32_t>(p.W); c += gridDim.y * kRowThreads * PER) {
    float acc[PER];
    const auto load = [&](const uint16_t* src, uint32_t (&v)[4]) {
      if constexpr (kVec) *reinterpret_cast<uint4*>(v) = __ldg(reinterpret_cast<const uint4*>(src));
      else v[0] = __ldg(src);
    };
    const auto value = [](const uint32_t (&v)[4], int i) {
      if constexpr (kVec) {
        const float2 f = pair_to_float2<kBF>(v[i >> 1]);
        return i & 1 ? f.y : f.x;
      } else {
        return elem_to_float<kBF>(static_cast<uint16_t>(v[0]));
      }
    };
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = 0.f;
    if (p.base) {
      uint32_t v[4];
      if constexpr (kVec) *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(p.base + t * p.W + c);  // out may be base
      else v[0] = p.base[t * p.W + c];
#pragma unroll
      for (int i = 0; i < PER; ++i) acc[i] = value(v, i);
    }
    for (int j0 = 0; j0 < p.k; j0 += BATCH) {
      uint32_t v[BATCH][4];
      float w[BATCH];
#pragma unroll
      for (int u = 0; u < BATCH; ++u) {
        w[u] = 0.f;
        v[u][0] = v[u][1] = v[u][2] = v[u][3] = 0u;
        if (j0 + u < p.k) {
          const int r = __ldg(p.rows + t * p.k + j0 + u);
          if (r >= 0 && r < p.R) {
            w[u] = __ldg(p.weights + t * p.k + j0 + u);
            load(p.y + static_cast<int64_t>(r) * p.W + c, v[u]);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < BATCH; ++u) {
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] += w[u] * value(v[u], i);
      }
    }
    if constexpr (kVec) {
      uint32_t v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = static_cast<uint32_t>(float_to_elem<kBF>(acc[2 * i])) | (static_cast<uint32_t>(float_to_elem<kBF>(acc[2 * i + 1])) << 16);
      *reinterpret_cast<uint4*>(p.out + t * p.W + c) = *reinterpret_cast<const uint4*>(v);
    } else {
      p.out[t * p.W + c] = float_to_elem<kBF>(acc[0]);
    }
  }
}

// Column runs of a row, one block each; beyond the most that a grid's second dimension takes, a block takes
// several.
unsigned runs(int64_t vectors) {
  const int64_t n = (vectors + kRowThreads - 1) / kRowThreads;
  return static_cast<unsigned>(n < 1 ? 1 : n < 65535 ? n : 65535);
}

// A launch that may be set up while the kernel before it on the stream still runs; the kernel waits
// for that one's results itself.
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename Vec>
cudaError_t run_dispatch(const DispatchProblem& p) {
  const int64_t R = p.T * p.k, vectors = p.W / static_cast<int>(sizeof(Vec) / 2);
  const dim3 rows(static_cast<unsigned>(p.T), runs(vectors));
  if (R <= kFewPlaces && p.k <= kFewK) {
    dispatch_few_kernel<Vec><<<rows, kRowThreads, (p.E + 1) * 4, p.stream>>>(p);
    return cudaGetLastError();
  }
  const int bins = p.E + 1, blocks = sort_blocks(R);
  int* dest = static_cast<int*>(p.workspace);
  int* hist = dest + R;
  const int smem = (kSortWarps + 2) * bins * 4;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(dispatch_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  dispatch_count_kernel<<<blocks, kSortThreads, bins * 4, p.stream>>>(p, hist);
  cudaError_t e = launch_early(dispatch_place_kernel, dim3(blocks), kSortThreads, smem, p.stream, p, hist, blocks, dest);
  if (e == cudaSuccess) e = launch_early(dispatch_copy_kernel<Vec>, rows, kRowThreads, 0, p.stream, p, dest);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

cudaError_t launch_route(const RouteProblem& p) {
  switch (p.dtype) {
    case 0: return launch_route_dt<0>(p);
    case 1: return launch_route_dt<1>(p);
    default: return launch_route_dt<2>(p);
  }
}

size_t dispatch_workspace_bytes(int64_t R, int E) {
  return static_cast<size_t>(sort_blocks(R)) * (E + 1) * 4 + static_cast<size_t>(R) * 4;
}

cudaError_t launch_dispatch(const DispatchProblem& p) {
  if (p.W % 8 == 0 && p.ld % 8 == 0 && aligned(p.x, 16) && aligned(p.routed, 16)) return run_dispatch<uint4>(p);
  return run_dispatch<uint16_t>(p);
}

cudaError_t launch_combine(const CombineProblem& p) {
  const bool vec = p.W % 8 == 0 && aligned(p.y, 16) && aligned(p.out, 16) && aligned(p.base, 16);
  const dim3 grid(static_cast<unsigned>(p.T), runs(vec ? p.W / 8 : p.W));
  if (vec) {
    if (p.bf16) combine_kernel<true, true><<<grid, kRowThreads, 0, p.stream>>>(p);
    else combine_kernel<false, true><<<grid, kRowThreads, 0, p.stream>>>(p);
  } else {
    if (p.bf16) combine_kernel<true, false><<<grid, kRowThreads, 0, p.stream>>>(p);
    else combine_kernel<false, false><<<grid, kRowThreads, 0, p.stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace awq
