// Around the grouped (mixture-of-experts) linears: routing of tokens to experts, the sort of the
// routed rows by expert (dispatch) and the weighted sum of a token's rows (combine).
#include "awq_layer.cuh"
#include "awq_ptx.cuh"

namespace awq {
namespace {

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

// One warp per token.  Lane l holds experts [l V, l V + V), V = ceil(E / 32) <= VT, so that the
// lowest lane and the lowest register of the equal keys is the lowest expert.
template <int DT, int VT>
__global__ void __launch_bounds__(128) route_kernel(const RouteProblem p) {
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const int V = (p.E + 31) / 32;
  const int e0 = lane * V;
  const int64_t row = t * p.ld;
  float x[VT];
#pragma unroll
  for (int i = 0; i < VT; ++i) x[i] = i < V && e0 + i < p.E ? load_logit<DT>(p.logits, row + e0 + i) : -INFINITY;

  // scores; an expert whose logit is -inf is out
  float score[VT];
  bool bad = false;
  if (p.sigmoid) {
#pragma unroll
    for (int i = 0; i < VT; ++i) score[i] = __fdiv_rn(1.f, 1.f + expf(-x[i]));
  } else {
    float top = -INFINITY;
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
#pragma unroll
    for (int i = 0; i < VT; ++i) score[i] = __fdiv_rn(score[i], sum);
  }
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
    uint32_t mine = 0u;  // lane g: group g's score
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
    uint32_t kept = 0u;
    for (int j = 0; j < p.topk_groups; ++j) {
      const uint32_t best = __reduce_max_sync(kAll, mine);
      if (!best) break;
      const int owner = __ffs(__ballot_sync(kAll, mine == best)) - 1;
      kept |= 1u << owner;
      if (lane == owner) mine = 0u;
    }
#pragma unroll
    for (int i = 0; i < VT; ++i) {
      const int e = e0 + i;
      if (i < V && e < p.E && !((kept >> (e / per)) & 1u)) key[i] = 0u;
    }
  }

  int chosen = -1;  // lane j: place j
  float weight = 0.f;
  if (bad) {
    chosen = lane;
    weight = __int_as_float(0x7fffffff);
  } else {
    for (int j = 0; j < p.k; ++j) {
      uint32_t first = 0u;
#pragma unroll
      for (int i = 0; i < VT; ++i) first = max(first, key[i]);
      const uint32_t best = __reduce_max_sync(kAll, first);
      if (!best) break;  // no expert left: the other places stay empty
      const int owner = __ffs(__ballot_sync(kAll, first == best)) - 1;
      int at = 0;
      float s = 0.f;
#pragma unroll
      for (int i = VT - 1; i >= 0; --i) {
        if (key[i] == best) {
          at = i;
          s = score[i];
        }
      }
      if (lane == owner) {
#pragma unroll
        for (int i = 0; i < VT; ++i) {
          if (i == at) key[i] = 0u;
        }
      }
      at = __shfl_sync(kAll, e0 + at, owner);
      s = __shfl_sync(kAll, s, owner);
      if (lane == j) {
        chosen = at;
        weight = s;
      }
    }
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

template <int DT>
cudaError_t launch_route_dt(const RouteProblem& p) {
  const unsigned grid = static_cast<unsigned>((p.T + 3) / 4);
  const int V = (p.E + 31) / 32;
  if (V <= 1) route_kernel<DT, 1><<<grid, 128, 0, p.stream>>>(p);
  else if (V <= 2) route_kernel<DT, 2><<<grid, 128, 0, p.stream>>>(p);
  else if (V <= 4) route_kernel<DT, 4><<<grid, 128, 0, p.stream>>>(p);
  else if (V <= 8) route_kernel<DT, 8><<<grid, 128, 0, p.stream>>>(p);
  else if (V <= 16) route_kernel<DT, 16><<<grid, 128, 0, p.stream>>>(p);
  else route_kernel<DT, 32><<<grid, 128, 0, p.stream>>>(p);
  return cudaGetLastError();
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
  extern __shared__ int cnt[];  // [kSortWarps][E + 1], then [E + 1] totals
  const int bins = p.E + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int* total = cnt + kSortWarps * bins;
  const int64_t R = p.T * p.k, chunk = sort_chunk(R), part = chunk / kSortWarps;
  const int64_t w0 = blockIdx.x * chunk + warp * part, w1 = min(R, w0 + part);
  for (int e = threadIdx.x; e < kSortWarps * bins; e += kSortThreads) cnt[e] = 0;
  __syncthreads();
  for (int64_t i = w0 + lane; i < w1; i += 32) atomicAdd(cnt + warp * bins + bin_of(__ldg(p.experts + i), p.E), 1);
  __syncthreads();
  for (int e = threadIdx.x; e < bins; e += kSortThreads) {
    int before = 0, all = 0;  // this bin's places of earlier blocks, of all blocks
    for (int b = 0; b < blocks; ++b) {
      const int c = __ldg(hist + static_cast<int64_t>(b) * bins + e);
      before += b < static_cast<int>(blockIdx.x) ? c : 0;
      all += c;
    }
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = cnt[w * bins + e];
      cnt[w * bins + e] = before;
      before += c;
    }
    total[e] = all;
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
      dest[i] = row;
      p.rows[i] = bin < p.E ? row : -1;
    }
    __syncwarp();
    if (in && lane == __ffs(same) - 1) cnt[warp * bins + bin] += __popc(same);
    __syncwarp();
  }
}

// Copies a token's row to the rows of its places; a token is read once.
template <typename Vec>
__global__ void __launch_bounds__(256) dispatch_copy_kernel(const DispatchProblem p, const int* dest) {
  constexpr int kPer = sizeof(Vec) / 2;
  const int64_t t = blockIdx.x;
  const int n = p.W / kPer;
  const Vec* src = reinterpret_cast<const Vec*>(p.x + t * p.ld);
  for (int c = threadIdx.x; c < n; c += 256) {
    const Vec v = __ldg(src + c);
    for (int j = 0; j < p.k; ++j) {
      const int64_t i = t * p.k + j;
      const int id = __ldg(p.experts + i);
      reinterpret_cast<Vec*>(p.routed + static_cast<int64_t>(__ldg(dest + i)) * p.W)[c] = id >= 0 && id < p.E ? v : Vec{};
    }
  }
}

// -------------------------------------------------------------------------------- combine ----

template <bool kBF>
__global__ void __launch_bounds__(256) combine_any_kernel(const CombineProblem p) {
  const int64_t t = blockIdx.x;
  for (int c = threadIdx.x; c < p.W; c += 256) {
    float a = p.base ? elem_to_float<kBF>(p.base[t * p.W + c]) : 0.f;
    for (int j = 0; j < p.k; ++j) {
      const int r = __ldg(p.rows + t * p.k + j);
      if (r >= 0 && r < p.R) a += __ldg(p.weights + t * p.k + j) * elem_to_float<kBF>(__ldg(p.y + static_cast<int64_t>(r) * p.W + c));
    }
    p.out[t * p.W + c] = float_to_elem<kBF>(a);
  }
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
  const int64_t R = p.T * p.k;
  const int bins = p.E + 1, blocks = sort_blocks(R);
  int* dest = static_cast<int*>(p.workspace);
  int* hist = dest + R;
  const int smem = (kSortWarps + 1) * bins * 4;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(dispatch_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  dispatch_count_kernel<<<blocks, kSortThreads, bins * 4, p.stream>>>(p, hist);
  dispatch_place_kernel<<<blocks, kSortThreads, smem, p.stream>>>(p, hist, blocks, dest);
  if (p.W % 8 == 0 && p.ld % 8 == 0 && aligned(p.x, 16) && aligned(p.routed, 16))
    dispatch_copy_kernel<uint4><<<static_cast<unsigned>(p.T), 256, 0, p.stream>>>(p, dest);
  else
    dispatch_copy_kernel<uint16_t><<<static_cast<unsigned>(p.T), 256, 0, p.stream>>>(p, dest);
  return cudaGetLastError();
}

cudaError_t launch_combine(const CombineProblem& p) {
  if (p.bf16) combine_any_kernel<true><<<static_cast<unsigned>(p.T), 256, 0, p.stream>>>(p);
  else combine_any_kernel<false><<<static_cast<unsigned>(p.T), 256, 0, p.stream>>>(p);
  return cudaGetLastError();
}

}  // namespace awq
