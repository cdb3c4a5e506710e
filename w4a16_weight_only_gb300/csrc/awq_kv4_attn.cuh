// Attention of the newest tokens of each sequence over a 4-bit key/value cache (awq_attention_kv4): the
// kernels, instantiated per head size by awq_kv4_attn_*.cu.
//
//   out[r] = sum_j p_j v_j / sum_j p_j,   p_j = 2^(z_j - max z),   z_j = scale log2(e) q[r] . k_j
//
// with k_j = s c + m per group of elements (codes c, scale s, minimum m), and v_j alike, so that
//
//   q . k_j = sum_g s_g (q_g . c_g) + m_g sum(q_g),    sum_j p_j v_j = sum_j (p_j s_j) (c_j - 8) + sum_j p_j (m_j + 8 s_j)
//
// and the codes themselves go to the tensor cores.  Some 400 instructions for a tile of 16 keys of a head of 128, most of
// them the codes' extraction, the softmax and the parameters.  No unit is full: 16 warps an SM, whose 128 registers spill
// 32 to 180 bytes, issue in 56 % of the schedulers' cycles, HBM is at 43 %, the tensor pipe at 18 % (counters of 32
// sequences); a warp waits for its own chain of words, first product, vote, exponentials and second product.  128
// sequences of up to 8197, 8 heads, 765 MB in 179 us, 4.3 TB/s.  A word of codes ANDed with 0x000f000f is a pair of fp16
// subnormals c 2^-24, with 0x00f000f0 a pair c 2^-20: an operand register of keys costs one logic operation, and
// every second one a shift; of values, ORed with 1024 and less 1032 (1024 + 128), one addition more.  The two kinds have
// accumulators of their own, scaled back at the end.
// Queries are fp16 for either element type (a bf16 row is scaled by a power of two first: exact down to 2^-18 of its
// largest element, in steps of 2^-28 below), p s is one fp16 number (fp16 elements: two) in a unit of its row and group.
#pragma once

#include <type_traits>

#include "awq_step.cuh"
#include "awq_attn.cuh"

namespace awq {
namespace kv4 {

using attn::exp2_approx;
using attn::kRaise;

constexpr int kWarps = 8;
constexpr int kTileKeys = 16;
constexpr int kCoarse = kWarps * 32;  // entries of a block's table of lengths, one per thread
constexpr unsigned int kStatusKv4Timeout = 0x10u;

constexpr int least(int a, int b) { return a < b ? a : b; }
constexpr int most(int a, int b) { return a > b ? a : b; }

// Blocks per SM of heads of D elements and 8 nt query rows: two, or one with twice the registers (16 rows of 64
// elements at two blocks spill: 16 x 4 over 2047 40 us, 34 at one).
__host__ __device__ constexpr int blocks_per_sm(int D, int nt) { return D <= 128 && nt == 1 ? 2 : 1; }

// Head size D, G groups of elements per head, 8 NT query rows.
template <int D, int G, int NT>
struct Shape {
  static constexpr int U = D / 32;                          // words of codes of a lane per key, and per pair of values
  static constexpr int PANELS = (D + 127) / 128, W = U / PANELS;
  static constexpr int TILE = 16 * (D + 8 * G);             // bytes
  static constexpr int ROWS = 8 * NT;
  static constexpr int PART = ROWS * (D + 2) * 4;           // bytes of a partial result: sums, then (max, sum of p)
  static constexpr int BLOCKS = blocks_per_sm(D, NT);
  // Two blocks per SM leave 128 registers: the queries' fragments are read from shared memory for every tile.
  static constexpr bool Q_SHARED = BLOCKS == 2;
  static constexpr int QUERIES = Q_SHARED ? NT * U * 512 : 0;  // bytes of a warp
  static constexpr int STAGES = least(8, (((228 / BLOCKS - 1) * 1024 - 4096) / kWarps - QUERIES) / TILE);
  static constexpr int RING = (most(STAGES * TILE, PART) + 127) / 128 * 128;  // of a warp
  static constexpr int QS = kWarps * RING;                  // offset of the queries
  static constexpr int BARS = QS + kWarps * QUERIES;        // of the barriers
  static constexpr int SMEM = BARS + kWarps * STAGES * 8;
  static_assert(STAGES >= 3 && SMEM + 4096 <= (228 / BLOCKS - 1) * 1024, "shared memory");
};

// How a call is cut.  A lane is a (key/value head, tile of query rows); a unit is a (lane, sequence) and
// has as many tiles of 16 keys as its rows see (Range).  All tiles of all units, lane by lane, sequence by
// sequence, form one line, of which warp w (of all) takes [w per, (w + 1) per); per is found on the device,
// where the lengths are.  A run is what a warp has of a unit.  A run that is a whole unit is written out at
// once; the others are joined, those of a block in the block, and a unit of several blocks by the join
// kernel: a block's part of a unit that goes on behind the block is at part 2 block + 1, of one that ends
// in it at 2 block.  Where the sequences' tables or windows are short and there are few units, a block takes
// one unit, and there is neither line nor join.
struct Args {
  AttentionKv4Problem p;
  int group;      // query heads per key/value head
  int row_tiles;  // of a sequence and key/value head
  int tiles_per_page;
  bool aligned;   // a unit per block instead: no line, nothing to join between blocks
  float* parts;   // [2 blocks] of PART bytes
  float* firsts;  // [blocks][warps] of PART bytes: a warp's first run, where others follow
  int64_t* line;  // per, then the sequences' first tiles (within a lane) and their number, [B + 1]
  unsigned int* status;
};

struct Range {
  int len;    // keys
  int sinks;  // tiles in front of the window's
  int first;  // the window's first tile
  int count;
  __device__ __forceinline__ int tile(int i) const { return i < sinks ? i : first + i - sinks; }
};

__device__ __forceinline__ Range range_of(const AttentionKv4Problem& p, int b) {
  Range r;
  const int64_t most_keys = static_cast<int64_t>(p.W) * p.cache.page_size;  // below 2^31
  r.len = static_cast<int>(min(static_cast<int64_t>(max(__ldg(p.lens + b), 0)), most_keys));
  r.sinks = r.first = 0;
  if (p.window > 0) {
    const int64_t low = static_cast<int64_t>(r.len) - p.n - p.window + 1;  // first key in the window of the first new token
    r.first = static_cast<int>(max(low, int64_t{0})) / kTileKeys;
    const int sink_tiles = static_cast<int>((static_cast<int64_t>(min(p.sinks, r.len)) + kTileKeys - 1) / kTileKeys);
    r.sinks = min(sink_tiles, r.first);
  }
  r.count = r.len == 0 ? 0 : r.sinks + (r.len - 1) / kTileKeys + 1 - r.first;
  return r;
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(ptx::smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(ptx::smem_u32(bar))
               : "memory");
}

// An 8 x 8 tile of 16-bit elements, one row per four lanes, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Two products, and two products with sums, in one instruction each.
__device__ __forceinline__ void mul2(float (&d)[2], float a0, float a1, float b0, float b1) {
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d[0]), "=f"(d[1])
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void fma2(float (&d)[2], float a0, float a1, float b0, float b1) {
  asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%0, %1};\n\t"
      "fma.rn.f32x2 c, a, b, c;\n\tmov.b64 {%0, %1}, c;\n\t}"
      : "+f"(d[0]), "+f"(d[1])
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fffffff); }

constexpr float kTwo24 = 16777216.f, kTwo20 = 1048576.f;

// A probability is kept as p = 2^(z - top), top a whole number that is raised only when a logit exceeds it by kRaise; the
// factor of a key's codes, p times its scale, as an fp16 number in units of 2^e, e a whole number for each query row
// and group of elements, raised only when a factor reaches 2^kFactorEnd, to where the largest is in 2^kFactorLog ..
// 2^(kFactorLog + 1).  Both change for those rows and groups alone whose own keys ask for it: neither a key that a row
// does not see nor one of no weight takes bits from the others.  64 over 8197, 64 / 8 heads of 128, groups of 32: 141 us,
// 149 us where one group's values are 2^-6 of another's or less (some 60 more if the bound alone decided, 5 more for all if
// each tile were looked at group by group); with one unit for all rows and groups 8 us less, and larger groups as now.
// fp16 numbers have their 11 bits down to 2^-14 and steps of 2^-24 below: 2^-21 and 2^-31 of a row's largest.  Units go
// from 2^-110 (values that small are near bf16's smallest number) to 2^126; 2^-e is kept as bf16, two groups to a word.
constexpr float kNoTop = -3.402823466e38f;
constexpr int kFactorLog = 7, kFactorEnd = 15;
constexpr float kLastFactor = kFactorEnd - 0.01f;  // its base-2 logarithm, by approximate ones
constexpr int kLeastUnit = -110, kMostUnit = 126;
constexpr uint32_t kLeastUnits = static_cast<uint32_t>(127 - kLeastUnit) << 23;

template <int G>
__device__ __forceinline__ float per_unit(const uint32_t* units, int group) {
  return __uint_as_float(G == 1 ? units[0] : group % 2 ? units[group / 2] << 16 : units[group / 2] & 0xffff0000u);
}
template <int G>
__device__ __forceinline__ int unit_log(const uint32_t* units, int group) {
  return 127 - static_cast<int>(__float_as_uint(per_unit<G>(units, group)) >> 23);
}

__device__ __forceinline__ float log2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^x for whole x up to 127, 0 where that is below the normal numbers.
__device__ __forceinline__ float whole_exp2(float x) {
  return x < -126.f ? 0.f : __uint_as_float(static_cast<uint32_t>(static_cast<int>(x) + 127) << 23);
}

// Codes of values count from 8.  Tensor cores cut off the last bits of a sum that they add to; a sum of codes that
// count from 0 grows with the keys, while results are small differences of it and of the minima's sum: 4 over 131072,
// fp16, had errors of 3.5 times the result's own rounding, all to one side (now: of its size; 115 -> 122 us, 128 over
// 8197 172 -> 179).  Sums started anew every four tiles, or every tile, had 2.2 and 2.1 times; a product with -8 ahead of
// the codes' instead of the subtraction 187 us for 128 over 8197, fp16 16 % more.
constexpr float kMiddle = 8.f;

__device__ __forceinline__ uint32_t from_middle(uint32_t words, bool high) {  // (c - 8) of the low nibbles, 16 (c - 8) of the high
  const uint32_t raw = ptx::and_or(words, high ? 0x00f000f0u : 0x000f000fu, 0x64006400u);
  const uint32_t middle = high ? 0xe480e480u : 0xe408e408u;  // -1152, -1032
  const __half2 h = __hadd2(*reinterpret_cast<const __half2*>(&raw), *reinterpret_cast<const __half2*>(&middle));
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Weight of a partial result (max m, sum l) against the maximum `top` of all.
__device__ __forceinline__ float weight(float m, float l, float top) { return l == 0.f ? 0.f : l * exp2_approx(m - top); }

template <bool kBF, int D, int G, int NT>
__global__ void __launch_bounds__(kWarps * 32, Shape<D, G, NT>::BLOCKS) attention_kernel(const __grid_constant__ Args a) {
  using S = Shape<D, G, NT>;
  // fp16 results show the rounding of p s (2.4 times the error of the result's own, 16 x 4 over 2047): it is taken
  // as two fp16 terms there.  bf16's own rounding hides it.
  constexpr int kTerms = kBF ? 1 : 2;
  constexpr int U = S::U, W = S::W, STAGES = S::STAGES, ROWS = S::ROWS, PER_GROUP = U / G;  // words of a group
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t coarse[kCoarse];
  __shared__ int64_t of_warp[kWarps];
  struct Entry {  // a unit to join in this block: from warp w on
    int valid, b, lane, last;  // last: its last warp here
    bool before, past;         // it begins before the block, goes on behind it
    bool in_first;             // its run in warp w is that warp's first of several
  };
  __shared__ Entry entries[kWarps][2];
  __shared__ bool several[kWarps];  // a warp's first run is followed by others: its part is in global memory
  const AttentionKv4Problem& p = a.p;
  const Kv4Cache& cache = p.cache;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;

  const int gran = (p.B + kCoarse - 2) / (kCoarse - 1);
  int64_t T = 0, total, per, X0;
  if (lane < 2) entries[warp][lane].valid = 0;
  if (lane == 2) several[warp] = false;
  if (a.aligned) {
    total = range_of(p, static_cast<int>(blockIdx.x % p.B)).count;
    per = max(int64_t{1}, (total + kWarps - 1) / kWarps);
    X0 = 0;
    __syncthreads();
  } else {
    // coarse[i]: tiles (of one lane) of the sequences before i * gran
    const int64_t b0 = static_cast<int64_t>(threadIdx.x) * gran, b1 = min(b0 + gran, static_cast<int64_t>(p.B));
    int64_t sum = 0;
    for (int64_t b = b0; b < b1; ++b) sum += range_of(p, static_cast<int>(b)).count;
    int64_t before = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, before, d);
      if (lane >= d) before += o;
    }
    if (lane == 31) of_warp[warp] = before;
    __syncthreads();
    before -= sum;
    for (int w = 0; w < warp; ++w) before += of_warp[w];
    coarse[threadIdx.x] = before;
    if (blockIdx.x == 0) {
      for (int64_t b = b0; b < b1; ++b) {
        a.line[1 + b] = before;
        before += range_of(p, static_cast<int>(b)).count;
      }
      if (threadIdx.x == kCoarse - 1) a.line[1 + p.B] = before;  // it has no sequences: (kCoarse - 1) gran >= B
    }
    __syncthreads();
    T = coarse[kCoarse - 1];
    total = T * (static_cast<int64_t>(cache.heads) * a.row_tiles);
    const int64_t warps = static_cast<int64_t>(gridDim.x) * kWarps;
    per = max(int64_t{1}, (total + warps - 1) / warps);
    if (blockIdx.x == 0 && threadIdx.x == 0) a.line[0] = per;
    X0 = static_cast<int64_t>(blockIdx.x) * kWarps * per;
  }
  ptx::launch_dependents();

  // sequences without keys: zeros
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (__ldg(p.lens + b) > 0 && p.W > 0) continue;
    const int64_t n = static_cast<int64_t>(p.n) * p.Hq * D / 8;
    uint4* dst = reinterpret_cast<uint4*>(p.out) + b * n;
    for (int64_t i = threadIdx.x; i < n; i += kWarps * 32) dst[i] = make_uint4(0u, 0u, 0u, 0u);
  }

  const int64_t X1 = min(total, X0 + kWarps * per);
  if (X0 >= total) return;
  const int64_t x0 = min(total, X0 + warp * per), x1 = min(total, x0 + per);

  uint8_t* ring = smem + warp * S::RING;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::BARS) + warp * STAGES;
  float* own_part = reinterpret_cast<float*>(ring);
  uint4* queries = reinterpret_cast<uint4*>(smem + S::QS + warp * S::QUERIES) + lane;  // [NT][U][32]
  const auto first_part = [&](int w) { return a.firsts + (static_cast<int64_t>(blockIdx.x) * kWarps + w) * (S::PART / 4); };

  if (x0 < x1) {
    if (lane == 0) {
      for (int s = 0; s < STAGES; ++s) ptx::mbar_init(&full[s], 1);
      ptx::fence_mbar_init();
    }
    __syncwarp();

    struct Cursor {
      int ln, b, at;  // lane, sequence, tile of the unit
      Range r;
    };
    Cursor cur;
    if (a.aligned) {
      cur.ln = static_cast<int>(blockIdx.x / p.B);
      cur.b = static_cast<int>(blockIdx.x - cur.ln * p.B);
      cur.at = static_cast<int>(x0);
      cur.r = range_of(p, cur.b);
    } else {  // the first tile's unit
      cur.ln = static_cast<int>(x0 / T);
      const int64_t rem = x0 - cur.ln * T;
      int lo = 0, hi = kCoarse - 1;  // coarse[lo] <= rem < coarse[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (coarse[mid] <= rem) lo = mid;
        else hi = mid;
      }
      int64_t before = coarse[lo];
      cur.b = 0;
      for (int b0 = lo * gran; b0 < p.B; b0 += 32) {  // 32 sequences at a time; rem lies below the last entry
        const int n = b0 + lane < p.B ? range_of(p, b0 + lane).count : 0;
        int64_t incl = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int64_t o = __shfl_up_sync(0xffffffffu, incl, d);
          if (lane >= d) incl += o;
        }
        const unsigned past = __ballot_sync(0xffffffffu, before + incl > rem);
        if (past) {
          const int l = __ffs(past) - 1;
          before += __shfl_sync(0xffffffffu, incl - n, l);
          cur.b = b0 + l;
          break;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
      }
      cur.r = range_of(p, cur.b);
      cur.at = static_cast<int>(rem - before);
    }
    const int lanes = cache.heads * a.row_tiles;
    const auto next_unit = [&](Cursor& c) {
      c.at = 0;
      do {
        if (++c.b == p.B) {
          c.b = 0;
          ++c.ln;
        }
        c.r = range_of(p, c.b);
      } while (c.r.count == 0 && c.ln < lanes);  // one has keys: the line is not at its end
    };

    // Copies run STAGES tiles ahead, across units.  Lane l holds where tile l of a batch of 32 begins, and
    // issues its copy; the next batch's pages are looked up half a batch earlier.
    Cursor ahead = cur;
    const int64_t tiles = x1 - x0;
    int64_t filled = 0;
    int page_of = -1;
    int64_t rest_of = 0;  // byte of the tile within the page
    const uint8_t* src = nullptr;
    const auto look_up = [&] {
      int n = 0;
      page_of = -1;
      while (n < 32 && filled < tiles) {
        const int take = static_cast<int>(min(static_cast<int64_t>(min(32 - n, ahead.r.count - ahead.at)), tiles - filled));
        if (lane >= n && lane < n + take) {
          const int tile = ahead.r.tile(ahead.at + lane - n), slot = tile / a.tiles_per_page;
          page_of = __ldg(p.pages + ahead.b * p.pages_ld + slot);
          rest_of = ahead.ln / a.row_tiles * cache.head_stride + static_cast<int64_t>(tile - slot * a.tiles_per_page) * S::TILE;
        }
        n += take;
        filled += take;
        ahead.at += take;
        if (ahead.at == ahead.r.count && filled < tiles) next_unit(ahead);
        if (take <= 0) break;
      }
    };
    const auto take_over = [&] {  // a page outside the cache: nothing is copied
      src = page_of >= 0 && page_of < cache.num_pages ? cache.data + page_of * cache.page_stride + rest_of : nullptr;
    };
    const auto issue = [&](int stage) {
      if (src) {
        ptx::mbar_arrive_expect_tx(&full[stage], S::TILE);
        bulk_load(ring + stage * S::TILE, src, S::TILE, &full[stage]);
      } else {
        ptx::mbar_arrive(&full[stage]);
      }
    };
    look_up();
    take_over();
    const int first_tiles = static_cast<int>(min(static_cast<int64_t>(STAGES), tiles));
    if (lane < first_tiles) issue(lane);
    __syncwarp();

    // The tile in a stage has arrived.  A bounded wait; the clock is read before the test that decides, so
    // that a pause between the two gives nothing up.
    const auto arrived = [&](int stage, uint32_t phase) -> bool {
      uint64_t* bar = &full[stage];
      const auto there = [&] { return __all_sync(0xffffffffu, ptx::mbar_try_wait(bar, phase)) != 0; };
      if (there()) return true;
      const uint64_t t0 = ptx::globaltimer_ns();
      while (true) {
        const bool late = __any_sync(0xffffffffu, ptx::globaltimer_ns() - t0 > attn::kWaitLimitNs);
        if (there()) return true;
        if (late) return false;
      }
    };

    bool gave_up = false;
    int64_t to_load = tiles - first_tiles;
    int in_flight = first_tiles;
    uint32_t next_load = first_tiles;  // its place in a batch: the low five bits
    int stage = 0;
    uint32_t phase = 0;
    for (int64_t x = x0; x < x1;) {
      // ---- one run ----
      const int hk = cur.ln / a.row_tiles, row0 = (cur.ln - hk * a.row_tiles) * ROWS, rows = p.n * a.group;
      const int len = cur.r.len, begin = cur.at;
      const int end = begin + static_cast<int>(min(static_cast<int64_t>(cur.r.count - begin), x1 - x));
      const int pos0 = len - p.n + row0 / a.group, pos1 = len - p.n + min(p.n - 1, (row0 + ROWS - 1) / a.group);
      // keys up to here are out of the window
      const int low0 = p.window > 0 ? static_cast<int>(max(static_cast<int64_t>(pos0) - p.window, int64_t{-1})) : -1;
      const int low1 = p.window > 0 ? static_cast<int>(max(static_cast<int64_t>(pos1) - p.window, int64_t{-1})) : -1;
      uint4 qf[S::Q_SHARED ? 1 : NT][S::Q_SHARED ? 1 : U];  // of a word: kind 0 (halves of the contraction), kind 1
      float qsum[NT][G][2];      // sums of the lane's two columns' queries over a group
      float zscale[NT][2];       // what takes a column's product to a base-2 logit
      int pos[NT][2];            // positions of the lane's two columns' tokens
#pragma unroll
      for (int m = 0; m < NT; ++m) {
        const int r = row0 + 8 * m + g, i = r / a.group;
        const uint16_t* src_q = p.q + cur.b * p.q_sb + i * p.q_sn + (hk * a.group + r - i * a.group) * p.q_sh + 8 * t;
        uint4 raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          raw[u] = r < rows ? __ldg(reinterpret_cast<const uint4*>(src_q + 32 * u)) : make_uint4(0u, 0u, 0u, 0u);
        float factor = 1.f, back = 1.f;
        if constexpr (kBF) {  // the row's largest element to 2^4 .. 2^5
          uint32_t top = 0;
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) top = max(top, max(w[j] & 0x7f80u, (w[j] >> 16) & 0x7f80u));
          }
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const int e = min(max(static_cast<int>(top >> 7), 8), 254);  // biased exponent
          factor = __uint_as_float(static_cast<uint32_t>(258 - e) << 23);
          back = __uint_as_float(static_cast<uint32_t>(e - 4) << 23);
        }
        float gs[G];
#pragma unroll
        for (int q = 0; q < G; ++q) gs[q] = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float2 e01 = ptx::pair_to_float2<kBF>(raw[u].x), e23 = ptx::pair_to_float2<kBF>(raw[u].y),
                       e45 = ptx::pair_to_float2<kBF>(raw[u].z), e67 = ptx::pair_to_float2<kBF>(raw[u].w);
          const float e[8] = {e01.x * factor, e01.y * factor, e23.x * factor, e23.y * factor,
                              e45.x * factor, e45.y * factor, e67.x * factor, e67.y * factor};
          const uint4 f = make_uint4(pack_half(e[0], e[4]), pack_half(e[2], e[6]), pack_half(e[1], e[5]), pack_half(e[3], e[7]));
          if constexpr (S::Q_SHARED) queries[(m * U + u) * 32] = f;  // a lane reads what it wrote
          else qf[m][u] = f;
          gs[u / PER_GROUP] += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
        }
#pragma unroll
        for (int q = 0; q < G; ++q) {
          gs[q] += __shfl_xor_sync(0xffffffffu, gs[q], 1);
          gs[q] += __shfl_xor_sync(0xffffffffu, gs[q], 2);
#pragma unroll
          for (int h = 0; h < 2; ++h) qsum[m][q][h] = __shfl_sync(0xffffffffu, gs[q], (2 * t + h) * 4);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          zscale[m][h] = __shfl_sync(0xffffffffu, back, (2 * t + h) * 4) * (p.scale * attn::kLog2e);
          pos[m][h] = len - p.n + min((row0 + 8 * m + 2 * t + h) / a.group, p.n - 1);
        }
      }
      float o[NT][U][2][4], top[NT][2], sum[NT][2], low[NT][G][2];  // low: sums of p times the values' code 8
      uint32_t units[NT][2][(G + 1) / 2];
      float least_unit[NT][2];  // of its groups, as e
#pragma unroll
      for (int m = 0; m < NT; ++m) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int c = 0; c < 2; ++c) o[m][u][c][0] = o[m][u][c][1] = o[m][u][c][2] = o[m][u][c][3] = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          top[m][h] = kNoTop;
#pragma unroll
          for (int w = 0; w < (G + 1) / 2; ++w) units[m][h][w] = G == 1 ? kLeastUnits : kLeastUnits | kLeastUnits >> 16;
          least_unit[m][h] = kLeastUnit;
          sum[m][h] = 0.f;
#pragma unroll
          for (int q = 0; q < G; ++q) low[m][q][h] = 0.f;
        }
      }

      for (int i = begin; i < end; ++i) {
        if (p.give_up || !arrived(stage, phase)) {
          gave_up = true;
          break;
        }
        const uint8_t* tile = ring + stage * S::TILE;
        const int k0 = cur.r.tile(i) * kTileKeys;
        // whether some row sees a key here, and whether all see all
        const bool any = k0 <= pos1 && (k0 + kTileKeys - 1 > low0 || k0 < p.sinks);
        const bool all = k0 + kTileKeys - 1 <= pos0 && (k0 > low1 || k0 + kTileKeys <= p.sinks);
        const auto body = [&](auto masked) {
          constexpr bool kMasked = decltype(masked)::value;
          uint32_t kw[2][U];  // keys g and g + 8
#pragma unroll
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int n = 0; n < S::PANELS; ++n) {
              const uint8_t* at = tile + n * 1024 + (g + 8 * half) * (16 * W) + t * (4 * W);
              if constexpr (W == 4) {
                *reinterpret_cast<uint4*>(&kw[half][n * W]) = *reinterpret_cast<const uint4*>(at);
              } else if constexpr (W == 2) {
                *reinterpret_cast<uint2*>(&kw[half][n * W]) = *reinterpret_cast<const uint2*>(at);
              } else {
#pragma unroll
                for (int w = 0; w < W; ++w) kw[half][n * W + w] = reinterpret_cast<const uint32_t*>(at)[w];
              }
            }
          // logits: z[m][half][h] of key g + 8 half and column 2 t + h
          const uint32_t* params = reinterpret_cast<const uint32_t*>(tile + 16 * D) + g * G;
          float z[NT][2][2];
#pragma unroll
          for (int m = 0; m < NT; ++m) z[m][0][0] = z[m][0][1] = z[m][1][0] = z[m][1][1] = 0.f;
#pragma unroll
          for (int q = 0; q < G; ++q) {
            float acc[NT][2][4];
#pragma unroll
            for (int w = q * PER_GROUP; w < (q + 1) * PER_GROUP; ++w) {
              const uint32_t x0w = kw[0][w], x1w = kw[1][w], y0w = x0w >> 8, y1w = x1w >> 8;
              uint4 f[NT];
#pragma unroll
              for (int m = 0; m < NT; ++m) {
                if constexpr (S::Q_SHARED) f[m] = queries[(m * U + w) * 32];
                else f[m] = qf[m][w];
              }
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const uint32_t mask = c ? 0x00f000f0u : 0x000f000fu;
                const uint32_t a0 = x0w & mask, a1 = x1w & mask, a2 = y0w & mask, a3 = y1w & mask;
#pragma unroll
                for (int m = 0; m < NT; ++m) {
                  const uint32_t b0 = c ? f[m].z : f[m].x, b1 = c ? f[m].w : f[m].y;
                  if (w == q * PER_GROUP) ptx::mma16816_zero(acc[m][c], a0, a1, a2, a3, b0, b1);
                  else ptx::mma16816(acc[m][c], a0, a1, a2, a3, b0, b1);
                }
              }
            }
            const float2 p0 = ptx::pair_to_float2<kBF>(params[q]), p1 = ptx::pair_to_float2<kBF>(params[8 * G + q]);
#pragma unroll
            for (int m = 0; m < NT; ++m)
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                const float2 sm = half ? p1 : p0;
                const float* a0 = acc[m][0] + 2 * half;
                const float* a1 = acc[m][1] + 2 * half;
                float both[2];
                mul2(both, a1[0], a1[1], kTwo20, kTwo20);
                fma2(both, a0[0], a0[1], kTwo24, kTwo24);
                fma2(z[m][half], both[0], both[1], sm.x, sm.x);
                fma2(z[m][half], qsum[m][q][0], qsum[m][q][1], sm.y, sm.y);
              }
          }
          uint32_t seen = 0xffffffffu;  // bit 4 m + 2 half + h
          if constexpr (kMasked) {
            seen = 0;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const int key = k0 + g + 8 * half;
#pragma unroll
              for (int m = 0; m < NT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  if (key <= pos[m][h] && (p.window == 0 || key > static_cast<int64_t>(pos[m][h]) - p.window || key < p.sinks))
                    seen |= 1u << (4 * m + 2 * half + h);
            }
          }
          float2 v[2][G];  // (scale, minimum) of the values
#pragma unroll
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int q = 0; q < G; ++q) v[half][q] = ptx::pair_to_float2<kBF>(params[16 * G + 8 * half * G + q]);
          float widest[2];  // of a key's scales, base-2 logarithm
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            widest[half] = v[half][0].x;
#pragma unroll
            for (int q = 1; q < G; ++q) widest[half] = fmaxf(widest[half], v[half][q].x);
            widest[half] = log2_approx(widest[half]);
          }
          bool raise = false;
#pragma unroll
          for (int m = 0; m < NT; ++m) {
            mul2(z[m][0], z[m][0][0], z[m][0][1], zscale[m][0], zscale[m][1]);
            mul2(z[m][1], z[m][1][0], z[m][1][1], zscale[m][0], zscale[m][1]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if constexpr (kMasked) {
#pragma unroll
                for (int half = 0; half < 2; ++half)
                  if (!((seen >> (4 * m + 2 * half + h)) & 1u)) z[m][half][h] = -INFINITY;
              }
              raise |= fmaxf(z[m][0][h], z[m][1][h]) - top[m][h] > kRaise;
              // a key's largest factor, of several groups at most; fmaxf leaves out the NaN of a masked key
              raise |= fmaxf(z[m][0][h] + widest[0], z[m][1][h] + widest[1]) - top[m][h] - least_unit[m][h] > kLastFactor;
            }
          }
          raise = __any_sync(0xffffffffu, raise);
          if constexpr (G > 1) {
            if (raise) {  // group by group: where one's values are 2^-6 of another's, that bound says yes for every tile
              raise = false;
#pragma unroll
              for (int m = 0; m < NT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  raise |= fmaxf(z[m][0][h], z[m][1][h]) - top[m][h] > kRaise;
                  float scaled[2] = {0.f, 0.f};
#pragma unroll
                  for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int q = 0; q < G; ++q) scaled[half] = fmaxf(scaled[half], per_unit<G>(units[m][h], q) * v[half][q].x);
                  raise |= fmaxf(z[m][0][h] + log2_approx(scaled[0]), z[m][1][h] + log2_approx(scaled[1])) - top[m][h] > kLastFactor;
                }
              raise = __any_sync(0xffffffffu, raise);
            }
          }
          if (raise) {
#pragma unroll
            for (int m = 0; m < NT; ++m)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float now = fmaxf(z[m][0][h], z[m][1][h]);
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, d));
                const float to = now - top[m][h] > kRaise ? ceilf(now) : top[m][h];
                const float down = top[m][h] - to, shrink = whole_exp2(down);
                top[m][h] = to;
                sum[m][h] *= shrink;
                const float p[2] = {exp2_approx(z[m][0][h] - to), exp2_approx(z[m][1][h] - to)};
                uint32_t kept[(G + 1) / 2] = {};
                float least = kMostUnit;
#pragma unroll
                for (int q = 0; q < G; ++q) {
                  low[m][q][h] *= shrink;
                  float wide = fmaxf(fmaxf(p[0] * v[0][q].x, p[1] * v[1][q].x), 0.f);
#pragma unroll
                  for (int d = 4; d < 32; d <<= 1) wide = fmaxf(wide, __shfl_xor_sync(0xffffffffu, wide, d));
                  const int log = static_cast<int>(__float_as_uint(wide) >> 23) - 127;
                  const float was = static_cast<float>(unit_log<G>(units[m][h], q)), moved = was + down;  // the same factors' unit
                  float unit = log - moved >= kFactorEnd ? static_cast<float>(log - kFactorLog) : moved;
                  unit = fminf(fmaxf(unit, static_cast<float>(kLeastUnit)), static_cast<float>(kMostUnit));
                  kept[q / 2] |= static_cast<uint32_t>(127 - static_cast<int>(unit)) << (q % 2 ? 7 : 23);
                  least = fminf(least, unit);
                  const float change = whole_exp2(moved - unit);
#pragma unroll
                  for (int u = q * PER_GROUP; u < (q + 1) * PER_GROUP; ++u)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                      o[m][u][c][h] *= change;
                      o[m][u][c][2 + h] *= change;
                    }
                }
#pragma unroll
                for (int w = 0; w < (G + 1) / 2; ++w) units[m][h][w] = kept[w];
                least_unit[m][h] = least;
              }
          }
#pragma unroll
          for (int m = 0; m < NT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              z[m][0][h] = exp2_approx(z[m][0][h] - top[m][h]);
              z[m][1][h] = exp2_approx(z[m][1][h] - top[m][h]);
              sum[m][h] += z[m][0][h] + z[m][1][h];
            }
          uint32_t vw[U][2];  // word, half of the keys
#pragma unroll
          for (int n = 0; n < U / 2; ++n) {
            const uint4 x4 = *reinterpret_cast<const uint4*>(tile + 8 * D + n * 512 + lane * 16);
            vw[2 * n][0] = x4.x;
            vw[2 * n][1] = x4.y;
            vw[2 * n + 1][0] = x4.z;
            vw[2 * n + 1][1] = x4.w;
          }
          if constexpr (U % 2) {
            const uint2 x2 = *reinterpret_cast<const uint2*>(tile + 8 * D + U / 2 * 512 + lane * 8);
            vw[U - 1][0] = x2.x;
            vw[U - 1][1] = x2.y;
          }
#pragma unroll
          for (int q = 0; q < G; ++q) {
            uint32_t pf[kTerms][NT][2];
#pragma unroll
            for (int m = 0; m < NT; ++m)
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                const float s = v[half][q].x, mn = v[half][q].y + kMiddle * s;
                float ps[2];
                mul2(ps, z[m][half][0], z[m][half][1], per_unit<G>(units[m][0], q), per_unit<G>(units[m][1], q));
                mul2(ps, ps[0], ps[1], s, s);
                if constexpr (kMasked) {  // zero times a value that is not finite
                  float pm[2] = {z[m][half][0] * mn, z[m][half][1] * mn};
#pragma unroll
                  for (int h = 0; h < 2; ++h)
                    if (!((seen >> (4 * m + 2 * half + h)) & 1u)) ps[h] = pm[h] = 0.f;
                  low[m][q][0] += pm[0];
                  low[m][q][1] += pm[1];
                } else {
                  fma2(low[m][q], z[m][half][0], z[m][half][1], mn, mn);
                }
                const uint32_t rounded = pack_half(ps[0], ps[1]);
                // P^T has keys along the lanes' rows; the second product wants them along the registers
                pf[0][m][half] = transpose8(rounded);
                if constexpr (kTerms == 2) {
                  const float2 kept = __half22float2(*reinterpret_cast<const __half2*>(&rounded));
                  pf[1][m][half] = transpose8(pack_half(ps[0] - kept.x, ps[1] - kept.y));
                }
              }
#pragma unroll
            for (int u = q * PER_GROUP; u < (q + 1) * PER_GROUP; ++u) {
              const uint32_t x0w = vw[u][0], x1w = vw[u][1], y0w = x0w >> 8, y1w = x1w >> 8;
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const uint32_t a0 = from_middle(x0w, c), a1 = from_middle(y0w, c), a2 = from_middle(x1w, c), a3 = from_middle(y1w, c);
#pragma unroll
                for (int m = 0; m < NT; ++m)
#pragma unroll
                  for (int k = 0; k < kTerms; ++k) ptx::mma16816(o[m][u][c], a0, a1, a2, a3, pf[k][m][0], pf[k][m][1]);
              }
            }
          }
        };
        if (all) body(std::false_type{});
        else if (any) body(std::true_type{});
        __syncwarp();  // the stage has been read
        if (to_load > 0) {
          const uint32_t owner = next_load & 31u;
          if (owner == 16) look_up();
          if (owner == 0) take_over();
          if (lane == static_cast<int>(owner)) issue(stage);
          --to_load;
          ++next_load;
        } else {
          --in_flight;
        }
        __syncwarp();
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (gave_up) break;

      // ---- the run's end ----
      const bool whole = begin == 0 && end == cur.r.count;
      const int64_t next = x + (end - begin);
      float* to = x > x0 || next == x1 ? own_part : first_part(warp);
#pragma unroll
      for (int m = 0; m < NT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float l = sum[m][h], lows[G];
#pragma unroll
          for (int q = 0; q < G; ++q) lows[q] = low[m][q][h];
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) {
            l += __shfl_xor_sync(0xffffffffu, l, d);
#pragma unroll
            for (int q = 0; q < G; ++q) lows[q] += __shfl_xor_sync(0xffffffffu, lows[q], d);
          }
          const int in_tile = 8 * m + 2 * t + h, r = row0 + in_tile;
          // a part holds quotients, so that nothing overflows; a whole row without weight is zero where it sees
          // no key and NaN where all its logits are -inf
          const float inv = l != 0.f ? 1.f / l : whole && pos[m][h] >= 0 ? quiet_nan() : 0.f;
          const int i = min(r, rows - 1) / a.group;
          uint16_t* out = p.out + ((static_cast<int64_t>(cur.b) * p.n + i) * p.Hq + hk * a.group + (r - i * a.group)) * D;
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const float lo = inv, hi = inv * 0.0625f, mn = lows[u / PER_GROUP] * inv;
            const float unit = __uint_as_float(static_cast<uint32_t>(127 + unit_log<G>(units[m][h], u / PER_GROUP)) << 23);
            const float e[4] = {o[m][u][0][h] * lo * unit + mn, o[m][u][1][h] * hi * unit + mn, o[m][u][0][2 + h] * lo * unit + mn,
                                o[m][u][1][2 + h] * hi * unit + mn};
            if (!whole) {
              *reinterpret_cast<float4*>(to + in_tile * D + 32 * u + 4 * g) = make_float4(e[0], e[1], e[2], e[3]);
            } else if (r < rows) {
              uint2 w;
              w.x = attn::pack2<kBF>(e[0], e[1]);
              w.y = attn::pack2<kBF>(e[2], e[3]);
              *reinterpret_cast<uint2*>(out + 32 * u + 4 * g) = w;
            }
          }
          if (!whole && g == 0)
            *reinterpret_cast<float2*>(to + ROWS * D + 2 * in_tile) = make_float2(top[m][h], l);
        }
      if (!whole && lane == 0) {
        const int64_t start = x - begin, stop = start + cur.r.count;  // of the unit on the line
        if (start >= x0 || warp == 0) {  // the block's first warp with this unit
          Entry& e = entries[warp][x > x0];
          e.valid = 1;
          e.b = cur.b;
          e.lane = cur.ln;
          e.last = static_cast<int>((min(stop, X1) - 1 - X0) / per);
          e.before = start < X0;
          e.past = stop > X1;
          e.in_first = x == x0 && next < x1;
        }
        if (x == x0) several[warp] = next < x1;
      }
      x = next;
      cur.at = end;
      if (x < x1) next_unit(cur);
    }
    if (gave_up) {
      if (lane == 0) atomicOr(a.status, kStatusKv4Timeout);
      for (; in_flight > 0; --in_flight) {
        arrived(stage, phase);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  }

  // ---- units of several warps ----
  __syncthreads();
  for (int n = 0; n < 2 * kWarps; ++n) {
    const int w0 = n >> 1;
    const Entry e = entries[w0][n & 1];
    if (!e.valid) continue;
    const auto part_of = [&](int w) -> const float* {
      return (w == w0 ? e.in_first : several[w]) ? first_part(w) : reinterpret_cast<const float*>(smem + w * S::RING);
    };
    const int hk = e.lane / a.row_tiles, row0 = (e.lane - hk * a.row_tiles) * ROWS, rows = p.n * a.group;
    const int last = min(e.last, kWarps - 1);
    for (int in_tile = warp; in_tile < ROWS; in_tile += kWarps) {
      const int r = row0 + in_tile;
      if (r >= rows) continue;
      float best = -INFINITY;
      for (int w = w0; w <= last; ++w) best = fmaxf(best, part_of(w)[ROWS * D + 2 * in_tile]);
      float acc[U], l = 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u) acc[u] = 0.f;
      for (int w = w0; w <= last; ++w) {
        const float* from = part_of(w);
        const float2 ml = *reinterpret_cast<const float2*>(from + ROWS * D + 2 * in_tile);
        const float wt = weight(ml.x, ml.y, best);
        l += wt;
        if (wt == 0.f) continue;
#pragma unroll
        for (int u = 0; u < U; ++u) acc[u] += wt * from[in_tile * D + 32 * u + lane];
      }
      const bool whole = !e.before && !e.past;
      const int i = r / a.group;
      const int at = range_of(p, e.b).len - p.n + i;
      const float inv = l != 0.f ? 1.f / l : whole && at >= 0 ? quiet_nan() : 0.f;
      if (whole) {
        uint16_t* out = p.out + ((static_cast<int64_t>(e.b) * p.n + i) * p.Hq + hk * a.group + (r - i * a.group)) * D;
#pragma unroll
        for (int u = 0; u < U; ++u) out[32 * u + lane] = float_to_elem<kBF>(acc[u] * inv);
      } else {
        float* to = a.parts + (2 * static_cast<int64_t>(blockIdx.x) + (e.past ? 1 : 0)) * (S::PART / 4);
#pragma unroll
        for (int u = 0; u < U; ++u) to[in_tile * D + 32 * u + lane] = acc[u] * inv;
        if (lane == 0) *reinterpret_cast<float2*>(to + ROWS * D + 2 * in_tile) = make_float2(best, l);
      }
    }
  }
}

// Joins the parts of units of several blocks.  One warp per row.
template <bool kBF, int D, int NT>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ Args a, int blocks) {
  constexpr int U = D / 32, ROWS = 8 * NT, PART = ROWS * (D + 2);
  const AttentionKv4Problem& p = a.p;
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (row >= static_cast<int64_t>(p.B) * p.n * p.Hq) return;
  const int h = static_cast<int>(row % p.Hq), i = static_cast<int>(row / p.Hq % p.n), b = static_cast<int>(row / p.Hq / p.n);
  const int hk = h / a.group, r = i * a.group + h - hk * a.group;
  ptx::grid_dependency_wait();
  const int64_t block = a.line[0] * kWarps, T = a.line[1 + p.B];
  const int64_t start = a.line[1 + b], stop = a.line[2 + b];
  if (start >= stop) return;
  const int64_t x0 = (static_cast<int64_t>(hk) * a.row_tiles + r / ROWS) * T;
  const int64_t c0 = (x0 + start) / block, c1 = min((x0 + stop - 1) / block, static_cast<int64_t>(blocks) - 1);
  if (c0 >= c1) return;
  const int in_tile = r % ROWS;
  const auto part = [&](int64_t c) -> const float* { return a.parts + (2 * c + (c < c1 ? 1 : 0)) * PART; };
  float best = -INFINITY, l = 0.f, acc[U];
  for (int64_t c = c0 + lane; c <= c1; c += 32) best = fmaxf(best, part(c)[ROWS * D + 2 * in_tile]);
#pragma unroll
  for (int d = 16; d; d >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, d));
#pragma unroll
  for (int u = 0; u < U; ++u) acc[u] = 0.f;
#pragma unroll 4
  for (int64_t c = c0; c <= c1; ++c) {
    const float* from = part(c);
    const float2 ml = *reinterpret_cast<const float2*>(from + ROWS * D + 2 * in_tile);
    const float wt = weight(ml.x, ml.y, best);
    l += wt;
#pragma unroll
    for (int u = 0; u < U; ++u) acc[u] += wt * from[in_tile * D + 32 * u + lane];
  }
  const bool sees = range_of(p, b).len - p.n + i >= 0;
  const float inv = l != 0.f ? 1.f / l : sees ? quiet_nan() : 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u) p.out[row * D + 32 * u + lane] = float_to_elem<kBF>(acc[u] * inv);
}

template <bool kBF, int D, int G, int NT>
cudaError_t run(const Args& a, int grid) {
  constexpr int smem = Shape<D, G, NT>::SMEM;
  const auto kernel = attention_kernel<kBF, D, G, NT>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kernel<<<grid, kWarps * 32, smem, a.p.stream>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (grid == 1 || a.aligned) return cudaSuccess;  // nothing to join
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((static_cast<int64_t>(a.p.B) * a.p.n * a.p.Hq + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = a.p.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<kBF, D, NT>, a, grid);
}

// Per head size, in a translation unit each; nt as planned.
cudaError_t run_64(const Args& a, int nt, int grid);
cudaError_t run_96(const Args& a, int nt, int grid);
cudaError_t run_128(const Args& a, int nt, int grid);
cudaError_t run_256(const Args& a, int nt, int grid);

}  // namespace kv4
}  // namespace awq
