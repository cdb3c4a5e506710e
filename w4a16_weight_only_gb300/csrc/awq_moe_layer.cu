// A mixture-of-experts layer of a few tokens on 4-bit experts, in two kernels (awq_moe_layer):
//
//   act[t, j] = silu(x[t] Wg) * (x[t] Wu)          of expert experts[t, j], as the sum of two elements
//   out[t]    = base[t] + sum_j weights[t, j] * (act[t, j] Wd)
//
// with  w = (code - zero) * scale  per group of G rows, sums in fp32, the result rounded once.  As one element act
// would double the variance of the result's own rounding.
#include "awq_step.cuh"
#include "awq_ptx.cuh"

namespace awq {
namespace {

constexpr int kMaxPlaces = kMoeLayerMaxT * 32;
// Columns of an m16n8k16: eight places of a job, in the second product four with their act's two elements.  An expert
// of more than four places is several jobs there: 16 tokens, 2 of 8, 4096 x 14336, fp16 252 us (211 with one element;
// 231 with eight places a job and products of their own for the second elements, which cost the others 2 to 5 %: 16
// tokens, 8 of 128, 236 and 242, one element 231; 3 tokens, 2 of 8, 131 and 136, 131).
constexpr int kRows = 8;
constexpr int kBlockK = 64;   // rows of a weight that a warp has in flight

struct Layout {
  size_t y, counters, bytes;  // offsets; act first
};

__host__ Layout layout(int T, int k, int H, int I) {
  Layout l;
  const auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  l.y = up(static_cast<size_t>(T) * k * I * 4);  // act: two elements, or fp32 in the kernels for any shape
  l.counters = l.y + up(static_cast<size_t>(T) * k * H * 4);
  l.bytes = l.counters + up(static_cast<size_t>((H + 127) / 128) * 4);
  return l;
}

// ---- any shape ----

// Sum over K of x[k] * w[k][8 c + j] of one expert for the eight columns of word column c.
template <bool kBF, typename F>
__device__ __forceinline__ void dot8(const Stacked& w, int64_t e, int K, int N, int G, int c, F&& x, float (&acc)[8]) {
  const uint32_t* qw = w.qw + (e * K) * (N / 8) + c;
  const int64_t g0 = e * (K / G);
  for (int j = 0; j < 8; ++j) acc[j] = 0.f;
  for (int g = 0; g < K / G; ++g) {
    const uint32_t z = w.qz[(g0 + g) * (N / 8) + c];
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int k = g * G; k < (g + 1) * G; ++k) {
      const uint32_t word = qw[static_cast<int64_t>(k) * (N / 8)];
      const float v = x(k);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        sum[nibble_column(i)] += v * static_cast<float>(static_cast<int>((word >> (4 * i)) & 15u) - static_cast<int>((z >> (4 * i)) & 15u));
    }
    for (int j = 0; j < 8; ++j) acc[j] += sum[j] * elem_to_float<kBF>(w.sc[(g0 + g) * N + 8 * c + j]);
  }
}

// One thread per (place, eight columns).  Slow: 2 of 8 experts of 2040 x 1400, groups of 8, 1.2 ms for 1 to 16 tokens (of
// 2048 x 1408, groups of 64, by the tensor-core kernels 20 to 34 us).
template <bool kBF>
__global__ void __launch_bounds__(128) moe_up_any_kernel(const MoeLayerProblem p, float* act) {
  const int c = blockIdx.x * 128 + threadIdx.x, place = blockIdx.y;
  if (c >= p.I / 8) return;
  const int e = p.experts[place];
  if (e < 0 || e >= p.E) return;
  const uint16_t* x = p.x + static_cast<int64_t>(place / p.k) * p.x_st;
  float gate[8], up[8];
  const auto at = [&](int k) { return elem_to_float<kBF>(x[k]); };
  dot8<kBF>(p.up, e, p.H, 2 * p.I, p.G, c, at, gate);
  dot8<kBF>(p.up, e, p.H, 2 * p.I, p.G, p.I / 8 + c, at, up);
  for (int j = 0; j < 8; ++j)
    act[static_cast<int64_t>(place) * p.I + 8 * c + j] = gate[j] / (1.f + expf(-gate[j])) * up[j];
}

// One thread per (token, eight columns).
template <bool kBF>
__global__ void __launch_bounds__(128) moe_down_any_kernel(const MoeLayerProblem p, const float* act) {
  const int c = blockIdx.x * 128 + threadIdx.x, t = blockIdx.y;
  if (c >= p.H / 8) return;
  float sum[8];
  for (int j = 0; j < 8; ++j)
    sum[j] = p.base ? elem_to_float<kBF>(p.base[static_cast<int64_t>(t) * p.H + 8 * c + j]) : 0.f;
  for (int j = 0; j < p.k; ++j) {
    const int place = t * p.k + j, e = p.experts[place];
    if (e < 0 || e >= p.E) continue;
    float y[8];
    const float* a = act + static_cast<int64_t>(place) * p.I;
    dot8<kBF>(p.down, e, p.I, p.H, p.G, c, [&](int k) { return a[k]; }, y);
    for (int i = 0; i < 8; ++i) sum[i] += p.weights[place] * y[i];
  }
  for (int j = 0; j < 8; ++j) p.out[static_cast<int64_t>(t) * p.H + 8 * c + j] = float_to_elem<kBF>(sum[j]);
}

// ---- tensor-core kernels ----

// The places, kPart of one expert at a time, in shared memory for T k of them.
struct Jobs {
  int* expert;
  int* rows;
  int* ids;                     // of the places
  uint16_t (*place)[kRows];
  int count;
  __device__ Jobs(uint8_t* at, int places)
      : expert(reinterpret_cast<int*>(at)), rows(expert + places), ids(rows + places),
        place(reinterpret_cast<uint16_t(*)[kRows]>(ids + places)), count(0) {}
  __host__ __device__ static constexpr int bytes(int places) { return places * (3 * 4 + kRows * 2); }
};

// Built by every block alike from the experts' ids: place p is row (rank % kPart) of its expert's job rank / kPart,
// jobs in the order of their first places.
template <int kThreads, int kPart>
__device__ __forceinline__ void build_jobs(const MoeLayerProblem& p, Jobs& jobs, int* head_job, int* count) {
  const int places = p.T * p.k;
  int* ids = jobs.ids;
  for (int i = threadIdx.x; i < places; i += kThreads) {
    ids[i] = __ldg(p.experts + i);
    jobs.rows[i] = 0;
  }
  __syncthreads();
  // head_job[i]: first the head of place i's job (i itself where it is one)
  constexpr int kPer = (kMaxPlaces + kThreads - 1) / kThreads;
  int row[kPer];
#pragma unroll
  for (int n = 0; n < kPer; ++n) {
    const int i = n * kThreads + threadIdx.x;
    row[n] = -1;
    if (i >= places) continue;
    const int e = ids[i];
    if (e < 0 || e >= p.E) {
      head_job[i] = -1;
      continue;
    }
    int rank = 0, head = i;
    for (int q = 0; q < i; ++q)
      if (ids[q] == e) {
        if ((rank & (kPart - 1)) == 0) head = q;
        ++rank;
      }
    row[n] = rank & (kPart - 1);
    head_job[i] = row[n] == 0 ? i : head;
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < kPer; ++n) {
    const int i = n * kThreads + threadIdx.x;
    if (row[n] < 0) continue;
    const int head = head_job[i];
    int job = 0;  // heads before this one
    for (int q = 0; q < head; ++q) job += head_job[q] == q;
    jobs.place[job][row[n]] = static_cast<uint16_t>(i);
    atomicAdd(&jobs.rows[job], 1);
    if (row[n] == 0) jobs.expert[job] = ids[i];
  }
  if (threadIdx.x < 32) {
    int n = 0;
    for (int q = threadIdx.x; q < places; q += 32) n += head_job[q] == q;
#pragma unroll
    for (int d = 16; d; d >>= 1) n += __shfl_xor_sync(0xffffffffu, n, d);
    if (threadIdx.x == 0) *count = n;
  }
  __syncthreads();
  jobs.count = *count;
}

__device__ __forceinline__ float silu(float v) { return v / (1.f + __expf(-v)); }

constexpr uint64_t kWaitLimitNs = 200ull * 1000 * 1000;
constexpr unsigned int kStatusMoeTimeout = 0x20u;

struct Args {
  MoeLayerProblem p;
  CUtensorMap map;  // the words of this product's weights
  uint16_t* act;
  float* y;
  int* counters;
  unsigned int* status;
};

// A stage: the words of 64 rows, two boxes of eight columns of words, and for their group of rows the scales
// and zeros of both boxes' columns.
struct Stage {
  static constexpr int BOX = 64 * 32, WORDS = 2 * BOX, PARAMS = 2 * 128 + 2 * 32;
  static constexpr int scales(int o) { return o * 128; }
  static constexpr int zeros(int o) { return 256 + o * 32; }
};

// Shared memory: the warps' sums, the rings' words, their parameters, barriers, then the jobs.
template <int kW>
struct Shared {
  static constexpr int STAGES = 2;
  static constexpr int WORDS = kW * 4096;
  static constexpr int PARAMS = WORDS + kW * STAGES * Stage::WORDS;
  static constexpr int BARS = PARAMS + kW * STAGES * Stage::PARAMS;
  static constexpr int JOBS = BARS + kW * STAGES * 8;
  static_assert(WORDS >= kMaxPlaces * 4, "the heads of the jobs are built in the sums' place");
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(ptx::smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(ptx::smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void box_load(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %4, %5}], [%2];" ::"r"(
          ptx::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(ptx::smem_u32(bar)), "r"(x), "r"(0), "r"(w)
      : "memory");
}

// One product of the layer.  A unit is a job times 128 columns (kUp: 64 gate columns and their 64 up
// columns); its K rows are cut over the block's warps.  The product is taken transposed, Y^T = W^T X^T:
// columns of the weight fill the 16 rows of an m16n8k16, the job's places its 8 columns.  Lane (g, t) has
// word columns g (a word is eight columns) of rows 8 t .. 8 t + 7 of every 32, so that an x fragment is part of
// one 16-byte load and a weight fragment is four words of one column octet, bytes exchanged between pairs of
// rows; the boxes come with the rows 8 t + i of the four t side by side, so that a warp reads 128 bytes in a
// row.  fp16: a pair of codes ANDed out of the words is c 2^-24 or c 2^-20, a subnormal number, exact;
// bf16: with the exponent ORed in it is 128 + c.  The zero (and 128) leaves with the sum of x, which an
// mma against ones gives in the same layout; a group's sums are scaled into fp32 totals.
// Each warp has a ring of stages of its own, filled by TMA across units: 16 tokens of 8 of 128 experts, 4096 x
// 1792, some 750 MB (66 distinct experts) in 236 us for both products, 3.2 TB/s (words loaded ahead into registers
// instead: 630 us, a warp waits for its newest load with its oldest).  No unit is full: at 15 warps an SM the schedulers
// issue in 59 and 54 % of their cycles, HBM is at 48 and 30 %, the tensor pipe at 21 and 14 %; a warp waits for its own
// chain of words, exchange and products, and a block for its slowest warp.
template <bool kBF, bool kUp, int kW>
__global__ void __launch_bounds__(kW * 32, 16 / kW) moe_kernel(const __grid_constant__ Args args) {
  using SH = Shared<kW>;
  constexpr int STAGES = SH::STAGES;
  extern __shared__ __align__(128) uint8_t smem[];
  float4* red = reinterpret_cast<float4*>(smem);  // [kW][8 quads][32 lanes]
  __shared__ int job_count;
  const MoeLayerProblem& p = args.p;
  Jobs jobs(smem + SH::JOBS, p.T * p.k);
  uint16_t* act = args.act;
  float* y = args.y;
  int* counters = args.counters;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  constexpr int kPart = kUp ? kRows : kRows / 2;  // places of a job
  const int K = kUp ? p.H : p.I, N = kUp ? 2 * p.I : p.H, words = N / 8;
  const Stacked& w = kUp ? p.up : p.down;
  ptx::launch_dependents();
  uint8_t* ring = smem + SH::WORDS + warp * (STAGES * Stage::WORDS);
  uint8_t* params = smem + SH::PARAMS + warp * (STAGES * Stage::PARAMS);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SH::BARS) + warp * STAGES;
  if (lane == 0) {
    for (int s = 0; s < STAGES; ++s) ptx::mbar_init(&full[s], 1);
    ptx::fence_mbar_init();
  }
  build_jobs<kW * 32, kPart>(p, jobs, reinterpret_cast<int*>(smem), &job_count);
  if (kUp && blockIdx.x == 0)
    for (int i = threadIdx.x; i < (p.H + 127) / 128; i += kW * 32) counters[i] = 0;
  const int tiles = kUp ? p.I / 64 : (p.H + 127) / 128, units = jobs.count * tiles;
  const int blocks = K / kBlockK, b0 = blocks * warp / kW, b1 = blocks * (warp + 1) / kW;
  const bool work = b1 > b0;

  // ---- what is loaded next: block pb of unit pu ----
  int pu = blockIdx.x, pb = b0;
  const auto issue = [&](int stage) {
    if (lane == 0) {
      const int job = pu / tiles, tile = pu - job * tiles, e = jobs.expert[job];
      const int c0 = kUp ? 8 * tile : 16 * tile;
      const int c1 = kUp ? p.I / 8 + c0 : c0 + 8 < words ? c0 + 8 : c0;  // half a tile at the end: its columns are not kept
      uint8_t* to = ring + stage * Stage::WORDS;
      uint8_t* to_params = params + stage * Stage::PARAMS;
      uint64_t* bar = &full[stage];
      ptx::mbar_arrive_expect_tx(bar, Stage::WORDS + Stage::PARAMS);
      const int slab = e * (K / 32) + pb * (kBlockK / 32);
      box_load(to, &args.map, bar, c0, slab);
      box_load(to + Stage::BOX, &args.map, bar, c1, slab);
      const int64_t at = static_cast<int64_t>(e) * (K / p.G) + pb * kBlockK / p.G;
      bulk_load(to_params + Stage::scales(0), w.sc + at * N + 8 * c0, 128, bar);
      bulk_load(to_params + Stage::scales(1), w.sc + at * N + 8 * c1, 128, bar);
      bulk_load(to_params + Stage::zeros(0), w.qz + at * words + c0, 32, bar);
      bulk_load(to_params + Stage::zeros(1), w.qz + at * words + c1, 32, bar);
    }
    __syncwarp();
    if (++pb == b1) {
      pb = b0;
      pu += gridDim.x;
    }
  };
  int loaded = 0, used = 0;
  if (work)
    for (; loaded < STAGES && pu < units; ++loaded) issue(loaded);

  // x of block b of a unit: eight elements of the lane's place per 32 rows
  const auto row_of = [&](int unit) -> const uint16_t* {
    const int job = unit / tiles, r = g & (kPart - 1);
    if (r >= jobs.rows[job]) return nullptr;
    const int place = jobs.place[job][r];
    const int64_t term = g / kPart;  // of act
    return (kUp ? p.x + static_cast<int64_t>(place / p.k) * p.x_st : act + (term * (p.T * p.k) + place) * p.I) + 8 * t;
  };
  const auto load_x = [&](const uint16_t* row, int b, uint4 (&v)[2]) {
#pragma unroll
    for (int half = 0; half < 2; ++half)
      v[half] = row ? *reinterpret_cast<const uint4*>(row + b * kBlockK + 32 * half) : make_uint4(0u, 0u, 0u, 0u);
  };
  // Block number n of this warp has arrived: a bounded wait, the clock read before the test that decides.
  const auto arrived = [&](int n) -> bool {
    const uint32_t parity = static_cast<uint32_t>(n / STAGES) & 1u;
    uint64_t* bar = &full[n % STAGES];
    const auto there = [&] { return __all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity)) != 0; };
    if (there()) return true;
    const uint64_t t0 = ptx::globaltimer_ns();
    while (true) {
      const bool late = __any_sync(0xffffffffu, ptx::globaltimer_ns() - t0 > kWaitLimitNs);
      if (there()) return true;
      if (late) return false;
    }
  };

  if (!kUp) ptx::grid_dependency_wait();  // act, and the counters' zeros
  bool gave_up = false;
  uint4 next_x[2];
  if (work && blockIdx.x < units) load_x(row_of(blockIdx.x), b0, next_x);
  for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int job = unit / tiles, tile = unit - job * tiles;
    float total[2][4][4];  // octet, mma, fragment
#pragma unroll
    for (int o = 0; o < 2; ++o)
#pragma unroll
      for (int i = 0; i < 4; ++i) total[o][i][0] = total[o][i][1] = total[o][i][2] = total[o][i][3] = 0.f;
    if (work && !gave_up) {
      const uint16_t* row_x = row_of(unit);
      float acc[2][4][4], ones[4];
      bool fresh = true;
      for (int b = b0; b < b1; ++b) {
        const uint4 xf[2] = {next_x[0], next_x[1]};
        if (b + 1 < b1) load_x(row_x, b + 1, next_x);
        else if (unit + gridDim.x < units) load_x(row_of(unit + gridDim.x), b0, next_x);
        if (p.give_up || !arrived(used)) {
          gave_up = true;
          break;
        }
        const int stage = used % STAGES;
        const uint8_t* at = ring + stage * Stage::WORDS;
        const uint8_t* from = params + stage * Stage::PARAMS;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (fresh) {
#pragma unroll
            for (int o = 0; o < 2; ++o)
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[o][i][0] = acc[o][i][1] = acc[o][i][2] = acc[o][i][3] = 0.f;
            ones[0] = ones[1] = ones[2] = ones[3] = 0.f;
          }
#pragma unroll
          for (int odd = 0; odd < 2; ++odd) {
            const uint32_t x0 = odd ? xf[half].z : xf[half].x, x1 = odd ? xf[half].w : xf[half].y;
            constexpr uint32_t one = kBF ? 0x3f803f80u : 0x3c003c00u;
            const auto mma = [&](float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
              if constexpr (kBF) ptx::mma16816_bf16(d, a0, a1, a2, a3, x0, x1);
              else ptx::mma16816(d, a0, a1, a2, a3, x0, x1);
            };
            mma(ones, one, one, one, one);
#pragma unroll
            for (int o = 0; o < 2; ++o) {
              const uint32_t* word = reinterpret_cast<const uint32_t*>(at + o * Stage::BOX + half * 1024 + odd * 512) + 8 * t + g;
              const uint32_t w0 = word[0], w1 = word[32], w2 = word[64], w3 = word[96];
#pragma unroll
              for (int high = 0; high < 2; ++high) {  // columns 0, 2, 4, 6; 1, 3, 5, 7
                const uint32_t sel = high ? 0x7632u : 0x5410u;
                const uint32_t u = ptx::prmt(w0, w1, sel), v = ptx::prmt(w2, w3, sel);
                if constexpr (kBF) {
                  const auto code = [](uint32_t q, int shift) { return ptx::and_or(q >> shift, 0x000f000fu, 0x43004300u); };
                  mma(acc[o][2 * high], code(u, 0), code(u, 8), code(v, 0), code(v, 8));
                  mma(acc[o][2 * high + 1], code(u, 4), code(u, 12), code(v, 4), code(v, 12));
                } else {
                  const uint32_t u8 = u >> 8, v8 = v >> 8;
                  mma(acc[o][2 * high], u & 0x000f000fu, u8 & 0x000f000fu, v & 0x000f000fu, v8 & 0x000f000fu);
                  mma(acc[o][2 * high + 1], u & 0x00f000f0u, u8 & 0x00f000f0u, v & 0x00f000f0u, v8 & 0x00f000f0u);
                }
              }
            }
          }
          fresh = (b * kBlockK + half * 32 + 32) % p.G == 0 || (half == 1 && b + 1 == b1);
          if (fresh) {  // the group's sums, or as much of them as is this warp's
#pragma unroll
            for (int o = 0; o < 2; ++o) {
              uint4 scale = *reinterpret_cast<const uint4*>(from + Stage::scales(o) + 16 * g);
              uint32_t zero = *reinterpret_cast<const uint32_t*>(from + Stage::zeros(o) + 4 * g);
              if (half && p.G == 32) {  // the block's second group
                const int64_t group = static_cast<int64_t>(jobs.expert[job]) * (K / 32) + 2 * b + 1;
                const int c = min((kUp ? 8 : 16) * tile + (o ? kUp ? p.I / 8 : 8 : 0) + g, words - 1);
                scale = __ldg(reinterpret_cast<const uint4*>(w.sc + group * N + 8 * c));
                zero = __ldg(w.qz + group * words + c);
              }
              const uint32_t sw[4] = {scale.x, scale.y, scale.z, scale.w};
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int second = 0; second < 2; ++second) {
                  // mma i has columns 2 (i % 2) + i / 2 and four further
                  const int col = 2 * (i & 1) + (i >> 1) + 4 * second, nibble = (col & 1) * 4 + (col >> 1);
                  const float2 s2 = ptx::pair_to_float2<kBF>(sw[col >> 1]);
                  const float s = col & 1 ? s2.y : s2.x;
                  const float z = static_cast<float>((zero >> (4 * nibble)) & 15u) + (kBF ? 128.f : 0.f);
                  const float lift = kBF ? 1.f : i & 1 ? 1048576.f : 16777216.f;
#pragma unroll
                  for (int h = 0; h < 2; ++h)
                    total[o][i][2 * second + h] += s * (acc[o][i][2 * second + h] * lift - z * ones[h]);
                }
            }
          }
        }
        __syncwarp();  // the stage has been read
        ++used;
        if (pu < units) {
          issue(stage);
          ++loaded;
        }
      }
    }
    // the warps' sums; warp n then has mma n % 4 of octet n / 4
    __syncthreads();  // the last unit's sums have been read
    float4* mine = red + warp * 256 + lane;
#pragma unroll
    for (int o = 0; o < 2; ++o)
#pragma unroll
      for (int i = 0; i < 4; ++i) mine[(4 * o + i) * 32] = make_float4(total[o][i][0], total[o][i][1], total[o][i][2], total[o][i][3]);
    __syncthreads();
    const auto sum = [&](int quad) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int n = 0; n < kW; ++n) {
        const float4 u = red[n * 256 + quad * 32 + lane];
        v.x += u.x;
        v.y += u.y;
        v.z += u.z;
        v.w += u.w;
      }
      return v;
    };
    if (warp < (kUp ? 4 : 8)) {
      const int i = warp & 3, col = 2 * (i & 1) + (i >> 1);
      const float4 a = sum(warp);
      const float first[4] = {a.x, a.y, a.z, a.w};
      if constexpr (kUp) {
        const float4 b = sum(4 + warp);
        const float second[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int r = 2 * t + (n & 1), column = 64 * tile + 8 * g + col + 4 * (n >> 1);
          if (r >= jobs.rows[job]) continue;
          const float v = silu(first[n]) * second[n];
          const uint16_t whole = float_to_elem<kBF>(v);
          const float rest = v - elem_to_float<kBF>(whole);
          const int64_t at = static_cast<int64_t>(jobs.place[job][r]) * p.I + column;
          act[at] = whole;
          // (infinities and NaN have no rest)
          act[at + static_cast<int64_t>(p.T * p.k) * p.I] = float_to_elem<kBF>(fabsf(rest) <= fabsf(v) ? rest : 0.f);
        }
      } else {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const float y_rc = first[n] + __shfl_xor_sync(0xffffffffu, first[n], 2);  // the places' rests are four columns further
          const int r = 2 * t + (n & 1), column = 128 * tile + 64 * (warp >> 2) + 8 * g + col + 4 * (n >> 1);
          if (r < jobs.rows[job] && column < p.H) y[static_cast<int64_t>(jobs.place[job][r]) * p.H + column] = y_rc;
        }
      }
    }
  }
  if (gave_up) {  // its copies in flight land first
    if (lane == 0) atomicOr(args.status, kStatusMoeTimeout);
    for (; used < loaded; ++used) arrived(used);
  }
  if constexpr (!kUp) {
    // The block that is the last with a tile of columns adds the places up, in their order.
    __shared__ int last[kW * 32];
    const int mine = (units - static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
    __threadfence();
    __syncthreads();
    for (int n0 = 0; n0 < mine; n0 += kW * 32) {
      const int n = n0 + threadIdx.x;
      last[threadIdx.x] = -1;
      if (n < mine) {
        const int tile = static_cast<int>((blockIdx.x + static_cast<int64_t>(n) * gridDim.x) % tiles);
        if (atomicAdd(counters + tile, 1) == jobs.count - 1) last[threadIdx.x] = tile;
      }
      __syncthreads();
      __threadfence();
      for (int i = 0; i < min(mine - n0, kW * 32); ++i) {
        const int tile = last[i];
        if (tile < 0) continue;
        for (int v = threadIdx.x; v < p.T * 128; v += kW * 32) {
          const int tok = v >> 7, column = 128 * tile + (v & 127);
          if (column >= p.H) continue;
          const int64_t at = static_cast<int64_t>(tok) * p.H + column;
          float total = p.base ? elem_to_float<kBF>(p.base[at]) : 0.f;
          for (int j = 0; j < p.k; ++j) {
            const int place = tok * p.k + j;
            if (jobs.ids[place] >= 0 && jobs.ids[place] < p.E) total += __ldg(p.weights + place) * __ldcg(y + static_cast<int64_t>(place) * p.H + column);
          }
          p.out[at] = float_to_elem<kBF>(total);
        }
      }
      __syncthreads();
    }
    if (jobs.count == 0)  // no place has an expert
      for (int64_t v = static_cast<int64_t>(blockIdx.x) * (kW * 32) + threadIdx.x; v < static_cast<int64_t>(p.T) * p.H;
           v += static_cast<int64_t>(gridDim.x) * (kW * 32))
        p.out[v] = p.base ? p.base[v] : 0;
  }
}

// The words of a product's weights as [32 rows][row % 8][row / 8 % 4][word] for boxes of 64 rows of eight words.
bool make_map(CUtensorMap* map, const Stacked& w, int E, int K, int N) {
  const uint64_t row = static_cast<uint64_t>(N) / 2;  // bytes
  const uint64_t dims[4] = {static_cast<uint64_t>(N) / 8, 4, 8, static_cast<uint64_t>(E) * (K / 32)};
  const uint64_t strides[3] = {8 * row, row, 32 * row};
  const uint32_t box[4] = {8, 4, 8, kBlockK / 32};
  return make_tmap_4d(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, w.qw, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}

template <bool kBF, bool kUp, int kW>
cudaError_t launch_product(const Args& args, int grid) {
  const auto kernel = moe_kernel<kBF, kUp, kW>;
  const int smem = Shared<kW>::JOBS + Jobs::bytes(args.p.T * args.p.k);
  // the attribute is the function's, not the call's: the most that any call needs, or another host thread's smaller
  // call would lower it between this call's attribute and its launch
  constexpr int most = Shared<kW>::JOBS + Jobs::bytes(kMaxPlaces);
  static_assert(most <= 227 * 1024, "shared memory of a block");
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];  // the second product's weights are on their way before the first has ended
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kW * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = args.p.stream;
  cfg.attrs = attr;
  cfg.numAttrs = kUp ? 0 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args);
}

bool tensor_cores_fit(const MoeLayerProblem& p) {
  const auto fits = [](const Stacked& w) { return aligned(w.qw, 16) && aligned(w.qz, 16) && aligned(w.sc, 16); };
  return p.k > 0 && p.H % kBlockK == 0 && p.I % kBlockK == 0 && (p.G == 32 || p.G % 64 == 0) && fits(p.up) && fits(p.down) &&
         aligned(p.x, 16) && (p.x_st % 8 == 0 || p.T == 1) && static_cast<int64_t>(p.E) * (p.H > p.I ? p.H : p.I) < (int64_t{1} << 31);
}

template <bool kBF>
cudaError_t launch(const MoeLayerProblem& p, int sms) {
  const Layout l = layout(p.T, p.k, p.H, p.I);
  uint8_t* ws = static_cast<uint8_t*>(p.workspace);
  Args up{}, down{};
  if (tensor_cores_fit(p)) {
    // First of all: it makes the device's context this host thread's, without which no tensor map is made.
    cudaError_t e = status_word_ptr(&up.status);
    if (e != cudaSuccess) return e;
    if (!make_map(&up.map, p.up, p.E, p.H, 2 * p.I) || !make_map(&down.map, p.down, p.E, p.I, p.H)) return cudaErrorInvalidValue;
    up.p = p;
    up.act = reinterpret_cast<uint16_t*>(ws);
    up.y = reinterpret_cast<float*>(ws + l.y);
    up.counters = reinterpret_cast<int*>(ws + l.counters);
    down.p = p;
    down.act = up.act;
    down.y = up.y;
    down.counters = up.counters;
    down.status = up.status;
    const auto grid = [&](int64_t tiles) {  // two blocks per SM: one computes while the other adds its warps up
      const int64_t units = tiles * p.T * p.k;
      return static_cast<int>(units < 2 * sms ? units : 2 * sms);
    };
    // (sixteen warps a block for few units, one block per SM: no faster, 25.2 us for one token of 8 of 128)
    e = launch_product<kBF, true, 8>(up, grid(p.I / 64));
    if (e != cudaSuccess) return e;
    return launch_product<kBF, false, 8>(down, grid((p.H + 127) / 128));
  }
  float* act = reinterpret_cast<float*>(ws);
  if (p.k > 0 && p.I > 0) {
    moe_up_any_kernel<kBF><<<dim3((p.I / 8 + 127) / 128, p.T * p.k), 128, 0, p.stream>>>(p, act);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  moe_down_any_kernel<kBF><<<dim3((p.H / 8 + 127) / 128, p.T), 128, 0, p.stream>>>(p, act);
  return cudaGetLastError();
}

}  // namespace

size_t moe_layer_workspace_bytes(int T, int k, int H, int I) { return T * k == 0 ? 0 : layout(T, k, H, I).bytes; }

cudaError_t launch_moe_layer(const MoeLayerProblem& p, int sms) { return p.bf16 ? launch<true>(p, sms) : launch<false>(p, sms); }

}  // namespace awq
