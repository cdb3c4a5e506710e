// The prefix of awq_attention_shared on the tensor cores: the query rows of all sequences that
// share a key/value head, stacked into tiles of 256, against the prefix's keys.
//
//   S = Q K^T (128 x 128 fp32 in TMEM),  P = exp2(scale log2(e) S - m),  O += P V (128 x D in TMEM)
//
// One block per SM.  The row tiles of a head run side by side in a group of blocks, which so read the
// same keys at the same time (cut one after the other, four tiles read 491 MB of HBM for the 134 MB
// there are); the 128-key steps of all heads form one sequence that is cut evenly over the groups (a
// head's keys cut between groups give one part each; the join kernel adds them), so the SMs finish
// together whatever the number of heads.
//
// Warps: 0-3 and 4-7 softmax of the tile's first and second 128 rows, one row per thread (a row's
// maximum and sum need no shuffles); 8 and 9 load keys and values into a ring of four 128-token slots
// (TMA boxes of whole runs of a page's tokens; cp.async where pages are odd and where the prefix
// ends); 10 issues the MMAs.  While one half's softmax runs, the tensor core works for the other half:
// PV(a), QK(a) of the next step, PV(b), QK(b).  P, rounded to the element type, overwrites the S it
// came from and is the MMA's A operand in TMEM; MMAs of one thread run in the order of issue, so the
// next QK into S starts after the PV that reads P.
//
// 128 sequences of 64 / 8 heads over 32768 keys of 128, bf16: 137 GFLOP in 92 us on all SMs, 1.49 PFLOP/s;
// 138 us on 100 SMs beside the streaming kernel, the same per SM.  Bound
// by the chain softmax - PV - QK of a half (about 1500 + 500 + 600 cycles of a step's 2900, the tensor
// core's share of a step being 2050) and by the issue of the MMAs, each of which takes its thread about
// as long as it runs.
//
// The running maximum m of a row is raised only when it is exceeded by more than 2^kRaise: until then
// nothing is rescaled (O and the sum l use the same m, so the result is unchanged; P keeps its relative
// accuracy).  A raise waits for the row's last PV and rescales O in
// TMEM.
#include "awq_attn.cuh"

namespace awq {
namespace {

using namespace ptx;
using namespace attn;

constexpr int kThreads = 384;
// Registers per thread at launch; the softmax warpgroups take 160, the third one 88: 2 x 160 + 88 = 3 x 136.
constexpr int kRegs = 136;
constexpr int kSlots = 4;  // ring of key / value tiles
constexpr uint32_t kTmemCols = 512;

// TMEM columns: S / P of the two halves, then O of the two halves.
constexpr uint32_t kColS = 0, kColO = 256;

template <int D>
struct Shape {
  static constexpr int PANELS = (D + 63) / 64;       // 64 elements (128 bytes) of every row
  static constexpr int PANEL = 128 * 128;            // 128 rows of 128 bytes, 128-byte swizzle
  static constexpr int TILE = PANELS * PANEL;        // 128 rows of Q, K or V
  static constexpr int Q_OFF = 0;
  static constexpr int RING_OFF = 2 * TILE;
  static constexpr int BAR_OFF = RING_OFF + kSlots * TILE;
  // full[kSlots], empty[kSlots], q_full[2], s_full[2], p_half[2], p_full[2], pv_done[2], drain
  static constexpr int NBARS = 2 * kSlots + 11;
  static constexpr int MISC_OFF = BAR_OFF + NBARS * 8;  // TMEM base, abort flag
  static constexpr int SMEM = 1024 + MISC_OFF + 16;
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)::"memory");
  return r != 0u;
}

__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Shared-memory operand descriptor, 128-byte swizzle.  K-major (Q, K: rows of 64 elements along the
// contraction): sbo = 1024 between 8-row groups, lbo unused.  MN-major (V: rows are the contraction,
// 64 elements along N): lbo between the 64-element panels, sbo = 1024 between 8-row groups.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr, uint32_t lbo) {
  uint64_t d = static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;  // descriptor version
  d |= static_cast<uint64_t>(2u) << 61;  // 128-byte swizzle
  return d;
}

// Instruction descriptor, kind::f16, fp32 accumulators, M = 128.
template <bool kBF, int N, bool kBMnMajor>
__host__ __device__ constexpr uint32_t idesc() {
  return (1u << 4) | (kBF ? (1u << 7) | (1u << 10) : 0u) | (kBMnMajor ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(128 >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]),
        "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]),
        "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]),
        "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr)
      : "memory");
}
// Waits for every tcgen05.ld before it; the registers pass through, so no use moves above the wait.
__device__ __forceinline__ void tmem_wait_ld32(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]),
                 "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]),
                 "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]),
                 "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
               :
               : "memory");
}
// 16 columns, complete on return.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]),
        "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
      "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two fp32 at a time.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

struct TcArgs : AttnArgs {
  CUtensorMap map_k, map_v;  // make_cache_map
  int box_tokens;
  bool tma;
};

template <bool kBF, int D>
__global__ void __maxnreg__(kRegs) attn_prefix_kernel(const __grid_constant__ TcArgs a) {
  using SH = Shape<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SH::BAR_OFF);
  uint64_t* empty = full + kSlots;
  uint64_t* q_full = empty + kSlots;
  uint64_t* s_full = q_full + 2;
  uint64_t* p_half = s_full + 2;
  uint64_t* p_full = p_half + 2;
  uint64_t* pv_done = p_full + 2;
  uint64_t* drain = pv_done + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SH::MISC_OFF);
  volatile uint32_t* abort_flag = tmem_slot + 1;

  const AttentionProblem& p = a.p;
  const Plan& pl = a.plan;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  launch_dependents();
  __shared__ int64_t own_steps[kThreads / 32];
  {
    int64_t own = 0;  // steps of the sequences' own keys
    if (pl.private_parts)
      for (int b = threadIdx.x; b < p.B; b += kThreads) own += stream_steps(own_length(p, b));
#pragma unroll
    for (int d = 16; d; d >>= 1) own += __shfl_xor_sync(0xffffffffu, own, d);
    if (lane == 0) own_steps[warp] = own;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(&q_full[h], 4);  // the half's softmax warps
      mbar_init(&s_full[h], 1);
      mbar_init(&p_half[h], 4);
      mbar_init(&p_full[h], 4);
      mbar_init(&pv_done[h], 1);
    }
    mbar_init(drain, 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 10) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "n"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  int64_t own = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) own += own_steps[w];
  const int per = split_sms(pl, p.kv.heads, own * pl.private_tiles, static_cast<int64_t>(p.B) * pl.private_tiles).per;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.tc_per = per;

  // Bounded waits; a role that gives up sets the flag, and the others leave at their next wait.
  // All lanes of a warp wait together and get one answer.  The clock is read before the test that
  // decides, so that a pause between the two (a context switch) gives nothing up.
  const auto give_up = [&] {
    atomicOr(a.status, kStatusAttnTimeout);
    *abort_flag = 1u;
  };
  const auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const uint64_t t0 = globaltimer_ns();
    while (true) {
      const bool late = globaltimer_ns() - t0 > kWaitLimitNs;
      if (__all_sync(0xffffffffu, mbar_try_wait_hint(bar, parity, AWQ_MBAR_SUSPEND_HINT_NS))) return true;
      if (__any_sync(0xffffffffu, *abort_flag != 0u)) return false;
      if (__any_sync(0xffffffffu, late)) {
        give_up();
        return false;
      }
    }
  };

  // this block's steps, tile by tile
  const int total = p.kv.heads * (pl.tc_tiles / pl.tc_lanes) * pl.tc_steps;
  const int group = blockIdx.x / pl.tc_lanes, tile_lane = blockIdx.x - group * pl.tc_lanes;
  const int s_begin = tc_first_step(group, per, total), s_end = min(total, s_begin + per);  // none for a group beyond the last
  const int stacked = p.B * p.n * pl.group;
  struct Segment {
    int hk, row0, halves, step0, steps, part;
  };
  const auto segment = [&](int at) {
    Segment s;
    const int u = at / pl.tc_steps;
    s.hk = pl.tc_lanes > 1 ? u : u / pl.tc_tiles;
    s.row0 = (pl.tc_lanes > 1 ? tile_lane : u - s.hk * pl.tc_tiles) * kTcRows;
    s.halves = stacked - s.row0 > 128 ? 2 : 1;
    s.step0 = at - u * pl.tc_steps;
    s.steps = min(pl.tc_steps - s.step0, s_end - at);
    s.part = group - tc_first_group(pl, u, per);
    return s;
  };

  if (warp < 8) {
    // ------------------------------------------------------------------ softmax ----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
    [&] {
      const int h = warp >> 2;
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t ts = tmem + lanes + kColS + h * 128, to = tmem + lanes + kColO + h * 128;
      uint8_t* q_tile = smem + SH::Q_OFF + h * SH::TILE;
      const int row = (warp & 3) * 32 + lane;  // of the half
      // a negative scale goes to the query's sign bits, so that the largest S is the largest logit
      const uint32_t flip = p.scale < 0.f ? 0x80008000u : 0u;
      // a scale of zero: the smallest factor, under which every finite logit is zero, but -inf stays
      const float sl = p.scale == 0.f ? 0x1p-126f : fabsf(p.scale) * kLog2e;
      uint32_t steps_done = 0, segs = 0;
      for (int at = s_begin; at < s_end;) {
        const Segment sg = segment(at);
        at += sg.steps;
        if (h >= sg.halves) continue;
        const int r = sg.row0 + h * 128 + row;
        const bool in = r < stacked;
        const int g = r % pl.group, bi = r / pl.group;
        {
          // the warp's 32 query rows, whole rows at a time
          const int64_t off = in ? static_cast<int64_t>(bi / p.n) * p.q_sb + static_cast<int64_t>(bi % p.n) * p.q_sn +
                                       static_cast<int64_t>(sg.hk * pl.group + g) * p.q_sh
                                 : -1;
          constexpr int CH = D / 8;
          uint4 v[CH];
#pragma unroll
          for (int i = 0; i < CH; ++i) {
            const int x = i * 32 + lane, k = x / CH, c = x % CH;  // chunk c of the warp's row k
            const int64_t o = __shfl_sync(0xffffffffu, off, k);
            v[i] = make_uint4(0u, 0u, 0u, 0u);
            if (sg.row0 + h * 128 + (warp & 3) * 32 + k < stacked) v[i] = __ldg(reinterpret_cast<const uint4*>(p.q + o) + c);
          }
#pragma unroll
          for (int i = 0; i < CH; ++i) {
            const int x = i * 32 + lane, k = x / CH, c = x % CH;
            const uint4 w = make_uint4(v[i].x ^ flip, v[i].y ^ flip, v[i].z ^ flip, v[i].w ^ flip);
            *reinterpret_cast<uint4*>(q_tile + (c >> 3) * SH::PANEL + ((warp & 3) * 32 + k) * 128 + (((c & 7) ^ (k & 7)) << 4)) = w;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&q_full[h]);
        }
        float m = -INFINITY;
        float2 sum0 = make_float2(0.f, 0.f), sum1 = make_float2(0.f, 0.f);
        for (int j = 0; j < sg.steps; ++j, ++steps_done) {
          if (!wait(&s_full[h], steps_done & 1u)) return;
          tc_fence_after();
          float s[128];
          float mx[4] = {m, m, m, m};
          const int left = static_cast<int>(p.prefix_len) - (sg.step0 + j) * kTcKeys;
          tmem_ld32(ts, s);
          tmem_ld32(ts + 32, s + 32);
          tmem_wait_ld32(s);
          tmem_wait_ld32(s + 32);
          tmem_ld32(ts + 64, s + 64);
          tmem_ld32(ts + 96, s + 96);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (c) {
              tmem_wait_ld32(s + 64);
              tmem_wait_ld32(s + 96);
            }
            if (left < 64 * c + 64) {
#pragma unroll
              for (int i = 64 * c; i < 64 * c + 64; ++i) s[i] = i < left ? s[i] : -INFINITY;
            }
#pragma unroll
            for (int i = 64 * c; i < 64 * c + 64; i += 8) {
#pragma unroll
              for (int x = 0; x < 4; ++x) mx[x] = fmaxf(mx[x], fmaxf(s[i + 2 * x], s[i + 2 * x + 1]));
            }
          }
          const float now = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          const bool raise = (now - m) * sl > kRaise || (m == -INFINITY && now > m);
          if (__any_sync(0xffffffffu, raise)) {
            const float next = raise ? now : m;
            const float f = raise ? exp2_approx((m - now) * sl) : 1.f;
            sum0.x *= f, sum0.y *= f, sum1.x *= f, sum1.y *= f;
            m = next;
            if (j > 0) {
              if (!wait(&pv_done[h], (steps_done - 1) & 1u)) return;
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                uint32_t o[16];
                tmem_ld16(to + 16 * c, o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tmem_st16(to + 16 * c, o);
              }
            }
          }
          const float ref = m == -INFINITY ? 0.f : kLift - m * sl;
          const float2 sl2 = make_float2(sl, sl), ref2 = make_float2(ref, ref);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t u[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 z = fma2(make_float2(s[32 * c + 2 * i], s[32 * c + 2 * i + 1]), sl2, ref2);
              const float2 e = make_float2(exp2_approx(z.x), exp2_approx(z.y));
              if (i & 1) sum1 = add2(sum1, e);
              else sum0 = add2(sum0, e);
              u[i] = pack2<kBF>(e.x, e.y);
            }
            tmem_st16(ts + 16 * c, u);
            if (c & 1) {  // the product of the first 64 keys starts while the others' P is made
              tmem_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(c == 1 ? &p_half[h] : &p_full[h]);
            }
          }
        }
        if (!wait(&pv_done[h], (steps_done - 1) & 1u)) return;
        tc_fence_after();
        const int64_t out_row = static_cast<int64_t>(bi) * p.Hq + sg.hk * pl.group + g;
        const int64_t slot = out_row * pl.parts + sg.part;
        // Rows are turned in shared memory, 32 columns at a time, so that a store writes four whole 128-byte
        // lines (a thread's own row would be 32 partial ones); the warp's share of the query tile is free.
        float4* turn = reinterpret_cast<float4*>(q_tile + (warp & 3) * 4096);
        const unsigned rows = __ballot_sync(0xffffffffu, in);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          tmem_ld32(to + 32 * c, o);
          tmem_wait_ld32(o);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) turn[lane * 8 + (i ^ (lane & 7))] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int k = 4 * i + (lane >> 3), x = lane & 7;  // piece x of row k
            const int64_t to_slot = __shfl_sync(0xffffffffu, slot, k);
            if ((rows >> k) & 1u) *reinterpret_cast<float4*>(a.part_o + to_slot * D + 32 * c + 4 * x) = turn[k * 8 + (x ^ (k & 7))];
          }
        }
        __syncwarp();
        tc_fence_before();
        if (in) a.part_ml[slot] = make_float2(m * sl - kLift, (sum0.x + sum0.y) + (sum1.x + sum1.y));
        ++segs;
      }
    }();
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");  // one instruction for the four warps
  }
  if (warp == 8 || warp == 9) {
    // ------------------------------------------------------------------- loads ----
    // warp 8 loads the steps' keys (ring tiles 0, 2, ...), warp 9 their values (1, 3, ...)
    const int kv = warp - 8;
    const uint16_t* base = kv ? p.kv.v : p.kv.k;
    const CUtensorMap* map = kv ? &a.map_v : &a.map_k;
    const int boxes = kTcKeys / a.box_tokens;  // TMA boxes of a whole step
    uint32_t item = kv, pending = ~0u;         // pending: tile copied by cp.async, not handed over yet
    const auto hand_over = [&](uint32_t i) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[i % kSlots]);
    };
    [&] {
      for (int at = s_begin; at < s_end;) {
        const Segment sg = segment(at);
        at += sg.steps;
        for (int j = 0; j < sg.steps; ++j, item += 2) {
          const int key0 = (sg.step0 + j) * kTcKeys;
          if (item >= kSlots) {
            if (p.give_up) return give_up();
            if (!wait(&empty[item % kSlots], (item / kSlots - 1) & 1u)) return;
          }
          uint8_t* tile = smem + SH::RING_OFF + (item % kSlots) * SH::TILE;
          if (a.tma && key0 + kTcKeys <= p.prefix_len) {
            // whole step: one box of 64 elements per panel and run of tokens within a page
            int page = 0, token = 0;
            if (lane < boxes) {
              const int key = key0 + lane * a.box_tokens, slot = key / p.kv.page_size;
              page = __ldg(p.prefix_pages + slot);
              token = key - slot * p.kv.page_size;
            }
            if (elect_one()) mbar_arrive_expect_tx(&full[item % kSlots], SH::TILE);
            __syncwarp();
            for (int i = 0; i < boxes; ++i) {
              const int pg = __shfl_sync(0xffffffffu, page, i), tk = __shfl_sync(0xffffffffu, token, i);
              if (elect_one()) {
#pragma unroll
                for (int n = 0; n < SH::PANELS; ++n)
                  tma_load_4d(tile + n * SH::PANEL + i * a.box_tokens * 128, map, &full[item % kSlots], 64 * n, tk, sg.hk, pg);
              }
              __syncwarp();
            }
            continue;
          }
          // odd pages, or the step the prefix ends in (zero-filled: what follows may be anything)
          constexpr int CH = D / 8;
          const uint32_t dst = smem_u32(tile);
#pragma unroll 1
          for (int b = 0; b < kTcKeys / 32; ++b) {
            const int key = key0 + 32 * b + lane;
            int64_t off = -1;
            if (key < p.prefix_len) {
              const int slot = key / p.kv.page_size, page = __ldg(p.prefix_pages + slot);
              if (page >= 0 && page < p.kv.num_pages)
                off = page * p.kv.page_stride + static_cast<int64_t>(key - slot * p.kv.page_size) * p.kv.token_stride +
                      sg.hk * p.kv.head_stride;
            }
#pragma unroll
            for (int i = 0; i < CH; ++i) {
              const int x = i * 32 + lane, k = x / CH, c = x % CH;  // chunk c of the batch's key k
              const int64_t o = __shfl_sync(0xffffffffu, off, k);
              cp_async16(dst + (32 * b + k) * 128 + (c >> 3) * SH::PANEL + (((c & 7) ^ (k & 7)) << 4),
                         base + (o < 0 ? 0 : o + c * 8), o >= 0);
            }
          }
          cp_async_commit();
          if (a.tma) {  // the prefix's last step: the next ones come by TMA
            cp_async_wait<0>();
            hand_over(item);
            continue;
          }
          if (pending != ~0u) {
            cp_async_wait<1>();
            hand_over(pending);
          }
          pending = item;
        }
      }
    }();
    cp_async_wait<0>();
    if (pending != ~0u) hand_over(pending);
    // No copy may outlive the block, and another role may give up after this one has issued its last: wait, a
    // bounded time, for the last of each slot (in a run to the end the products have waited for them anyway).
    static_assert(kSlots % 2 == 0, "a warp's copies alternate between kSlots / 2 slots");
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t d = 2; d <= kSlots && item >= d; d += 2) {
      const uint32_t i = item - d;
      while (!mbar_try_wait(&full[i % kSlots], (i / kSlots) & 1u) && globaltimer_ns() - t0 < kWaitLimitNs) {
      }
    }
  } else if (warp == 10) {
    // -------------------------------------------------------------------- MMAs ----
    // The whole warp runs the loop and one elected lane issues: every operand is the same in all
    // lanes, so it lives in uniform registers (inside a one-lane branch each MMA would cost a loop
    // over the lanes' values, 130 cycles instead of the tensor core's 64).
    [&] {
      constexpr uint32_t kQK = idesc<kBF, kTcKeys, false>(), kPV = idesc<kBF, D, true>();
      const uint32_t q_addr = smem_u32(smem + SH::Q_OFF), ring = smem_u32(smem + SH::RING_OFF);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      uint32_t slot = 0, phase = 0;  // of the next ring tile
      uint32_t segs0 = 0, segs1 = 0, done0 = 0, done1 = 0;
      const auto next = [&] {
        if (++slot == kSlots) slot = 0, phase ^= 1u;
      };
      const auto qk = [&](uint32_t h, uint32_t sl, bool last) {
        const uint64_t ad = sw128_desc(q_addr + h * SH::TILE, 0), bd = sw128_desc(ring + sl * SH::TILE, 0);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t o = ((k >> 2) * SH::PANEL + (k & 3) * 32) >> 4;
            mma_ss(tm + kColS + h * 128, ad + o, bd + o, kQK, k > 0);
          }
          mma_commit(&s_full[h]);
          if (last) mma_commit(&empty[sl]);
        }
        __syncwarp();
      };
      // the products of the step's first (part 0) or last 64 keys
      const auto pv = [&](uint32_t h, uint32_t sl, uint32_t part, bool accumulate, bool last) {
        const uint64_t bd = sw128_desc(ring + sl * SH::TILE + part * 4 * 2048, SH::PANEL);
        const uint32_t o = tm + kColO + h * 128, pa = tm + kColS + h * 128 + part * 32;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kTcKeys / 32; ++k) mma_ts(o, pa + 8 * k, bd + ((k * 2048) >> 4), kPV, accumulate || k > 0);
          if (part) {
            mma_commit(&pv_done[h]);
            if (last) mma_commit(&empty[sl]);
          }
        }
        __syncwarp();
      };
      // Three waits at the price of one (some 120 cycles each, even if they pass at once; issuing an MMA
      // takes as long as executing one, so they are lost to the tensor core).
      const auto wait3 = [&](uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb, uint64_t* c, uint32_t pc) {
        const bool x = mbar_try_wait(a, pa), y = mbar_try_wait(b, pb), z = mbar_try_wait(c, pc);
        return __all_sync(0xffffffffu, x && y && z) || (wait(a, pa) && wait(b, pb) && wait(c, pc));
      };
      for (int at = s_begin; at < s_end;) {
        const Segment sg = segment(at);
        at += sg.steps;
        const bool two = sg.halves == 2;
        if (!wait(&q_full[0], segs0++ & 1u)) return;
        if (two && !wait(&q_full[1], segs1++ & 1u)) return;
        if (!wait(&full[slot], phase)) return;
        tc_fence_after();
        qk(0, slot, !two);
        if (two) qk(1, slot, true);
        next();
        for (int j = 0; j < sg.steps; ++j) {
          const bool more = j + 1 < sg.steps;
          const uint32_t v = slot, v_phase = phase;
          next();
          const uint32_t k = more ? slot : v, k_phase = more ? phase : v_phase;
          if (more) next();
          if (!wait3(&full[v], v_phase, &full[k], k_phase, &p_half[0], done0 & 1u)) return;
          tc_fence_after();
          pv(0, v, 0, j > 0, !two);
          if (!wait(&p_full[0], done0++ & 1u)) return;
          tc_fence_after();
          pv(0, v, 1, true, !two);
          if (more) qk(0, k, !two);
          if (two) {
            if (!wait(&p_half[1], done1 & 1u)) return;
            tc_fence_after();
            pv(1, v, 0, j > 0, true);
            if (!wait(&p_full[1], done1++ & 1u)) return;
            tc_fence_after();
            pv(1, v, 1, true, true);
            if (more) qk(1, k, true);
          }
        }
      }
    }();
    // nothing of this block may still run when TMEM is freed
    if (elect_one()) mma_commit(drain);
    __syncwarp();
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait_hint(drain, 0u, AWQ_MBAR_SUSPEND_HINT_NS) && globaltimer_ns() - t0 < kWaitLimitNs) {
    }
    __syncwarp();
  }
  __syncthreads();
  if (warp == 10) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols) : "memory");
  }
}

// Tokens of a TMA box: a step is whole boxes and no box crosses a page; 0: the pages do not allow it
// (a box's rows must start at a multiple of 8, where the swizzle pattern repeats).
int box_tokens(int page_size) {
  if (page_size % kTcKeys == 0) return kTcKeys;
  return page_size >= 8 && kTcKeys % page_size == 0 ? page_size : 0;
}

template <bool kBF, int D>
cudaError_t run(const AttnArgs& attn) {
  TcArgs a{};
  static_cast<AttnArgs&>(a) = attn;
  a.box_tokens = box_tokens(attn.p.kv.page_size);
  a.tma = a.box_tokens > 0 && attn.p.prefix_len >= kTcKeys &&
          make_cache_map(&a.map_k, attn.p.kv.k, attn.p, a.box_tokens) && make_cache_map(&a.map_v, attn.p.kv.v, attn.p, a.box_tokens);
  if (!a.tma) a.box_tokens = kTcKeys;
  const cudaError_t e =
      cudaFuncSetAttribute(attn_prefix_kernel<kBF, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<D>::SMEM);
  if (e != cudaSuccess) return e;
  attn_prefix_kernel<kBF, D><<<a.plan.tc_groups * a.plan.tc_lanes, kThreads, Shape<D>::SMEM, a.p.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

bool attn::make_cache_map(CUtensorMap* map, const void* base, const AttentionProblem& p, int box) {
  const uint64_t dims[4] = {static_cast<uint64_t>(p.kv.head_dim), static_cast<uint64_t>(p.kv.page_size),
                            static_cast<uint64_t>(p.kv.heads), static_cast<uint64_t>(p.kv.num_pages)};
  const uint64_t strides[3] = {static_cast<uint64_t>(p.kv.token_stride) * 2, static_cast<uint64_t>(p.kv.head_stride) * 2,
                               static_cast<uint64_t>(p.kv.page_stride) * 2};
  const uint32_t boxes[4] = {64, static_cast<uint32_t>(box), 1, 1};
  return make_tmap_4d(map, p.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, base, dims, strides,
                      boxes, CU_TENSOR_MAP_SWIZZLE_128B);
}

bool attn::tc_head_dim_supported(int D) { return D == 64 || D == 96 || D == 128; }

cudaError_t attn::launch_prefix_tc(const AttnArgs& a) {
  switch (a.p.kv.head_dim) {
    case 64: return a.p.bf16 ? run<true, 64>(a) : run<false, 64>(a);
    case 96: return a.p.bf16 ? run<true, 96>(a) : run<false, 96>(a);
    default: return a.p.bf16 ? run<true, 128>(a) : run<false, 128>(a);
  }
}

}  // namespace awq
