// Attention of a batch whose sequences share a prefix (awq_attention_shared).
//
//   out[r] = sum_j exp(z[r][j]) v[j] / sum_j exp(z[r][j]),   z[r][j] = scale * q[r] . k[j]
//
// over the prefix's keys and the sequence's own ("private") keys.  The sum splits over any
// partition of the keys: a part contributes (m, l, o) = (max z, sum exp(z - m), sum exp(z - m) v),
// and parts join as  M = max m, l = sum l_i exp(m_i - M), o likewise.  So the prefix is taken
// once for the query rows of all sequences (a matrix product with many rows), each sequence's own
// keys once for that sequence's rows, both cut along the keys to fill the GPU, and a last kernel
// joins the parts.
//
// Statistics, sums and parts are fp32; probabilities are rounded to the element type for the
// second matrix product (the first factor of an mma has that type; the sum l uses the unrounded
// ones), and the result is rounded once.
#include "awq_attn.cuh"

namespace awq {
namespace {

using namespace ptx;
using namespace attn;

// ------------------------------------------------------------------------ streaming kernel ----

// An 8 x 8 tile of 16-bit elements, one row per four lanes, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

template <int D, bool kTma>
struct Stream {
  // a step in shared memory: rows of PITCH elements, so that eight rows of a fragment fall into different
  // banks; or (kTma) panels of 64 elements, 16 rows of 128 bytes in the 128-byte swizzle
  static constexpr int PITCH = D + 8, PANELS = (D + 63) / 64;
  static constexpr int HALF = kStreamKeys * (kTma ? PANELS * 64 : PITCH);  // elements of the keys or values
  static constexpr int STEP = 2 * HALF;                               // keys, then values
  static constexpr int STAGES = D <= 64 ? 5 : D <= 96 && !kTma ? 4 : 3;       // steps in flight per warp
  static constexpr int BLOCKS = D <= 128 ? 2 : 1;                     // blocks per SM
  static constexpr int COARSE = 256;                                  // entries of the table of lengths
  static constexpr int RING = kStreamWarps * STAGES * STEP * 2;
  static constexpr int BARS_OFF = RING + COARSE * 8;                  // full[kStreamWarps][STAGES]
  static constexpr int SMEM = BARS_OFF + kStreamWarps * STAGES * 8 + 16 + (kTma ? 1024 : 0);
  static_assert(BLOCKS * (SMEM + 1024) <= 228 * 1024, "shared memory");
};

// n / d for 0 <= n < 2^31 by a multiplication: m = ceil(2^(31 + l) / d), l = ceil(log2 d), is below
// 2^32, and n m / 2^(31 + l) exceeds n / d by less than 1 / d (Granlund and Montgomery, 1994).
struct Divider {
  uint32_t m, shift;
  static Divider by(uint32_t d) {
    uint32_t l = 0;
    while ((uint64_t{1} << l) < d) ++l;
    return {static_cast<uint32_t>(((uint64_t{1} << (31 + l)) + d - 1) / d), 31 + l};
  }
  __device__ __forceinline__ int of(int n) const {
    return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * m) >> shift);
  }
};

struct StreamArgs : AttnArgs {
  CUtensorMap map_k, map_v;  // kTma
  Divider page, group, n;  // by the page size, the heads of a group, the new tokens of a sequence
};

// Whether one of two elements is infinite or NaN (all bits of its exponent set).
template <bool kBF>
__device__ __forceinline__ bool any_not_finite(uint32_t pair) {
  constexpr uint32_t lo = kBF ? 0x7f80u : 0x7c00u, hi = lo << 16;
  return (pair & lo) == lo || (pair & hi) == hi;
}


// Where a warp stands: a unit and a step of it.
struct Cursor {
  int b;       // sequence, -1: the prefix
  int tile;    // row tile
  int step, steps;
  int len;
};

// Each warp works alone: it copies its own keys and values into a ring, keeps its own (m, l, o), and writes
// a part when its unit or its share ends.  Pages of whole steps come by TMA, boxes of 16 tokens of 64
// elements (kTma); other pages by cp.async, whole rows by all lanes (128 sequences as below: 192 and 199 us a
// call, the kernels one after the other).  What follows a sequence's end may be anything: it is zero-filled.
// The copies run ahead across units, so the memory system is busy from the first step to the last; 2 blocks
// of 4 warps per SM keep about 130 KB per SM in flight.  HBM-bound on all SMs: 128 sequences of 1024 own keys
// on average, 8 heads of 128, 537 MB in 90 us (5.9 TB/s).  On 40 SMs alone 151 us (3.6 TB/s), of which the
// copies are 110: so it shares the SMs with the tensor-core kernel (split_sms).
//
// The products are taken transposed, S^T = K Q^T and O^T += V^T P^T: keys (then elements) fill the 16
// rows of an m16n8k16 and 8 query rows its columns, so that the usual 8 heads of a group waste
// nothing and the accumulators are half those of Q K^T.
template <bool kBF, int D, int NT, bool kTma>
__global__ void __launch_bounds__(kStreamWarps * 32, Stream<D, kTma>::BLOCKS) attn_stream_kernel(const __grid_constant__ StreamArgs a) {
  using ST = Stream<D, kTma>;
  constexpr int STAGES = ST::STAGES;
  extern __shared__ __align__(16) uint16_t smem_raw[];
  uint16_t* smem = kTma ? smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u) / 2 : smem_raw;
  // bytes from a step's keys or values to 16-byte chunk c of row k
  const auto at_chunk = [](int k, int c) {
    return kTma ? (c >> 3) * (kStreamKeys * 128) + k * 128 + (((c & 7) ^ (k & 7)) << 4) : k * (ST::PITCH * 2) + c * 16;
  };
  const AttentionProblem& p = a.p;
  const Plan& pl = a.plan;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t* coarse = reinterpret_cast<int64_t*>(reinterpret_cast<uint8_t*>(smem) + ST::RING);
  const int heads = p.kv.heads, prefix_len = static_cast<int>(p.prefix_len);
  const auto length = [&](int b) { return b < p.B ? own_length(p, b) : 0; };
  const auto steps_of = [](int len) { return stream_steps(len); };

  // coarse[g]: steps (of one unit each) of the sequences before g * gran; its last entry: of all
  const int gran = (p.B + ST::COARSE - 2) / (ST::COARSE - 1);
  if (pl.private_parts) {
    for (int g = threadIdx.x; g < ST::COARSE; g += kStreamWarps * 32) {
      int64_t n = 0;
      const int b1 = min(p.B, (g + 1) * gran);
      for (int b = g * gran; b < b1; ++b) n += steps_of(length(b));
      coarse[g] = n;
    }
    __syncthreads();
    if (warp == 0) {
      constexpr int E = ST::COARSE / 32;
      int64_t v[E], run = 0;
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = coarse[lane * E + i];
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int64_t c = v[i];
        v[i] = run;
        run += c;
      }
      int64_t before = run;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, before, d);
        if (lane >= d) before += o;
      }
      before -= run;
#pragma unroll
      for (int i = 0; i < E; ++i) coarse[lane * E + i] = before + v[i];
    }
    __syncthreads();
  }
  const int64_t prefix_total = pl.tc ? 0 : static_cast<int64_t>(steps_of(prefix_len)) * pl.prefix_tiles;
  const int64_t total = prefix_total + (pl.private_parts ? coarse[ST::COARSE - 1] * pl.private_tiles : 0);
  int shares = pl.shares;
  if (pl.tc) {
    const int left = split_sms(pl, heads, total, static_cast<int64_t>(p.B) * pl.private_tiles).left;
    if (left > 0) shares = max(1, min(shares, left * (ST::BLOCKS * kStreamWarps) / heads));
  }
  const int64_t per = max(static_cast<int64_t>(pl.per_min), (total + shares - 1) / shares);
  const int w = blockIdx.x * kStreamWarps + warp, hk = w % heads, share = w / heads;
  const int64_t x0 = share * per, x1 = share < shares ? min(total, x0 + per) : x0;
  launch_dependents();
  if (x0 >= x1) {
    if (pl.tc && blockIdx.x == gridDim.x - 1) grid_dependency_wait();
    return;
  }

  // the first step's unit
  Cursor at;
  int64_t unit_start;  // of the unit's first step, among all
  {
    int64_t rem = x0;
    if (x0 < prefix_total) {
      at.b = -1;
      at.len = prefix_len;
    } else {
      const int64_t own = x0 - prefix_total;
      const int64_t q = pl.private_tiles == 1 ? own : own / pl.private_tiles;  // in steps of one tile per sequence
      int lo = 0, hi = ST::COARSE - 1;                           // coarse[lo] <= q < coarse[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (coarse[mid] <= q) lo = mid;
        else hi = mid;
      }
      int64_t before = coarse[lo];
      for (int b0 = lo * gran;; b0 += 32) {  // 32 sequences at a time; q lies below the last entry
        const int n = steps_of(length(b0 + lane));
        int incl = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, incl, d);
          if (lane >= d) incl += o;
        }
        const unsigned past = __ballot_sync(0xffffffffu, before + incl > q);
        if (past) {
          const int l = __ffs(past) - 1;
          before += __shfl_sync(0xffffffffu, incl - n, l);
          at.b = b0 + l;
          break;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
      }
      at.len = length(at.b);
      rem = x0 - prefix_total - before * pl.private_tiles;
    }
    at.steps = steps_of(at.len);
    at.tile = rem < at.steps ? 0 : static_cast<int>(rem / at.steps);
    at.step = static_cast<int>(rem - static_cast<int64_t>(at.tile) * at.steps);
  }
  unit_start = x0 - at.step;
  const auto advance = [&](Cursor& c) {  // to the first step of the next unit
    c.step = 0;
    if (++c.tile < (c.b < 0 ? pl.prefix_tiles : pl.private_tiles)) return;
    c.tile = 0;
    do {
      ++c.b;
      c.len = length(c.b);
    } while (c.len == 0 && c.b < p.B);
    c.steps = steps_of(c.len);
  };

  // Copies: 32 lanes take whole rows, so that every line is asked for once.  Lane l < 16 holds where
  // key l of the next step to load starts; its page was read a step earlier.
  constexpr int CH = D / 8;  // 16-byte chunks of a row
  uint16_t* ring = smem + warp * STAGES * ST::STEP;
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(smem) + ST::BARS_OFF) + warp * STAGES;
  if constexpr (kTma) {
    if (lane == 0) {
      for (int s = 0; s < STAGES; ++s) mbar_init(&full[s], 1);
      fence_mbar_init();
    }
    __syncwarp();
  }
  Cursor ahead = at;
  int64_t to_load = x1 - x0;
  uint32_t loaded = 0;  // steps
  int page_next = 0, token_next = 0;
  const auto fetch_page = [&] {
    const int key = ahead.step * kStreamKeys + (kTma ? 0 : lane & 15), slot = a.page.of(key);
    const int* table = ahead.b < 0 ? p.prefix_pages : p.pages + ahead.b * p.pages_ld;
    page_next = key < ahead.len ? __ldg(table + slot) : -1;
    token_next = key - slot * p.kv.page_size;
  };
  const auto load_step = [&] {
    if (kTma && to_load > 0) {  // a step lies in one page
      const int page = page_next, token = token_next;
      --to_load;
      if (++ahead.step == ahead.steps && to_load > 0) advance(ahead);
      if (to_load > 0) fetch_page();
      if (lane == 0) {
        uint64_t* bar = &full[loaded % STAGES];
        uint16_t* dst = ring + loaded % STAGES * ST::STEP;
        mbar_arrive_expect_tx(bar, ST::STEP * 2);
#pragma unroll
        for (int n = 0; n < ST::PANELS; ++n) {  // a page outside the cache: zeros
          tma_load_4d(dst + n * kStreamKeys * 64, &a.map_k, bar, 64 * n, token, hk, page);
          tma_load_4d(dst + ST::HALF + n * kStreamKeys * 64, &a.map_v, bar, 64 * n, token, hk, page);
        }
      }
      __syncwarp();
      ++loaded;
    } else if (to_load > 0) {
      const int page = page_next;
      const bool valid = page >= 0 && page < p.kv.num_pages;
      const int64_t off = page * p.kv.page_stride + static_cast<int64_t>(token_next) * p.kv.token_stride +
                          hk * p.kv.head_stride;
      const uint32_t live = __ballot_sync(0xffffffffu, valid);
      --to_load;
      if (++ahead.step == ahead.steps && to_load > 0) advance(ahead);
      if (to_load > 0) fetch_page();
      const uint32_t dk = smem_u32(ring + loaded % STAGES * ST::STEP);
#pragma unroll
      for (int i = 0; i < kStreamKeys * CH / 32; ++i) {
        const int t = i * 32 + lane, k = t / CH, c = t % CH;  // chunk c of key k
        const int64_t o = __shfl_sync(0xffffffffu, off, k);
        const bool in = (live >> k) & 1u;
        const int64_t from = in ? o + c * 8 : 0;
        cp_async16(dk + at_chunk(k, c), p.kv.k + from, in);
        cp_async16(dk + ST::HALF * 2 + at_chunk(k, c), p.kv.v + from, in);
      }
      ++loaded;
    }
    if constexpr (!kTma) cp_async_commit();
  };
  fetch_page();
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) load_step();

  const float scale = p.scale * kLog2e;
  const auto mma = [](float(&d)[4], const uint32_t(&x)[4], uint32_t b0, uint32_t b1) {
    if constexpr (kBF) mma16816_bf16(d, x[0], x[1], x[2], x[3], b0, b1);
    else mma16816(d, x[0], x[1], x[2], x[3], b0, b1);
  };

  // Step `used` has arrived.  A bounded wait: one that gives up sets the status word, and the warp leaves
  // once its copies in flight have landed (waiting for each a bounded time too).  The clock is read before
  // the test that decides, so that a pause between the two (a context switch) gives nothing up.
  const auto arrived = [&](uint32_t used) -> bool {
    const auto there = [&] { return __all_sync(0xffffffffu, mbar_try_wait(&full[used % STAGES], (used / STAGES) & 1u)) != 0; };
    if (there()) return true;
    const uint64_t t0 = globaltimer_ns();
    while (true) {
      const bool late = __any_sync(0xffffffffu, globaltimer_ns() - t0 > kWaitLimitNs);
      if (there()) return true;
      if (late) return false;
    }
  };
  uint32_t used = 0;  // steps
  bool gave_up = false;
  for (int64_t x = x0; x < x1 && !gave_up;) {
    // one run of a unit
    const int row0 = at.tile * (8 * NT);
    const int rows = at.b < 0 ? p.B * pl.own_rows : pl.own_rows, b0 = max(at.b, 0);
    const int end = at.step + static_cast<int>(min(static_cast<int64_t>(at.steps - at.step), x1 - x));
    uint32_t qf[NT][D / 16][2];
    const bool causal = at.b >= 0 && p.n > 1;
    int limit[NT][2];  // keys that the lane's two rows of each column tile see
#pragma unroll
    for (int m = 0; m < NT; ++m) {
      const int r = row0 + m * 8 + (lane >> 2), bi = a.group.of(r), g = r - bi * pl.group;  // bi: query token within the rows' sequences
      const int s = a.n.of(bi);
      const uint16_t* src = p.q + (b0 + s) * p.q_sb + (bi - s * p.n) * p.q_sn + (hk * pl.group + g) * p.q_sh + (lane & 3) * 2;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        qf[m][c][0] = r < rows ? __ldg(reinterpret_cast<const uint32_t*>(src + c * 16)) : 0u;
        qf[m][c][1] = r < rows ? __ldg(reinterpret_cast<const uint32_t*>(src + c * 16 + 8)) : 0u;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // an own unit's query token is its row's: b0 + 0
        const int i = a.group.of(row0 + m * 8 + (lane & 3) * 2 + h);
        limit[m][h] = at.b < 0 ? at.len : min(at.len, at.len - p.n + 1 + i);
      }
    }
    float o[NT][D / 16][4];
    float top[NT][2], sum[NT][2];
#pragma unroll
    for (int m = 0; m < NT; ++m) {
#pragma unroll
      for (int c = 0; c < D / 16; ++c) o[m][c][0] = o[m][c][1] = o[m][c][2] = o[m][c][3] = 0.f;
      top[m][0] = top[m][1] = -INFINITY;
      sum[m][0] = sum[m][1] = 0.f;
    }

    for (int step = at.step; step < end; ++step, ++used) {
      load_step();
      uint16_t* st = ring + used % STAGES * ST::STEP;
      const uint32_t ks = smem_u32(st), vs = ks + ST::HALF * 2;
      if constexpr (kTma) {
        if (p.give_up || !arrived(used)) {
          gave_up = true;
          break;
        }
        const int live = at.len - step * kStreamKeys;  // what follows the last key may be anything: values to zero
        if (live < kStreamKeys) {
          for (int i = live * CH + lane; i < kStreamKeys * CH; i += 32)
            *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(st + ST::HALF) + at_chunk(i / CH, i % CH)) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();  // before the copy that overwrites them
        }
      } else {
        cp_async_wait<STAGES - 1>();
      }
      __syncwarp();
      float s[NT][2][4];  // two chains
#pragma unroll
      for (int m = 0; m < NT; ++m)
#pragma unroll
        for (int t = 0; t < 2; ++t) s[m][t][0] = s[m][t][1] = s[m][t][2] = s[m][t][3] = 0.f;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        uint32_t kf[4];  // (keys 0-7, low), (keys 8-15, low), (keys 0-7, high), (keys 8-15, high)
        ldmatrix_x4(kf, ks + at_chunk(lane & 15, 2 * c + (lane >> 4)));
#pragma unroll
        for (int m = 0; m < NT; ++m) mma(s[m][c & 1], kf, qf[m][c][0], qf[m][c][1]);
      }
      const int k0 = step * kStreamKeys + (lane >> 2);
      float z[NT][2][2];  // [row][keys lane / 4, + 8]
      bool raise = false;
#pragma unroll
      for (int m = 0; m < NT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const float v = s[m][0][2 * t + h] + s[m][1][2 * t + h];
            z[m][h][t] = k0 + 8 * t < limit[m][h] ? v * scale : -INFINITY;
          }
          raise |= fmaxf(z[m][h][0], z[m][h][1]) > top[m][h] + kRaise;  // always where no key was seen yet
        }
      // a row's maximum is raised when a logit exceeds it by kRaise
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int m = 0; m < NT; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float now = fmaxf(z[m][h][0], z[m][h][1]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, d));
            now = fmaxf(now, top[m][h]);
            const float shrink = now == -INFINITY ? 1.f : exp2_approx(top[m][h] - now);
            top[m][h] = now;
            sum[m][h] *= shrink;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              o[m][c][h] *= shrink;
              o[m][c][2 + h] *= shrink;
            }
          }
      }
      uint32_t pf[NT][2];
#pragma unroll
      for (int m = 0; m < NT; ++m) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float ref = top[m][h] == -INFINITY ? 0.f : top[m][h] - kLift;  // a row that has seen no key yet: 0
          z[m][h][0] = exp2_approx(z[m][h][0] - ref);
          z[m][h][1] = exp2_approx(z[m][h][1] - ref);
          sum[m][h] += z[m][h][0] + z[m][h][1];
        }
        // P^T has keys along the lanes' rows; the second product wants them along the registers
        pf[m][0] = transpose8(pack2<kBF>(z[m][0][0], z[m][1][0]));
        pf[m][1] = transpose8(pack2<kBF>(z[m][0][1], z[m][1][1]));
      }
      // A key that some of the rows do not see (new tokens among themselves) has p = 0 there, and 0 times
      // a value that is not finite would be NaN: with such a value among them, the step's products are
      // made one by one.
      bool odd = false;
      if (causal && (step + 1) * kStreamKeys > at.len - p.n + 1) {
#pragma unroll 1
        for (int i = lane; i < kStreamKeys * CH; i += 32) {
          const uint4 v = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(st + ST::HALF) + at_chunk(i / CH, i % CH));
          odd |= any_not_finite<kBF>(v.x) | any_not_finite<kBF>(v.y) | any_not_finite<kBF>(v.z) | any_not_finite<kBF>(v.w);
        }
        odd = __any_sync(0xffffffffu, odd);
      }
      if (odd) {
#pragma unroll 1
        for (int k = 0; k < kStreamKeys; ++k) {
          const auto value = [&](int c) {  // element c 8 + lane / 4 of the key
            return elem_to_float<kBF>(*reinterpret_cast<const uint16_t*>(reinterpret_cast<const uint8_t*>(st + ST::HALF) +
                                                                         at_chunk(k, c) + (lane >> 2) * 2));
          };
#pragma unroll
          for (int m = 0; m < NT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float w = __shfl_sync(0xffffffffu, k < 8 ? z[m][h][0] : z[m][h][1], (k & 7) * 4 + (lane & 3));
              if (step * kStreamKeys + k < limit[m][h]) {
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                  o[m][c][h] += w * value(2 * c);
                  o[m][c][2 + h] += w * value(2 * c + 1);
                }
              }
            }
        }
        __syncwarp();
        continue;
      }
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        uint32_t vf[4];  // (elements 0-7, keys 0-7), (8-15, 0-7), (0-7, 8-15), (8-15, 8-15)
        // rows are keys, so the transposed tile's first 8 columns are keys 0-7
        ldmatrix_x4_trans(vf, vs + at_chunk((lane & 7) + (lane >> 4) * 8, 2 * c + ((lane >> 3) & 1)));
#pragma unroll
        for (int m = 0; m < NT; ++m) mma(o[m][c], vf, pf[m][0], pf[m][1]);
      }
      __syncwarp();  // the next load_step overwrites a stage read here
    }

    if (gave_up) break;
    // the part: slot = this share's number among those that meet in the unit
    const int part = unit_start < x0 ? static_cast<int>(share - unit_start / per) : 0;
#pragma unroll
    for (int m = 0; m < NT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float l = sum[m][h];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
        const int r = row0 + m * 8 + (lane & 3) * 2 + h;
        if (r >= rows) continue;
        const int bi = a.group.of(r);
        const int64_t out_row = (static_cast<int64_t>(b0) * p.n + bi) * p.Hq + hk * pl.group + (r - bi * pl.group);
        const int64_t slot = out_row * pl.parts + (at.b < 0 ? 0 : pl.prefix_parts) + part;
        if (lane < 4) a.part_ml[slot] = make_float2(top[m][h] - kLift, l);
        float* dst = a.part_o + slot * D + (lane >> 2);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          dst[c * 16] = o[m][c][h];
          dst[c * 16 + 8] = o[m][c][2 + h];
        }
      }
    if (end == at.steps && lane == 0)
      a.counts[(at.b < 0 ? at.tile : pl.prefix_tiles + static_cast<int64_t>(at.b) * pl.private_tiles + at.tile) * heads + hk] = part + 1;
    x += end - at.step;
    if (x < x1) {
      advance(at);
      unit_start = x;
    }
  }
  if constexpr (!kTma) cp_async_wait<0>();
  if (kTma && gave_up) {
    if (lane == 0) atomicOr(a.status, kStatusAttnTimeout);
    for (; used < loaded; ++used) arrived(used);
  }
  // One block waits, so that this kernel's end is also the tensor-core kernel's; the others make room.
  if (pl.tc && blockIdx.x == gridDim.x - 1) grid_dependency_wait();
}

// Joins a row's parts.  One warp per row; a lane holds the (m, l) of every 32nd part and D / 32
// elements of the sums, and the parts' elements are read BATCH parts at a time.
template <bool kBF, int D, int BATCH>
__global__ void __launch_bounds__(128) attn_join_kernel(const AttnArgs a) {
  const AttentionProblem& p = a.p;
  const Plan& pl = a.plan;
  const int lane = threadIdx.x & 31;
  const int rows = p.B * p.n * p.Hq, r = blockIdx.x * 4 + (threadIdx.x >> 5);  // below 2^31
  if (r >= rows) return;
  const int bi = r / p.Hq, h = r - bi * p.Hq, hk = h / pl.group, b = bi / p.n;
  grid_dependency_wait();  // the parts
  int first = 0, own = 0;  // parts of the prefix, at slots 0 ..; own parts, at slots prefix_parts ..
  if (p.prefix_len > 0) {
    const int stacked = bi * pl.group + h - hk * pl.group;
    if (pl.tc) {
      const int u = tc_unit(pl, hk, stacked / kTcRows), per = *a.tc_per;
      first = tc_last_group(pl, u, per) - tc_first_group(pl, u, per) + 1;
    } else {
      first = a.counts[stacked / pl.tile * p.kv.heads + hk];
    }
    first = parts_within(first, pl.prefix_parts);
  }
  bool sees = p.prefix_len > 0;  // any key at all
  const int own_len = pl.private_parts ? own_length(p, b) : 0;
  if (own_len > 0) {
    sees |= own_len - p.n + 1 + bi - b * p.n > 0;
    const int own_row = (bi - b * p.n) * pl.group + h - hk * pl.group;
    own = parts_within(a.counts[pl.prefix_tiles * p.kv.heads +
                                (static_cast<int64_t>(b) * pl.private_tiles + own_row / pl.tile) * p.kv.heads + hk],
                       pl.private_parts);
  }
  const int parts = first + own, skip = pl.prefix_parts - first;
  const float2* ml = a.part_ml + static_cast<int64_t>(r) * pl.parts;
  constexpr int V = D % 128 == 0 ? 4 : D % 64 == 0 ? 2 : 1, N = D / 32 / V;  // elements of a load, loads of a row
  const float* src = a.part_o + static_cast<int64_t>(r) * pl.parts * D + lane * V;
  float acc[N][V] = {}, l = 0.f, all = -INFINITY;
  for (int s0 = 0; s0 < parts; s0 += 32) {
    const int s = s0 + lane, n = min(32, parts - s0);
    const float2 mine = s < parts ? ml[s < first ? s : s + skip] : make_float2(-INFINITY, 0.f);
    float v[BATCH][N][V];
    const auto load = [&](int i0) {  // a batch of parts; past the last one it is read again, with weight 0
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const int t = s0 + min(i0 + i, n - 1);
        const float* from = src + static_cast<int64_t>(t < first ? t : t + skip) * D;
#pragma unroll
        for (int c = 0; c < N; ++c) {
          if constexpr (V == 4) *reinterpret_cast<float4*>(v[i][c]) = *reinterpret_cast<const float4*>(from + c * 128);
          else if constexpr (V == 2) *reinterpret_cast<float2*>(v[i][c]) = *reinterpret_cast<const float2*>(from + c * 64);
          else v[i][c][0] = from[c * 32];
        }
      }
    };
    load(0);
    float best = mine.x;
#pragma unroll
    for (int d = 16; d; d >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, d));
    const float now = fmaxf(all, best), ref = now == -INFINITY ? 0.f : now;
    const float shrink = exp2_approx(all - ref), f = exp2_approx(mine.x - ref);  // 0 past the last part
    all = now;
    l = l * shrink + mine.y * f;  // this lane's parts
#pragma unroll
    for (int c = 0; c < N; ++c)
#pragma unroll
      for (int e = 0; e < V; ++e) acc[c][e] *= shrink;
    for (int i0 = 0; i0 < n; i0 += BATCH) {
      if (i0) load(i0);
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const float g = __shfl_sync(0xffffffffu, f, i0 + i);
        if (i0 + i < n) {
#pragma unroll
          for (int c = 0; c < N; ++c)
#pragma unroll
            for (int e = 0; e < V; ++e) acc[c][e] += v[i][c][e] * g;
        }
      }
    }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  // l is at least 2^kLift where a logit is finite.  A row that sees no key is zero, one whose logits are all
  // -inf 0 / 0; NaN stays.
  const float inv = l > 0.f ? 1.f / l : l == 0.f && sees ? __int_as_float(0x7fffffff) : l;
  uint16_t* out = p.out + static_cast<int64_t>(r) * D + lane * V;
#pragma unroll
  for (int c = 0; c < N; ++c) {
    if constexpr (V == 4)
      *reinterpret_cast<uint2*>(out + c * 128) =
          make_uint2(pack2<kBF>(acc[c][0] * inv, acc[c][1] * inv), pack2<kBF>(acc[c][2] * inv, acc[c][3] * inv));
    else if constexpr (V == 2) *reinterpret_cast<uint32_t*>(out + c * 64) = pack2<kBF>(acc[c][0] * inv, acc[c][1] * inv);
    else out[c * 32] = float_to_elem<kBF>(acc[c][0] * inv);
  }
}

int ceil_div(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

Plan make_plan(const AttentionProblem& p, int sms) {
  Plan pl{};
  pl.sms = sms;
  pl.group = p.Hq / p.kv.heads;
  pl.own_rows = p.n * pl.group;
  const int64_t stacked = static_cast<int64_t>(p.B) * pl.own_rows;  // rows that share a prefix key
  // Tensor cores from 33 rows on; their steps are counted in 32 bits.  Both sides measured (us a call, tensor
  // cores and streaming kernel; 64 own keys per row's sequence): 40 rows of one head of 128 over 256, 2048 and
  // 16384 keys 13.7 / 14.6, 13.3 / 17.3, 16.3 / 41.8, of eight heads 13.4 / 15.8, 14.5 / 25.1, 27.3 / 65.6; 8 rows
  // of eight heads 13.3 / 10.2, 13.6 / 12.8, 23.6 / 23.5.  Between 17 and 32 rows the tensor cores are the faster
  // ones already (24 rows of eight heads: 13.4 / 15.5, 14.1 / 21.0, 26.4 / 49.8), which this rule leaves.
  pl.tc = p.prefix_len > 0 && tc_head_dim_supported(p.kv.head_dim) && stacked > 32 &&
          static_cast<int64_t>(p.kv.heads) * ceil_div(stacked, kTcRows) * ceil_div(p.prefix_len, kTcKeys) < (int64_t{1} << 30);
  const int64_t rows = pl.tc || p.prefix_len == 0 ? pl.own_rows : stacked;
  pl.tile = rows <= 8 ? 8 : rows <= 16 || p.kv.head_dim > 128 ? 16 : 32;
  const int tile = pl.tile;
  if (pl.tc) {
    pl.tc_tiles = ceil_div(stacked, kTcRows);
    pl.tc_steps = ceil_div(p.prefix_len, kTcKeys);
    pl.tc_lanes = pl.tc_tiles <= sms ? pl.tc_tiles : 1;
    const int total = p.kv.heads * (pl.tc_tiles / pl.tc_lanes) * pl.tc_steps;
    pl.tc_per = max(2, ceil_div(total, sms / pl.tc_lanes));
    pl.tc_groups = ceil_div(total, pl.tc_per);
    pl.prefix_parts = min((pl.tc_steps - 1) / pl.tc_per + 2, pl.tc_groups);
  } else if (p.prefix_len > 0) {
    pl.prefix_tiles = ceil_div(stacked, tile);
  }
  if (p.max_len > 0) pl.private_tiles = ceil_div(pl.own_rows, tile);
  // most steps that the streaming kernel can have per head; the lengths, known on the device only, may
  // add up to less, so shares go down to a quarter of what this many would give each warp
  const int64_t prefix_steps = pl.tc ? 0 : ceil_div(p.prefix_len, kStreamKeys);
  const int64_t own_steps = ceil_div(p.max_len, kStreamKeys);
  const int64_t total = prefix_steps * pl.prefix_tiles + own_steps * p.B * pl.private_tiles;
  const int64_t warps = static_cast<int64_t>(sms) * (p.kv.head_dim <= 128 ? 2 : 1) * kStreamWarps;
  const int64_t shares = max(int64_t{1}, warps / p.kv.heads);
  pl.per_min = static_cast<int>(max(int64_t{2}, min((total + shares - 1) / shares / 4, int64_t{1} << 20)));
  pl.shares = static_cast<int>(min(shares, (total + pl.per_min - 1) / pl.per_min));
  pl.blocks = ceil_div(static_cast<int64_t>(pl.shares) * p.kv.heads, kStreamWarps);
  if (pl.prefix_tiles) pl.prefix_parts = static_cast<int>((prefix_steps - 1) / pl.per_min + 2);
  if (p.max_len > 0) pl.private_parts = static_cast<int>((own_steps - 1) / pl.per_min + 2);
  pl.parts = pl.prefix_parts + pl.private_parts;
  return pl;
}

struct Layout {
  size_t ml, per, counts, bytes;  // offsets; part_o first
};

Layout layout(const AttentionProblem& p, const Plan& pl) {
  const size_t slots = static_cast<size_t>(p.B) * p.n * p.Hq * pl.parts;
  const size_t units = (static_cast<size_t>(pl.prefix_tiles) + static_cast<size_t>(p.B) * pl.private_tiles) * p.kv.heads;
  Layout l;
  l.ml = slots * p.kv.head_dim * 4;
  l.per = l.ml + slots * 8;
  l.counts = l.per + 4;
  l.bytes = l.counts + units * 4;
  return l;
}

// The kernel, set up and where there is room run while the one before it still runs; it waits for that
// one's end itself.  Behind the tensor-core kernel: the streaming kernel runs beside it.  Without that one
// only the join could be early: 0.2 us of 12.0 for 3 over 1000, lost in a call's host time of 22 us.
template <typename A>
cudaError_t launch_early(void (*kernel)(A), unsigned blocks, int threads, size_t smem, cudaStream_t stream, const A& a, bool early) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <bool kBF, int D, int NT, bool kTma>
cudaError_t launch_stream(const AttnArgs& attn, StreamArgs& a) {
  constexpr int smem = Stream<D, kTma>::SMEM;
  const auto kernel = attn_stream_kernel<kBF, D, NT, kTma>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  static_cast<AttnArgs&>(a) = attn;
  a.page = Divider::by(static_cast<uint32_t>(attn.p.kv.page_size));
  a.group = Divider::by(static_cast<uint32_t>(attn.plan.group));
  a.n = Divider::by(static_cast<uint32_t>(attn.p.n));
  return launch_early(kernel, attn.plan.blocks, kStreamWarps * 32, smem, attn.p.stream, a, attn.plan.tc);
}

template <bool kBF, int D, int NT>
cudaError_t run_stream(const AttnArgs& attn) {
  if (attn.plan.blocks == 0) return cudaSuccess;
  StreamArgs a{};
  if (attn.p.kv.page_size % kStreamKeys == 0 && make_cache_map(&a.map_k, attn.p.kv.k, attn.p, kStreamKeys) &&
      make_cache_map(&a.map_v, attn.p.kv.v, attn.p, kStreamKeys))
    return launch_stream<kBF, D, NT, true>(attn, a);
  return launch_stream<kBF, D, NT, false>(attn, a);
}

template <bool kBF, int D>
cudaError_t run(const AttnArgs& a) {
  cudaError_t e = a.plan.tc ? launch_prefix_tc(a) : cudaSuccess;
  if (e != cudaSuccess) return e;
  if (a.plan.tile == 8) e = run_stream<kBF, D, 1>(a);
  else if (a.plan.tile == 16) e = run_stream<kBF, D, 2>(a);
  else if constexpr (D <= 128) e = run_stream<kBF, D, 4>(a);
  if (e != cudaSuccess) return e;
  const int64_t rows = static_cast<int64_t>(a.p.B) * a.p.n * a.p.Hq;
  // few rows: more parts in flight per row (96 rows of 34 parts 5.1 us, 6.1 with eight); many: more rows
  // (8192 rows 10.4 us, 12.1 with sixteen)
  const auto join = D <= 128 && rows <= 2048 ? attn_join_kernel<kBF, D, 16> : attn_join_kernel<kBF, D, 8>;
  return launch_early(join, static_cast<unsigned>((rows + 3) / 4), 128, 0, a.p.stream, a, a.plan.tc && a.plan.blocks > 0);
}

template <bool kBF>
cudaError_t run_dim(const AttnArgs& a) {
  switch (a.p.kv.head_dim) {
    case 64: return run<kBF, 64>(a);
    case 96: return run<kBF, 96>(a);
    case 128: return run<kBF, 128>(a);
    default: return run<kBF, 256>(a);
  }
}

}  // namespace

bool attention_head_dim_supported(int64_t D) { return D == 64 || D == 96 || D == 128 || D == 256; }

size_t attention_workspace_bytes(const AttentionProblem& p, int sms) { return layout(p, make_plan(p, sms)).bytes; }

cudaError_t launch_attention(const AttentionProblem& p, int sms) {
  AttnArgs a{};
  a.p = p;
  a.plan = make_plan(p, sms);
  const cudaError_t e = status_word_ptr(&a.status);
  if (e != cudaSuccess) return e;
  const Layout l = layout(p, a.plan);
  uint8_t* ws = static_cast<uint8_t*>(p.workspace);
  a.part_o = reinterpret_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float2*>(ws + l.ml);
  a.tc_per = reinterpret_cast<int*>(ws + l.per);
  a.counts = reinterpret_cast<int*>(ws + l.counts);
  return p.bf16 ? run_dim<true>(a) : run_dim<false>(a);
}

}  // namespace awq
