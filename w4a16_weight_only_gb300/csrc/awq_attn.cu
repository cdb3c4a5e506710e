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

constexpr int kWarps = 4;
constexpr int kKeys = 16;    // keys of one warp's step
constexpr int kStages = 3;   // steps in flight per warp

// One block: one row tile (16 MT query rows that share a key/value head) against one run of keys.
// Warp w takes the steps w, w + 4, ...; it copies its own keys and values (cp.async, zero-filled
// past the run's end: what lies there may be anything) and keeps its own (m, l, o), so that warps
// meet only at the end.  Shared rows are padded by 16 bytes: eight rows of a matrix fragment fall
// into different banks for every head size.
template <bool kBF, int D, int MT>
__global__ void __launch_bounds__(kWarps * 32) attn_stream_kernel(const AttnArgs a) {
  constexpr int PITCH = D + 8;
  constexpr int STEP = 2 * kKeys * PITCH;  // elements of one stage: keys, then values
  extern __shared__ __align__(16) uint16_t smem[];
  const AttentionProblem& p = a.p;
  const Plan& pl = a.plan;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // which rows, which keys
  int unit = blockIdx.x;
  const int prefix_units = pl.tc ? 0 : p.kv.heads * pl.prefix_tiles * pl.prefix_parts;
  int b, hk, tile, part, rows, key0, key1, limit0;
  const int* table;
  if (unit < prefix_units) {
    part = unit % pl.prefix_parts;
    unit /= pl.prefix_parts;
    tile = unit % pl.prefix_tiles;
    hk = unit / pl.prefix_tiles;
    b = 0;
    rows = p.B * p.n * pl.group;
    key0 = part * pl.prefix_chunk;
    key1 = min(static_cast<int>(p.prefix_len), key0 + pl.prefix_chunk);
    limit0 = key1;  // every row sees the whole run
    table = p.prefix_pages;
  } else {
    unit -= prefix_units;
    hk = unit % p.kv.heads;
    unit /= p.kv.heads;
    tile = unit % pl.private_tiles;
    unit /= pl.private_tiles;
    part = unit % pl.private_parts;
    b = unit / pl.private_parts;
    rows = p.n * pl.group;
    const int len = min(max(__ldg(p.lens + b), 0), static_cast<int>(p.max_len));
    key0 = part * pl.chunk;
    key1 = min(len, key0 + pl.chunk);
    limit0 = len - p.n + 1;  // query token i sees keys below limit0 + i
    if (key0 >= key1) return;
    part += pl.prefix_parts;
    table = p.pages + b * p.pages_ld;
  }
  const bool own = part >= pl.prefix_parts;
  const int row0 = tile * 16 * MT;

  // address of a key's elements, or of any valid memory with valid = false
  const auto locate = [&](int key, const uint16_t* base, bool* valid) -> const uint16_t* {
    *valid = false;
    if (key >= key1) return base;
    const int slot = key / p.kv.page_size, page = __ldg(table + slot);
    if (page < 0 || page >= p.kv.num_pages) return base;
    *valid = true;
    return base + page * p.kv.page_stride + static_cast<int64_t>(key - slot * p.kv.page_size) * p.kv.token_stride +
           hk * p.kv.head_stride;
  };
  uint16_t* ring = smem + warp * kStages * STEP;
  const auto load_step = [&](int step) {  // step: index among all of the run's 16-key steps
    const int k0 = key0 + step * kKeys;
    if (k0 < key1) {
      uint16_t* st = ring + (step / kWarps) % kStages * STEP;
      constexpr int CH = D / 8;
      // each lane copies half of a key's and half of a value's elements
      const int key = lane >> 1, half = lane & 1;
      bool valid;
      const uint16_t* base = locate(k0 + key, p.kv.k, &valid);
      const int64_t off = base - p.kv.k;
      const uint32_t dk = smem_u32(st + key * PITCH), dv = smem_u32(st + (kKeys + key) * PITCH);
#pragma unroll
      for (int c = 0; c < CH / 2; ++c) {
        const int e = (2 * c + half) * 8;
        const int64_t from = valid ? off + e : 0;
        cp_async16(dk + e * 2, p.kv.k + from, valid);
        cp_async16(dv + e * 2, p.kv.v + from, valid);
      }
    }
    cp_async_commit();
  };
  const int steps = (key1 - key0 + kKeys - 1) / kKeys;
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) load_step(warp + s * kWarps);

  // query fragments, from global memory (rows past the end read as zero)
  uint32_t qf[MT][D / 16][4];
  int limit[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = row0 + m * 16 + h * 8 + (lane >> 2);
      const bool in = r < rows;
      const int g = r % pl.group, bi = r / pl.group;  // bi: query token within the rows' sequences
      const int i = bi % p.n, bb = b + bi / p.n;
      limit[m][h] = own ? min(key1, limit0 + i) : limit0;
      const uint16_t* src = p.q + bb * p.q_sb + i * p.q_sn + (hk * pl.group + g) * p.q_sh + (lane & 3) * 2;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        qf[m][c][h] = in ? *reinterpret_cast<const uint32_t*>(src + c * 16) : 0u;
        qf[m][c][h + 2] = in ? *reinterpret_cast<const uint32_t*>(src + c * 16 + 8) : 0u;
      }
    }
  }

  float o[MT][D / 8][4];
  float top[MT][2], sum[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int c = 0; c < D / 8; ++c) o[m][c][0] = o[m][c][1] = o[m][c][2] = o[m][c][3] = 0.f;
    top[m][0] = top[m][1] = -INFINITY;
    sum[m][0] = sum[m][1] = 0.f;
  }
  const float scale = p.scale * kLog2e;
  const auto mma = [](float(&d)[4], const uint32_t(&x)[4], uint32_t b0, uint32_t b1) {
    if constexpr (kBF) mma16816_bf16(d, x[0], x[1], x[2], x[3], b0, b1);
    else mma16816(d, x[0], x[1], x[2], x[3], b0, b1);
  };

  for (int step = warp; step < steps; step += kWarps) {
    load_step(step + (kStages - 1) * kWarps);
    cp_async_wait<kStages - 1>();
    __syncwarp();
    const uint16_t* st = ring + (step / kWarps) % kStages * STEP;
    const uint32_t ks = smem_u32(st), vs = smem_u32(st + kKeys * PITCH);
    float s[MT][2][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < 2; ++t) s[m][t][0] = s[m][t][1] = s[m][t][2] = s[m][t][3] = 0.f;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      uint32_t kf[4];  // (keys 0-7, low), (keys 0-7, high), (keys 8-15, low), (keys 8-15, high)
      const int r = (lane & 7) + (lane >> 4) * 8, e = c * 16 + ((lane >> 3) & 1) * 8;
      ldmatrix_x4(kf, ks + (r * PITCH + e) * 2);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        mma(s[m][0], qf[m][c], kf[0], kf[1]);
        mma(s[m][1], qf[m][c], kf[2], kf[3]);
      }
    }
    const int k0 = key0 + step * kKeys;
    uint32_t pf[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float z[4] = {s[m][0][2 * h], s[m][0][2 * h + 1], s[m][1][2 * h], s[m][1][2 * h + 1]};
        float best = -INFINITY;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int key = k0 + (t >> 1) * 8 + (lane & 3) * 2 + (t & 1);
          z[t] = key < limit[m][h] ? z[t] * scale : -INFINITY;
          best = fmaxf(best, z[t]);
        }
        best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 1));
        best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 2));
        const float now = fmaxf(top[m][h], best);
        const float ref = now == -INFINITY ? 0.f : now;  // a row that has seen no key yet
        const float shrink = exp2_approx(top[m][h] - ref);
        top[m][h] = now;
        sum[m][h] *= shrink;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          o[m][c][2 * h] *= shrink;
          o[m][c][2 * h + 1] *= shrink;
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          z[t] = exp2_approx(z[t] - ref);
          sum[m][h] += z[t];
        }
        pf[m][h] = pack2<kBF>(z[0], z[1]);
        pf[m][h + 2] = pack2<kBF>(z[2], z[3]);
      }
    }
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      uint32_t vf[4];  // (keys 0-7, low), (keys 8-15, low), (keys 0-7, high), (keys 8-15, high)
      const int r = lane & 15, e = c * 16 + (lane >> 4) * 8;
      ldmatrix_x4_trans(vf, vs + (r * PITCH + e) * 2);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        mma(o[m][2 * c], pf[m], vf[0], vf[1]);
        mma(o[m][2 * c + 1], pf[m], vf[2], vf[3]);
      }
    }
    __syncwarp();  // the next load_step overwrites the stage read here
  }
  cp_async_wait<0>();
  __syncthreads();

  // join the four warps: (m, l) first, then each warp's o scaled to the common maximum
  float* ml = reinterpret_cast<float*>(smem);            // [kWarps][16 MT][2]
  float* acc = ml + kWarps * 16 * MT * 2;                // [kWarps][16 MT][D + 4]
  constexpr int OP = D + 4;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float l = sum[m][h];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      if ((lane & 3) == 0) {
        const int r = m * 16 + h * 8 + (lane >> 2);
        ml[(warp * 16 * MT + r) * 2] = top[m][h];
        ml[(warp * 16 * MT + r) * 2 + 1] = l;
      }
    }
  __syncthreads();
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = m * 16 + h * 8 + (lane >> 2);
      float all = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) all = fmaxf(all, ml[(w * 16 * MT + r) * 2]);
      const float f = exp2_approx(top[m][h] - (all == -INFINITY ? 0.f : all));
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        float2* dst = reinterpret_cast<float2*>(acc + (warp * 16 * MT + r) * OP + c * 8 + (lane & 3) * 2);
        *dst = make_float2(o[m][c][2 * h] * f, o[m][c][2 * h + 1] * f);
      }
    }
  __syncthreads();
  for (int x = threadIdx.x; x < 16 * MT * (D / 4); x += kWarps * 32) {
    const int r = x / (D / 4), c = x % (D / 4) * 4;
    if (row0 + r >= rows) break;
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
    float all = -INFINITY, l = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 u = *reinterpret_cast<const float4*>(acc + (w * 16 * MT + r) * OP + c);
      t.x += u.x, t.y += u.y, t.z += u.z, t.w += u.w;
      all = fmaxf(all, ml[(w * 16 * MT + r) * 2]);
    }
    const int rr = row0 + r, g = rr % pl.group, bi = rr / pl.group;
    const int64_t out_row = (static_cast<int64_t>(b) * p.n + bi) * p.Hq + hk * pl.group + g;
    const int64_t at = out_row * pl.parts + part;
    *reinterpret_cast<float4*>(a.part_o + at * D + c) = t;
    if (c == 0) {
      const float ref = all == -INFINITY ? 0.f : all;
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        l += ml[(w * 16 * MT + r) * 2 + 1] * exp2_approx(ml[(w * 16 * MT + r) * 2] - ref);
      a.part_ml[at] = make_float2(all, l);
    }
  }
}

// Joins a row's parts.  One warp per row.
template <bool kBF, int D>
__global__ void __launch_bounds__(128) attn_join_kernel(const AttnArgs a) {
  const AttentionProblem& p = a.p;
  const Plan& pl = a.plan;
  const int lane = threadIdx.x & 31;
  const int64_t rows = static_cast<int64_t>(p.B) * p.n * p.Hq;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (r >= rows) return;
  const int b = static_cast<int>(r / (static_cast<int64_t>(p.n) * p.Hq));
  int len = 0;
  if (pl.private_parts) len = min(max(__ldg(p.lens + b), 0), static_cast<int>(p.max_len));
  int first = pl.prefix_parts;  // parts of the prefix; the private ones follow at slot prefix_parts
  if (pl.tc) {
    const int h = static_cast<int>(r % p.Hq), hk = h / pl.group;
    const int64_t stacked = r / p.Hq * pl.group + h % pl.group;
    const int t = hk * pl.tc_tiles + static_cast<int>(stacked / kTcRows);
    first = tc_last_block(pl, t) - tc_first_block(pl, t) + 1;
  }
  const int own = pl.chunk ? (len + pl.chunk - 1) / pl.chunk : 0;
  const int parts = first + own, skip = pl.prefix_parts - first;  // slot of part s: s, from `first` on s + skip
  const float2* ml = a.part_ml + r * pl.parts;
  const float* src = a.part_o + r * pl.parts * D;
  float all = -INFINITY;
  for (int s = 0; s < parts; ++s) all = fmaxf(all, ml[s < first ? s : s + skip].x);
  const float ref = all == -INFINITY ? 0.f : all;
  constexpr int N = D / 32;
  float acc[N] = {}, l = 0.f;
  for (int s = 0; s < parts; ++s) {
    const int slot = s < first ? s : s + skip;
    const float f = exp2_approx(ml[slot].x - ref);
    l += ml[slot].y * f;
#pragma unroll
    for (int c = 0; c < N; ++c) acc[c] += src[static_cast<int64_t>(slot) * D + c * 32 + lane] * f;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;  // a row that sees no key is zero
#pragma unroll
  for (int c = 0; c < N; ++c) p.out[r * D + c * 32 + lane] = float_to_elem<kBF>(acc[c] * inv);
}

int ceil_div(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

Plan make_plan(const AttentionProblem& p, int sms) {
  Plan pl{};
  pl.group = p.Hq / p.kv.heads;
  const int own_rows = p.n * pl.group;
  pl.mt = own_rows > 16 && p.kv.head_dim <= 128 ? 2 : 1;
  const int tile = 16 * pl.mt;
  const int64_t want = 2 * sms;  // blocks that fill the GPU
  const int64_t stacked = static_cast<int64_t>(p.B) * own_rows;  // rows that share a prefix key
  pl.tc = p.prefix_len > 0 && tc_head_dim_supported(p.kv.head_dim) && stacked > 32;
  if (pl.tc) {
    pl.tc_tiles = ceil_div(stacked, kTcRows);
    pl.tc_steps = ceil_div(p.prefix_len, kTcKeys);
    const int64_t total = static_cast<int64_t>(p.kv.heads) * pl.tc_tiles * pl.tc_steps;
    pl.tc_per = max(2, ceil_div(total, sms));
    pl.tc_blocks = ceil_div(total, pl.tc_per);
    pl.prefix_parts = min((pl.tc_steps - 1) / pl.tc_per + 2, pl.tc_blocks);
  } else if (p.prefix_len > 0) {
    pl.prefix_tiles = ceil_div(stacked, tile);
    const int64_t units = static_cast<int64_t>(p.kv.heads) * pl.prefix_tiles;
    const int cuts = static_cast<int>(max(int64_t{1}, min(static_cast<int64_t>(ceil_div(want, units)),
                                                          static_cast<int64_t>(ceil_div(p.prefix_len, 128)))));
    pl.prefix_chunk = (ceil_div(p.prefix_len, cuts) + 63) / 64 * 64;
    pl.prefix_parts = ceil_div(p.prefix_len, pl.prefix_chunk);
  }
  if (p.max_len > 0) {
    pl.private_tiles = ceil_div(own_rows, tile);
    const int64_t units = static_cast<int64_t>(p.B) * p.kv.heads * pl.private_tiles;
    const int cuts = static_cast<int>(max(int64_t{1}, min(static_cast<int64_t>(ceil_div(4 * want, units)),
                                                          static_cast<int64_t>(ceil_div(p.max_len, 128)))));
    pl.chunk = (ceil_div(p.max_len, cuts) + 63) / 64 * 64;
    pl.private_parts = ceil_div(p.max_len, pl.chunk);
  }
  pl.parts = pl.prefix_parts + pl.private_parts;
  return pl;
}

template <bool kBF, int D, int MT>
cudaError_t run_stream(const AttnArgs& a) {
  constexpr int ring = kWarps * kStages * 2 * kKeys * (D + 8) * 2;
  constexpr int join = kWarps * 16 * MT * (2 + D + 4) * 4;
  constexpr int smem = ring > join ? ring : join;
  const Plan& pl = a.plan;
  const int64_t units = (pl.tc ? 0 : static_cast<int64_t>(a.p.kv.heads) * pl.prefix_tiles * pl.prefix_parts) +
                        static_cast<int64_t>(a.p.B) * a.p.kv.heads * pl.private_tiles * pl.private_parts;
  if (units == 0) return cudaSuccess;
  if (units > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cudaError_t e = cudaFuncSetAttribute(attn_stream_kernel<kBF, D, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  attn_stream_kernel<kBF, D, MT><<<static_cast<unsigned>(units), kWarps * 32, smem, a.p.stream>>>(a);
  return cudaGetLastError();
}

template <bool kBF, int D>
cudaError_t run(const AttnArgs& a) {
  cudaError_t e = a.plan.tc ? launch_prefix_tc(a) : cudaSuccess;
  if (e != cudaSuccess) return e;
  if constexpr (D <= 128) e = a.plan.mt == 2 ? run_stream<kBF, D, 2>(a) : run_stream<kBF, D, 1>(a);
  else e = run_stream<kBF, D, 1>(a);
  if (e != cudaSuccess) return e;
  const int64_t rows = static_cast<int64_t>(a.p.B) * a.p.n * a.p.Hq;
  attn_join_kernel<kBF, D><<<static_cast<unsigned>((rows + 3) / 4), 128, 0, a.p.stream>>>(a);
  return cudaGetLastError();
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

size_t attention_workspace_bytes(const AttentionProblem& p, int sms) {
  const Plan pl = make_plan(p, sms);
  const size_t slots = static_cast<size_t>(p.B) * p.n * p.Hq * pl.parts;
  return slots * p.kv.head_dim * 4 + slots * 8;
}

cudaError_t launch_attention(const AttentionProblem& p, int sms) {
  AttnArgs a{p, make_plan(p, sms), nullptr, nullptr, nullptr};
  if (a.plan.tc) {
    const cudaError_t e = status_word_ptr(&a.status);
    if (e != cudaSuccess) return e;
  }
  const size_t slots = static_cast<size_t>(p.B) * p.n * p.Hq * a.plan.parts;
  a.part_o = static_cast<float*>(p.workspace);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + slots * p.kv.head_dim);
  return p.bf16 ? run_dim<true>(a) : run_dim<false>(a);
}

}  // namespace awq
