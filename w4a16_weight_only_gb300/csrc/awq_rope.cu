// Rotary positions: the table of cosines and sines, and the rotation of query and key heads with
// an optional append of keys and values to a paged cache.
//
//   (a, b) -> (a c - b s, b c + a s),  c = cos(p f_i) m,  s = sin(p f_i) m
//
// for pair i of the rotated part of a head (the first `rot` elements; pairs (i, i + rot / 2) or,
// interleaved, (2 i, 2 i + 1)) at position p.  Arithmetic is fp32, rounded once to the element
// type; the table is fp32, its angles are formed in 64 bits (an fp32 product p f loses the angle
// at long contexts: at p = 10^5 its last bit is worth 0.008 radians).
#include "awq_layer.cuh"
#include "awq_ptx.cuh"

namespace awq {
namespace {

// ---- table ----

// f_i = base^(-2 i / rot), scaled for a context `factor` times the trained one:
//   1 linear   f / factor (positions interpolated)
//   2 ntk      base grown so that the slowest pair is stretched by `factor`
//   3 yarn     pairs that turn more than p0 times over the trained context keep f, those that
//              turn less than p1 times take f / factor, a linear ramp over the pair index between
//   4 banded   wavelengths below original / p1 keep f, above original / p0 take f / factor, a
//              blend linear in original / wavelength between
__device__ double scaled_frequency(const RopeTableProblem& p, int i) {
  const double rot = p.rot;
  if (p.scaling == 2) {
    const double base = p.base * pow(p.factor, rot / (rot - 2.0));
    return pow(base, -2.0 * i / rot);
  }
  const double f = pow(p.base, -2.0 * i / rot);
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  if (p.scaling == 1) return f / p.factor;
  if (p.scaling == 3) {
    const double at0 = rot * log(p.original / (p.p0 * kTwoPi)) / (2.0 * log(p.base));
    const double at1 = rot * log(p.original / (p.p1 * kTwoPi)) / (2.0 * log(p.base));
    const double low = fmax(floor(at0), 0.0), high = fmin(ceil(at1), rot - 1.0);
    const double ramp = fmin(fmax((i - low) / fmax(high - low, 0.001), 0.0), 1.0);
    return f / p.factor * ramp + f * (1.0 - ramp);
  }
  if (p.scaling == 4) {
    const double turns = p.original * f / kTwoPi;  // original / wavelength
    if (turns > p.p1) return f;
    if (turns < p.p0) return f / p.factor;
    const double blend = (turns - p.p0) / (p.p1 - p.p0);
    return (1.0 - blend) * f / p.factor + blend * f;
  }
  return f;
}

// One thread per (position, pair), pairs fastest.  Written once per model, so fp64 throughout.
__global__ void __launch_bounds__(256) rope_table_kernel(const RopeTableProblem p) {
  const int half = p.rot / 2;
  const int64_t total = p.max_position * half;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; t < total;
       t += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t pos = t / half;
    const int i = static_cast<int>(t - pos * half);
    double s, c;
    sincos(static_cast<double>(pos) * scaled_frequency(p, i), &s, &c);
    float* line = p.table + pos * p.rot;
    line[i] = static_cast<float>(c * p.attention_factor);
    line[half + i] = static_cast<float>(s * p.attention_factor);
  }
}

// ---- rotation ----

// Where head `h` of token t is read and written: query heads first, then key heads, then (append)
// value heads.  A null destination means that nothing of the head is kept.
struct Row {
  const uint16_t* src;
  uint16_t* dst;
  bool turn;  // value heads are copied
};

__device__ __forceinline__ Row row_of(const RopeProblem& p, int64_t t, int h, int64_t cell) {
  Row r;
  r.turn = true;
  if (h < p.Hq) {
    r.src = p.q + t * p.q_st + h * p.q_sh;
    r.dst = p.q_out + t * p.qo_st + h * p.qo_sh;
    return r;
  }
  h -= p.Hq;
  if (h < p.Hkv) {
    r.src = p.k + t * p.k_st + h * p.k_sh;
    r.dst = p.append ? (cell < 0 ? nullptr : p.kv.k + cell + h * p.kv.head_stride)
                     : p.k_out + t * p.ko_st + h * p.ko_sh;
    return r;
  }
  h -= p.Hkv;
  r.turn = false;
  r.src = p.v + t * p.v_st + h * p.v_sh;
  r.dst = cell < 0 ? nullptr : p.kv.v + cell + h * p.kv.head_stride;
  return r;
}

// First element of token t's cache cell, -1 when the slot lies outside the cache.
__device__ __forceinline__ int64_t cell_of(const RopeProblem& p, int64_t t) {
  if (!p.append) return -1;
  const int slot = __ldg(p.slots + t);
  if (slot < 0 || slot >= static_cast<int64_t>(p.kv.num_pages) * p.kv.page_size) return -1;
  const int page = slot / p.kv.page_size;
  return page * p.kv.page_stride + static_cast<int64_t>(slot - page * p.kv.page_size) * p.kv.token_stride;
}

template <bool kBF>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  return static_cast<uint32_t>(float_to_elem<kBF>(lo)) | (static_cast<uint32_t>(float_to_elem<kBF>(hi)) << 16);
}

// Any size, stride and alignment: one thread per pair or copied element.
template <bool kBF>
__global__ void __launch_bounds__(128) rope_any_kernel(const RopeProblem p) {
  const int half = p.rot / 2, items = half + (p.D - p.rot);
  const int heads = p.Hq + p.Hkv * (p.append ? 2 : 1);
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    const int64_t cell = cell_of(p, t);
    const int pos = __ldg(p.positions + t);
    const bool inside = pos >= 0 && pos < p.max_position;
    const float* line = p.table + static_cast<int64_t>(inside ? pos : 0) * p.rot;
    for (int w = threadIdx.x; w < heads * items; w += 128) {
      const int h = w / items, i = w - h * items;
      const Row r = row_of(p, t, h, cell);
      if (!r.dst) continue;
      if (i >= half) {
        r.dst[p.rot + i - half] = r.src[p.rot + i - half];
        continue;
      }
      const int ia = p.interleaved ? 2 * i : i, ib = p.interleaved ? 2 * i + 1 : i + half;
      const uint16_t ua = r.src[ia], ub = r.src[ib];
      if (!r.turn) {
        r.dst[ia] = ua;
        r.dst[ib] = ub;
        continue;
      }
      const float c = inside ? __ldg(line + i) : __int_as_float(0x7fffffff);
      const float s = inside ? __ldg(line + half + i) : __int_as_float(0x7fffffff);
      const float a = elem_to_float<kBF>(ua), b = elem_to_float<kBF>(ub);
      r.dst[ia] = float_to_elem<kBF>(a * c - b * s);
      r.dst[ib] = float_to_elem<kBF>(b * c + a * s);
    }
  }
}

// Aligned tensors, rotated part and head size multiples of 16.  A thread owns 16 elements of a head, two
// 16-byte vectors: eight pairs (the vectors at 8 c and rot / 2 + 8 c, or 16 c and 16 c + 8 when
// interleaved), or 16 elements behind the rotated part.  It keeps its eight cosines and sines and
// goes through the heads, kUnroll of them in flight, so a table line is read once per token and the
// tensors once: HBM-bound for many tokens (8191 tokens of 64 heads of 128, fp16, 271 MB: 44 us, 6.1
// TB/s; kUnroll 4 and 8: 50 and 68 us, fewer threads fit), a
// single round trip for few (8 tokens: 2.5 us).
constexpr int kRopeThreads = 128;
constexpr int kUnroll = 2;

template <bool kBF, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) rope_vec_kernel(const RopeProblem p, int heads_per_block) {
  const int chunks = p.D / 16, lanes = kRopeThreads / chunks;  // head lanes of the block
  const int c = threadIdx.x % chunks, lane = threadIdx.x / chunks;
  if (lane >= lanes) return;
  const int64_t t = blockIdx.x;
  const int heads = p.Hq + p.Hkv * (p.append ? 2 : 1);
  const int h0 = blockIdx.y * heads_per_block, h1 = min(heads, h0 + heads_per_block);
  const int64_t cell = cell_of(p, t);
  const bool turns = 16 * c < p.rot;
  const int ea = turns && !kInterleaved ? 8 * c : 16 * c, eb = turns && !kInterleaved ? p.rot / 2 + 8 * c : 16 * c + 8;
  float cs[8], sn[8];
  if (turns) {
    const int pos = __ldg(p.positions + t);
    if (pos >= 0 && pos < p.max_position) {
      const float* line = p.table + static_cast<int64_t>(pos) * p.rot + 8 * c;
      *reinterpret_cast<float4*>(cs) = __ldg(reinterpret_cast<const float4*>(line));
      *reinterpret_cast<float4*>(cs + 4) = __ldg(reinterpret_cast<const float4*>(line + 4));
      *reinterpret_cast<float4*>(sn) = __ldg(reinterpret_cast<const float4*>(line + p.rot / 2));
      *reinterpret_cast<float4*>(sn + 4) = __ldg(reinterpret_cast<const float4*>(line + p.rot / 2 + 4));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) cs[i] = sn[i] = __int_as_float(0x7fffffff);
    }
  }
  for (int h = h0 + lane; h < h1; h += kUnroll * lanes) {
    Row r[kUnroll];
    uint4 va[kUnroll], vb[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      r[u].dst = nullptr;
      if (h + u * lanes < h1) r[u] = row_of(p, t, h + u * lanes, cell);
      if (r[u].dst) {
        va[u] = *reinterpret_cast<const uint4*>(r[u].src + ea);
        vb[u] = *reinterpret_cast<const uint4*>(r[u].src + eb);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (!r[u].dst) continue;
      if (turns && r[u].turn) {
        uint32_t* a = reinterpret_cast<uint32_t*>(&va[u]);
        uint32_t* b = reinterpret_cast<uint32_t*>(&vb[u]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 x = ptx::pair_to_float2<kBF>(a[i]), y = ptx::pair_to_float2<kBF>(b[i]);
          if constexpr (kInterleaved) {  // a[i] is pair i, b[i] pair 4 + i
            a[i] = pack<kBF>(x.x * cs[i] - x.y * sn[i], x.y * cs[i] + x.x * sn[i]);
            b[i] = pack<kBF>(y.x * cs[4 + i] - y.y * sn[4 + i], y.y * cs[4 + i] + y.x * sn[4 + i]);
          } else {  // a[i] and b[i] are the first and second elements of pairs 2 i, 2 i + 1
            a[i] = pack<kBF>(x.x * cs[2 * i] - y.x * sn[2 * i], x.y * cs[2 * i + 1] - y.y * sn[2 * i + 1]);
            b[i] = pack<kBF>(y.x * cs[2 * i] + x.x * sn[2 * i], y.y * cs[2 * i + 1] + x.y * sn[2 * i + 1]);
          }
        }
      }
      *reinterpret_cast<uint4*>(r[u].dst + ea) = va[u];
      *reinterpret_cast<uint4*>(r[u].dst + eb) = vb[u];
    }
  }
}

bool vectors_fit(const RopeProblem& p) {
  const int64_t strides = p.q_st | p.q_sh | p.k_st | p.k_sh | p.v_st | p.v_sh | p.qo_st | p.qo_sh |
                          (p.append ? p.kv.page_stride | p.kv.token_stride | p.kv.head_stride : p.ko_st | p.ko_sh);
  return p.rot % 16 == 0 && p.D % 16 == 0 && p.D / 16 <= kRopeThreads && strides % 8 == 0 && aligned(p.q, 16) && aligned(p.k, 16) &&
         aligned(p.v, 16) && aligned(p.q_out, 16) && aligned(p.k_out, 16) && aligned(p.table, 16) && aligned(p.kv.k, 16) &&
         aligned(p.kv.v, 16);
}

template <bool kBF, bool kInterleaved>
cudaError_t launch_vec(const RopeProblem& p) {
  const int heads = p.Hq + p.Hkv * (p.append ? 2 : 1), lanes = kRopeThreads / (p.D / 16);
  // few tokens: a token's heads over as many blocks as give each thread one head
  int per = kUnroll * lanes;
  if (p.T * ((heads + per - 1) / per) < 304) per = lanes;
  else per = heads;
  per = per > (heads + 65534) / 65535 ? per : (heads + 65534) / 65535;
  rope_vec_kernel<kBF, kInterleaved>
      <<<dim3(static_cast<unsigned>(p.T), static_cast<unsigned>((heads + per - 1) / per)), kRopeThreads, 0, p.stream>>>(p, per);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_table(const RopeTableProblem& p) {
  const int64_t blocks = (p.max_position * (p.rot / 2) + 255) / 256;
  rope_table_kernel<<<static_cast<unsigned>(blocks < 4096 ? blocks : 4096), 256, 0, p.stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_rope(const RopeProblem& p) {
  if (vectors_fit(p)) {
    if (p.bf16) return p.interleaved ? launch_vec<true, true>(p) : launch_vec<true, false>(p);
    return p.interleaved ? launch_vec<false, true>(p) : launch_vec<false, false>(p);
  }
  const unsigned grid = static_cast<unsigned>(p.T < (1 << 20) ? p.T : (1 << 20));
  if (p.bf16) rope_any_kernel<true><<<grid, 128, 0, p.stream>>>(p);
  else rope_any_kernel<false><<<grid, 128, 0, p.stream>>>(p);
  return cudaGetLastError();
}

}  // namespace awq
