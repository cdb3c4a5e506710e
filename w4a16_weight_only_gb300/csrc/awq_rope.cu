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

}  // namespace

cudaError_t launch_rope_table(const RopeTableProblem& p) {
  const int64_t blocks = (p.max_position * (p.rot / 2) + 255) / 256;
  rope_table_kernel<<<static_cast<unsigned>(blocks < 4096 ? blocks : 4096), 256, 0, p.stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_rope(const RopeProblem& p) {
  const unsigned grid = static_cast<unsigned>(p.T < (1 << 20) ? p.T : (1 << 20));
  if (p.bf16) rope_any_kernel<true><<<grid, 128, 0, p.stream>>>(p);
  else rope_any_kernel<false><<<grid, 128, 0, p.stream>>>(p);
  return cudaGetLastError();
}

}  // namespace awq
