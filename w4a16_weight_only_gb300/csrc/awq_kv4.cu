// The 4-bit key/value cache: the append that rotates and quantizes, and the read.
//
// A group of `group` neighbouring elements x of a head is kept as 4-bit codes, a scale and a minimum:
//
//   m = min x,  s = rn16((max x - m) / 15),  c = clamp(rint((x - m) / s), 0, 15),  x ~ c s + m
//
// Keys are rotated first and rounded to the element type, as the 16-bit cache would hold them.  Every
// operation is rounded to fp32 by itself (no fused product and sum), so that a code is a function of the
// inputs that any implementation can follow bit for bit.  Differences are taken of halves, (x / 2 - m / 2)
// / (s / 2): the same quotient, without overflow for bf16.  A group with an infinity or a NaN has no
// codes: its minimum and scale are NaN, and all of it reads NaN.
#include "awq_step.cuh"

namespace awq {
namespace {

constexpr uint32_t kFull = 0xffffffffu;

// First byte of the tile of a slot's token and head, nullptr when the slot lies outside the cache; row: the
// token's row in the tile.
__device__ __forceinline__ uint8_t* tile_of(const Kv4Cache& c, int slot, int head, int* row) {
  if (slot < 0 || slot >= static_cast<int64_t>(c.num_pages) * c.page_size) return nullptr;
  const int page = slot / c.page_size, token = slot - page * c.page_size;
  *row = token & 15;
  return c.data + page * c.page_stride + head * c.head_stride + static_cast<int64_t>(token >> 4) * c.tile_bytes();
}

__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fffffff); }

// Elements 4 x .. 4 x + 3 of a head of token t, rotated and rounded to the element type.
template <bool kBF>
__device__ __forceinline__ void load_quad(const AppendKv4Problem& p, const uint16_t* src, int x, bool turn, const float* line,
                                          uint16_t (&out)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int e = 4 * x + j;
    out[j] = src[e];
    if (!turn || e >= p.rot) continue;
    const int half = p.rot / 2, i = p.interleaved ? e >> 1 : e % half;
    const bool second = p.interleaved ? e & 1 : e >= half;
    const float own = elem_to_float<kBF>(out[j]);
    const float other = elem_to_float<kBF>(src[p.interleaved ? e ^ 1 : second ? e - half : e + half]);
    const float c = line ? __ldg(line + i) : quiet_nan(), s = line ? __ldg(line + half + i) : quiet_nan();
    const float a = __fmul_rn(own, c), b = __fmul_rn(other, s);
    out[j] = float_to_elem<kBF>(second ? __fadd_rn(a, b) : __fsub_rn(a, b));
  }
}

// One warp per (token, head): query heads first, then key heads, then value heads.  A lane owns quads of
// elements, so a group is 8, 16 or 32 neighbouring lanes.
template <bool kBF>
__global__ void __launch_bounds__(256) append_kernel(const AppendKv4Problem p) {
  const int heads = p.Hq + 2 * p.Hkv, lane = threadIdx.x & 31;
  const int64_t item = blockIdx.x * int64_t{8} + (threadIdx.x >> 5);
  const int64_t t = item / heads;
  if (t >= p.T) return;
  int h = static_cast<int>(item - t * heads);
  const float* line = nullptr;
  const bool turning = p.table != nullptr;
  if (turning) {
    const int pos = __ldg(p.positions + t);
    if (pos >= 0 && pos < p.max_position) line = p.table + static_cast<int64_t>(pos) * p.rot;
  }
  if (h < p.Hq) {
    const uint16_t* src = p.q + t * p.q_st + h * p.q_sh;
    uint16_t* dst = p.q_out + t * p.qo_st + h * p.qo_sh;
    for (int x0 = 0; x0 < p.D / 4; x0 += 32) {
      const int x = x0 + lane;
      uint16_t e[4];
      if (x < p.D / 4) load_quad<kBF>(p, src, x, turning, line, e);
      __syncwarp();  // in place: a quad's partner is read before it is written
      if (x0 == 0 && p.D > 128) {  // two quads per lane: both are read before either is written
        uint16_t f[4];
        load_quad<kBF>(p, src, x + 32, turning, line, f);
        __syncwarp();
        for (int j = 0; j < 4; ++j) dst[4 * (x + 32) + j] = f[j];
        for (int j = 0; j < 4; ++j) dst[4 * x + j] = e[j];
        break;
      }
      if (x < p.D / 4)
        for (int j = 0; j < 4; ++j) dst[4 * x + j] = e[j];
    }
    return;
  }
  h -= p.Hq;
  const bool value = h >= p.Hkv;
  if (value) h -= p.Hkv;
  int row = 0;
  uint8_t* tile = tile_of(p.cache, __ldg(p.slots + t), h, &row);
  if (!tile) return;
  const uint16_t* src = value ? p.v + t * p.v_st + h * p.v_sh : p.k + t * p.k_st + h * p.k_sh;
  const int G = p.cache.groups(), per = p.cache.group / 4;  // lanes of a group
  uint8_t* codes = tile + (value ? 8 * p.D : 0);
  uint16_t* params = reinterpret_cast<uint16_t*>(tile + 16 * p.D + (value ? 64 * G : 0)) + 2 * (row * G);
  for (int x0 = 0; x0 < p.D / 4; x0 += 32) {
    const int x = x0 + lane;
    const bool in = x < p.D / 4;
    uint16_t e[4] = {0, 0, 0, 0};
    if (in) load_quad<kBF>(p, src, x, turning && !value, line, e);
    float f[4], low, high;
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[j] = elem_to_float<kBF>(e[j]);
      bad |= !(fabsf(f[j]) <= 3.4028235e38f);
    }
    low = fminf(fminf(f[0], f[1]), fminf(f[2], f[3]));
    high = fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3]));
    for (int d = 1; d < per; d <<= 1) {
      low = fminf(low, __shfl_xor_sync(kFull, low, d));
      high = fmaxf(high, __shfl_xor_sync(kFull, high, d));
      bad |= __shfl_xor_sync(kFull, bad ? 1 : 0, d) != 0;
    }
    const float range = __fsub_rn(high * 0.5f, low * 0.5f);
    const uint16_t sb = bad ? float_to_elem<kBF>(quiet_nan()) : float_to_elem<kBF>(__fdiv_rn(range, 7.5f));
    const float s = elem_to_float<kBF>(sb);
    uint32_t word = 0;
    if (s > 0.f) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float c = rintf(__fdiv_rn(__fsub_rn(f[j] * 0.5f, low * 0.5f), s * 0.5f));
        word |= static_cast<uint32_t>(fminf(fmaxf(c, 0.f), 15.f)) << (4 * j);
      }
    }
    if (!in) continue;
    *reinterpret_cast<uint16_t*>(codes + (value ? Kv4::value_byte(p.D, row, 2 * x) : Kv4::key_byte(p.D, row, 2 * x))) =
        static_cast<uint16_t>(word);
    if (x % per == 0) {
      params[2 * (x / per)] = sb;
      params[2 * (x / per) + 1] = bad ? sb : float_to_elem<kBF>(low);
    }
  }
}

// One warp per (token, head).
template <bool kBF>
__global__ void __launch_bounds__(256) read_kernel(const ReadKv4Problem p) {
  const Kv4Cache& c = p.cache;
  const int lane = threadIdx.x & 31, D = c.head_dim, G = c.groups();
  const int64_t item = blockIdx.x * int64_t{8} + (threadIdx.x >> 5);
  const int64_t t = item / c.heads;
  if (t >= p.T) return;
  const int h = static_cast<int>(item - t * c.heads);
  int row = 0;
  const uint8_t* tile = tile_of(c, __ldg(p.slots + t), h, &row);
  for (int value = 0; value < 2; ++value) {
    uint16_t* dst = (value ? p.v : p.k) + item * D;
    for (int x = lane; x < D / 4; x += 32) {
      uint16_t out[4] = {0, 0, 0, 0};
      if (tile) {
        const uint32_t word = *reinterpret_cast<const uint16_t*>(
            tile + (value ? 8 * D + Kv4::value_byte(D, row, 2 * x) : Kv4::key_byte(D, row, 2 * x)));
        const uint16_t* params = reinterpret_cast<const uint16_t*>(tile + 16 * D + (value ? 64 * G : 0)) +
                                 2 * (row * G + 4 * x / c.group);
        const float s = elem_to_float<kBF>(params[0]), m = elem_to_float<kBF>(params[1]);
#pragma unroll
        for (int j = 0; j < 4; ++j)  // the product is exact
          out[j] = float_to_elem<kBF>(__fadd_rn(static_cast<float>((word >> (4 * j)) & 15u) * s, m));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) dst[4 * x + j] = out[j];
    }
  }
}

}  // namespace

bool kv4_shape_supported(int64_t D, int64_t group) {
  return (D == 64 || D == 96 || D == 128 || D == 256) && (group == 32 || group == 64 || group == 128) && D % group == 0;
}

cudaError_t launch_append_kv4(const AppendKv4Problem& p) {
  const int64_t items = p.T * (p.Hq + 2 * p.Hkv);
  const unsigned blocks = static_cast<unsigned>((items + 7) / 8);
  if (p.bf16) append_kernel<true><<<blocks, 256, 0, p.stream>>>(p);
  else append_kernel<false><<<blocks, 256, 0, p.stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_read_kv4(const ReadKv4Problem& p) {
  const unsigned blocks = static_cast<unsigned>((p.T * p.cache.heads + 7) / 8);
  if (p.bf16) read_kernel<true><<<blocks, 256, 0, p.stream>>>(p);
  else read_kernel<false><<<blocks, 256, 0, p.stream>>>(p);
  return cudaGetLastError();
}

}  // namespace awq
