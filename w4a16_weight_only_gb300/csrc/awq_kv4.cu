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
#include "awq_ptx.cuh"

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

// Codes of a group of elements within low .. high.
template <bool kBF>
struct Quantizer {
  uint16_t sb, mb;
  float low, s;
  __device__ __forceinline__ Quantizer(float lo, float hi, bool bad) : low(lo) {
    const uint16_t nan = float_to_elem<kBF>(quiet_nan());
    sb = bad ? nan : float_to_elem<kBF>(__fdiv_rn(__fsub_rn(hi * 0.5f, lo * 0.5f), 7.5f));
    mb = bad ? nan : float_to_elem<kBF>(lo);
    s = elem_to_float<kBF>(sb);
  }
  __device__ __forceinline__ uint32_t code(float x) const {
    if (!(s > 0.f)) return 0u;
    const float c = rintf(__fdiv_rn(__fsub_rn(x * 0.5f, low * 0.5f), s * 0.5f));
    return static_cast<uint32_t>(fminf(fmaxf(c, 0.f), 15.f));
  }
  // The codes of eight elements.  The quotient by a reciprocal is within 2^-22 of the rounded one's 16, so both
  // round to the same code unless they are near the middle between two: then, rarely, the division decides
  // (8191 tokens, keys and values of 8 heads of 128: 66 us with eight divisions, which bound the kernel).
  __device__ __forceinline__ uint32_t codes(const float (&x)[8]) const {
    if (!(s > 0.f)) return 0u;
    const float half = low * 0.5f, per = __frcp_rn(s * 0.5f);
    constexpr float kWhole = 12582912.f;  // 1.5 2^23: a sum with it is rounded to a whole number
    uint32_t word = 0;
    bool near = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float c = __fmul_rn(__fsub_rn(x[j] * 0.5f, half), per), w = __fadd_rn(c, kWhole), r = __fsub_rn(w, kWhole);
      near |= !(fabsf(c - r) < 0.4999f);
      word |= (min(__float_as_uint(w), __float_as_uint(kWhole) + 15u) & 15u) << (4 * j);
    }
    if (near) {
      word = 0;
#pragma unroll 1
      for (int j = 0; j < 8; ++j) word |= code(x[j]) << (4 * j);
    }
    return word;
  }
  __device__ __forceinline__ uint32_t params() const { return sb | (static_cast<uint32_t>(mb) << 16); }
};

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

// Any size, stride and alignment: one warp per (token, head), query heads first, then key heads, then value heads.  A lane owns quads of
// elements, so a group is 8, 16 or 32 neighbouring lanes.
template <bool kBF>
__global__ void __launch_bounds__(256) append_any_kernel(const AppendKv4Problem p) {
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
    const Quantizer<kBF> quantizer(low, high, bad);
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) word |= quantizer.code(f[j]) << (4 * j);
    if (!in) continue;
    *reinterpret_cast<uint16_t*>(codes + (value ? Kv4::value_byte(p.D, row, 2 * x) : Kv4::key_byte(p.D, row, 2 * x))) =
        static_cast<uint16_t>(word);
    if (x % per == 0) {
      params[2 * (x / per)] = quantizer.sb;
      params[2 * (x / per) + 1] = quantizer.mb;
    }
  }
}

// Any alignment: one warp per (token, head).
template <bool kBF>
__global__ void __launch_bounds__(256) read_any_kernel(const ReadKv4Problem p) {
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

// Aligned tensors, a rotated part of whole vector pairs.  A thread owns vector x (eight elements) of a head
// and keeps its cosines and sines; it goes through the heads, rows of D / 8 threads side by side, first the
// query heads (rotated and written), then keys and values, whose groups are 4, 8 or 16 neighbouring lanes.  A
// vector's codes are one word of the keys, half a word each of two of the values.  Many tokens are near the issue rate
// (8191 of 32 + 8 heads of 128, fp16, 176 MB in 56 us: the schedulers issue in 76 % of their cycles, HBM is at 35 %), few a
// round trip; ten blocks of an SM leave 48 registers a thread, of which 4 bytes (interleaved) to 48 spill (twelve blocks:
// more, 2 us).
constexpr int kThreads = 128;
constexpr int kFlight = 2;

template <bool kBF>
__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 e = ptx::pair_to_float2<kBF>(w[j]);
    f[2 * j] = e.x;
    f[2 * j + 1] = e.y;
  }
}

template <bool kBF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (kBF) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

template <bool kBF, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 10) append_vec_kernel(const AppendKv4Problem p, int q_parts, int q_per, int kv_per) {
  const int L = p.D / 8, R = kThreads / L;  // threads of a row, rows of the block
  const int x = threadIdx.x % L, row = threadIdx.x / L;
  const int64_t t = blockIdx.x;
  const bool turns = p.table && 8 * x < p.rot;
  const int half = p.rot / 16;  // vectors of half the rotated part
  const bool second = !kInterleaved && x >= half;
  float cs[8], sn[8];  // interleaved: four of each
  const auto load_line = [&](int pos) {
    if (!turns) return;
    if (pos >= 0 && pos < p.max_position) {
      const float* line = p.table + static_cast<int64_t>(pos) * p.rot + (kInterleaved ? 4 * x : 8 * (second ? x - half : x));
      *reinterpret_cast<float4*>(cs) = __ldg(reinterpret_cast<const float4*>(line));
      *reinterpret_cast<float4*>(sn) = __ldg(reinterpret_cast<const float4*>(line + p.rot / 2));
      if constexpr (!kInterleaved) {
        *reinterpret_cast<float4*>(cs + 4) = __ldg(reinterpret_cast<const float4*>(line + 4));
        *reinterpret_cast<float4*>(sn + 4) = __ldg(reinterpret_cast<const float4*>(line + p.rot / 2 + 4));
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) cs[j] = sn[j] = quiet_nan();
    }
  };
  const int pos = turns ? __ldg(p.positions + t) : 0;
  const auto own = [&](const uint16_t* src) { return *(reinterpret_cast<const uint4*>(src) + x); };
  const auto other = [&](const uint16_t* src) {  // the vector of the pairs' other elements
    return !kInterleaved && turns ? *(reinterpret_cast<const uint4*>(src) + (second ? x - half : x + half)) : make_uint4(0u, 0u, 0u, 0u);
  };
  const auto rotate = [&](const uint4& a, const uint4& b) {
    uint4 out;
    uint32_t* w = reinterpret_cast<uint32_t*>(&out);
    float f[8], o[8];
    unpack8<kBF>(a, f);
    if constexpr (kInterleaved) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = pack2<kBF>(__fsub_rn(__fmul_rn(f[2 * j], cs[j]), __fmul_rn(f[2 * j + 1], sn[j])),
                          __fadd_rn(__fmul_rn(f[2 * j + 1], cs[j]), __fmul_rn(f[2 * j], sn[j])));
    } else {
      unpack8<kBF>(b, o);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float m = __fmul_rn(f[j], cs[j]), n = __fmul_rn(o[j], sn[j]);
        f[j] = second ? __fadd_rn(m, n) : __fsub_rn(m, n);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = pack2<kBF>(f[2 * j], f[2 * j + 1]);
    }
    return out;
  };

  if (static_cast<int>(blockIdx.y) < q_parts) {
    // Query heads, kFlight of them in flight, the first ones before the position's line.  In place, a vector's partner is read by one thread and written by another:
    // all of a step's reads come before its writes.
    const int h0 = blockIdx.y * q_per, h1 = min(p.Hq, h0 + q_per);
    for (int base = h0; base < h1; base += kFlight * R) {
      uint4 a[kFlight], b[kFlight];
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        const int h = base + u * R + row;
        if (row >= R || h >= h1) continue;
        const uint16_t* src = p.q + t * p.q_st + h * p.q_sh;
        a[u] = own(src);
        b[u] = other(src);
      }
      if (base == h0) load_line(pos);
      if (p.q_out == p.q) __syncthreads();
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        const int h = base + u * R + row;
        if (row >= R || h >= h1) continue;
        *(reinterpret_cast<uint4*>(p.q_out + t * p.qo_st + h * p.qo_sh) + x) = turns ? rotate(a[u], b[u]) : a[u];
      }
    }
    return;
  }
  const int h0 = (blockIdx.y - q_parts) * kv_per, h1 = min(2 * p.Hkv, h0 + kv_per);  // key heads, then value heads
  const int per = p.cache.group / 8, G = p.cache.groups(), slot = __ldg(p.slots + t);
  uint4 next[2];  // the next head's vector, and its pairs' others
  const auto load = [&](int base) {
    const int n = base + row;
    next[0] = next[1] = make_uint4(0u, 0u, 0u, 0u);
    if (row >= R || n >= h1) return;
    const uint16_t* src = n >= p.Hkv ? p.v + t * p.v_st + (n - p.Hkv) * p.v_sh : p.k + t * p.k_st + n * p.k_sh;
    next[0] = own(src);
    if (n < p.Hkv) next[1] = other(src);
  };
  load(h0);
  load_line(pos);
  for (int base = h0; base < h1; base += R) {
    const int n = base + row;
    const bool in = row < R && n < h1, value = n >= p.Hkv;
    const int h = value ? n - p.Hkv : n;
    const uint4 mine[2] = {next[0], next[1]};
    load(base + R);
    const uint4 e = turns && !value ? rotate(mine[0], mine[1]) : mine[0];
    float f[8];
    unpack8<kBF>(e, f);
    float low = f[0], high = f[0];
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      low = fminf(low, f[j]);
      high = fmaxf(high, f[j]);
      bad |= !(fabsf(f[j]) <= 3.4028235e38f);
    }
    for (int d = 1; d < per; d <<= 1) {
      low = fminf(low, __shfl_xor_sync(kFull, low, d));
      high = fmaxf(high, __shfl_xor_sync(kFull, high, d));
      bad |= __shfl_xor_sync(kFull, bad ? 1 : 0, d) != 0;
    }
    int r = 0;
    uint8_t* tile = in ? tile_of(p.cache, slot, h, &r) : nullptr;
    if (!tile) continue;
    const Quantizer<kBF> quantizer(low, high, bad);
    const uint32_t word = quantizer.codes(f);
    if (value) {
      uint8_t* codes = tile + 8 * p.D;
      *reinterpret_cast<uint16_t*>(codes + Kv4::value_byte(p.D, r, 4 * x)) = static_cast<uint16_t>(word);
      *reinterpret_cast<uint16_t*>(codes + Kv4::value_byte(p.D, r, 4 * x + 2)) = static_cast<uint16_t>(word >> 16);
    } else {
      *reinterpret_cast<uint32_t*>(tile + Kv4::key_byte(p.D, r, 4 * x)) = word;
    }
    if (x % per == 0)
      *(reinterpret_cast<uint32_t*>(tile + 16 * p.D + (value ? 64 * G : 0)) + r * G + x / per) = quantizer.params();
  }
}

bool vectors_fit(const AppendKv4Problem& p) {
  return (p.q_st | p.q_sh | p.k_st | p.k_sh | p.v_st | p.v_sh | p.qo_st | p.qo_sh) % 8 == 0 && p.rot % 16 == 0 && aligned(p.q, 16) &&
         aligned(p.k, 16) && aligned(p.v, 16) && aligned(p.q_out, 16) && aligned(p.table, 16);
}

template <bool kBF, bool kInterleaved>
cudaError_t launch_vec(const AppendKv4Problem& p, int sms) {
  const int R = kThreads / (p.D / 8);
  // Few tokens: as many blocks as give a thread one head; many: a block for a token's query heads, one for its others.
  // By the former's blocks, 16 per SM (ten run at a time): 64 + 8 heads of 128, 64 tokens (640 blocks) 4.1 and 5.3 us, 160
  // (1600) 5.3 and 5.5, 256 (2560) 6.4 and 6.1, 1024 16.5 and 12.5; 32 + 8 of 128, 256 tokens (1536) 5.2 and 5.9, 512
  // (3072) 7.8 and 7.1; 40 + 40 of 96, 128 tokens (1536) 6.2 and 13.3, 512 (6144) 15.9 and 17.3; 16 + 1 of 256, 160
  // tokens (800) 4.0 and 3.6.
  const bool few = p.T * ((p.Hq + R - 1) / R + (2 * p.Hkv + R - 1) / R) < int64_t{16} * sms;
  const int q_per = few ? R : p.Hq, kv_per = few ? R : 2 * p.Hkv;
  const int q_parts = p.Hq ? (p.Hq + q_per - 1) / q_per : 0, kv_parts = (2 * p.Hkv + kv_per - 1) / kv_per;
  append_vec_kernel<kBF, kInterleaved>
      <<<dim3(static_cast<unsigned>(p.T), static_cast<unsigned>(q_parts + kv_parts)), kThreads, 0, p.stream>>>(p, q_parts, q_per, kv_per);
  return cudaGetLastError();
}

// Aligned outputs: a thread has a vector of a key head and the same of the value head, behind a slot and a tile that it
// reads one after the other: 8191 tokens of 8 heads of 128, 43 MB in 15 us.
template <bool kBF>
__global__ void __launch_bounds__(kThreads) read_vec_kernel(const ReadKv4Problem p) {
  const Kv4Cache& c = p.cache;
  const int L = c.head_dim / 8, D = c.head_dim, G = c.groups();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x, item = i / L;
  if (item >= p.T * c.heads) return;
  const int x = static_cast<int>(i - item * L);
  const int64_t t = item / c.heads;
  const int h = static_cast<int>(item - t * c.heads);
  int r = 0;
  const uint8_t* tile = tile_of(c, __ldg(p.slots + t), h, &r);
  uint32_t word[2] = {0u, 0u}, params[2] = {0u, 0u};
  if (tile) {
    word[0] = *reinterpret_cast<const uint32_t*>(tile + Kv4::key_byte(D, r, 4 * x));
    word[1] = *reinterpret_cast<const uint16_t*>(tile + 8 * D + Kv4::value_byte(D, r, 4 * x)) |
              (static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(tile + 8 * D + Kv4::value_byte(D, r, 4 * x + 2))) << 16);
    const uint32_t* at = reinterpret_cast<const uint32_t*>(tile + 16 * D) + r * G + 8 * x / c.group;
    params[0] = at[0];
    params[1] = at[16 * G];
  }
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    const float2 sm = ptx::pair_to_float2<kBF>(params[v]);
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // the products are exact
      const float a = static_cast<float>((word[v] >> (8 * j)) & 15u) * sm.x, b = static_cast<float>((word[v] >> (8 * j + 4)) & 15u) * sm.x;
      w[j] = pack2<kBF>(__fadd_rn(a, sm.y), __fadd_rn(b, sm.y));
    }
    *(reinterpret_cast<uint4*>((v ? p.v : p.k) + item * D) + x) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

}  // namespace

bool kv4_shape_supported(int64_t D, int64_t group) {
  return (D == 64 || D == 96 || D == 128 || D == 256) && (group == 32 || group == 64 || group == 128) && D % group == 0;
}

cudaError_t launch_append_kv4(const AppendKv4Problem& p, int sms) {
  if (vectors_fit(p)) {
    if (p.bf16) return p.interleaved ? launch_vec<true, true>(p, sms) : launch_vec<true, false>(p, sms);
    return p.interleaved ? launch_vec<false, true>(p, sms) : launch_vec<false, false>(p, sms);
  }
  const int64_t items = p.T * (p.Hq + 2 * p.Hkv);
  const unsigned blocks = static_cast<unsigned>((items + 7) / 8);
  if (p.bf16) append_any_kernel<true><<<blocks, 256, 0, p.stream>>>(p);
  else append_any_kernel<false><<<blocks, 256, 0, p.stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_read_kv4(const ReadKv4Problem& p) {
  if (aligned(p.k, 16) && aligned(p.v, 16)) {
    const unsigned blocks = static_cast<unsigned>((p.T * p.cache.heads * (p.cache.head_dim / 8) + kThreads - 1) / kThreads);
    if (p.bf16) read_vec_kernel<true><<<blocks, kThreads, 0, p.stream>>>(p);
    else read_vec_kernel<false><<<blocks, kThreads, 0, p.stream>>>(p);
    return cudaGetLastError();
  }
  const unsigned blocks = static_cast<unsigned>((p.T * p.cache.heads + 7) / 8);
  if (p.bf16) read_any_kernel<true><<<blocks, 256, 0, p.stream>>>(p);
  else read_any_kernel<false><<<blocks, 256, 0, p.stream>>>(p);
  return cudaGetLastError();
}

}  // namespace awq
