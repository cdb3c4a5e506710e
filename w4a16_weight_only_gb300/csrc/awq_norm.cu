// The norms before and after a block, around its residual sum (awq_residual_norm):
//
//   t = norm(x) post_weight (+ post_bias), or x;   h = residual + scale gate t;   y = norm(h) weight (+ bias)
//
//   norm(z) = z / sqrt(mean(z^2) + eps), for layer norms of z - mean(z)
//
// in fp32, each output rounded once; y is formed from the unrounded h.
#include "awq_step.cuh"
#include "awq_ptx.cuh"

namespace awq {
namespace {

// Sum over the block; `shared` has room for 32 numbers and is free again at the next call's first barrier.
__device__ __forceinline__ float block_sum(float v, float* shared) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (threadIdx.x & 31) < warps ? shared[threadIdx.x & 31] : 0.f;
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// Any width, stride and alignment: the row is read again for every sum (8191 rows of 5121, norms on either side, a gate per
// row, 227 us; of 5120 by vectors 75).
template <bool kBF>
__global__ void __launch_bounds__(256) norm_any_kernel(const ResidualNormProblem p) {
  __shared__ float shared[32];
  const float inv = 1.f / p.W;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    const uint16_t* x = p.x + t * p.x_st;
    const uint16_t* r = p.residual ? p.residual + t * p.r_st : nullptr;
    const uint16_t* g = p.gate ? p.gate + t * p.g_st : nullptr;
    const auto stats = [&](auto&& at, float* mean, float* rstd) {
      float s = 0.f;
      *mean = 0.f;
      if (p.layer) {
        for (int i = threadIdx.x; i < p.W; i += 256) s += at(i);
        *mean = block_sum(s, shared) * inv;
      }
      s = 0.f;
      for (int i = threadIdx.x; i < p.W; i += 256) {
        const float d = at(i) - *mean;
        s += d * d;
      }
      *rstd = rsqrtf(block_sum(s, shared) * inv + p.eps);
    };
    float pm = 0.f, pr = 1.f, m, rs;
    if (p.post_weight) stats([&](int i) { return elem_to_float<kBF>(x[i]); }, &pm, &pr);
    const auto h_at = [&](int i) {
      float v = elem_to_float<kBF>(x[i]);
      if (p.post_weight) {
        v = (v - pm) * pr * elem_to_float<kBF>(p.post_weight[i]);
        if (p.post_bias) v += elem_to_float<kBF>(p.post_bias[i]);
      }
      if (g) v *= elem_to_float<kBF>(g[i]);
      v *= p.scale;
      return r ? elem_to_float<kBF>(r[i]) + v : v;
    };
    if (p.weight) stats(h_at, &m, &rs);
    for (int i = threadIdx.x; i < p.W; i += 256) {
      const float v = h_at(i);
      p.h[t * p.W + i] = float_to_elem<kBF>(v);
      if (!p.weight) continue;
      float w = (v - m) * rs * elem_to_float<kBF>(p.weight[i]);
      if (p.bias) w += elem_to_float<kBF>(p.bias[i]);
      p.y[t * p.W + i] = float_to_elem<kBF>(w);
    }
    __syncthreads();
  }
}

// Rows of whole aligned 16-byte vectors: one block per row, the row in registers (V vectors a thread), read
// and written once.  HBM-bound for many rows: 8191 of 5120, norms on either side, a gate per row, 419 MB in 72 us,
// 5.8 TB/s (205 us reading the row again for every sum); a round trip for few.  Four vectors a thread, above 16384
// elements, spill 56 bytes.
template <bool kBF, int V>
__global__ void __launch_bounds__(1024) norm_vec_kernel(const ResidualNormProblem p) {
  __shared__ float shared[32];
  const int vectors = p.W / 8;
  const float inv = 1.f / p.W;
  const int64_t t = blockIdx.x;
  const auto at = [&](int v) { return static_cast<int>(threadIdx.x + v * blockDim.x); };
  const auto load = [](const uint16_t* row, int i) { return *(reinterpret_cast<const uint4*>(row) + i); };
  const auto weights = [](const uint16_t* row, int i) { return __ldg(reinterpret_cast<const uint4*>(row) + i); };
  const auto unpack = [](const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 e = ptx::pair_to_float2<kBF>(w[j]);
      f[2 * j] = e.x;
      f[2 * j + 1] = e.y;
    }
  };
  const auto pack = [](const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = static_cast<uint32_t>(float_to_elem<kBF>(f[2 * j])) | (static_cast<uint32_t>(float_to_elem<kBF>(f[2 * j + 1])) << 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
  };
  uint4 raw[V], res[V], gate[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = at(v);
    if (i >= vectors) continue;
    raw[v] = load(p.x + t * p.x_st, i);
    if (p.residual) res[v] = load(p.residual + t * p.r_st, i);
    if (p.gate) gate[v] = load(p.gate + t * p.g_st, i);
  }
  float h[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (at(v) < vectors) {
      unpack(raw[v], h[v]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) h[v][j] = 0.f;
    }
  }
  const auto stats = [&](float* mean, float* rstd) {
    float s = 0.f;
    *mean = 0.f;
    if (p.layer) {
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) s += h[v][j];
      *mean = block_sum(s, shared) * inv;
      s = 0.f;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (at(v) >= vectors) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = h[v][j] - *mean;
        s += d * d;
      }
    }
    *rstd = rsqrtf(block_sum(s, shared) * inv + p.eps);
  };
  const auto normalize = [&](int v, const uint16_t* weight, const uint16_t* bias, float mean, float rstd, float (&to)[8]) {
    float w[8];
    unpack(weights(weight, at(v)), w);
#pragma unroll
    for (int j = 0; j < 8; ++j) to[j] = (h[v][j] - mean) * rstd * w[j];
    if (bias) {
      unpack(weights(bias, at(v)), w);
#pragma unroll
      for (int j = 0; j < 8; ++j) to[j] += w[j];
    }
  };
  float mean, rstd;
  if (p.post_weight) {
    stats(&mean, &rstd);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (at(v) < vectors) normalize(v, p.post_weight, p.post_bias, mean, rstd, h[v]);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (at(v) >= vectors) continue;
    float f[8];
    if (p.gate) {
      unpack(gate[v], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[v][j] *= f[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) h[v][j] *= p.scale;
    if (p.residual) {
      unpack(res[v], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[v][j] += f[j];
    }
    *(reinterpret_cast<uint4*>(p.h + t * p.W) + at(v)) = pack(h[v]);
  }
  if (!p.weight) return;
  stats(&mean, &rstd);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (at(v) >= vectors) continue;
    float f[8];
    normalize(v, p.weight, p.bias, mean, rstd, f);
    *(reinterpret_cast<uint4*>(p.y + t * p.W) + at(v)) = pack(f);
  }
}

bool vectors_fit(const ResidualNormProblem& p) {
  return p.W % 8 == 0 && p.W <= 32768 && (p.x_st | p.r_st | p.g_st) % 8 == 0 && aligned(p.x, 16) && aligned(p.residual, 16) &&
         aligned(p.gate, 16) && aligned(p.post_weight, 16) && aligned(p.post_bias, 16) && aligned(p.weight, 16) &&
         aligned(p.bias, 16) && aligned(p.h, 16) && aligned(p.y, 16);
}

template <bool kBF, int V>
cudaError_t launch_vec(const ResidualNormProblem& p) {
  const int threads = ((p.W / 8 + V - 1) / V + 31) / 32 * 32;
  norm_vec_kernel<kBF, V><<<static_cast<unsigned>(p.T), threads, 0, p.stream>>>(p);
  return cudaGetLastError();
}

template <bool kBF>
cudaError_t launch(const ResidualNormProblem& p, int sms) {
  if (vectors_fit(p)) {
    // One vector a thread where there are few rows (at most two blocks an SM), two where there are many.  Launches back to
    // back, norms on either side, a gate per row: 1 row of 8192 3.7 us with one and 4.2 with two, 304 of 2048 3.1 and 3.9,
    // 304 of 8192 5.6 and 5.3; 608 of 4096 5.4 and 5.3, 1024 of 8192 18.3 and 19.4, 8192 of 4096 57.6 and 58.4, of 8192
    // 119.3 and 116.7.
    const int vectors = p.W / 8, v = vectors <= 1024 && p.T <= 2 * sms ? 1 : vectors <= 2048 ? 2 : 4;
    switch (v) {
      case 1: return launch_vec<kBF, 1>(p);
      case 2: return launch_vec<kBF, 2>(p);
      default: return launch_vec<kBF, 4>(p);
    }
  }
  const unsigned blocks = static_cast<unsigned>(p.T < (1 << 20) ? p.T : (1 << 20));
  norm_any_kernel<kBF><<<blocks, 256, 0, p.stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_residual_norm(const ResidualNormProblem& p, int sms) { return p.bf16 ? launch<true>(p, sms) : launch<false>(p, sms); }

}  // namespace awq
