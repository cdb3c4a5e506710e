// The norms before and after a block, around its residual sum (awq_residual_norm):
//
//   t = norm(x) post_weight (+ post_bias), or x;   h = residual + scale gate t;   y = norm(h) weight (+ bias)
//
//   norm(z) = z / sqrt(mean(z^2) + eps), for layer norms of z - mean(z)
//
// in fp32, each output rounded once; y is formed from the unrounded h.
#include "awq_step.cuh"

namespace awq {
namespace {

template <int kThreads>
__device__ __forceinline__ float block_sum(float v, float* shared) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  if constexpr (kThreads > 32) {
    __syncthreads();
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (threadIdx.x & 31) < kThreads / 32 ? shared[threadIdx.x & 31] : 0.f;
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  }
  return v;
}

// Any width, stride and alignment: the row is read again for every sum.
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
        *mean = block_sum<256>(s, shared) * inv;
      }
      s = 0.f;
      for (int i = threadIdx.x; i < p.W; i += 256) {
        const float d = at(i) - *mean;
        s += d * d;
      }
      *rstd = rsqrtf(block_sum<256>(s, shared) * inv + p.eps);
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

}  // namespace

cudaError_t launch_residual_norm(const ResidualNormProblem& p) {
  const unsigned blocks = static_cast<unsigned>(p.T < (1 << 20) ? p.T : (1 << 20));
  if (p.bf16) norm_any_kernel<true><<<blocks, 256, 0, p.stream>>>(p);
  else norm_any_kernel<false><<<blocks, 256, 0, p.stream>>>(p);
  return cudaGetLastError();
}

}  // namespace awq
