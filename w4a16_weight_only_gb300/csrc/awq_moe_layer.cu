// A mixture-of-experts layer of a few tokens on 4-bit experts, in two kernels (awq_moe_layer):
//
//   act[t, j] = silu(x[t] Wg) * (x[t] Wu)          of expert experts[t, j], fp32 to the workspace
//   out[t]    = base[t] + sum_j weights[t, j] * (act[t, j] Wd)
//
// with  w = (code - zero) * scale  per group of G rows, sums in fp32, the result rounded once.
#include "awq_step.cuh"

namespace awq {
namespace {

// Sum over K of x[k] * w[k][8 c + j] of one expert for the eight columns of word column c.
template <typename F>
__device__ __forceinline__ void dot8(const Stacked& w, int64_t e, int K, int N, int G, int c, bool bf16, F&& x, float (&acc)[8]) {
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
    for (int j = 0; j < 8; ++j) {
      const uint16_t s = w.sc[(g0 + g) * N + 8 * c + j];
      acc[j] += sum[j] * (bf16 ? elem_to_float<true>(s) : elem_to_float<false>(s));
    }
  }
}

// Any shape: one thread per (place, eight columns).
template <bool kBF>
__global__ void __launch_bounds__(128) moe_up_any_kernel(const MoeLayerProblem p, float* act) {
  const int c = blockIdx.x * 128 + threadIdx.x, place = blockIdx.y;
  if (c >= p.I / 8) return;
  const int e = p.experts[place];
  if (e < 0 || e >= p.E) return;
  const uint16_t* x = p.x + static_cast<int64_t>(place / p.k) * p.x_st;
  float gate[8], up[8];
  const auto at = [&](int k) { return elem_to_float<kBF>(x[k]); };
  dot8(p.up, e, p.H, 2 * p.I, p.G, c, kBF, at, gate);
  dot8(p.up, e, p.H, 2 * p.I, p.G, p.I / 8 + c, kBF, at, up);
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
    dot8(p.down, e, p.I, p.H, p.G, c, kBF, [&](int k) { return a[k]; }, y);
    for (int i = 0; i < 8; ++i) sum[i] += p.weights[place] * y[i];
  }
  for (int j = 0; j < 8; ++j) p.out[static_cast<int64_t>(t) * p.H + 8 * c + j] = float_to_elem<kBF>(sum[j]);
}

template <bool kBF>
cudaError_t launch(const MoeLayerProblem& p) {
  float* act = static_cast<float*>(p.workspace);
  if (p.k > 0 && p.I > 0) {
    moe_up_any_kernel<kBF><<<dim3((p.I / 8 + 127) / 128, p.T * p.k), 128, 0, p.stream>>>(p, act);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  moe_down_any_kernel<kBF><<<dim3((p.H / 8 + 127) / 128, p.T), 128, 0, p.stream>>>(p, act);
  return cudaGetLastError();
}

}  // namespace

size_t moe_layer_workspace_bytes(int T, int k, int I) { return static_cast<size_t>(T) * k * I * 4; }

cudaError_t launch_moe_layer(const MoeLayerProblem& p, int sms) {
  (void)sms;
  return p.bf16 ? launch<true>(p) : launch<false>(p);
}

}  // namespace awq
