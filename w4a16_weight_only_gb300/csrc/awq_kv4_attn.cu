// Attention of the newest tokens of each sequence over a 4-bit key/value cache (awq_attention_kv4).
#include "awq_step.cuh"

namespace awq {
namespace {

// One warp per output row; a lane owns quads of elements.
template <bool kBF>
__global__ void __launch_bounds__(128) attention_any_kernel(const AttentionKv4Problem p) {
  const Kv4Cache& c = p.cache;
  const int lane = threadIdx.x & 31, D = c.head_dim, G = c.groups(), quads = D / 4;
  const int64_t row = blockIdx.x * int64_t{4} + (threadIdx.x >> 5);
  if (row >= static_cast<int64_t>(p.B) * p.n * p.Hq) return;
  const int h = static_cast<int>(row % p.Hq), i = static_cast<int>(row / p.Hq % p.n), b = static_cast<int>(row / p.Hq / p.n);
  const int hk = h / (p.Hq / c.heads);
  const uint16_t* q = p.q + b * p.q_sb + i * p.q_sn + h * p.q_sh;
  const int len = static_cast<int>(min(static_cast<int64_t>(max(p.lens[b], 0)), static_cast<int64_t>(p.W) * c.page_size));
  const int at = len - p.n + i;
  float qv[2][4], o[2][4], top = -INFINITY, sum = 0.f;
  for (int u = 0; u < 2; ++u)
    for (int j = 0; j < 4; ++j) {
      const int x = lane + 32 * u;
      qv[u][j] = x < quads ? elem_to_float<kBF>(q[4 * x + j]) : 0.f;
      o[u][j] = 0.f;
    }
  for (int key = 0; key <= at; ++key) {
    if (p.window && key <= at - p.window && key >= p.sinks) {
      key = max(p.sinks, at - p.window + 1) - 1;
      continue;
    }
    const int page = p.pages[b * p.pages_ld + key / c.page_size];
    if (page < 0 || page >= c.num_pages) continue;
    const int token = key % c.page_size, r = token & 15;
    const uint8_t* tile = c.data + page * c.page_stride + hk * c.head_stride + static_cast<int64_t>(token >> 4) * c.tile_bytes();
    float v[2][4], z = 0.f;
    for (int u = 0; u < 2; ++u) {
      const int x = lane + 32 * u;
      if (x >= quads) continue;
      const uint32_t kw = *reinterpret_cast<const uint16_t*>(tile + Kv4::key_byte(D, r, 2 * x));
      const uint32_t vw = *reinterpret_cast<const uint16_t*>(tile + 8 * D + Kv4::value_byte(D, r, 2 * x));
      const uint16_t* kp = reinterpret_cast<const uint16_t*>(tile + 16 * D) + 2 * (r * G + 4 * x / c.group);
      const uint16_t* vp = kp + 32 * G;
      const float ks = elem_to_float<kBF>(kp[0]), km = elem_to_float<kBF>(kp[1]);
      const float vs = elem_to_float<kBF>(vp[0]), vm = elem_to_float<kBF>(vp[1]);
      for (int j = 0; j < 4; ++j) {
        z += qv[u][j] * (static_cast<float>((kw >> (4 * j)) & 15u) * ks + km);
        v[u][j] = static_cast<float>((vw >> (4 * j)) & 15u) * vs + vm;
      }
    }
    for (int d = 16; d; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
    z *= p.scale;
    const float now = fmaxf(top, z);
    const float shrink = top == -INFINITY ? 0.f : expf(top - now), e = expf(z - now);
    top = now;
    sum = sum * shrink + e;
    for (int u = 0; u < 2; ++u)
      for (int j = 0; j < 4; ++j)
        if (lane + 32 * u < quads) o[u][j] = o[u][j] * shrink + e * v[u][j];
  }
  for (int u = 0; u < 2; ++u)
    for (int j = 0; j < 4; ++j) {
      const int x = lane + 32 * u;
      if (x < quads) p.out[row * D + 4 * x + j] = float_to_elem<kBF>(at >= 0 ? o[u][j] / sum : 0.f);
    }
}

}  // namespace

size_t attention_kv4_workspace_bytes(const AttentionKv4Problem& p, int sms) {
  (void)p;
  (void)sms;
  return 0;
}

cudaError_t launch_attention_kv4(const AttentionKv4Problem& p, int sms) {
  (void)sms;
  const int64_t rows = static_cast<int64_t>(p.B) * p.n * p.Hq;
  const unsigned blocks = static_cast<unsigned>((rows + 3) / 4);
  if (p.bf16) attention_any_kernel<true><<<blocks, 128, 0, p.stream>>>(p);
  else attention_any_kernel<false><<<blocks, 128, 0, p.stream>>>(p);
  return cudaGetLastError();
}

}  // namespace awq
