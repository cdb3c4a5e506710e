// awq_attention_kv4 for heads of 128.
#include "awq_kv4_attn.cuh"

namespace awq {
namespace kv4 {

cudaError_t run_128(const Args& a, int nt, int grid) {
  const int groups = a.p.cache.groups();
  if (groups == 1) {
    if (a.p.bf16) return nt == 1 ? run<true, 128, 1, 1>(a, grid) : run<true, 128, 1, 2>(a, grid);
    return nt == 1 ? run<false, 128, 1, 1>(a, grid) : run<false, 128, 1, 2>(a, grid);
  }
  if (groups == 2) {
    if (a.p.bf16) return nt == 1 ? run<true, 128, 2, 1>(a, grid) : run<true, 128, 2, 2>(a, grid);
    return nt == 1 ? run<false, 128, 2, 1>(a, grid) : run<false, 128, 2, 2>(a, grid);
  }
  if (a.p.bf16) return nt == 1 ? run<true, 128, 4, 1>(a, grid) : run<true, 128, 4, 2>(a, grid);
  return nt == 1 ? run<false, 128, 4, 1>(a, grid) : run<false, 128, 4, 2>(a, grid);
}

}  // namespace kv4
}  // namespace awq
