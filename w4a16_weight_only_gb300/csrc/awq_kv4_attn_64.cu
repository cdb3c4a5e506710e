// awq_attention_kv4 for heads of 64.
#include "awq_kv4_attn.cuh"

namespace awq {
namespace kv4 {

cudaError_t run_64(const Args& a, int nt, int grid) {
  const int groups = a.p.cache.groups();
  if (groups == 1) {
    if (a.p.bf16) return nt == 1 ? run<true, 64, 1, 1>(a, grid) : run<true, 64, 1, 2>(a, grid);
    return nt == 1 ? run<false, 64, 1, 1>(a, grid) : run<false, 64, 1, 2>(a, grid);
  }
  if (a.p.bf16) return nt == 1 ? run<true, 64, 2, 1>(a, grid) : run<true, 64, 2, 2>(a, grid);
  return nt == 1 ? run<false, 64, 2, 1>(a, grid) : run<false, 64, 2, 2>(a, grid);
}

}  // namespace kv4
}  // namespace awq
