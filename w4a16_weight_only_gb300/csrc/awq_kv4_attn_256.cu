// awq_attention_kv4 for heads of 256.
#include "awq_kv4_attn.cuh"

namespace awq {
namespace kv4 {

cudaError_t run_256(const Args& a, int nt, int grid) {
  (void)nt;
  const int groups = a.p.cache.groups();
  if (groups == 2) {
    return a.p.bf16 ? run<true, 256, 2, 1>(a, grid) : run<false, 256, 2, 1>(a, grid);
  }
  if (groups == 4) {
    return a.p.bf16 ? run<true, 256, 4, 1>(a, grid) : run<false, 256, 4, 1>(a, grid);
  }
  return a.p.bf16 ? run<true, 256, 8, 1>(a, grid) : run<false, 256, 8, 1>(a, grid);
}

}  // namespace kv4
}  // namespace awq
