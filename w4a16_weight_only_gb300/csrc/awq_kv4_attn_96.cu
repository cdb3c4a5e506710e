// awq_attention_kv4 for heads of 96.
#include "awq_kv4_attn.cuh"

namespace awq {
namespace kv4 {

cudaError_t run_96(const Args& a, int nt, int grid) {
  if (a.p.bf16) return nt == 1 ? run<true, 96, 3, 1>(a, grid) : run<true, 96, 3, 2>(a, grid);
  return nt == 1 ? run<false, 96, 3, 1>(a, grid) : run<false, 96, 3, 2>(a, grid);
}

}  // namespace kv4
}  // namespace awq
