// kv_q4_attend_tree's kernels for head dimension 256.
#include "attn_q4.cuh"

namespace mtp {

cudaError_t launch_q4_tree_256(const Q4AttnArgs& a, int n, bool wide, int blocks, cudaStream_t s) {
  return launch_q4_attn<256, true>(a, n, wide, blocks, s);
}

}  // namespace mtp
