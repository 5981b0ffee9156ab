// kv_q4_attend's kernels for head dimension 64.
#include "attn_q4.cuh"

namespace mtp {

cudaError_t launch_q4_attn_64(const Q4AttnArgs& a, int n, bool wide, int blocks, cudaStream_t s) {
  return launch_q4_attn<64, false>(a, n, wide, blocks, s);
}

}  // namespace mtp
