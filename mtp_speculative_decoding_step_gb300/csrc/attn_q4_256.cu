// kv_q4_attend's kernels for head dimension 256.
#include "attn_q4.cuh"

namespace mtp {

cudaError_t launch_q4_attn_256(const Q4AttnArgs& a, int n, bool wide, int blocks, cudaStream_t s) {
  return launch_q4_attn<256, false>(a, n, wide, blocks, s);
}

}  // namespace mtp
