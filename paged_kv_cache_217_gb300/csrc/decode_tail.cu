// Decode grids over what remains of sequences: of a batch of prompts those with a single
// query token, and the members of groups behind a prefix that is computed apart.
#include "decode_launch.cuh"

namespace pkv {
cudaError_t launch_decode_tail(const DecodeArgs& a, bool bf16, int head_dim, int gpad, const CUtensorMap* kmap,
                               const CUtensorMap* vmap, cudaStream_t stream) {
  return bf16 ? launch_decode_tail_t<__nv_bfloat16>(a, head_dim, gpad, kmap, vmap, stream)
              : launch_decode_tail_t<__half>(a, head_dim, gpad, kmap, vmap, stream);
}
}  // namespace pkv
