// attn_decode_score.cu -- the single-token attention's kernels with changed
// scores (attn_decode.cuh).  Kernels of their own: the test for a cap and for
// slopes is made once a step, but what it guards takes registers that the
// plain kernels' loads need.
#include "attn_decode.cuh"

namespace attn {

cudaError_t launch_decode_score(const DecodeArgs& a, cudaStream_t stream) {
  if (a.c.type == kCacheInt4) return launch_type<kCacheInt4, true>(a, stream);
  return a.c.type == kCacheE4m3 ? launch_type<kCacheE4m3, true>(a, stream)
                                : launch_type<kCacheBf16, true>(a, stream);
}

}  // namespace attn
