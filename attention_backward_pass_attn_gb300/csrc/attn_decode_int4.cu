// attn_decode_int4.cu -- the single-token attention's kernels for 4-bit caches
// (attn_decode.cuh).
#include "attn_decode.cuh"

namespace attn {

cudaError_t launch_decode_int4(const DecodeArgs& a, cudaStream_t stream) {
  return launch_type<kCacheInt4, false>(a, stream);
}

}  // namespace attn
