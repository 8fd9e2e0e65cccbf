// attn_decode.cu -- the single-token attention's launcher, and its kernels for
// bf16 and e4m3 caches whose scores are not changed (attn_decode.cuh).
#include "attn_decode.cuh"

namespace attn {

cudaError_t launch_decode(const DecodeArgs& args, cudaStream_t stream) {
  DecodeArgs a = args;
  a.group = a.Hq / a.c.Hkv;
  a.group_blocks = (a.group + kDecodeHeads - 1) / kDecodeHeads;
  a.block_heads = (a.group + a.group_blocks - 1) / a.group_blocks;
  a.head_blocks = a.c.Hkv * a.group_blocks;
  a.block_div = make_fast_div(a.group_blocks);
  if (a.score.cap_log2 > 0.f || a.score.slopes) return launch_decode_score(a, stream);
  if (a.c.type == kCacheInt4) return launch_decode_int4(a, stream);
  return a.c.type == kCacheE4m3 ? launch_type<kCacheE4m3, false>(a, stream)
                                : launch_type<kCacheBf16, false>(a, stream);
}

}  // namespace attn
