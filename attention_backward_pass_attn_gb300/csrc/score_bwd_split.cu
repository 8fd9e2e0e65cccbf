// score_bwd_split.cu -- the backward's main kernel for key heads whose query heads
// are dealt to several items (score_bwd.cuh).
#include "score_bwd.cuh"

namespace attn {

cudaError_t launch_score_bwd_split(const ScoreBwdMaps& m, const Workspace& ws, float* sums,
                                   const ScoreProblem& p, float scale, int* err,
                                   cudaStream_t stream) {
  return p.d == 64 ? score_bwd::launch_d<64, true>(m, ws, sums, p, scale, err, stream)
                   : score_bwd::launch_d<128, true>(m, ws, sums, p, scale, err, stream);
}

}  // namespace attn
