// score.h -- attention with changed scores (a tanh cap, a bias that falls with
// distance) and shared key heads: the problem, its launchers and their C ABI's
// helpers, shared between score_fwd.cu, score_bwd.cu and score_api.cu.
// Internal to the library.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kernels.h"
#include "score_tanh.h"

namespace attn {

// The current device's error word (attn_api.cu); null if it has none.
int* error_word_ptr();

// The backward's dx, and what is summed of it, are 2^14 times themselves
// (score_bwd.cuh).
constexpr float kPxUp = 16384.f, kPxDown = 1.f / 16384.f, kPxUpLog2 = 14.f;

// What turns a raw product u = <q, k> into a score in base 2.
struct ScoreMap {
  float scale_log2;   // scale log2(e)
  float poly[kTanhTerms];  // x = u (poly[0] + poly[1] u^2 + ...), for |u| <= poly_limit
  float poly_limit;   // negative: never
  float far_poly[kTanhFarTerms];  // the same for |u| <= far_limit
  float far_limit;
  float exp_scale;    // 2 log2(e) scale / cap
  float cap_log2;     // cap log2(e)
  float der_sq;       // -kPxUp / cap_log2^2: times x^2 it is -kPxUp tanh^2
  const float* slopes;  // [Hq] or null
};

struct ScoreProblem {
  int B, Hq, Hkv, group;  // group = Hq / Hkv
  int split;              // backward: items that share a group's heads, a divisor of group
  int N, d;
  int n_tiles, Npad;
  int causal, window;     // window 0: none
  const int* doc;         // [B][N] or null
  const int* prefix;      // [B] or null
  bool cap;
  ScoreMap map;
};

// Fills the map's constants; false if one of them is not finite.
bool make_score_map(float scale, float softcap, const float* slopes, ScoreMap* m);

// 4-D bf16 tensor map over [B][H][N][d] rows with element strides (batch,
// head, token; the head dim is contiguous), 64 x 128 boxes, 128-byte swizzle.
// Returns 0 on success.
int make_rows_map(CUtensorMap* map, const void* ptr, const int64_t strides[3], int B, int H, int N,
                  int d);

cudaError_t launch_score_fwd(const CUtensorMap& tmQ, const CUtensorMap& tmK,
                             const CUtensorMap& tmV, void* O, float* L, const ScoreProblem& p,
                             int* err, cudaStream_t stream);

// The backward's workspace is the plain one's for Hq heads (L2, D, acc); with
// documents its tables hold, per batch element: items [B][n_tiles].x, the last
// query tile that sees a key tile; qend [B][Npad], per key one past its
// document's last query; order [B * n_tiles], the key tiles by their number of
// query tiles, most first (launch_bwd_order).
cudaError_t launch_score_bwd_tables(const Workspace& ws, const ScoreProblem& p,
                                    cudaStream_t stream);

struct ScoreBwdMaps {
  CUtensorMap q, k, v;       // make_rows_map
  CUtensorMap dout, dk, dv;  // make_tile_map
  CUtensorMap acc;           // make_acc_map
};
// sums: with split > 1, fp32 [2][B][Hkv][split][Npad][d], dV's and dK's parts.
int score_bwd_split(const ScoreProblem& p, int sms);
cudaError_t launch_score_bwd_main(const ScoreBwdMaps& m, const Workspace& ws, float* sums,
                                  const ScoreProblem& p, float scale, int* err,
                                  cudaStream_t stream);
cudaError_t launch_score_bwd_split(const ScoreBwdMaps& m, const Workspace& ws, float* sums,
                                   const ScoreProblem& p, float scale, int* err,
                                   cudaStream_t stream);  // the former's, with split > 1
cudaError_t launch_score_bwd_join(void* dK, void* dV, const float* sums, const ScoreProblem& p,
                                  float scale, cudaStream_t stream);

}  // namespace attn
