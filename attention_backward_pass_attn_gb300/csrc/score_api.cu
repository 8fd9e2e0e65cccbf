// score_api.cu -- the C ABI of attention with changed scores (declared in
// include/attn.h): argument validation, the constants of the score map, tensor
// maps, and the calls into the kernel launchers.
#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/attn.h"
#include "score.h"

namespace attn {

static constexpr double kLog2e = 1.4426950408889634;

bool make_score_map(float scale, float softcap, const float* slopes, ScoreMap* m) {
  *m = {};
  m->scale_log2 = float(scale * kLog2e);
  m->slopes = slopes;
  m->poly_limit = m->far_limit = -1.f;
  if (!std::isfinite(m->scale_log2) || softcap == 0.f) return std::isfinite(m->scale_log2);
  const double c = double(scale) / softcap;
  m->exp_scale = float(2 * kLog2e * c);
  m->cap_log2 = float(softcap * kLog2e);
  m->der_sq = float(-kPxUp / (softcap * kLog2e * softcap * kLog2e));
  if (!std::isfinite(m->exp_scale) || !std::isfinite(2 * m->cap_log2)) return false;
  const double s = scale * kLog2e;  // x = u s sum_k c_k (c u)^2k
  bool good = std::isfinite(m->der_sq);
  for (int k = 0; k < kTanhTerms; ++k) {
    m->poly[k] = float(tanh_poly(k) * s * std::pow(c, 2 * k));
    good = good && std::isfinite(m->poly[k]);
  }
  bool far = good;
  for (int k = 0; k < kTanhFarTerms; ++k) {
    m->far_poly[k] = float(tanh_far_poly(k) * s * std::pow(c, 2 * k));
    far = far && std::isfinite(m->far_poly[k]);
  }
  const auto limit = [&](double reach) {
    const float u = float(reach / c);
    return std::isfinite(u) ? u : 3.4e38f;
  };
  if (good) m->poly_limit = limit(kTanhReach);
  m->far_limit = far ? limit(kTanhFarReach) : m->poly_limit;
  return true;
}

namespace {

constexpr int kSms = 152;  // what the backward's items are dealt to

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool good(const void* p, uintptr_t n) { return p && aligned(p, n); }
int status_of(cudaError_t e) { return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA; }

// Sizes, masks and the score map; *empty: nothing to do.
int make_problem(int B, int Hq, int Hkv, int N, int d, int causal, int window, const int* doc,
                 const int* prefix, float softcap, const float* slopes, float scale,
                 ScoreProblem* p, bool* empty) {
  if (B < 0 || Hq < 0 || Hkv < 1 || Hq % Hkv || N < 0 || d < 0) return ATTN_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return ATTN_ERR_INVALID_ARG;
  if (window < 0 || (!causal && (window || doc || prefix))) return ATTN_ERR_INVALID_ARG;
  if (prefix && (window || doc)) return ATTN_ERR_INVALID_ARG;
  if (!aligned(doc, 4) || !aligned(prefix, 4) || !aligned(slopes, 4)) return ATTN_ERR_INVALID_ARG;
  if (!(std::isfinite(scale) && scale > 0.f) || !(std::isfinite(softcap) && softcap >= 0.f))
    return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  *p = {};
  if (!make_score_map(scale, softcap, slopes, &p->map)) return ATTN_ERR_INVALID_ARG;
  *empty = B == 0 || Hq == 0 || N == 0;
  if (*empty) return ATTN_OK;
  const long long n_tiles = (N + 127LL) / 128;
  // every row index, and the grid, inside 31 bits
  if ((long long)B * Hq > INT_MAX || (long long)B * Hq * n_tiles * 128 > INT_MAX)
    return ATTN_ERR_UNSUPPORTED;
  p->B = B;
  p->Hq = Hq;
  p->Hkv = Hkv;
  p->group = Hq / Hkv;
  p->N = N;
  p->d = d;
  p->n_tiles = int(n_tiles);
  p->Npad = int(n_tiles * 128);
  p->causal = causal;
  p->window = window >= N ? 0 : window;
  p->doc = doc;
  p->prefix = prefix;
  p->cap = softcap > 0.f;
  p->split = 1;
  return ATTN_OK;
}

// The plain kernels' shape for H heads.
Shape shape_of(const ScoreProblem& p, int H) {
  Shape s = {};
  s.BH = p.B * H;
  s.N = p.N;
  s.d = p.d;
  s.causal = p.causal;
  s.n_tiles = p.n_tiles;
  s.Npad = p.Npad;
  s.H = H;
  return s;
}

// Where the backward's split sums begin in its workspace, and where they end.
size_t sums_offset(const ScoreProblem& p) {
  return (workspace_bytes(shape_of(p, p.Hq)) + 255) & ~size_t(255);
}
size_t score_workspace_bytes(const ScoreProblem& p) {
  const size_t sums = size_t(p.B) * p.Hkv * p.split * p.Npad * p.d * 2 * sizeof(float);
  return sums_offset(p) + (p.split > 1 ? sums : 0);
}

// Strides of Q, K and V (batch, head, token): the caller's, or contiguous rows'.
struct RowStrides {
  int64_t s[3][3];
};
int set_strides(const int64_t* given, const ScoreProblem& p, RowStrides* out) {
  for (int w = 0; w < 3; ++w) {
    const int H = w ? p.Hkv : p.Hq;
    const int64_t rows[3] = {int64_t(H) * p.N * p.d, int64_t(p.N) * p.d, p.d};
    const int n[3] = {p.B, H, p.N};
    for (int k = 0; k < 3; ++k) {
      // a dimension of one index has no stride to speak of
      const int64_t s = given && n[k] > 1 ? given[3 * w + k] : rows[k];
      if (s < 1 || s % 8) return ATTN_ERR_INVALID_ARG;
      if (s >= int64_t(1) << 39) return ATTN_ERR_UNSUPPORTED;  // 2^40 bytes
      out->s[w][k] = s;
    }
  }
  return ATTN_OK;
}

// The three operands' maps; false if one cannot be encoded.
bool make_maps(CUtensorMap* q, CUtensorMap* k, CUtensorMap* v, const void* Q, const void* K,
               const void* V, const RowStrides& st, const ScoreProblem& p) {
  return !make_rows_map(q, Q, st.s[0], p.B, p.Hq, p.N, p.d) &&
         !make_rows_map(k, K, st.s[1], p.B, p.Hkv, p.N, p.d) &&
         !make_rows_map(v, V, st.s[2], p.B, p.Hkv, p.N, p.d);
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" {

int attn_fwd_score(const void* Q, const void* K, const void* V, const int64_t* strides, void* O,
                   float* L, int B, int Hq, int Hkv, int N, int d, int causal, int window,
                   const int* doc_start, const int* prefix, float softcap, const float* slopes,
                   float scale, void* stream) {
  ScoreProblem p;
  bool empty = false;
  int st = make_problem(B, Hq, Hkv, N, d, causal, window, doc_start, prefix, softcap, slopes,
                        scale, &p, &empty);
  if (st != ATTN_OK || empty) return st;
  if (!good(Q, 16) || !good(K, 16) || !good(V, 16) || !good(O, 16) || !good(L, 4))
    return ATTN_ERR_INVALID_ARG;
  RowStrides rows;
  if ((st = set_strides(strides, p, &rows)) != ATTN_OK) return st;
  int* err = error_word_ptr();
  CUtensorMap mq, mk, mv;
  if (!err || !make_maps(&mq, &mk, &mv, Q, K, V, rows, p)) return ATTN_ERR_CUDA;
  return status_of(launch_score_fwd(mq, mk, mv, O, L, p, err, (cudaStream_t)stream));
}

size_t attn_bwd_score_workspace_size(int B, int Hq, int Hkv, int N, int d, int causal,
                                     int window) {
  ScoreProblem p;
  bool empty = false;
  if (make_problem(B, Hq, Hkv, N, d, causal, window, nullptr, nullptr, 0.f, nullptr, 1.f, &p,
                   &empty) != ATTN_OK || empty)
    return 0;
  p.split = score_bwd_split(p, kSms);
  return score_workspace_bytes(p);
}

int attn_bwd_score(const void* Q, const void* K, const void* V, const int64_t* strides,
                   const void* O, const void* dO, const float* L, void* dQ, void* dK, void* dV,
                   int B, int Hq, int Hkv, int N, int d, int causal, int window,
                   const int* doc_start, const int* prefix, float softcap, const float* slopes,
                   float scale, void* workspace, size_t bytes, void* stream) {
  ScoreProblem p;
  bool empty = false;
  int st = make_problem(B, Hq, Hkv, N, d, causal, window, doc_start, prefix, softcap, slopes,
                        scale, &p, &empty);
  if (st != ATTN_OK) return st;
  // without query heads there is no gradient for the keys to sum
  if (empty) return B > 0 && N > 0 ? ATTN_ERR_INVALID_ARG : ATTN_OK;
  for (const void* x : {Q, K, V, O, dO, (const void*)dQ, (const void*)dK, (const void*)dV})
    if (!good(x, 16)) return ATTN_ERR_INVALID_ARG;
  if (!good(L, 4)) return ATTN_ERR_INVALID_ARG;
  RowStrides operands;
  if ((st = set_strides(strides, p, &operands)) != ATTN_OK) return st;
  const Shape rows = shape_of(p, p.Hq), keys = shape_of(p, p.Hkv);
  p.split = score_bwd_split(p, kSms);
  if (!good(workspace, 256) || bytes < score_workspace_bytes(p)) return ATTN_ERR_WORKSPACE;
  float* sums = reinterpret_cast<float*>(static_cast<char*>(workspace) + sums_offset(p));
  const Workspace ws = carve_workspace(workspace, rows);
  int* err = error_word_ptr();
  ScoreBwdMaps m;
  if (!err || !make_maps(&m.q, &m.k, &m.v, Q, K, V, operands, p)) return ATTN_ERR_CUDA;
  if (make_tile_map(&m.dout, dO, rows) || make_tile_map(&m.dk, dK, keys) ||
      make_tile_map(&m.dv, dV, keys) || make_acc_map(&m.acc, ws.acc, rows))
    return ATTN_ERR_CUDA;
  const cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = launch_bwd_preprocess(O, dO, L, ws, rows, true, s);
  if (e == cudaSuccess && p.doc) e = launch_score_bwd_tables(ws, p, s);
  if (e == cudaSuccess && p.doc) e = launch_bwd_order(ws, shape_of(p, 1), s);
  if (e == cudaSuccess) e = launch_score_bwd_main(m, ws, sums, p, scale, err, s);
  if (e == cudaSuccess && p.split > 1) e = launch_score_bwd_join(dK, dV, sums, p, scale, s);
  if (e == cudaSuccess) e = launch_bwd_dq_convert(dQ, ws, rows, scale * kPxDown, s);
  return status_of(e);
}

}  // extern "C"
