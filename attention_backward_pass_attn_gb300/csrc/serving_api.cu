// serving_api.cu -- the C ABI of the answering path (declared in
// include/attn.h): rotary positions, the paged key/value cache and attention
// of one new token.  Argument validation, workspace carve-up, and the calls
// into the kernel launchers.
#include <atomic>
#include <chrono>
#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/attn.h"
#include "kernels.h"
#include "paged.cuh"
#include "score_tanh.h"
#include "serving.h"

namespace attn {
static_assert(int(kCacheBf16) == int(ATTN_CACHE_BF16) && int(kCacheE4m3) == int(ATTN_CACHE_E4M3) &&
                  int(kCacheInt4) == int(ATTN_CACHE_INT4),
              "the public cache types are the kernels'");
namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool good(const void* p, uintptr_t n) { return p && aligned(p, n); }
int launch_status(cudaError_t e) { return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA; }

// Element strides (batch, head, token) of a [B][H][N][d] operand: the
// caller's, or contiguous ones.  A dimension of one index has no stride to
// speak of.  16-byte loads need every other stride to be a multiple of 8.
bool set_strides(const int64_t* given, int B, int H, int N, int d, int64_t* sb, int64_t* sh,
                 int64_t* sn) {
  *sb = B > 1 ? (given ? given[0] : int64_t(H) * N * d) : 0;
  *sh = H > 1 ? (given ? given[1] : int64_t(N) * d) : 0;
  *sn = N > 1 ? (given ? given[2] : d) : 0;
  for (int64_t s : {*sb, *sh, *sn})
    if (s < 0 || s % 8) return false;
  return true;
}

int rope(const void* Q, const void* K, const int* pos, const float* inv_freq, const int* sections,
         int axes, int interleaved, const int64_t* strides, void* Q_out, void* K_out, int B, int H,
         int Hk, int N, int d, int pos_batches, int backward, void* stream) {
  if (B < 0 || H < 0 || Hk < 0 || N < 0 || d < 0) return ATTN_ERR_INVALID_ARG;
  if (axes < 1 || axes > kMaxAxes || !sections) return ATTN_ERR_INVALID_ARG;
  if (interleaved != 0 && interleaved != 1) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (pos_batches != 1 && pos_batches != B) return ATTN_ERR_INVALID_ARG;
  RopeArgs a = {};
  int end = 0;
  for (int x = 0; x < kMaxAxes; ++x) {
    if (x < axes) {
      if (sections[x] < 0 || sections[x] > d / 2) return ATTN_ERR_INVALID_ARG;
      end += sections[x];
    }
    a.axis_end[x] = end;
  }
  if (end != d / 2) return ATTN_ERR_INVALID_ARG;
  if (B == 0 || N == 0 || (H == 0 && Hk == 0)) return ATTN_OK;
  if ((long long)B * N > INT_MAX || (long long)H + Hk > INT_MAX) return ATTN_ERR_UNSUPPORTED;
  if (!good(pos, 4) || !good(inv_freq, 4)) return ATTN_ERR_INVALID_ARG;
  const void* in[2] = {Q, K};
  void* out[2] = {Q_out, K_out};
  a.heads[0] = H;
  a.heads[1] = Hk;
  for (int w = 0; w < 2; ++w) {
    if (a.heads[w] == 0) continue;
    if (!good(in[w], 16) || !good(out[w], 16)) return ATTN_ERR_INVALID_ARG;
    a.x[w] = in[w];
    a.y[w] = out[w];
    if (!set_strides(strides ? strides + 3 * w : nullptr, B, a.heads[w], N, d, &a.sb[w], &a.sh[w],
                     &a.sn[w]))
      return ATTN_ERR_INVALID_ARG;
  }
  a.pos = pos;
  a.pos_axis = int64_t(pos_batches) * N;
  a.pos_batch = pos_batches == 1 ? 0 : N;
  a.inv_freq = inv_freq;
  a.axes = axes;
  a.B = B;
  a.N = N;
  a.N_div = make_fast_div(N);
  a.d = d;
  a.interleaved = interleaved;
  a.backward = backward;
  return launch_status(launch_rope(a, (cudaStream_t)stream));
}

// Sizes of a paged cache; pointers are looked at by set_cache.
int check_cache(int B, int Hkv, int d, int page_size, int num_pages, int max_pages) {
  if (B < 0 || Hkv < 1 || d < 0 || page_size < 1 || num_pages < 1 || max_pages < 1)
    return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (page_size % kPageQuantum) return ATTN_ERR_UNSUPPORTED;
  // a key index one unit of work past the last position stays in 31 bits
  if ((long long)max_pages * page_size > INT_MAX - 4096) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

int set_cache(CacheArgs* c, const void* kc, const void* vc, const float* kd, const float* vd,
              const int* table, int B, int Hkv, int d, int page_size, int num_pages,
              int max_pages) {
  if (!good(kc, 16) || !good(vc, 16) || !good(table, 4)) return ATTN_ERR_INVALID_ARG;
  if (!kd != !vd || !aligned(kd, 4) || !aligned(vd, 4)) return ATTN_ERR_INVALID_ARG;
  c->kc = const_cast<void*>(kc);
  c->vc = const_cast<void*>(vc);
  c->kd = const_cast<float*>(kd);
  c->vd = const_cast<float*>(vd);
  c->type = kd ? kCacheE4m3 : kCacheBf16;
  c->table = table;
  c->num_pages = num_pages;
  c->Hkv = Hkv;
  c->page_size = page_size;
  c->d = d;
  c->max_pages = max_pages;
  c->B = B;
  c->capacity = max_pages * page_size;
  c->page_div = make_fast_div(page_size);
  return ATTN_OK;
}

// A cache of any type, its factors as it has them.
int set_cache_of(CacheArgs* c, int type, const void* kc, const void* vc, const void* kf,
                 const void* vf, const int* table, int B, int Hkv, int d, int page_size,
                 int num_pages, int max_pages) {
  if (type != kCacheInt4) {
    if ((type == kCacheE4m3) != (kf && vf) || !kf != !vf) return ATTN_ERR_INVALID_ARG;
    return set_cache(c, kc, vc, static_cast<const float*>(kf), static_cast<const float*>(vf),
                     table, B, Hkv, d, page_size, num_pages, max_pages);
  }
  // a row's factors are 2 d / 32 bytes, read a factor at a time
  if (!good(kf, 2) || !good(vf, 2)) return ATTN_ERR_INVALID_ARG;
  const int st = set_cache(c, kc, vc, nullptr, nullptr, table, B, Hkv, d, page_size, num_pages,
                           max_pages);
  c->kf = static_cast<uint16_t*>(const_cast<void*>(kf));
  c->vf = static_cast<uint16_t*>(const_cast<void*>(vf));
  c->type = kCacheInt4;
  return st;
}

// Appends to a cache of any type.
int write_rows(int type, const void* K, const void* V, const int64_t* strides, void* K_cache,
               void* V_cache, void* kf, void* vf, const int* page_table, const int* start,
               const int* count, int B, int Hkv, int T, int d, int page_size, int num_pages,
               int max_pages, void* stream) {
  int st = check_cache(B, Hkv, d, page_size, num_pages, max_pages);
  if (st != ATTN_OK) return st;
  if (T < 0) return ATTN_ERR_INVALID_ARG;
  if (B == 0 || T == 0) return ATTN_OK;
  CacheArgs c = {};
  if ((st = set_cache_of(&c, type, K_cache, V_cache, kf, vf, page_table, B, Hkv, d, page_size,
                         num_pages, max_pages)) != ATTN_OK)
    return st;
  if (!good(K, 16) || !good(V, 16) || !good(start, 4) || !aligned(count, 4))
    return ATTN_ERR_INVALID_ARG;
  if ((long long)B * Hkv > INT_MAX || (long long)B * Hkv * T > INT_MAX) return ATTN_ERR_UNSUPPORTED;
  CacheRows r = {};
  const void* in[2] = {K, V};
  for (int s = 0; s < 2; ++s) {
    r.x[s] = const_cast<void*>(in[s]);
    if (!set_strides(strides ? strides + 3 * s : nullptr, B, Hkv, T, d, &r.sb[s], &r.sh[s],
                     &r.st[s]))
      return ATTN_ERR_INVALID_ARG;
  }
  r.start = start;
  r.count = count;
  r.T = T;
  r.T_div = make_fast_div(T);
  r.head_div = make_fast_div(Hkv);
  int* err = error_word_ptr();
  if (!err) return ATTN_ERR_CUDA;
  return launch_status(launch_kv_write(c, r, err, (cudaStream_t)stream));
}

// Reads rows of a cache of any type.
int read_rows(int type, const void* K_cache, const void* V_cache, const void* kf, const void* vf,
              const int* page_table, const int* start, const int* count, void* K, void* V, int B,
              int Hkv, int T, int d, int page_size, int num_pages, int max_pages, void* stream) {
  int st = check_cache(B, Hkv, d, page_size, num_pages, max_pages);
  if (st != ATTN_OK) return st;
  if (T < 0) return ATTN_ERR_INVALID_ARG;
  if (B == 0 || T == 0) return ATTN_OK;
  CacheArgs c = {};
  if ((st = set_cache_of(&c, type, K_cache, V_cache, kf, vf, page_table, B, Hkv, d, page_size,
                         num_pages, max_pages)) != ATTN_OK)
    return st;
  if (!good(K, 16) || !good(V, 16) || !good(start, 4) || !aligned(count, 4))
    return ATTN_ERR_INVALID_ARG;
  if ((long long)B * Hkv > INT_MAX || (long long)B * Hkv * T > INT_MAX) return ATTN_ERR_UNSUPPORTED;
  CacheRows r = {};
  r.x[0] = K;
  r.x[1] = V;
  r.start = start;
  r.count = count;
  r.T = T;
  r.T_div = make_fast_div(T);
  r.head_div = make_fast_div(Hkv);
  int* err = error_word_ptr();
  if (!err) return ATTN_ERR_CUDA;
  return launch_status(launch_kv_read(c, r, err, (cudaStream_t)stream));
}

// Constants of the decode's changed scores; false if one is not finite.
bool set_score(DecodeScore* s, float softcap, const float* slopes) {
  *s = {};
  s->slopes = slopes;
  if (softcap == 0.f) return true;
  const double cap = softcap * 1.4426950408889634;
  s->cap_log2 = float(cap);
  s->inv_cap_log2 = float(1 / cap);
  s->exp_scale = float(2.0 / softcap);
  s->reach = float(kTanhReach * cap);
  return s->cap_log2 > 0.f && std::isfinite(2 * s->cap_log2) && std::isfinite(s->inv_cap_log2) &&
         std::isfinite(s->exp_scale);
}

// A 48-bit number that no earlier call of this process had, and another
// process's calls hardly: what the decode's arrival words are told apart by.
unsigned long long next_tag() {
  static std::atomic<unsigned long long> tag{
      (unsigned long long)std::chrono::steady_clock::now().time_since_epoch().count() *
      0x9E3779B97F4A7C15ull};
  return tag.fetch_add(1, std::memory_order_relaxed) & 0xFFFFFFFFFFFFull;
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" {

int rope_fwd(const void* Q, const void* K, const int* pos, const float* inv_freq,
             const int* sections, int axes, int interleaved, const int64_t* strides, void* Q_out,
             void* K_out, int B, int H, int Hk, int N, int d, int pos_batches, void* stream) {
  return rope(Q, K, pos, inv_freq, sections, axes, interleaved, strides, Q_out, K_out, B, H, Hk, N,
              d, pos_batches, 0, stream);
}

int rope_bwd(const void* dQ, const void* dK, const int* pos, const float* inv_freq,
             const int* sections, int axes, int interleaved, const int64_t* strides, void* dQ_out,
             void* dK_out, int B, int H, int Hk, int N, int d, int pos_batches, void* stream) {
  return rope(dQ, dK, pos, inv_freq, sections, axes, interleaved, strides, dQ_out, dK_out, B, H,
              Hk, N, d, pos_batches, 1, stream);
}

int kv_cache_write(const void* K, const void* V, const int64_t* strides, void* K_cache,
                   void* V_cache, float* k_descale, float* v_descale, const int* page_table,
                   const int* start, const int* count, int B, int Hkv, int T, int d, int page_size,
                   int num_pages, int max_pages, void* stream) {
  return write_rows(k_descale || v_descale ? kCacheE4m3 : kCacheBf16, K, V, strides, K_cache,
                    V_cache, k_descale, v_descale, page_table, start, count, B, Hkv, T, d,
                    page_size, num_pages, max_pages, stream);
}

int int4_cache_write(const void* K, const void* V, const int64_t* strides, void* K_cache,
                     void* V_cache, void* k_factor, void* v_factor, const int* page_table,
                     const int* start, const int* count, int B, int Hkv, int T, int d,
                     int page_size, int num_pages, int max_pages, void* stream) {
  return write_rows(kCacheInt4, K, V, strides, K_cache, V_cache, k_factor, v_factor, page_table,
                    start, count, B, Hkv, T, d, page_size, num_pages, max_pages, stream);
}

int kv_cache_read(const void* K_cache, const void* V_cache, const float* k_descale,
                  const float* v_descale, const int* page_table, const int* start,
                  const int* count, void* K, void* V, int B, int Hkv, int T, int d, int page_size,
                  int num_pages, int max_pages, void* stream) {
  return read_rows(k_descale || v_descale ? kCacheE4m3 : kCacheBf16, K_cache, V_cache, k_descale,
                   v_descale, page_table, start, count, K, V, B, Hkv, T, d, page_size, num_pages,
                   max_pages, stream);
}

int int4_cache_read(const void* K_cache, const void* V_cache, const void* k_factor,
                    const void* v_factor, const int* page_table, const int* start,
                    const int* count, void* K, void* V, int B, int Hkv, int T, int d,
                    int page_size, int num_pages, int max_pages, void* stream) {
  return read_rows(kCacheInt4, K_cache, V_cache, k_factor, v_factor, page_table, start, count, K,
                   V, B, Hkv, T, d, page_size, num_pages, max_pages, stream);
}

size_t attn_decode_workspace_size(int d) {
  if (d != 64 && d != 128) return 0;
  return 2 * decode_arrival_bytes() + 2 * decode_ml_bytes() + decode_o_bytes(d);
}

int attn_decode(const void* Q, const void* K_cache, const void* V_cache, const float* k_descale,
                const float* v_descale, const int* page_table, const int* seq_lens, void* O,
                float* L, int B, int Hq, int Hkv, int d, int page_size, int num_pages,
                int max_pages, int window, float scale, void* workspace, size_t workspace_bytes,
                void* stream) {
  return attn_score_decode(Q, K_cache, V_cache, k_descale, v_descale,
                           k_descale || v_descale ? ATTN_CACHE_E4M3 : ATTN_CACHE_BF16, page_table,
                           seq_lens, O, L, B, Hq, Hkv, d, page_size, num_pages, max_pages, window,
                           0.f, nullptr, scale, workspace, workspace_bytes, stream);
}

int attn_score_decode(const void* Q, const void* K_cache, const void* V_cache,
                      const void* k_factor, const void* v_factor, int cache_type,
                      const int* page_table, const int* seq_lens, void* O, float* L, int B, int Hq,
                      int Hkv, int d, int page_size, int num_pages, int max_pages, int window,
                      float softcap, const float* slopes, float scale, void* workspace,
                      size_t workspace_bytes, void* stream) {
  int st = check_cache(B, Hkv, d, page_size, num_pages, max_pages);
  if (st != ATTN_OK) return st;
  if (cache_type < ATTN_CACHE_BF16 || cache_type > ATTN_CACHE_INT4) return ATTN_ERR_INVALID_ARG;
  if (Hq < 0 || Hq % Hkv || window < 0) return ATTN_ERR_INVALID_ARG;
  if (!(std::isfinite(softcap) && softcap >= 0.f) || !aligned(slopes, 4))
    return ATTN_ERR_INVALID_ARG;
  if (!(std::isfinite(scale) && scale > 0.f)) return ATTN_ERR_INVALID_ARG;
  if (B == 0 || Hq == 0) return ATTN_OK;
  if ((long long)B * Hq > INT_MAX) return ATTN_ERR_UNSUPPORTED;
  DecodeArgs a = {};
  if ((st = set_cache_of(&a.c, cache_type, K_cache, V_cache, k_factor, v_factor, page_table, B,
                         Hkv, d, page_size, num_pages, max_pages)) != ATTN_OK)
    return st;
  if (!set_score(&a.score, softcap, slopes)) return ATTN_ERR_INVALID_ARG;
  if (!good(Q, 16) || !good(O, 16) || !good(L, 4) || !good(seq_lens, 4))
    return ATTN_ERR_INVALID_ARG;
  if (!good(workspace, 256) || workspace_bytes < attn_decode_workspace_size(d))
    return ATTN_ERR_WORKSPACE;
  a.q = Q;
  a.lens = seq_lens;
  a.o = O;
  a.lse = L;
  a.Hq = Hq;
  a.window = window;
  a.scale_log2 = scale * 1.4426950408889634f;
  if (!std::isfinite(a.scale_log2)) return ATTN_ERR_INVALID_ARG;
  char* ws = static_cast<char*>(workspace);
  a.arrivals = reinterpret_cast<unsigned long long*>(ws);
  a.arrivals2 = reinterpret_cast<unsigned long long*>(ws + decode_arrival_bytes());
  a.tag = next_tag();
  a.part_ml = reinterpret_cast<float*>(ws + 2 * decode_arrival_bytes());
  a.part_ml2 = reinterpret_cast<float*>(ws + 2 * decode_arrival_bytes() + decode_ml_bytes());
  a.part_o = reinterpret_cast<float*>(ws + 2 * decode_arrival_bytes() + 2 * decode_ml_bytes());
  a.err = error_word_ptr();
  if (!a.err) return ATTN_ERR_CUDA;
  return launch_status(launch_decode(a, (cudaStream_t)stream));
}

}  // extern "C"
