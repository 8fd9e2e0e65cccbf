// serving.h -- host-side launchers of the answering path (rotary positions,
// the paged key/value cache, attention of one new token), shared between the
// kernel translation units and their C ABI in serving_api.cu.  Internal to
// the library.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "paged.cuh"

namespace attn {

// The current device's error word (attn_api.cu); null if it has none.
int* error_word_ptr();

// Device error code of a page-table entry or a length outside the cache (the
// other codes are in ptx.cuh).
constexpr int kDevBadIndex = 4;
// What the index belonged to, in the error word's low bits.
constexpr int kSiteLength = 0x501;     // a length or start outside the page table
constexpr int kSiteDecodePage = 0x502;
constexpr int kSiteWritePage = 0x503;
constexpr int kSiteReadPage = 0x504;

constexpr int kMaxAxes = 4;

// Rotary positions (rope.cu).  x has H heads from `q` then Hk from `k`, each
// with its own element strides (batch, head, token; the head dim is
// contiguous); outputs are contiguous [B][heads][N][d].
struct RopeArgs {
  const void* x[2];
  void* y[2];
  int64_t sb[2], sh[2], sn[2];
  int heads[2];
  const int* pos;       // [axes][B or 1][N]
  int64_t pos_axis;     // elements between axes
  int64_t pos_batch;    // elements between batch rows; 0 = shared
  const float* inv_freq;  // [d / 2]
  int axis_end[kMaxAxes];  // first pair index past each axis's pairs
  int axes;
  int B, N, d;
  FastDiv N_div;  // by N
  int interleaved;
  int backward;
};
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t stream);

// The paged cache as the kernels see it.  descale pointers are null for bf16.
struct CacheArgs {
  void* kc;
  void* vc;
  float* kd;
  float* vd;
  const int* table;  // [B][max_pages]
  int num_pages, Hkv, page_size, d, max_pages, B;
  int capacity;      // max_pages * page_size
  FastDiv page_div;  // by page_size
};

// kv_cache.cu.  Rows of k and v: [B][Hkv][T][d], read with element strides
// (batch, head, token), written contiguous.
struct CacheRows {
  void* x[2];  // k, v
  int64_t sb[2], sh[2], st[2];
  const int* start;  // [B]
  const int* count;  // [B] or null = T
  int T;
  FastDiv T_div, head_div;  // by T and by the cache's Hkv
};
cudaError_t launch_kv_write(const CacheArgs& c, const CacheRows& r, int* err, cudaStream_t stream);
cudaError_t launch_kv_read(const CacheArgs& c, const CacheRows& r, int* err, cudaStream_t stream);

// attn_decode.cu.
struct DecodeArgs {
  CacheArgs c;
  const void* q;         // [B][Hq][d] bf16
  const int* lens;       // [B]
  void* o;               // [B][Hq][d] bf16
  float* lse;            // [B][Hq]
  int Hq;
  int window;
  float scale_log2;      // scale * log2(e)
  // set by launch_decode: the query heads of a key head, cut into blocks of at
  // most kDecodeHeads (the last may have fewer)
  int group, group_blocks, block_heads;
  int head_blocks;       // of a sequence
  FastDiv block_div;     // by group_blocks
  unsigned long long *arrivals, *arrivals2;  // workspace: a word per slot each, see arrive()
  unsigned long long tag;        // 48 bits, another one for every call
  float *part_ml, *part_ml2;  // workspace: [2 * blocks][16][2] running maximum and sum
  float* part_o;         // workspace: [2 * blocks][16][d] unnormalised output
  int* err;
};
// Thread blocks the split's workspace provides for: three for each of 152 SMs.
constexpr int kDecodeMaxBlocks = 456;
constexpr int kDecodeHeads = 16;  // heads of one key/value head a block works on at most
inline size_t decode_arrival_bytes() {
  return sizeof(unsigned long long) * 2 * size_t(kDecodeMaxBlocks);  // one of the two arrays
}
inline size_t decode_ml_bytes() {
  return sizeof(float) * 2 * kDecodeHeads * 2 * size_t(kDecodeMaxBlocks);
}
inline size_t decode_o_bytes(int d) {
  return sizeof(float) * d * kDecodeHeads * 2 * size_t(kDecodeMaxBlocks);
}
cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t stream);

}  // namespace attn
