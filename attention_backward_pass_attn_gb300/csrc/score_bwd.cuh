// score_bwd.cuh -- attention backward with changed scores (see score_fwd.cu); the
// main kernel, instantiated in score_bwd.cu and score_bwd_split.cu:
//
//   P_ij = exp(x_ij - l_i),  D_i = <do_i, o_i>
//   dx_ij = P_ij (<do_i, v_j> - D_i) x'_ij,  x' = 1 - tanh^2 under a cap, else 1
//   dq_i = s sum_j dx_ij k_j,  dk_j = s sum_i dx_ij q_i,  dv_j = sum_i P_ij do_i
//
// dk_j and dv_j also summed over the query heads that share the key head.  The
// bias adds a constant to a score and leaves no trace but P's.
//
// The frame is the plain backward's main kernel (attn_bwd_main.cuh): per
// 128-row key/value tile five tcgen05.mma contractions for every query tile
// that sees it, dK and dV in tensor memory until the tile is done, dQ's
// partial tiles added into an fp32 accumulator by TMA reduce-adds (their order
// varies: dQ repeats to fp32 rounding, dK and dV bit for bit).  Warps 0-3
// drain dQ, 4-19 own 32 query columns each of S^T and dP^T, a thread to a key
// row, 20 issues copies and 21 the tensor core's instructions.  The steps
// before and after (D, L log2 e and zeroed accumulators; dQ to bf16) are the
// plain backward's.  What differs:
//
//  * An item is a tile of a key head and walks the query tiles of every query
//    head that reads it, one head after another: dK and dV are summed over the
//    group where they lie, with no further pass and no atomics.  Where that
//    leaves too few items for the GPU, or one too heavy (score_bwd_split), a
//    group's heads are dealt to several items, whose fp32 sums a last kernel
//    adds in the order of the heads.
//  * Which queries see a key is an interval [q_lo, q_lim) under every mask,
//    held by the thread that owns the key's row; tiles that cut no row of a
//    warp skip the test.
//  * dx is formed in fp32 from P x' held in fp16 and rounded to bf16 once.  P x'
//    is held times 2^14 (kPxUp), dx, the sums of dQ and dK and all: 11 bits down
//    to P = 2^-28, and 2^-39 off below, where 2^0 would leave the keys that
//    every row sees a little of, 2^-20 in a million, four bits.  (N=4096 b4 h16
//    d=128: 1,162 us became 1,171, with a cap 1,280 and 1,300.)  P is at most 1
//    and some roundings of the scores more, fp16 ends at 4: what a cap of 10^7
//    may leave above, whose scores differ by more, stays there.
#pragma once

#include <cuda_fp16.h>

#include <type_traits>

#include "score.cuh"

namespace attn {
namespace score_bwd {

// d = 128 takes two idle warps more, to make the last four a warpgroup that can
// hand its registers to the drain's (see setmaxnreg below).
template <int HD>
constexpr int kThreads = HD == 128 ? 768 : 704;
constexpr int kSoftmaxThreads = 512;
constexpr int kProducerWarp = 20;
constexpr int kMmaWarp = 21;
constexpr uint32_t kTmemCols = 512;

// Item-level barriers (one phase per work item of the CTA).
constexpr int kBarKFull = 0;
constexpr int kBarVFull = 1;
constexpr int kBarKEmpty = 2;
constexpr int kBarVEmpty = 3;
constexpr int kBarAccFull = 4;   // dK, dV complete in tensor memory
constexpr int kBarAccEmpty = 5;  // dK, dV read out by the epilogue
// Tile-level barriers (one phase per query tile the CTA processes).
constexpr int kBarQFull = 6;     // + stage
constexpr int kBarQEmpty = 8;    // + stage
constexpr int kBarDOFull = 10;   // + dO stage
constexpr int kBarDOEmpty = 12;  // + dO stage
constexpr int kBarSFull = 14;
constexpr int kBarPReady = 15;
constexpr int kBarDPFull = 16;
constexpr int kBarDSReady = 17;
constexpr int kBarDSFree = 18;
constexpr int kBarDQFull = 19;
constexpr int kBarDQFree = 20;
constexpr int kBarDrain = 21;
// The item epilogue stages dV and dK through the shared dS^T tile (two turns
// for d = 128, one for d = 64): written by the softmax warps of a turn, then
// stored by TMA, after which the tile is free again.
constexpr int kBarEpiFull = 22;  // + turn
constexpr int kBarEpiFree = 24;  // + turn
constexpr int kNumBars = 26;
constexpr int kDrainBarrierId = 1;  // named barrier of the 128 dQ-drain threads

template <int HD>
struct Layout {
  static constexpr int kTileBytes = 128 * HD * 2;
  static constexpr int kK = 0;
  static constexpr int kV = kK + kTileBytes;
  static constexpr int kQ = kV + kTileBytes;  // + stage * kTileBytes
  // dO: two stages for d = 64; for d = 128 the dQ staging buffers take the
  // room of the second.
  static constexpr int kDOStages = HD == 64 ? 2 : 1;
  static constexpr int kDO = kQ + 2 * kTileBytes;           // + stage * kTileBytes
  static constexpr int kDS = kDO + kDOStages * kTileBytes;  // 128 x 128 bf16, two 16 KB blocks
  static constexpr int kStage = kDS + 32768;                // 2 x (128 rows x 32 fp32), swizzled
  static constexpr int kVec = kStage + 32768;  // stage s: L2 at +1024 s, D at +1024 s + 512
  static constexpr int kBar = kVec + 2048;
  static constexpr int kTmemSlot = kBar + kNumBars * 8;
  static constexpr int kAbort = kTmemSlot + 4;
  // At least half of the SM's shared memory: one CTA (owning all 512
  // tensor-memory columns) per SM.
  static constexpr int kRaw = (kAbort + 4 + 15) / 16 * 16;
  static constexpr int kBytes = kRaw > 118784 ? kRaw : 118784;
  static constexpr uint32_t kColDV = 0;
  static constexpr uint32_t kColDK = HD;
  static constexpr uint32_t kColS = 2 * HD;
  static constexpr uint32_t kColDP = 2 * HD + 128;
  // d = 64 leaves 128 of the 512 columns free: dQ gets its own, and dK reads
  // dS^T from the dP^T columns.  With d = 128 dQ reuses the dP^T columns and
  // is issued before dK, which reads dS^T from shared memory, so that dQ's
  // drain overlaps dK's contraction.
  static constexpr bool kSeparateDq = HD == 64;
  static constexpr uint32_t kColDQ = kSeparateDq ? 2 * HD + 256 : kColDP;
  // Turns of the item epilogue through the 32 KB dS^T tile: dV then dK for
  // d = 128 (32 KB each), both at once for d = 64.
  static constexpr int kEpiTurns = HD == 128 ? 2 : 1;
};

// A work item: tile jt of key head hk of batch element b, the first of the
// heads whose query tiles it0 .. it0 + n_it - 1 it walks (group / split of
// them), and which part of the group they are, counted over all key heads.
struct Item {
  int b, hk, h0, part, jt, it0, n_it;
};

// Items, heaviest first under the causal mask: tiles by their start (an
// earlier one is seen by more queries), with documents in the order that
// attn_bwd_order_kernel sorted them into.  Without the mask all cost the same,
// and (parts of) key heads are taken in groups of HG whose query, dO and
// dQ-accumulator tiles fit in L2 together.
template <bool SPLIT>
struct ItemMap {
  const ScoreProblem& p;
  const Workspace& ws;
  int HG;
  __device__ __forceinline__ Item item(int i) const {
    Item t;
    const int split = SPLIT ? p.split : 1;
    const int parts = p.Hkv * split;  // of a batch element
    int part;
    if (p.doc) {
      const int rank = i / parts, id = __ldg(ws.order + rank);
      part = i - rank * parts;
      t.b = id / p.n_tiles;
      t.jt = id - t.b * p.n_tiles;
    } else {
      const int per_group = HG * p.n_tiles;
      const int gr = i / per_group, r = i - gr * per_group;
      const int hg = min(HG, p.B * parts - gr * HG);  // parts in this group
      t.jt = r / hg;
      part = gr * HG + (r - t.jt * hg);
      t.b = part / parts;
      part -= t.b * parts;
    }
    t.hk = part / split;
    t.h0 = part * (p.group / split);
    t.part = t.b * parts + part;
    int last = p.n_tiles - 1;
    t.it0 = 0;
    if (p.causal) {
      t.it0 = p.prefix && __ldg(p.prefix + t.b) > t.jt * 128 ? 0 : t.jt;
      // the last query that still sees a key of the tile: jt 128 + 127 +
      // window - 1 under a window, tabulated with documents
      if (p.doc)
        last = min(last, max(t.jt, __ldg(&ws.items[size_t(t.b) * p.n_tiles + t.jt].x)));
      else if (p.window > 0)
        last = int(min((long long)last, ((long long)t.jt * 128 + 126 + p.window) >> 7));
    }
    t.n_it = last - t.it0 + 1;
    return t;
  }
};

// CTA b of G takes items b, 2G-1-b, 2G+b, 4G-1-b, ... (a snake over rounds,
// which evens out the heavy-first order); -1 past the last item.
__device__ __forceinline__ int snake_item(int k, int b, int G, int n_items) {
  const long long idx = (k & 1) ? (long long)k * G + (G - 1 - b) : (long long)k * G + b;
  return idx < n_items ? int(idx) : -1;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t w;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}
__device__ __forceinline__ uint64_t unpack_f16x2(uint32_t w) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return f32x2(f.x, f.y);
}

// Slopes alone: the bias brings the 2^14 along, and P too is held times that (a
// product for every pair of scores more took N=8192 h16 d=64 from 870 us to 916).
template <bool CAP, bool SLOPES>
constexpr bool kUpP = SLOPES && !CAP;

// Descriptor conventions (128-byte swizzle, tiles of 128 rows in 64-column
// blocks of 16 KB): a K-major operand advances 32 bytes per 16-element k-step
// within a block and 16 KB across blocks; an MN-major operand advances 2 KB
// (16 rows) per k-step, its MN extent spanning blocks 16 KB apart (LBO).

// SPLIT: several items share a group's heads (a kernel of its own: its
// epilogue's registers cost the others' loops 7 % with d = 64).
template <int HD, bool CAP, bool SLOPES, bool SPLIT>
__global__ void __launch_bounds__(kThreads<HD>, 1)
    score_bwd_kernel(const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ CUtensorMap tmdO,
                     const __grid_constant__ CUtensorMap tmAcc,
                     const __grid_constant__ CUtensorMap tmDK,
                     const __grid_constant__ CUtensorMap tmDV,
                     const __grid_constant__ Workspace ws,
                     const __grid_constant__ ScoreProblem p, float* __restrict__ sums,
                     int head_group, float scale, int* err) {
  using Ly = Layout<HD>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (sbase & 1023u) {
    if (threadIdx.x == 0) report_error(err, kDevSmemAlign, 0x700);
    return;
  }

  constexpr float kUpLog2 = kUpP<CAP, SLOPES> ? kPxUpLog2 : 0.f;
  const int split = SPLIT ? p.split : 1;
  const int n_items = p.B * p.Hkv * split * p.n_tiles;
  const int group = p.group / split;  // query heads of an item
  const ItemMap<SPLIT> imap{p, ws, head_group};
  const int G = gridDim.x, cta = blockIdx.x;

  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Ly::kAbort);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Ly::kTmemSlot);
  auto bar = [&](int i) -> uint32_t { return sbase + Ly::kBar + 8 * i; };

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < kNumBars; ++i) {
      // arrivals per phase: the softmax threads, the 128 drain threads, or one
      // (a TMA transaction or a tcgen05.commit)
      const uint32_t count =
          (i == kBarPReady || i == kBarDSReady || i == kBarAccEmpty) ? kSoftmaxThreads
          : (i == kBarDQFree)                                          ? 128
          : (i == kBarEpiFull || i == kBarEpiFull + 1) ? kSoftmaxThreads / Ly::kEpiTurns
                                                       : 1;
      mbar_init(bar(i), count);
    }
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  if (warp == kProducerWarp && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmdO);
    tma_prefetch_desc(&tmAcc);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  const WaitCtx ctx{abort_flag, err, kWaitLimitNs};
  // Everything above overlaps the previous kernel; its results are read below.
  grid_dep_wait();
  grid_dep_launch();

  // Registers for d = 128: 80 for each of 768 threads at the launch.  The last
  // warpgroup (copies and tensor core) gives 32 of them back and the drain's
  // takes 32 more, so that three of dQ's four 32-column chunks leave tensor
  // memory at once: 4 x 80 + 112 + 48 = 6 x 80.
  if (warp >= kProducerWarp) {
    if constexpr (HD == 128) asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (warp == kProducerWarp) {
      // ------------------------------------------------------------ TMA producer
      // The whole warp runs the loop (warp-uniform operands); one lane issues.
      // Per item: V (free once the previous item's last dP is done), K (free
      // once its last dK/dQ is done); per query tile g: dO(g) (its stage is free
      // once the dV of the tile that last held it is done) and Q(g+1) with its
      // L and D vectors (two stages, free once dK(g-1) is done), which for the
      // last tile of an item is the first of the next.
      auto load_q = [&](int g, int b, int h, int qt) {  // elected lane only
        const int s = g & 1;
        mbar_arrive_expect_tx(bar(kBarQFull + s), Ly::kTileBytes + 1024);
#pragma unroll
        for (int cb = 0; cb < HD / 64; ++cb)
          tma_load_4d(sbase + Ly::kQ + s * Ly::kTileBytes + cb * 16384, &tmQ, bar(kBarQFull + s),
                      cb * 64, qt * 128, h, b);
        const size_t vo = (size_t(b) * p.Hq + h) * p.Npad + size_t(qt) * 128;
        bulk_load(sbase + Ly::kVec + s * 1024, ws.L2 + vo, 512, bar(kBarQFull + s));
        bulk_load(sbase + Ly::kVec + s * 1024 + 512, ws.D + vo, 512, bar(kBarQFull + s));
      };
      bool ok = true;
      int g = 0;
      for (int k = 0, i = snake_item(0, cta, G, n_items); ok && i >= 0; ++k) {
        const Item t = imap.item(i);
        const int h0 = t.h0;
        const int next = snake_item(k + 1, cta, G, n_items);
        const Item nt = next >= 0 ? imap.item(next) : t;
        if (k > 0 && !(ok = mbar_wait_warp(bar(kBarVEmpty), (k - 1) & 1, ctx, 0x712))) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(bar(kBarVFull), Ly::kTileBytes);
#pragma unroll
          for (int cb = 0; cb < HD / 64; ++cb)
            tma_load_4d(sbase + Ly::kV + cb * 16384, &tmV, bar(kBarVFull), cb * 64, t.jt * 128,
                        t.hk, t.b);
        }
        __syncwarp();
        if (k > 0 && !(ok = mbar_wait_warp(bar(kBarKEmpty), (k - 1) & 1, ctx, 0x713))) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(bar(kBarKFull), Ly::kTileBytes);
#pragma unroll
          for (int cb = 0; cb < HD / 64; ++cb)
            tma_load_4d(sbase + Ly::kK + cb * 16384, &tmK, bar(kBarKFull), cb * 64, t.jt * 128,
                        t.hk, t.b);
          if (k == 0) load_q(0, t.b, h0, t.it0);
          // Warm L2 (and the address translation) for the next item: a new head
          // is often a cold region, and its first tiles are needed right at the
          // item switch.
          if (next >= 0) {
            const int nh = nt.h0;
#pragma unroll
            for (int cb = 0; cb < HD / 64; ++cb) {
              tma_prefetch_4d(&tmK, cb * 64, nt.jt * 128, nt.hk, nt.b);
              tma_prefetch_4d(&tmV, cb * 64, nt.jt * 128, nt.hk, nt.b);
              tma_prefetch_4d(&tmQ, cb * 64, nt.it0 * 128, nh, nt.b);
              tma_prefetch_3d(&tmdO, cb * 64, nt.it0 * 128, nt.b * p.Hq + nh);
            }
            const size_t vo = (size_t(nt.b) * p.Hq + nh) * p.Npad + size_t(nt.it0) * 128;
            bulk_prefetch(ws.L2 + vo, 512);
            bulk_prefetch(ws.D + vo, 512);
          }
        }
        __syncwarp();
        for (int h = 0, it = 0; h < group; ++g) {
          const int ds_ = g % Ly::kDOStages, dn = g / Ly::kDOStages;
          if (dn > 0 &&
              !(ok = mbar_wait_warp(bar(kBarDOEmpty + ds_), (dn - 1) & 1, ctx, 0x711)))
            break;
          if (elect_one()) {
            mbar_arrive_expect_tx(bar(kBarDOFull + ds_), Ly::kTileBytes);
#pragma unroll
            for (int cb = 0; cb < HD / 64; ++cb)
              tma_load_3d(sbase + Ly::kDO + ds_ * Ly::kTileBytes + cb * 16384, &tmdO,
                          bar(kBarDOFull + ds_), cb * 64, (t.it0 + it) * 128,
                          t.b * p.Hq + h0 + h);
          }
          __syncwarp();
          if (++it == t.n_it) it = 0, ++h;
          int qb = t.b, qh = h0 + h, qt = t.it0 + it;
          if (h == group) {
            if (next < 0) continue;
            qb = nt.b;
            qh = nt.h0;
            qt = nt.it0;
          }
          const int gn = g + 1;
          if (gn >= 2 &&
              !(ok = mbar_wait_warp(bar(kBarQEmpty + (gn & 1)), ((gn >> 1) - 1) & 1, ctx, 0x710)))
            break;
          if (elect_one()) load_q(gn, qb, qh, qt);
          __syncwarp();
        }
        i = next;
      }
    } else if (warp == kMmaWarp) {
      // ------------------------------------------------------------ MMA issuer
      // The whole warp runs the loop and waits; one elected lane issues.  Every
      // descriptor is a per-tile base plus a compile-time k-step offset.
      constexpr uint32_t kIdS = make_idesc_bf16(128, 128, 0, 0);  // S^T, dP^T
      constexpr uint32_t kIdV = make_idesc_bf16(128, HD, 0, 1);   // dV, dK
      constexpr uint32_t kIdQ = make_idesc_bf16(128, HD, 1, 1);   // dQ = dS K
      const uint64_t dK_k = make_sdesc_sw128(sbase + Ly::kK, 16, 1024);       // K, K-major
      const uint64_t dK_mn = make_sdesc_sw128(sbase + Ly::kK, 16384, 1024);   // K, MN-major
      const uint64_t dV_k = make_sdesc_sw128(sbase + Ly::kV, 16, 1024);
      const uint64_t dS_k = make_sdesc_sw128(sbase + Ly::kDS, 16, 1024);      // dS^T, K-major
      const uint64_t dS_mn = make_sdesc_sw128(sbase + Ly::kDS, 16384, 1024);  // dS, MN-major
      const uint32_t tS = tbase + Ly::kColS, tDP = tbase + Ly::kColDP;
      const uint32_t tDV = tbase + Ly::kColDV, tDK = tbase + Ly::kColDK;
      const uint32_t tDQ = tbase + Ly::kColDQ;
      // Issue order per query tile:  dP, dV, S(next), dQ, dK (d = 128; else dK,
      // dQ).  S(next) goes right behind dV (which has consumed P from the S
      // columns; the softmax warps keep P in registers), so the softmax warps
      // compute the next tile's P while the tensor core runs dK and dQ.  The
      // first S of an item waits for its K.
      auto issue_s = [&](int stage) {  // S^T = K Q^T; elected lane only
        const uint64_t dq = make_sdesc_sw128(sbase + Ly::kQ + stage * Ly::kTileBytes, 16, 1024);
#pragma unroll
        for (int k = 0; k < HD / 16; ++k) {
          const uint32_t off = (k >> 2) * 16384 + (k & 3) * 32;
          mma_ss(tS, sdesc_add(dK_k, off), sdesc_add(dq, off), kIdS, k > 0 ? 1u : 0u);
        }
        tc_commit(bar(kBarSFull));
      };
      bool ok = true;
      int g = 0;
      for (int k = 0, i = snake_item(0, cta, G, n_items); ok && i >= 0; ++k) {
        const int total = imap.item(i).n_it * group;
        if (!(ok = mbar_wait_warp(bar(kBarKFull), k & 1, ctx, 0x720))) break;
        if (!(ok = mbar_wait_warp(bar(kBarQFull + (g & 1)), (g >> 1) & 1, ctx, 0x721))) break;
        tc_fence_after();
        if (elect_one()) issue_s(g & 1);
        __syncwarp();
        if (!(ok = mbar_wait_warp(bar(kBarVFull), k & 1, ctx, 0x727))) break;
        for (int it = 0; it < total; ++it, ++g) {
          const int s = g & 1;
          const bool last = it + 1 == total;
          const uint32_t sQ = sbase + Ly::kQ + s * Ly::kTileBytes;
          const int ds_ = g % Ly::kDOStages;
          const uint32_t sDO = sbase + Ly::kDO + ds_ * Ly::kTileBytes;
          const uint64_t dQ_mn = make_sdesc_sw128(sQ, 16384, 1024);
          const uint64_t dO_k = make_sdesc_sw128(sDO, 16, 1024);
          const uint64_t dO_mn = make_sdesc_sw128(sDO, 16384, 1024);
          const uint32_t acc0 = it > 0 ? 1u : 0u;
          // dP^T = V dO^T.  When dQ shares the dP columns, they held the previous
          // dQ: wait for its drain.  (Otherwise the previous dP has been read:
          // the softmax warps signalled DS_READY, which the last tile waited on.)
          if (!(ok = mbar_wait_warp(bar(kBarDOFull + ds_), (g / Ly::kDOStages) & 1, ctx, 0x722)))
            break;
          if (!Ly::kSeparateDq && g > 0 &&
              !(ok = mbar_wait_warp(bar(kBarDQFree), (g - 1) & 1, ctx, 0x723)))
            break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk) {
              const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
              mma_ss(tDP, sdesc_add(dV_k, off), sdesc_add(dO_k, off), kIdS, kk > 0 ? 1u : 0u);
            }
            tc_commit(bar(kBarDPFull));
            if (last) tc_commit(bar(kBarVEmpty));
          }
          __syncwarp();
          // dV += P^T dO, P^T read from tensor memory: the softmax warps of 32
          // query columns packed them into the first 16 of their own.  The first
          // dV of an item overwrites the accumulator: the previous item's
          // epilogue must have read it.
          if (!(ok = mbar_wait_warp(bar(kBarPReady), g & 1, ctx, 0x724))) break;
          if (it == 0 && k > 0 &&
              !(ok = mbar_wait_warp(bar(kBarAccEmpty), (k - 1) & 1, ctx, 0x728)))
            break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_ts(tDV, tS + 32 * (kk >> 1) + 8 * (kk & 1), sdesc_add(dO_mn, kk * 2048), kIdV,
                     kk > 0 ? 1u : acc0);
            tc_commit(bar(kBarDOEmpty + ds_));
          }
          __syncwarp();
          // S of the item's next query tile into the S columns, behind dV
          if (!last) {
            const int s1 = (g + 1) & 1;
            if (!(ok = mbar_wait_warp(bar(kBarQFull + s1), ((g + 1) >> 1) & 1, ctx, 0x726)))
              break;
            tc_fence_after();
            if (elect_one()) issue_s(s1);
            __syncwarp();
          }
          if (!(ok = mbar_wait_warp(bar(kBarDSReady), g & 1, ctx, 0x725))) break;
          tc_fence_after();
          if constexpr (Ly::kSeparateDq) {
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)  // dS^T packed like P^T, in the dP^T columns
                mma_ts(tDK, tDP + 32 * (kk >> 1) + 8 * (kk & 1), sdesc_add(dQ_mn, kk * 2048), kIdV,
                       kk > 0 ? 1u : acc0);
              tc_commit(bar(kBarQEmpty + s));
            }
            __syncwarp();
            // With its own columns, dQ waits only for the previous dQ's drain.
            if (g > 0 && !(ok = mbar_wait_warp(bar(kBarDQFree), (g - 1) & 1, ctx, 0x723))) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                mma_ss(tDQ, sdesc_add(dS_mn, kk * 2048), sdesc_add(dK_mn, kk * 2048), kIdQ,
                       kk > 0 ? 1u : 0u);
              tc_commit(bar(kBarDQFull));
            }
            __syncwarp();
          } else {
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                mma_ss(tDQ, sdesc_add(dS_mn, kk * 2048), sdesc_add(dK_mn, kk * 2048), kIdQ,
                       kk > 0 ? 1u : 0u);
              tc_commit(bar(kBarDQFull));
#pragma unroll
              for (int kk = 0; kk < 8; ++kk) {
                const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
                mma_ss(tDK, sdesc_add(dS_k, off), sdesc_add(dQ_mn, kk * 2048), kIdV,
                       kk > 0 ? 1u : acc0);
              }
              tc_commit(bar(kBarQEmpty + s));
            }
            __syncwarp();
          }
          // dK and dQ have read the dS^T tile; the item's last tile also
          // releases K and hands the accumulators to the epilogue.
          if (elect_one()) {
            tc_commit(bar(kBarDSFree));
            if (last) {
              tc_commit(bar(kBarKEmpty));
              tc_commit(bar(kBarAccFull));
            }
          }
          __syncwarp();
        }
        i = snake_item(k + 1, cta, G, n_items);
      }
      if (elect_one()) tc_commit(bar(kBarDrain));
      __syncwarp();
      volatile int never = 0;  // this wait ignores the CTA abort flag
      const WaitCtx own{&never, err, kWaitLimitNs};
      mbar_wait_warp(bar(kBarDrain), 0, own, 0x72F);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax / dS
    const int quarter = (warp - 4) >> 2;  // query columns 32 quarter .. 32 quarter + 31
    const int r = threadIdx.x & 127;      // key row within the tile = TMEM lane
    const uint32_t lane_off = uint32_t((warp & 3) * 32) << 16;
    const uint32_t tS = tbase + lane_off + Ly::kColS + 32 * quarter;
    const uint32_t tDP = tbase + lane_off + Ly::kColDP + 32 * quarter;
    const uint32_t sDSrow = sbase + Ly::kDS + (quarter >> 1) * 16384 + r * 128;
    const ScoreMap& mp = p.map;
    bool ok = true;
    int g = 0;
    for (int k = 0, i = snake_item(0, cta, G, n_items); ok && i >= 0; ++k) {
      const Item t = imap.item(i);
      const int key = t.jt * 128 + r;
      // Queries q_lo <= q < q_lim see this thread's key; rows past N, the
      // zero-filled tail of the last tile, are seen by none.  (Queries past N
      // have L log2 e = +inf and P = 0.)
      int q_lo = 0, q_lim = p.Npad;
      if (p.causal) {
        q_lo = p.prefix && key < __ldg(p.prefix + t.b) ? 0 : key;
        if (p.doc) q_lim = __ldg(ws.qend + size_t(t.b) * p.Npad + key);
        if (p.window > 0 && p.window < q_lim - key) q_lim = key + p.window;
      }
      if (key >= p.N) q_lim = 0;
      // every key row of the warp is seen by queries [all_lo, all_lim)
      const int all_lo = __reduce_max_sync(0xffffffffu, q_lo);
      const int all_lim = __reduce_min_sync(0xffffffffu, q_lim);
      for (int h = 0, it = 0; h < group; ++g) {
        const int s = g & 1, q0 = (t.it0 + it) * 128 + 32 * quarter;  // the first column's query
        const bool first = it == 0 && h == 0;
        if (!(ok = mbar_wait_warp(bar(kBarQFull + s), (g >> 1) & 1, ctx, 0x730))) break;
        if (!(ok = mbar_wait_warp(bar(kBarSFull), g & 1, ctx, 0x731))) break;
        tc_fence_after();
        const float4* L2v4 =
            reinterpret_cast<const float4*>(smem + Ly::kVec + s * 1024) + 8 * quarter;
        const float4* Dv4 =
            reinterpret_cast<const float4*>(smem + Ly::kVec + s * 1024 + 512) + 8 * quarter;
        // P x' stays in registers (fp16) for the dS phase: the tensor core
        // overwrites these S columns with the next S once dV has read P.
        uint32_t px[16];
        {
          uint32_t u[32], pk[16];
          tmem_ld32(tS, u);
          tmem_wait_ld();
          auto pair = [&](int e) {
            return f32x2(__uint_as_float(u[e]), __uint_as_float(u[e + 1]));
          };
          float slope = 0.f, d0 = 0.f, sl = 0.f, row = 0.f;
          bool linear = true;
          if constexpr (SLOPES) {
            slope = __ldg(mp.slopes + t.h0 + h) * 1.4426950408889634f;
            d0 = float(q0 - key);
            const int w0 = t.jt * 128 + 32 * (warp & 3);  // the warp's first key
            const bool past = q0 >= w0 + 31;
            linear = past || q0 + 31 <= w0;  // one sign for every distance of the warp
            sl = past ? slope : -slope;
            row = fmaf(sl, d0, -kUpLog2);
          }
          // Two columns: L - x, P and P x'.
          auto columns = [&](int e, float l0, float l1, auto by_poly, auto edge) {
            uint64_t der = f32x2(kPxUp);  // x' times 2^14, where P is not
            // y = L - x of two columns, so that no sign has to be changed: the
            // exponential takes -y for nothing.
            uint64_t y, off = f32x2(l0, l1);
            if constexpr (SLOPES) {  // distances are whole numbers, exact below 2^24
              if (!decltype(edge)::value || linear)
                off = f32x2(fmaf(sl, float(e), l0 + row), fmaf(sl, float(e + 1), l1 + row));
              else
                off = f32x2(fmaf(slope, fabsf(d0 + float(e)), l0 - kUpLog2),
                            fmaf(slope, fabsf(d0 + float(e + 1)), l1 - kUpLog2));
            }
            if constexpr (!CAP) {
              y = fma_f32x2(pair(e), f32x2(-mp.scale_log2), off);
            } else if constexpr (decltype(by_poly)::value) {
              const uint64_t x = cap_poly(mp, pair(e));
              der = fma_f32x2(mul_f32x2(x, x), f32x2(mp.der_sq), f32x2(kPxUp));
              y = fma_f32x2(x, f32x2(-1.f), off);
            } else {
              // e^2y and r = 1 / (1 + e^2y): 1 - tanh^2 = 4 r (r e^2y), a product of
              // numbers with all their digits on either side (1 - r has none far
              // below zero).  The limit keeps r e^2y from infinity times zero.
              // (Scores of 12 under a cap of 5, N=8192 h16 d=128: 661 us, where 4 r
              // (1 - r) took 644.)
              const auto e2y = [&](float w) {
                float z;
                asm("min.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(w * mp.exp_scale), "f"(126.f));
                return ex2(z);
              };
              const float e0 = e2y(__uint_as_float(u[e])), e1 = e2y(__uint_as_float(u[e + 1]));
              const uint64_t rr = f32x2(rcp_approx(1.f + e0), rcp_approx(1.f + e1));
              der = mul_f32x2(mul_f32x2(rr, f32x2(4.f * kPxUp)), mul_f32x2(rr, f32x2(e0, e1)));
              y = fma_f32x2(fma_f32x2(rr, f32x2(-2.f * mp.cap_log2), f32x2(mp.cap_log2)),
                            f32x2(-1.f), off);
            }
            float p0, p1;
            f32x2_split(y, p0, p1);
            p0 = ex2(-p0);
            p1 = ex2(-p1);
            if constexpr (decltype(edge)::value) {
              const int q = q0 + e;
              if (q < q_lo || q >= q_lim) p0 = 0.f;
              if (q + 1 < q_lo || q + 1 >= q_lim) p1 = 0.f;
            }
            pk[e / 2] = pack_bf16x2(p0, p1);
            if constexpr (!kUpP<CAP, SLOPES>) f32x2_split(mul_f32x2(f32x2(p0, p1), der), p0, p1);
            px[e / 2] = pack_f16x2(p0, p1);
          };
          auto all = [&](auto by_poly, auto edge) {
#pragma unroll
            for (int c4 = 0; c4 < 8; ++c4) {
              const float4 l = L2v4[c4];  // one broadcast load for four query columns
              columns(4 * c4, l.x, l.y, by_poly, edge);
              columns(4 * c4 + 2, l.z, l.w, by_poly, edge);
            }
          };
          auto paths = [&](auto edge) {
            bool poly = true;
            if constexpr (CAP) poly = all_within(top_of(u), mp.poly_limit);
            if (poly)
              all(std::true_type(), edge);
            else
              all(std::false_type(), edge);
          };
          // (a piece with distances of both signs takes the masked path too,
          // which is the rare one)
          if (q0 < all_lo || q0 + 32 > all_lim || !linear)
            paths(std::true_type());
          else
            paths(std::false_type());
          tmem_st16(tS, pk);
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(bar(kBarPReady));
        }
        if (!(ok = mbar_wait_warp(bar(kBarDPFull), g & 1, ctx, 0x732))) break;
        // dQ reads dS from the shared-memory tile: the previous one must be done,
        // and at an item's first tile so must the previous item's epilogue
        if (g > 0 && !(ok = mbar_wait_warp(bar(kBarDSFree), (g - 1) & 1, ctx, 0x733))) break;
        if (!SPLIT && first && k > 0 &&
            !(ok = mbar_wait_warp(bar(kBarEpiFree + Ly::kEpiTurns - 1), (k - 1) & 1, ctx, 0x734)))
          break;
        tc_fence_after();
        // dS^T goes into row r of the shared dS^T tile (128-byte swizzle:
        // 16-byte chunk c lands at c ^ (r % 8)), and where dK reads it from
        // tensor memory also back into the dP^T columns this warp has read,
        // packed two queries per column as P^T is.
        {
          uint32_t u[32], ds[16];
          tmem_ld32(tDP, u);
          tmem_wait_ld();
          auto dx = [&](int c, float da, float db) {  // columns 2c, 2c + 1
            const uint64_t e = fma_f32x2(f32x2(da, db), f32x2(-1.f),
                                         f32x2(__uint_as_float(u[2 * c]),
                                               __uint_as_float(u[2 * c + 1])));
            float a, b;
            f32x2_split(mul_f32x2(e, unpack_f16x2(px[c])), a, b);
            ds[c] = pack_bf16x2(a, b);
          };
#pragma unroll
          for (int c4 = 0; c4 < 8; ++c4) {
            const float4 dd = Dv4[c4];  // one broadcast load for four columns
            dx(2 * c4, dd.x, dd.y);
            dx(2 * c4 + 1, dd.z, dd.w);
          }
          if constexpr (Ly::kSeparateDq) tmem_st16(tDP, ds);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            st_shared_v4(sDSrow + (((4 * (quarter & 1) + c) ^ (r & 7)) << 4), ds[4 * c],
                         ds[4 * c + 1], ds[4 * c + 2], ds[4 * c + 3]);
        }
        tmem_wait_st();
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(bar(kBarDSReady));
        if (++it == t.n_it) it = 0, ++h;
      }
      if (!ok) break;
      // Epilogue of the item: dV (quarters 0 and 1, half of its columns each)
      // and dK (2 and 3; times the softmax scale) from tensor memory, rounded
      // to bf16 into the shared dS^T tile (its two 16 KB blocks are the
      // 64-column boxes of the output tile map, with the same 128-byte swizzle)
      // and written by TMA tile stores, which leave out the rows past N.  One
      // elected warp per turn issues them; their shared-memory reads complete
      // before the tile is used again.
      if (!(ok = mbar_wait_warp(bar(kBarAccFull), k & 1, ctx, 0x738))) break;
      tc_fence_after();
      const int which = quarter >> 1, part = quarter & 1;  // dV or dK; half of its columns
      const uint32_t tAcc =
          tbase + lane_off + (which == 0 ? Ly::kColDV : Ly::kColDK) + (HD / 2) * part;
      if constexpr (SPLIT) {  // one of several sums: as they are, a thread's columns of its row
        float4* dst = reinterpret_cast<float4*>(
            sums +
            ((size_t(which) * p.B * p.Hkv * split + t.part) * p.Npad + t.jt * 128 + r) * HD +
            (HD / 2) * part);
#pragma unroll
        for (int c4 = 0; c4 < HD / 64; ++c4) {
          uint32_t o[32];
          tmem_ld32(tAcc + 32 * c4, o);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 8; ++c)
            dst[8 * c4 + c] = make_float4(__uint_as_float(o[4 * c]), __uint_as_float(o[4 * c + 1]),
                                          __uint_as_float(o[4 * c + 2]),
                                          __uint_as_float(o[4 * c + 3]));
        }
        tc_fence_before();
        mbar_arrive(bar(kBarAccEmpty));
      } else {
        const float mult = which == 0 ? (kUpP<CAP, SLOPES> ? kPxDown : 1.f) : scale * kPxDown;
        for (int turn = 0; ok && turn < Ly::kEpiTurns; ++turn) {
          if (Ly::kEpiTurns == 1 || which == turn) {
            // The tile's previous contents: this item's dS^T (the contractions
            // have completed: AccFull), then the previous turn's store -- of this
            // item for turn 1, of the previous item for turn 0.
            const int prev_turn = turn > 0 ? turn - 1 : Ly::kEpiTurns - 1;
            const int prev_item = turn > 0 ? k : k - 1;
            if (prev_item >= 0 &&
                !(ok = mbar_wait_warp(bar(kBarEpiFree + prev_turn), prev_item & 1, ctx, 0x73A)))
              break;
            // d = 128: block `part` of the tensor's two; d = 64: half of block `which`
            const uint32_t row =
                sbase + Ly::kDS + (HD == 128 ? part : which) * 16384 + r * 128;
#pragma unroll
            for (int c4 = 0; c4 < HD / 64; ++c4) {
              uint32_t o[32];
              tmem_ld32(tAcc + 32 * c4, o);
              tmem_wait_ld();
#pragma unroll
              for (int c8 = 0; c8 < 4; ++c8) {  // 16-byte chunk j of the 64-column block
                const int j = (HD == 128 ? 4 * c4 : 4 * part) + c8;
                uint32_t w4[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  w4[e] = pack_bf16x2(__uint_as_float(o[8 * c8 + 2 * e]) * mult,
                                      __uint_as_float(o[8 * c8 + 2 * e + 1]) * mult);
                st_shared_v4(row + ((j ^ (r & 7)) << 4), w4[0], w4[1], w4[2], w4[3]);
              }
            }
            tc_fence_before();
            mbar_arrive(bar(kBarAccEmpty));  // this thread's accumulator columns are read
            fence_proxy_async_smem();
            mbar_arrive(bar(kBarEpiFull + turn));
          }
          if (warp == 4 + 8 * turn) {  // the turn's issuing warp, one of those that wrote
            if (!(ok = mbar_wait_warp(bar(kBarEpiFull + turn), k & 1, ctx, 0x73B))) break;
            if (elect_one()) {
              const int bh = t.b * p.Hkv + t.hk;
              if constexpr (HD == 128) {
                const CUtensorMap* map = turn == 0 ? &tmDV : &tmDK;
                tma_store_3d(map, sbase + Ly::kDS, 0, t.jt * 128, bh);
                tma_store_3d(map, sbase + Ly::kDS + 16384, 64, t.jt * 128, bh);
              } else {
                tma_store_3d(&tmDV, sbase + Ly::kDS, 0, t.jt * 128, bh);
                tma_store_3d(&tmDK, sbase + Ly::kDS + 16384, 0, t.jt * 128, bh);
              }
              bulk_commit_group();
              bulk_wait_group_read<0>();
              mbar_arrive(bar(kBarEpiFree + turn));
            }
            __syncwarp();
          }
        }
      }
      if (!ok) break;
      i = snake_item(k + 1, cta, G, n_items);
    }
    bulk_wait_group_all();  // the epilogue's stores complete before the CTA retires
  } else {
    if constexpr (HD == 128) asm volatile("setmaxnreg.inc.sync.aligned.u32 112;");
    // ------------------------------------------------------------ dQ drain
    // Tensor memory -> registers -> swizzled fp32 staging tile -> TMA
    // reduce-add into the accumulator, 32 columns (16 KB) per box, two
    // staging buffers.  Thread 0 issues the reductions and owns their groups.
    const int r = threadIdx.x;  // query row within the tile = TMEM lane
    const uint32_t tDQ = tbase + (uint32_t(warp * 32) << 16) + Ly::kColDQ;
    const bool issuer = threadIdx.x == 0;
    bool ok = true;
    int g = 0;
    for (int k = 0, i = snake_item(0, cta, G, n_items); ok && i >= 0; ++k) {
      const Item t = imap.item(i);
      for (int h = 0, it = 0; h < group; ++g) {
        const int row0 = (t.b * p.Hq + t.h0 + h) * p.Npad + (t.it0 + it) * 128;
        // The four drain warps agree before any named barrier below, so that a
        // wait that gave up in one warp stops all of them.
        const bool got = mbar_wait_warp(bar(kBarDQFull), g & 1, ctx, 0x740);
        if (!(ok = named_barrier_and(kDrainBarrierId, 128, got))) break;
        tc_fence_after();
        // 32-column chunks.  For d = 128 the registers hold three: chunk 3
        // follows when chunk 0 is staged, and then the columns are released to
        // the MMA warp.
        auto stage = [&](int c, const uint32_t (&v)[32]) {
          const uint32_t buf = sbase + Ly::kStage + (c & 1) * 16384;
          // the reduction that last read this buffer (two boxes ago) is done
          if (issuer) bulk_wait_group_read<1>();
          named_barrier_sync(kDrainBarrierId, 128);
          const uint32_t row = buf + r * 128;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            st_shared_v4(row + ((j ^ (r & 7)) << 4), v[4 * j], v[4 * j + 1], v[4 * j + 2],
                         v[4 * j + 3]);
          fence_proxy_async_smem();
          named_barrier_sync(kDrainBarrierId, 128);
          if (issuer) {
            tma_reduce_add_2d(&tmAcc, buf, 32 * c, row0);
            bulk_commit_group();
          }
        };
        uint32_t a0[32], a1[32];
        tmem_ld32(tDQ, a0);
        tmem_ld32(tDQ + 32, a1);
        if constexpr (HD == 128) {
          uint32_t a2[32];
          tmem_ld32(tDQ + 64, a2);
          tmem_wait_ld();
          stage(0, a0);
          tmem_ld32(tDQ + 96, a0);
          tmem_wait_ld();
          tc_fence_before();
          mbar_arrive(bar(kBarDQFree));
          stage(1, a1);
          stage(2, a2);
          stage(3, a0);
        } else {
          tmem_wait_ld();
          tc_fence_before();
          mbar_arrive(bar(kBarDQFree));
          stage(0, a0);
          stage(1, a1);
        }
        if (++it == t.n_it) it = 0, ++h;
      }
      i = snake_item(k + 1, cta, G, n_items);
    }
    if (issuer) bulk_wait_group_all();  // reductions complete before the CTA retires
  }

  // ---------------------------------------------------------------- teardown
  if (*abort_flag && threadIdx.x == 0) {
    // Give copies still in flight time to land before the CTA retires.
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000ull) {
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tbase, kTmemCols);
  }
}

// Parts of key heads per work-item group without the mask: as many as keep
// their Q, dO (bf16) and dQ accumulators (fp32), 8 bytes per element of a query
// head, within 64 MB, half the L2.
inline int heads_per_group(const ScoreProblem& p) {
  const int heads = p.B * p.Hkv * p.split;
  if (p.causal) return heads;
  const size_t per_head = size_t(p.Npad) * p.d * 8 * (p.group / p.split);
  const size_t hg = (size_t(64) << 20) / per_head;
  return int(hg < 1 ? 1 : hg > size_t(heads) ? heads : hg);
}

template <int HD, bool CAP, bool SLOPES, bool SPLIT>
cudaError_t launch_t(const ScoreBwdMaps& m, const Workspace& ws, float* sums,
                     const ScoreProblem& p, float scale, int* err, cudaStream_t stream) {
  using Ly = Layout<HD>;
  cudaError_t e = set_smem_limit_once<score_bwd_kernel<HD, CAP, SLOPES, SPLIT>>(Ly::kBytes);
  if (e != cudaSuccess) return e;
  // Persistent grid: at most one CTA per SM, each walking its work items.
  const long long n_items = (long long)p.n_tiles * p.B * p.Hkv * p.split;
  const int sms = device_sm_count();
  const dim3 grid(unsigned(n_items < sms ? n_items : sms));
  return launch_kernel(score_bwd_kernel<HD, CAP, SLOPES, SPLIT>, grid, dim3(kThreads<HD>),
                       Ly::kBytes, stream, m.q, m.k, m.v, m.dout, m.acc, m.dk, m.dv, ws, p, sums,
                       heads_per_group(p), scale, err);
}

template <int HD, bool SPLIT>
cudaError_t launch_d(const ScoreBwdMaps& m, const Workspace& ws, float* sums,
                     const ScoreProblem& p, float scale, int* err, cudaStream_t stream) {
  if (p.cap)
    return p.map.slopes ? launch_t<HD, true, true, SPLIT>(m, ws, sums, p, scale, err, stream)
                        : launch_t<HD, true, false, SPLIT>(m, ws, sums, p, scale, err, stream);
  return p.map.slopes ? launch_t<HD, false, true, SPLIT>(m, ws, sums, p, scale, err, stream)
                      : launch_t<HD, false, false, SPLIT>(m, ws, sums, p, scale, err, stream);
}

}  // namespace score_bwd
}  // namespace attn
