// score_fwd.cu -- attention forward with changed scores: capped by a tanh, with
// a bias that falls with distance, a prefix that sees itself whole, and key
// heads that several query heads share.
//
//   x_ij = f(<q_i, k_j>),  f(u) = s u, or cap tanh(s u / cap)
//   x_ij -= slope_h |i - j|            (with slopes)
//   l_i = logsumexp_j x_ij,  o_i = sum_j exp(x_ij - l_i) v_j
//
// over the keys j that row i sees (RowMask in score.cuh).
//
// The frame is the plain forward's (attn_fwd.cu): a task is two 128-row query
// tiles of one head, whose 128-row key/value tiles run through a two-stage TMA
// ring; S and P share tensor-memory columns, and the grid is fwd_grid's.  What
// differs:
//
//  * Scores are changed where they lie, in registers, before the row maximum.
//  * A cap bounds the scores, |x| <= cap log2(e) in base 2, and the bias of a
//    row is largest at its own key or, with a negative slope, at the farthest
//    one it sees.  Less that bias, up to kBoundedLog2 (a cap of 55) every 2^x
//    and their sums are fp32 (and bf16) numbers without a maximum to subtract:
//    no maximum and no rescaling, so a row's halves need not wait for one
//    another, and sixteen warps, each with half the columns of 32 rows, take
//    the place of eight.
//  * The bias -slope |i - j| of a tile wholly in its rows' past or future is a
//    number of the row plus or minus slope times the column, whose number the
//    multiply-add has as an immediate operand.  (From a table in shared memory
//    the same took N=4096 b4 h16 d=128 from 380 us without a bias to 520.)
//  * A query head reads key head h / group, through 4-D tensor maps with the
//    caller's strides: heads of a fused projection are taken as they lie.  The
//    heads of a group run side by side, so the L2 serves all but one of them.
#include <type_traits>

#include "score.cuh"

namespace attn {
namespace score_fwd {

constexpr int kTileBarrier = 1;  // named barriers of the tiles' softmax threads, + tile
constexpr int kStages = 2;
constexpr uint32_t kTmemCols = 512;
// Scores of at most this in base 2 need no maximum: weights from 2^-80 to 2^80,
// sums of 2^31 of them, and their products with values up to 2^15, are finite.
constexpr float kBoundedLog2 = 80.f;
constexpr int kBoundedKeys = 256;

// Barrier indices.
constexpr int kBarQFull = 0;
constexpr int kBarQEmpty = 1;
constexpr int kBarKFull = 2;                     // + stage
constexpr int kBarKEmpty = kBarKFull + kStages;  // + stage
constexpr int kBarVFull = kBarKEmpty + kStages;  // + stage
constexpr int kBarVEmpty = kBarVFull + kStages;  // + stage
constexpr int kBarSFull = kBarVEmpty + kStages;  // + tile (0 = A, 1 = B)
constexpr int kBarPReady = kBarSFull + 2;        // + tile
constexpr int kBarOFull = kBarPReady + 2;        // + tile
constexpr int kBarDrain = kBarOFull + 2;
constexpr int kNumBars = kBarDrain + 1;

template <int HD>
struct Layout {
  static constexpr int kTileBytes = 128 * HD * 2;  // one 128-row bf16 tile
  static constexpr int kQ = 0;                      // two query tiles
  static constexpr int kK = kQ + 2 * kTileBytes;    // kStages key tiles
  static constexpr int kV = kK + kStages * kTileBytes;
  static constexpr int kBar = kV + kStages * kTileBytes;
  static constexpr int kSum = kBar + (kNumBars * 8 + 15) / 16 * 16;  // [tile][half][128] fp32
  static constexpr int kTmemSlot = kSum + 2 * 2 * 128 * 4;
  static constexpr int kAbort = kTmemSlot + 4;
  // Padded past half of the SM's shared memory: one CTA, which allocates all
  // 512 tensor-memory columns, per SM.
  static constexpr int kRaw = (kAbort + 4 + 15) / 16 * 16;
  static constexpr int kBytes = kRaw > 118784 ? kRaw : 118784;
  static constexpr uint32_t kColO = 0;       // + tile * HD
  static constexpr uint32_t kColS = 2 * HD;  // + tile * 128
};

// One task: query tiles qt_a (A) and qt_a + 1 (B, when N reaches it and a task
// has two) of query head h of batch element b against key/value tiles kv_lo ..
// kv_lo + n_kv - 1.
struct Task {
  int b, h, qt_a, kv_lo, n_kv;
  bool has_b;
};

// Query tiles of a task, and tasks of a head.
constexpr int tasks_of(int n_tiles, int tiles) { return (n_tiles + tiles - 1) / tiles; }

// Task i of B * Hq * tasks_of(n_tiles, tiles).  Causal: heaviest first (a later
// one sees more key/value tiles), heads interleaved, a group's side by side.
// Without the mask every task costs the same and tasks run head by head.
struct TaskMap {
  const ScoreProblem& p;
  int tiles, n;  // a task's query tiles; a head's tasks

  __device__ __forceinline__ RowMask mask(int b) const {
    return {p.N, p.causal, p.window, p.doc ? p.doc + size_t(b) * p.N : nullptr,
            p.prefix ? __ldg(p.prefix + b) : 0};
  }
  __device__ __forceinline__ Task task(int i) const {
    const int BH = p.B * p.Hq;
    const int bh = p.causal ? i % BH : i / n;
    const int x = p.causal ? n - 1 - i / BH : i % n;
    Task t;
    t.b = bh / p.Hq;
    t.h = bh - t.b * p.Hq;
    t.qt_a = tiles * x;
    t.has_b = tiles == 2 && t.qt_a + 1 < p.n_tiles;
    // The first row of tile A bounds the first key tile (lower bounds never
    // decrease), the last row of the last tile the last one.
    const RowMask m = mask(t.b);
    const int last = min(p.N, (t.qt_a + (t.has_b ? 2 : 1)) * 128) - 1;
    t.kv_lo = m.lo(t.qt_a * 128) / 128;
    t.n_kv = (m.hi(last) + 127) / 128 - t.kv_lo;
    return t;
  }
};

// CTA b of G takes tasks b, 2G-1-b, 2G+b, 4G-1-b, ...: a snake over rounds,
// which evens out the heavy-first order; -1 past the last task.
__device__ __forceinline__ int snake_task(int k, int b, int G, int n_tasks) {
  const long long idx = (k & 1) ? (long long)k * G + (G - 1 - b) : (long long)k * G + b;
  return idx < n_tasks ? int(idx) : -1;
}

// Descriptor conventions (128-byte swizzle, tiles of 128 rows in 64-column
// blocks of 16 KB): a K-major operand advances 32 bytes per 16-element k-step
// within a block and 16 KB across blocks; an MN-major operand advances 2 KB
// (16 rows) per k-step, its MN extent spanning blocks 16 KB apart (LBO).

// CAP, SLOPES: how scores are changed; BOUNDED: by a cap of at most
// kBoundedLog2, in rows that may see kBoundedKeys.
template <bool BOUNDED>
struct Warps {
  static constexpr int kSoftmax = BOUNDED ? 16 : 8;
  static constexpr int kTileThreads = 16 * kSoftmax;  // softmax threads of a query tile
  static constexpr int kProducer = kSoftmax;
  static constexpr int kMma = kSoftmax + 1;
  static constexpr int kThreads = 32 * (kSoftmax + 2);
};

template <int HD, bool CAP, bool SLOPES, bool BOUNDED>
__global__ void __launch_bounds__(Warps<BOUNDED>::kThreads, 1)
    score_fwd_kernel(const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, __nv_bfloat16* __restrict__ O,
                     float* __restrict__ Lout, const __grid_constant__ ScoreProblem p, int tiles,
                     int* err) {
  using Ly = Layout<HD>;
  constexpr int kProducerWarp = Warps<BOUNDED>::kProducer, kMmaWarp = Warps<BOUNDED>::kMma;
  constexpr int kTileThreads = Warps<BOUNDED>::kTileThreads;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (sbase & 1023u) {  // uniform over the CTA: every thread returns here
    if (threadIdx.x == 0) report_error(err, kDevSmemAlign, 0x600);
    return;
  }

  const int N = p.N;
  const int n_tasks = p.B * p.Hq * tasks_of(p.n_tiles, tiles);
  const int G = int(gridDim.x), cta = int(blockIdx.x);
  const TaskMap tm{p, tiles, tasks_of(p.n_tiles, tiles)};

  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Ly::kAbort);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Ly::kTmemSlot);
  auto bar = [&](int i) -> uint32_t { return sbase + Ly::kBar + 8 * i; };

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < kNumBars; ++i)
      mbar_init(bar(i), i == kBarPReady || i == kBarPReady + 1 ? kTileThreads : 1);
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
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  const WaitCtx ctx{abort_flag, err, kWaitLimitNs};
  // Everything above overlaps the previous kernel; its results are read below.
  grid_dep_wait();
  grid_dep_launch();
  if (warp == kProducerWarp) {
    // ------------------------------------------------------------ TMA producer
    // The whole warp runs the loop (warp-uniform operands); one lane issues.
    // Key/value tiles run through the ring across tasks (g counts them), so
    // the next task's first tiles load while this one finishes.
    bool ok = true;
    int g = 0;
    for (int k = 0, i = snake_task(0, cta, G, n_tasks); ok && i >= 0;
         i = snake_task(++k, cta, G, n_tasks)) {
      const Task tk = tm.task(i);
      const int hk = tk.h / p.group;
      // Both query tiles are free once the previous task's last S completed.
      if (k > 0 && !(ok = mbar_wait_warp(bar(kBarQEmpty), (k - 1) & 1, ctx, 0x612))) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(bar(kBarQFull), (tk.has_b ? 2 : 1) * Ly::kTileBytes);
        for (int t = 0; t < (tk.has_b ? 2 : 1); ++t)
#pragma unroll
          for (int cb = 0; cb < HD / 64; ++cb)
            tma_load_4d(sbase + Ly::kQ + t * Ly::kTileBytes + cb * 16384, &tmQ, bar(kBarQFull),
                        cb * 64, (tk.qt_a + t) * 128, tk.h, tk.b);
      }
      __syncwarp();
      for (int j = 0; j < tk.n_kv; ++j, ++g) {
        const int s = g % kStages, n = g / kStages;
        if (g >= kStages && !(ok = mbar_wait_warp(bar(kBarKEmpty + s), (n - 1) & 1, ctx, 0x610)))
          break;
        if (elect_one()) {
          mbar_arrive_expect_tx(bar(kBarKFull + s), Ly::kTileBytes);
#pragma unroll
          for (int cb = 0; cb < HD / 64; ++cb)
            tma_load_4d(sbase + Ly::kK + s * Ly::kTileBytes + cb * 16384, &tmK,
                        bar(kBarKFull + s), cb * 64, (tk.kv_lo + j) * 128, hk, tk.b);
        }
        __syncwarp();
        if (g >= kStages && !(ok = mbar_wait_warp(bar(kBarVEmpty + s), (n - 1) & 1, ctx, 0x611)))
          break;
        if (elect_one()) {
          mbar_arrive_expect_tx(bar(kBarVFull + s), Ly::kTileBytes);
#pragma unroll
          for (int cb = 0; cb < HD / 64; ++cb)
            tma_load_4d(sbase + Ly::kV + s * Ly::kTileBytes + cb * 16384, &tmV,
                        bar(kBarVFull + s), cb * 64, (tk.kv_lo + j) * 128, hk, tk.b);
        }
        __syncwarp();
      }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp runs the loop and waits; one elected lane issues.  Every
    // descriptor is a per-tile base plus a compile-time k-step offset.
    constexpr uint32_t kIdS = make_idesc_bf16(128, 128, 0, 0);  // S = Q K^T
    constexpr uint32_t kIdO = make_idesc_bf16(128, HD, 0, 1);   // O += P V
    const uint64_t dQa = make_sdesc_sw128(sbase + Ly::kQ, 16, 1024);
    const uint64_t dQb = make_sdesc_sw128(sbase + Ly::kQ + Ly::kTileBytes, 16, 1024);
    auto issue_s = [&](int t, int stage) {  // elected lane only
      const uint64_t dq = t == 0 ? dQa : dQb;
      const uint64_t dk = make_sdesc_sw128(sbase + Ly::kK + stage * Ly::kTileBytes, 16, 1024);
      const uint32_t d = tbase + Ly::kColS + 128 * t;
#pragma unroll
      for (int k = 0; k < HD / 16; ++k) {
        const uint32_t off = (k >> 2) * 16384 + (k & 3) * 32;
        mma_ss(d, sdesc_add(dq, off), sdesc_add(dk, off), kIdS, k > 0 ? 1u : 0u);
      }
      tc_commit(bar(kBarSFull + t));
    };
    auto issue_pv = [&](int t, int stage, uint32_t acc) {  // elected lane only
      const uint64_t dv = make_sdesc_sw128(sbase + Ly::kV + stage * Ly::kTileBytes, 16384, 1024);
      const uint32_t d = tbase + Ly::kColO + HD * t;
      const uint32_t pc = tbase + Ly::kColS + 128 * t;
#pragma unroll
      for (int k = 0; k < 8; ++k)  // 128 keys, 16 per step; P packed 2 per column of its half
        mma_ts(d, pc + 64 * (k >> 2) + 8 * (k & 3), sdesc_add(dv, k * 2048), kIdO,
               k > 0 ? 1u : acc);
    };
    // Handshake counts across tasks: g key/value tiles, ca (cb) S/P rounds of
    // tile A (B).  A task's first P V overwrites O_t; the softmax warps of
    // tile t read the previous task's O_t before they signal the first P of
    // this one, so the P-ready wait covers that hazard.  Tensor-core
    // instructions of this thread run in issue order, so an S written into
    // the columns that hold P comes after the P V that reads them.
    bool ok = true;
    int g = 0, ca = 0, cb = 0;
    for (int k = 0, i = snake_task(0, cta, G, n_tasks); ok && i >= 0;
         i = snake_task(++k, cta, G, n_tasks)) {
      const Task tk = tm.task(i);
      const int n_kv = tk.n_kv;
      if (!(ok = mbar_wait_warp(bar(kBarQFull), k & 1, ctx, 0x620))) break;
      if (!(ok = mbar_wait_warp(bar(kBarKFull + g % kStages), (g / kStages) & 1, ctx, 0x621)))
        break;
      tc_fence_after();
      if (elect_one()) {
        issue_s(0, g % kStages);
        if (tk.has_b) issue_s(1, g % kStages);
        if (n_kv == 1) tc_commit(bar(kBarQEmpty));  // the task's last S
        tc_commit(bar(kBarKEmpty + g % kStages));
      }
      __syncwarp();
      for (int j = 0; j < n_kv; ++j, ++g) {
        const int s = g % kStages;
        const bool next = j + 1 < n_kv;
        const int s1 = (g + 1) % kStages, n1 = (g + 1) / kStages;
        const uint32_t acc = j > 0 ? 1u : 0u;
        if (!(ok = mbar_wait_warp(bar(kBarVFull + s), (g / kStages) & 1, ctx, 0x622))) break;
        if (!(ok = mbar_wait_warp(bar(kBarPReady + 0), (ca + j) & 1, ctx, 0x623))) break;
        tc_fence_after();
        if (elect_one()) issue_pv(0, s, acc);
        __syncwarp();
        if (next) {
          if (!(ok = mbar_wait_warp(bar(kBarKFull + s1), n1 & 1, ctx, 0x624))) break;
          tc_fence_after();
          if (elect_one()) issue_s(0, s1);
          __syncwarp();
        }
        if (tk.has_b) {
          if (!(ok = mbar_wait_warp(bar(kBarPReady + 1), (cb + j) & 1, ctx, 0x625))) break;
          tc_fence_after();
          if (elect_one()) {
            issue_pv(1, s, acc);
            if (next) issue_s(1, s1);
          }
          __syncwarp();
        }
        if (elect_one()) {
          if (j + 2 == n_kv) tc_commit(bar(kBarQEmpty));  // the task's last S was issued above
          tc_commit(bar(kBarVEmpty + s));
          if (next) tc_commit(bar(kBarKEmpty + s1));
        }
        __syncwarp();
      }
      if (!ok) break;
      if (elect_one()) {
        tc_commit(bar(kBarOFull + 0));
        if (tk.has_b) tc_commit(bar(kBarOFull + 1));
      }
      __syncwarp();
      ca += n_kv;
      if (tk.has_b) cb += n_kv;
    }
    // Wait until every MMA issued above has completed before teardown.
    if (elect_one()) tc_commit(bar(kBarDrain));
    __syncwarp();
    volatile int never = 0;  // this wait ignores the CTA abort flag
    const WaitCtx own{&never, err, kWaitLimitNs};
    mbar_wait_warp(bar(kBarDrain), 0, own, 0x62F);
  } else {
    // ------------------------------------------------------------ softmax
    // 0 = tile A, 1 = tile B; without BOUNDED a thread has its whole row, with
    // it columns 64 half .. 64 half + 63.
    const int t = (warp / (Warps<BOUNDED>::kSoftmax / 2)) & 1;
    const int half = BOUNDED ? (warp >> 2) & 1 : 0;
    const int r = threadIdx.x & 127;
    const uint32_t lane_off = uint32_t((warp & 3) * 32) << 16;
    const uint32_t tS = tbase + lane_off + Ly::kColS + 128 * t + 64 * half;
    const uint32_t tO = tbase + lane_off + Ly::kColO + HD * t;
    const ScoreMap& mp = p.map;
    bool ok = true;
    int c = 0;   // S/P rounds of this tile so far
    int no = 0;  // outputs of this tile so far
    for (int k = 0, i = snake_task(0, cta, G, n_tasks); ok && i >= 0;
         i = snake_task(++k, cta, G, n_tasks)) {
      const Task tk = tm.task(i);
      if (t == 1 && !tk.has_b) continue;
      const int q_tile0 = (tk.qt_a + t) * 128;
      const int q = q_tile0 + r;
      const RowMask mask = tm.mask(tk.b);
      // The row sees keys lo_q <= j < hi_q; every row of the warp sees those
      // of [all_lo, all_hi).
      const int lo_q = mask.lo(q), hi_q = mask.hi(q);
      const int all_lo = __reduce_max_sync(0xffffffffu, lo_q);
      const int all_hi = __reduce_min_sync(0xffffffffu, hi_q);
      float m = BOUNDED ? 0.f : -INFINITY;  // running max of the base-2 scores
      float l = 0.f;                        // running sum of 2^(x - m)
      if constexpr (BOUNDED) {
        float slope = 0.f;
        if constexpr (SLOPES) {
          slope = __ldg(mp.slopes + tk.h) * 1.4426950408889634f;
          // the largest bias of the row, whose own key it sees
          m = slope < 0.f ? -slope * float(max(q - lo_q, hi_q - 1 - q)) : 0.f;
        }
        for (int j = 0; j < tk.n_kv; ++j) {
          if (!(ok = mbar_wait_warp(bar(kBarSFull + t), (c + j) & 1, ctx, 0x630 + t))) break;
          tc_fence_after();
          const int kv0 = (tk.kv_lo + j) * 128 + 64 * half;  // this half's first key
          const int e_lo = lo_q - kv0, e_hi = hi_q - kv0;    // the row's columns
          uint64_t sum[2] = {0, 0};
#pragma unroll
          for (int ch = 0; ch < 2; ++ch) {
            uint32_t u[32], pk[16];
            tmem_ld32(tS + 32 * ch, u);
            tmem_wait_ld();
            // Two columns' biases less m.
            float sl = 0.f, row = 0.f, d0 = 0.f;
            bool linear = true;
            if constexpr (SLOPES) {
              d0 = float(q - kv0 - 32 * ch);
              const int w0 = q_tile0 + 32 * (warp & 3);  // the warp's first row
              const bool past = kv0 + 32 * ch + 31 <= w0;
              linear = past || kv0 + 32 * ch >= w0 + 31;  // one sign for the warp's distances
              sl = past ? slope : -slope;
              row = fmaf(-sl, d0, -m);
            }
            auto bias = [&](int e, auto edge) {  // distances are whole numbers, exact below 2^24
              if (!decltype(edge)::value || linear)
                return f32x2(fmaf(sl, float(e), row), fmaf(sl, float(e + 1), row));
              return f32x2(fmaf(-slope, fabsf(d0 - float(e)), -m),
                           fmaf(-slope, fabsf(d0 - float(e + 1)), -m));
            };
            float far[kTanhFarTerms];
            auto weigh = [&](int e, auto near, auto edge) {
              const uint64_t v = f32x2(__uint_as_float(u[e]), __uint_as_float(u[e + 1]));
              uint64_t x;
              if constexpr (decltype(near)::value > 0) {
                const uint64_t h = decltype(near)::value == 1 ? cap_factor(mp.poly, v)
                                                              : cap_factor(far, v);
                x = SLOPES ? fma_f32x2(v, h, bias(e, edge)) : mul_f32x2(v, h);
              } else {
                x = fma_f32x2(f32x2(cap_r(mp, __uint_as_float(u[e])),
                                    cap_r(mp, __uint_as_float(u[e + 1]))),
                              f32x2(-2.f * mp.cap_log2), f32x2(mp.cap_log2));
                if constexpr (SLOPES) x = add_f32x2(x, bias(e, edge));
              }
              float p0, p1;
              f32x2_split(x, p0, p1);
              p0 = ex2(p0);
              p1 = ex2(p1);
              if constexpr (decltype(edge)::value) {
                const int col = 32 * ch + e;
                if (col < e_lo || col >= e_hi) p0 = 0.f;
                if (col + 1 < e_lo || col + 1 >= e_hi) p1 = 0.f;
              }
              sum[(e >> 1) & 1] = add_f32x2(sum[(e >> 1) & 1], f32x2(p0, p1));
              pk[e / 2] = pack_bf16x2(p0, p1);
            };
            auto all = [&](auto edge) {
              const float top = top_of(u);
              if (all_within(top, mp.poly_limit)) {
#pragma unroll
                for (int e = 0; e < 32; e += 2) weigh(e, std::integral_constant<int, 1>(), edge);
              } else if (all_within(top, mp.far_limit)) {
                // Read here and nowhere earlier: held through the loop, these
                // constants' registers cost the nearer path 5 % (N=16384 h16
                // d=128, one set of inputs: 885 in place of 841 us; 820 without
                // this path, which takes sharp heads, scores up to the cap, from
                // 1,218 to 1,040).
#pragma unroll
                for (int k = 0; k < kTanhFarTerms; ++k) {
                  far[k] = mp.far_poly[k];
                  asm volatile("" : "+f"(far[k]));
                }
#pragma unroll
                for (int e = 0; e < 32; e += 2) weigh(e, std::integral_constant<int, 2>(), edge);
              } else {
#pragma unroll
                for (int e = 0; e < 32; e += 2) weigh(e, std::integral_constant<int, 0>(), edge);
              }
            };
            // (a piece with distances of both signs takes the masked path too,
            // which is the rare one)
            if (kv0 + 32 * ch < all_lo || kv0 + 32 * ch + 32 > all_hi || !linear)
              all(std::true_type());
            else
              all(std::false_type());
            tmem_st16(tS + 16 * ch, pk);  // onto columns that have been read
          }
          float s0, s1;
          f32x2_split(add_f32x2(sum[0], sum[1]), s0, s1);
          l += s0 + s1;
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(bar(kBarPReady + t));
        }
        // The halves' sums, written behind the wait for O: O is complete once all
        // threads of the tile have signalled this task's P, and each of them had
        // read the other half's sum of the task before by then.  (Ahead of that
        // wait nothing orders the two where a task has one key tile: its S comes
        // without a signal from the softmax warps.)  A wait that gave up in one
        // warp stops the tile's eight.
        ok = ok && mbar_wait_warp(bar(kBarOFull + t), no & 1, ctx, 0x638 + t);
        float* sums = reinterpret_cast<float*>(smem + Ly::kSum) + 256 * t + r;
        if (ok) sums[128 * half] = l;
        if (!(ok = named_barrier_and(kTileBarrier + t, kTileThreads, ok))) break;
        l += sums[128 * (1 - half)];
      } else {
        // Under a cap u becomes the score in base 2, else it stays a raw product,
        // to which the bias, divided by the scale, is added.
        float slope = 0.f;
        if constexpr (SLOPES) {
          slope = __ldg(mp.slopes + tk.h) * 1.4426950408889634f;
          if (!CAP) slope /= mp.scale_log2;
        }
        for (int j = 0; j < tk.n_kv; ++j) {
          if (!(ok = mbar_wait_warp(bar(kBarSFull + t), (c + j) & 1, ctx, 0x630 + t))) break;
          tc_fence_after();
          uint32_t u[128];
          tmem_ld32(tS + 0, *reinterpret_cast<uint32_t(*)[32]>(&u[0]));
          tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&u[32]));
          tmem_ld32(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(&u[64]));
          tmem_ld32(tS + 96, *reinterpret_cast<uint32_t(*)[32]>(&u[96]));
          tmem_wait_ld();
          const int kv0 = (tk.kv_lo + j) * 128;
          const bool edge = kv0 < all_lo || kv0 + 128 > all_hi;
          auto f = [&](int e) { return __uint_as_float(u[e]); };
          auto pair = [&](int e) { return f32x2(f(e), f(e + 1)); };
          auto put = [&](int e, uint64_t x) {
            float a, b;
            f32x2_split(x, a, b);
            u[e] = __float_as_uint(a);
            u[e + 1] = __float_as_uint(b);
          };
          const uint64_t sc = f32x2(mp.scale_log2);
          if constexpr (CAP) {
            if (all_within(top_of(u), mp.poly_limit)) {
#pragma unroll
              for (int e = 0; e < 128; e += 2) put(e, cap_poly(mp, pair(e)));
            } else {
#pragma unroll
              for (int e = 0; e < 128; ++e)
                u[e] = __float_as_uint(fmaf(cap_r(mp, f(e)), -2.f * mp.cap_log2, mp.cap_log2));
            }
          }
          float row = 0.f;  // the row's share of the bias: x = u + row
          if constexpr (SLOPES) {
            const float d0 = float(q - kv0);
            const int w0 = q_tile0 + 32 * (warp & 3);  // the warp's first row
            const bool past = kv0 + 127 <= w0;
            if (past || kv0 >= w0 + 31) {  // one sign for every distance of the warp
              const float sl = past ? slope : -slope;
              row = -sl * d0;
#pragma unroll
              for (int e = 0; e < 128; ++e) u[e] = __float_as_uint(fmaf(sl, float(e), f(e)));
            } else {  // distances are whole numbers, exact below 2^24
#pragma unroll
              for (int e = 0; e < 128; ++e)
                u[e] = __float_as_uint(fmaf(-slope, fabsf(d0 - float(e)), f(e)));
            }
            if (!CAP) row *= mp.scale_log2;
          }
          if (edge) {
            const int e_lo = lo_q - kv0, e_hi = hi_q - kv0;
#pragma unroll
            for (int e = 0; e < 128; ++e)
              if (e >= e_hi || e < e_lo) u[e] = __float_as_uint(-INFINITY);
          }
          // row maximum: eight chains of three-input maxima (two scores each)
          float m8[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) m8[e] = f(e);
#pragma unroll
          for (int e = 8; e < 128; e += 2)
            m8[(e >> 1) & 7] = max3f(m8[(e >> 1) & 7], f(e), f(e + 1));
          const float mx = max3f(max3f(m8[0], m8[1], m8[2]), max3f(m8[3], m8[4], m8[5]),
                                 fmaxf(m8[6], m8[7]));
          // scale > 0, so the maximum commutes with it
          const float m_new = fmaxf(m, CAP ? mx + row : fmaf(mx, mp.scale_log2, row));
          // Lazy rescale: move the reference maximum (and rescale l and O by
          // 2^(m - m_new)) only when the maximum grew by more than 8 in base 2.
          const bool rescale = m_new > m + 8.f;
          const float alpha = rescale ? ex2(m - m_new) : 1.f;
          if (rescale) {
            l *= alpha;
            m = m_new;
          }
          const uint64_t mb = f32x2(m == -INFINITY ? 0.f : row - m);
          uint64_t sum[2] = {0, 0};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t pk[32];
#pragma unroll
            for (int e = 0; e < 64; e += 2) {
              float p0, p1;
              f32x2_split(CAP ? add_f32x2(pair(64 * h + e), mb)
                              : fma_f32x2(pair(64 * h + e), sc, mb), p0, p1);
              p0 = ex2(p0);
              p1 = ex2(p1);
              sum[(e >> 1) & 1] = add_f32x2(sum[(e >> 1) & 1], f32x2(p0, p1));
              pk[e / 2] = pack_bf16x2(p0, p1);
            }
            tmem_st32(tS + 64 * h, pk);
          }
          float s0, s1;
          f32x2_split(add_f32x2(sum[0], sum[1]), s0, s1);
          l += s0 + s1;
          // tcgen05.ld/st are warp-collective: if any row of the warp moved its
          // maximum, the whole warp rescales (alpha = 1 leaves the other rows
          // unchanged).  O holds P V of earlier tiles; PV(j-1) has completed.
          if (j > 0 && __any_sync(0xffffffffu, rescale)) {
#pragma unroll
            for (int c4 = 0; c4 < HD / 32; ++c4) {
              uint32_t o[32];
              tmem_ld32(tO + 32 * c4, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32(tO + 32 * c4, o);
            }
          }
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(bar(kBarPReady + t));
        }
        if (!ok || !(ok = mbar_wait_warp(bar(kBarOFull + t), no & 1, ctx, 0x638 + t))) break;
      }
      c += tk.n_kv;
      ++no;
      tc_fence_after();
      // Without a maximum a row that sees one key weighs it by its 2^x, which met V
      // rounded to bf16: divided by that, O is v, and D then <do, v>, as the
      // gradient of such a row, zero, needs it.  (For rows of more keys the sum of
      // the rounded weights is no better a divisor: it moves O by 2^-8 of sum p |v
      // - o| where l moves it by as much of sum p |v|.)
      const float inv_l =
          1.f / (BOUNDED && hi_q - lo_q == 1 ? bf16lo_to_f32(pack_bf16x2(l, 0.f)) : l);
      const size_t row = (size_t(tk.b) * p.Hq + tk.h) * N + q;
      constexpr int kCols = BOUNDED ? HD / 2 : HD;  // of this thread
      __nv_bfloat16* orow = O + row * HD + kCols * half;
#pragma unroll
      for (int c4 = 0; c4 < kCols / 32; ++c4) {
        uint32_t o[32];
        tmem_ld32(tO + kCols * half + 32 * c4, o);
        tmem_wait_ld();
        if (q < N) {
#pragma unroll
          for (int c8 = 0; c8 < 4; ++c8) {
            uint32_t w4[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w4[e] = pack_bf16x2(__uint_as_float(o[8 * c8 + 2 * e]) * inv_l,
                                  __uint_as_float(o[8 * c8 + 2 * e + 1]) * inv_l);
            st_global_v4(orow + 32 * c4 + 8 * c8, w4[0], w4[1], w4[2], w4[3]);
          }
        }
      }
      if (q < N && half == 0) Lout[row] = (m + log2f(l)) * 0.69314718055994530942f;
      // O_t has been read into registers (tmem_wait_ld above) before this
      // warp signals the next task's first P.
      tc_fence_before();
    }
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

template <int HD, bool CAP, bool SLOPES, bool BOUNDED>
static cudaError_t launch_t(const CUtensorMap& tmQ, const CUtensorMap& tmK,
                            const CUtensorMap& tmV, void* O, float* L, const ScoreProblem& p,
                            int* err, cudaStream_t stream) {
  using Ly = Layout<HD>;
  constexpr auto kern = score_fwd_kernel<HD, CAP, SLOPES, BOUNDED>;
  constexpr int kThreads = Warps<BOUNDED>::kThreads;
  cudaError_t e = set_smem_limit_once<kern>(Ly::kBytes);
  if (e != cudaSuccess) return e;
  const long long heads = (long long)p.B * p.Hq;
  const long long pairs = tasks_of(p.n_tiles, 2) * heads;
  // One query tile a task where tasks of two would leave SMs idle: a step of one
  // takes two thirds of the time of two.  Under the mask, where half of a
  // task's tiles is what the mean has, up to one pair an SM (128 pairs of
  // N=2048 d=128 with a cap: 38 and 30 us), without it while all single tiles
  // run at once (64 pairs: 36 and 30 us; 96 pairs: 37 and 56).
  const int tiles = (p.causal ? pairs : 2 * pairs) <= device_sm_count() ? 1 : 2;
  const long long n_tasks = tasks_of(p.n_tiles, tiles) * heads;
  const dim3 grid(unsigned(fwd_grid(n_tasks, p.causal)));
  return launch_kernel(kern, grid, dim3(kThreads), Ly::kBytes, stream, tmQ, tmK, tmV,
                       static_cast<__nv_bfloat16*>(O), L, p, tiles, err);
}

template <int HD>
static cudaError_t launch_d(const CUtensorMap& tmQ, const CUtensorMap& tmK,
                            const CUtensorMap& tmV, void* O, float* L, const ScoreProblem& p,
                            int* err, cudaStream_t stream) {
  const bool slopes = p.map.slopes;
  // Calls whose rows all see few keys keep the maximum: its weight is 1,
  // exactly, where 2^x rounded to bf16 is off by up to 2^-8 of itself, which many
  // keys average out.
  const int seen = p.window > 0 ? p.window : p.N;
  if (p.cap && p.map.cap_log2 <= kBoundedLog2 && seen >= kBoundedKeys)
    return slopes ? launch_t<HD, true, true, true>(tmQ, tmK, tmV, O, L, p, err, stream)
                  : launch_t<HD, true, false, true>(tmQ, tmK, tmV, O, L, p, err, stream);
  if (p.cap)
    return slopes ? launch_t<HD, true, true, false>(tmQ, tmK, tmV, O, L, p, err, stream)
                  : launch_t<HD, true, false, false>(tmQ, tmK, tmV, O, L, p, err, stream);
  return slopes ? launch_t<HD, false, true, false>(tmQ, tmK, tmV, O, L, p, err, stream)
                : launch_t<HD, false, false, false>(tmQ, tmK, tmV, O, L, p, err, stream);
}

}  // namespace score_fwd

cudaError_t launch_score_fwd(const CUtensorMap& tmQ, const CUtensorMap& tmK,
                             const CUtensorMap& tmV, void* O, float* L, const ScoreProblem& p,
                             int* err, cudaStream_t stream) {
  return p.d == 64 ? score_fwd::launch_d<64>(tmQ, tmK, tmV, O, L, p, err, stream)
                   : score_fwd::launch_d<128>(tmQ, tmK, tmV, O, L, p, err, stream);
}

}  // namespace attn
