// score_bwd.cu -- the launchers of attention's backward with changed scores, its
// main kernel for key heads whose query heads one item walks (score_bwd.cuh),
// and the small kernels before and after it.
#include "score_bwd.cuh"

namespace attn {
namespace score_bwd {

// With documents, per batch element: for each key/value tile the last query
// tile whose first row still sees one of its keys (row lower bounds never
// decrease, so a binary search over query tiles), and for each key one past
// its document's last query.
__global__ void __launch_bounds__(256)
    score_bwd_tables_kernel(const __grid_constant__ Workspace ws,
                            const __grid_constant__ ScoreProblem p) {
  grid_dep_wait();
  grid_dep_launch();
  const size_t nthreads = size_t(gridDim.x) * blockDim.x;
  const size_t gt = size_t(blockIdx.x) * blockDim.x + threadIdx.x;
  for (size_t i = gt; i < size_t(p.B) * p.n_tiles; i += nthreads) {
    const int b = int(i / p.n_tiles), jt = int(i % p.n_tiles);
    const int* doc = p.doc + size_t(b) * p.N;
    int a = jt, z = p.n_tiles - 1;
    while (a < z) {
      const int mid = (a + z + 1) >> 1;
      if (first_visible_key(mid * 128, doc, p.window, p.N) <= jt * 128 + 127)
        a = mid;
      else
        z = mid - 1;
    }
    ws.items[i] = make_int2(a, 0);
  }
  for (size_t i = gt; i < size_t(p.B) * p.Npad; i += nthreads) {
    const int b = int(i / p.Npad), k = int(i % p.Npad);
    const int* doc = p.doc + size_t(b) * p.N;
    int a = k + 1, z = p.N;  // answer in [k + 1, N]
    if (k >= p.N) a = z = p.N;
    while (a < z) {
      const int mid = (a + z) >> 1;
      if (first_visible_key(mid, doc, 0, p.N) > k)
        z = mid;
      else
        a = mid + 1;
    }
    ws.qend[i] = a;
  }
}

// dK and dV of split groups: the parts' sums, added in their order, rounded to
// bf16.  Eight values a thread.
template <int HD>
__global__ void __launch_bounds__(256)
    score_bwd_join_kernel(const float* __restrict__ sums, __nv_bfloat16* __restrict__ dK,
                          __nv_bfloat16* __restrict__ dV, const __grid_constant__ ScoreProblem p,
                          float mult_v, float mult_k) {
  grid_dep_wait();
  grid_dep_launch();
  const size_t heads = size_t(p.B) * p.Hkv, units = heads * p.N * (HD / 8);
  const size_t nthreads = size_t(gridDim.x) * blockDim.x;
  for (size_t i = size_t(blockIdx.x) * blockDim.x + threadIdx.x; i < 2 * units; i += nthreads) {
    const int which = i >= units;  // dV, dK
    const size_t u = which ? i - units : i;
    const size_t row = u / (HD / 8), head = row / p.N;
    const int n = int(row - head * p.N), c = int(u % (HD / 8)) * 8;
    const float* src =
        sums + ((which * heads * p.split + head * p.split) * p.Npad + n) * HD + c;
    float a[8] = {};
    for (int s = 0; s < p.split; ++s, src += size_t(p.Npad) * HD) {
      const float4 x = __ldcs(reinterpret_cast<const float4*>(src));
      const float4 y = __ldcs(reinterpret_cast<const float4*>(src + 4));
      a[0] += x.x, a[1] += x.y, a[2] += x.z, a[3] += x.w;
      a[4] += y.x, a[5] += y.y, a[6] += y.z, a[7] += y.w;
    }
    const float m = which ? mult_k : mult_v;
    st_global_v4((which ? dK : dV) + row * HD + c, pack_bf16x2(a[0] * m, a[1] * m),
                 pack_bf16x2(a[2] * m, a[3] * m), pack_bf16x2(a[4] * m, a[5] * m),
                 pack_bf16x2(a[6] * m, a[7] * m));
  }
}

}  // namespace score_bwd

cudaError_t launch_score_bwd_tables(const Workspace& ws, const ScoreProblem& p,
                                    cudaStream_t stream) {
  const size_t blocks = (size_t(p.B) * p.Npad + 255) / 256;
  return launch_kernel(score_bwd::score_bwd_tables_kernel,
                       dim3(unsigned(blocks < 2432 ? blocks : 2432)), dim3(256), 0, stream, ws, p);
}

// How many items share a group's heads: the divisor of the group with the
// shortest estimate, in query tiles that one CTA walks (2.7 us each; 2 us with
// d = 64).  With the items heaviest first the total spreads evenly over the
// SMs, but none ends before its heaviest item; without the mask all items are
// equal and go in whole rounds.  Split sums cost a launch, some 3 tiles, and 5
// (3) tiles an item for their way to memory.  Measured, one batch element, d =
// 128, causal, one item a tile and split: 8 query heads on 1 key head, N=4096,
// 560 and 105 us (8 items); 32 on 4, N=4096, 611 and 359 us (4); 32 on 8, 342
// and 363 us (2), which this leaves alone.
int score_bwd_split(const ScoreProblem& p, int sms) {
  // tiles of the heaviest item for one head, and of all items for all heads
  const long long n = p.n_tiles, seen = p.window > 0 ? (p.window + 254LL) / 128 + 1 : n;
  const long long heaviest = seen < n ? seen : n;
  const long long total = (p.causal ? heaviest * n - heaviest * (heaviest - 1) / 2 : n * n) *
                          p.B * p.Hq;
  int best = 1;
  double least = 0;
  for (int s = 1; s <= p.group; ++s) {
    if (p.group % s) continue;
    const double item = double(heaviest) * (p.group / s);
    double t = double(total) / sms;
    if (!p.causal) {  // equal items: whole rounds
      const long long items = n * p.B * p.Hkv * s;
      t = double((items + sms - 1) / sms) * item;
    }
    if (t < item) t = item;
    if (s > 1) t += 3 + (p.d == 128 ? 5.0 : 3.0) * n * p.B * p.Hkv * s / sms;
    if (s == 1 || t < 0.95 * least) best = s, least = t;
  }
  return best;
}

cudaError_t launch_score_bwd_join(void* dK, void* dV, const float* sums, const ScoreProblem& p,
                                  float scale, cudaStream_t stream) {
  const size_t blocks = (size_t(p.B) * p.Hkv * p.N * (p.d / 8) * 2 + 255) / 256;
  const auto k = static_cast<__nv_bfloat16*>(dK);
  const auto v = static_cast<__nv_bfloat16*>(dV);
  return launch_kernel(p.d == 64 ? score_bwd::score_bwd_join_kernel<64>
                                 : score_bwd::score_bwd_join_kernel<128>,
                       dim3(unsigned(blocks < 2432 ? blocks : 2432)), dim3(256), 0, stream, sums, k,
                       v, p, p.map.slopes && !p.cap ? kPxDown : 1.f, scale * kPxDown);
}

cudaError_t launch_score_bwd_main(const ScoreBwdMaps& m, const Workspace& ws, float* sums,
                                  const ScoreProblem& p, float scale, int* err,
                                  cudaStream_t stream) {
  if (p.split > 1) return launch_score_bwd_split(m, ws, sums, p, scale, err, stream);
  return p.d == 64 ? score_bwd::launch_d<64, false>(m, ws, sums, p, scale, err, stream)
                   : score_bwd::launch_d<128, false>(m, ws, sums, p, scale, err, stream);
}

}  // namespace attn
