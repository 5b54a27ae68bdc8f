// Joins the partial softmaxes of units that the division cut between CTAs
// (paged_common.cuh): out = sum_i O_i 2^(m_i - M) / sum_i l_i 2^(m_i - M),
// M = max m_i, partials in CTA order.
//
// One CTA row of the grid looks at one part boundary; the first boundary inside
// a cut unit joins all of it.  A unit of many partials (one long sequence over
// all CTAs) is a short, wide reduction: its rows go to different CTAs and the
// partials of a row to the eight warps of a CTA.
#include "paged_common.cuh"

namespace fkv {

constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;

template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const PagedArgs a) {
  pdl_wait();
  const int c = int(blockIdx.x) + 1;
  const PlanRec r = a.rec[c];
  // boundary c cuts the steps of a unit, and the previous one does not
  if (r.count == 0 || r.j <= a.extra || r.j - r.per > a.extra) return;
  constexpr int kVec = D / 32;
  __shared__ float s_o[kJoinWarps][D];
  __shared__ float2 s_ml[kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int parts = 1 + (r.n - r.j + r.per - 1) / r.per;
  const Seq s = load_seq(a, r.b);
  for (int row = blockIdx.y; row < a.R; row += gridDim.y) {
    int token, head;
    if (!row_place(a, s, r.qt, r.hm, row, &token, &head)) continue;
    float m = -INFINITY, l = 0.f, o[kVec];
#pragma unroll
    for (int v = 0; v < kVec; ++v) o[v] = 0.f;
    for (int i = warp; i < parts; i += kJoinWarps) {
      const int64_t at = int64_t(i == 0 ? 2 * c - 1 : 2 * (c - 1 + i)) * a.R + row;
      const float2 ml = a.part_ml[at];
      float x[kVec];
      const float* src = a.part_o + at * D + lane * kVec;
#pragma unroll
      for (int v = 0; v < kVec; v += 2)
        *reinterpret_cast<float2*>(&x[v]) = *reinterpret_cast<const float2*>(src + v);
      if (ml.x == -INFINITY) continue;
      const float mn = fmaxf(m, ml.x);
      const float ca = exp2f(m - mn), cb = exp2f(ml.x - mn);
      m = mn;
      l = l * ca + ml.y * cb;
#pragma unroll
      for (int v = 0; v < kVec; ++v) o[v] = o[v] * ca + x[v] * cb;
    }
#pragma unroll
    for (int v = 0; v < kVec; ++v) s_o[warp][lane * kVec + v] = o[v];
    if (lane == 0) s_ml[warp] = make_float2(m, l);
    __syncthreads();
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) M = fmaxf(M, s_ml[w].x);
    const float Ms = M == -INFINITY ? 0.f : M;
    float L = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) L += s_ml[w].y * exp2f(s_ml[w].x - Ms);
    if (threadIdx.x < D) {
      float x = 0.f;
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w) x += s_o[w][threadIdx.x] * exp2f(s_ml[w].x - Ms);
      const float y = L > 0.f || L != L ? x / L : 0.f;
      T* dst = static_cast<T*>(a.out) + int64_t(s.q0 + token) * a.o_ts + int64_t(head) * a.o_hs;
      dst[threadIdx.x] = from_f32<T>(y);
    }
    if (a.lse && threadIdx.x == 0)
      a.lse[int64_t(s.q0 + token) * a.Hq + head] =
          L > 0.f || L != L ? (Ms + log2f(L)) * 0.6931471805599453f : -INFINITY;
    __syncthreads();
  }
}

cudaError_t launch_paged_join(const PagedArgs& a, int D, bool bf16, int grid, cudaStream_t s) {
  if (grid < 2) return cudaSuccess;
  const dim3 g(unsigned(grid - 1), 16);
  auto* k = bf16 ? (D == 128 ? paged_join_kernel<__nv_bfloat16, 128> : paged_join_kernel<__nv_bfloat16, 64>)
                 : (D == 128 ? paged_join_kernel<float, 128> : paged_join_kernel<float, 64>);
  return launch_kernel(k, g, dim3(kJoinThreads), 0, s, true, a);
}

}  // namespace fkv
