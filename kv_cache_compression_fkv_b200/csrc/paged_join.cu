// Joins the partial softmaxes of units that the division cut between CTAs
// (paged_common.cuh): out = sum_i O_i 2^(m_i - M) / sum_i l_i 2^(m_i - M),
// M = max m_i, partials in CTA order.
//
// One CTA column of the grid looks at one part boundary; the first boundary
// inside a cut unit joins all of it.  Bound by latency: a unit of few partials (the
// usual case) takes a warp per row, one of many (one long sequence over all CTAs)
// the eight warps of a CTA per row, each with an eighth of the partials.
#include "paged_common.cuh"

namespace fkv {

constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kJoinFew = 16;  // partials that one warp takes alone

// A row's running sums: maximum, sum and D / 32 output dims per lane.
template <int D, bool kColumns>
struct RowSum {
  static constexpr int kVec = D / 32;
  float m, l, o[kVec];

  __device__ __forceinline__ RowSum() : m(-INFINITY), l(0.f) {
#pragma unroll
    for (int v = 0; v < kVec; ++v) o[v] = 0.f;
  }
  // Adds the partials first, first + step, ... < parts of a row.
  __device__ __forceinline__ void add(const PagedArgs& a, int c, int row, int first, int step,
                                      int parts, int lane) {
#pragma unroll 4
    for (int i = first; i < parts; i += step) {
      const int64_t slot = i == 0 ? 2 * c - 1 : 2 * (c - 1 + i);
      const float2 ml = a.part_ml[slot * a.R + row];
      float x[kVec];
      const int d = lane * kVec;
      const float* src = a.part_o + slot * a.R * D +
                         (kColumns ? ((d >> 2) * a.R + row) * 4 + (d & 3) : row * D + d);
#pragma unroll
      for (int v = 0; v < kVec; v += 2)
        *reinterpret_cast<float2*>(&x[v]) = *reinterpret_cast<const float2*>(src + v);
      const float mn = fmaxf(m, ml.x), ms = mn == -INFINITY ? 0.f : mn;
      const float ca = exp2f(m - ms), cb = exp2f(ml.x - ms);
      m = mn;
      l = l * ca + ml.y * cb;
#pragma unroll
      for (int v = 0; v < kVec; ++v) o[v] = o[v] * ca + x[v] * cb;
    }
  }
};

template <typename T, int D, bool kColumns>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const PagedArgs a) {
  pdl_wait();
  const int c = int(blockIdx.x) + 1;
  const PlanRec& r = a.rec[c];
  // boundary c cuts the steps of a unit, and the previous one does not
  const int count = r.count, j = r.j, per = r.per;
  if (count == 0 || j <= r.extra || j - per > r.extra) return;
  constexpr int kVec = D / 32;
  __shared__ float s_o[kJoinWarps][D];
  __shared__ float2 s_ml[kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int parts = 1 + (r.n - j + per - 1) / per;
  const Seq s = r.s;
  const int qt = r.qt, hm = r.hm;
  int token, head;
  if (parts <= kJoinFew) {
    for (int row = int(blockIdx.y) * kJoinWarps + warp; row < a.R; row += int(gridDim.y) * kJoinWarps) {
      if (!row_place(a, s, qt, hm, row, &token, &head)) continue;
      RowSum<D, kColumns> sum;
      sum.add(a, c, row, 0, 1, parts, lane);
      const bool some = sum.l > 0.f || sum.l != sum.l;
      const float f = some ? 1.f / sum.l : 0.f;
      T* dst = static_cast<T*>(a.out) + int64_t(s.q0 + token) * a.o_ts + int64_t(head) * a.o_hs;
#pragma unroll
      for (int v = 0; v < kVec; ++v) dst[lane * kVec + v] = from_f32<T>(sum.o[v] * f);
      if (a.lse && lane == 0)
        a.lse[int64_t(s.q0 + token) * a.Hq + head] =
            some ? (sum.m + log2f(sum.l)) * 0.6931471805599453f : -INFINITY;
    }
    return;
  }
  for (int row = blockIdx.y; row < a.R; row += gridDim.y) {
    if (!row_place(a, s, qt, hm, row, &token, &head)) continue;
    RowSum<D, kColumns> sum;
    sum.add(a, c, row, warp, kJoinWarps, parts, lane);
#pragma unroll
    for (int v = 0; v < kVec; ++v) s_o[warp][lane * kVec + v] = sum.o[v];
    if (lane == 0) s_ml[warp] = make_float2(sum.m, sum.l);
    __syncthreads();
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) M = fmaxf(M, s_ml[w].x);
    const float Ms = M == -INFINITY ? 0.f : M;
    float L = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) L += s_ml[w].y * exp2f(s_ml[w].x - Ms);
    const bool some = L > 0.f || L != L;
    if (threadIdx.x < D) {
      float x = 0.f;
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w) x += s_o[w][threadIdx.x] * exp2f(s_ml[w].x - Ms);
      T* dst = static_cast<T*>(a.out) + int64_t(s.q0 + token) * a.o_ts + int64_t(head) * a.o_hs;
      dst[threadIdx.x] = from_f32<T>(some ? x / L : 0.f);
    }
    if (a.lse && threadIdx.x == 0)
      a.lse[int64_t(s.q0 + token) * a.Hq + head] = some ? (Ms + log2f(L)) * 0.6931471805599453f : -INFINITY;
    __syncthreads();
  }
}

cudaError_t launch_paged_join(const PagedArgs& a, int D, bool bf16, bool columns, int grid,
                              cudaStream_t s) {
  if (grid < 2) return cudaSuccess;
  const dim3 g(unsigned(grid - 1), 16);
  using B = __nv_bfloat16;
  auto* k = paged_join_kernel<float, 128, false>;
  if (!bf16) k = D == 128 ? k : paged_join_kernel<float, 64, false>;
  else if (columns) k = D == 128 ? paged_join_kernel<B, 128, true> : paged_join_kernel<B, 64, true>;
  else k = D == 128 ? paged_join_kernel<B, 128, false> : paged_join_kernel<B, 64, false>;
  return launch_kernel(k, g, dim3(kJoinThreads), 0, s, true, a);
}

}  // namespace fkv
