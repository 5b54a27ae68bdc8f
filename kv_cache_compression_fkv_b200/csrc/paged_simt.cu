// Paged attention on the CUDA cores (fp32, the library's accuracy mode; one
// kernel for single tokens and chunks): fp32 products and sums throughout.
//
// Each warp owns R / 4 query rows: the running maximum and sum of a row, its
// probabilities and its output stay with the warp, so the four warps meet only
// to exchange K / V tiles.  A lane scores one key of the 32-key tile and owns
// D / 32 output dims.
#include "paged_common.cuh"

namespace fkv {

constexpr int kSimtThreads = 128;
constexpr int kSimtKeys = 32;

template <typename T, int D, int R>
__global__ void __launch_bounds__(kSimtThreads) paged_simt_kernel(const PagedArgs a) {
  constexpr int kRows = R / 4;       // rows per warp
  constexpr int kLd = D + 4;         // padded row: a warp reads 32 rows at one column
  constexpr int kDims = D / 32;      // output dims per lane
  constexpr int kVec = 16 / int(sizeof(T));
  extern __shared__ __align__(16) float sm[];
  float* Qs = sm;                    // [R][D]
  float* Ks = Qs + R * D;            // [32][kLd]
  float* Vs = Ks + kSimtKeys * kLd;  // [32][D]
  __shared__ PlanRec rec;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  plan_part<kSimtThreads>(a, reinterpret_cast<int64_t*>(sm), &rec);
  const float log2e = 1.4426950408889634f;
  Walk w;
  for (w.begin(a, rec); !w.done(); w.next(a)) {
    const int h = w.hm / a.mt;
    __syncthreads();
    for (int i = threadIdx.x; i < R * D; i += kSimtThreads) {
      const int r = i / D, d = i - r * D;
      int token, head;
      float x = 0.f;
      if (row_place(a, w.s, w.qt, w.hm, r, &token, &head))
        x = to_f32(static_cast<const T*>(a.q)[int64_t(w.s.q0 + token) * a.q_ts + int64_t(head) * a.q_hs + d]);
      Qs[i] = x;
    }
    float m[kRows], l[kRows], o[kRows][kDims], slope[kRows];
    RowSpan span[kRows];
    int pos[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
      int token, head;
      const bool ok = row_place(a, w.s, w.qt, w.hm, warp * kRows + i, &token, &head);
      pos[i] = w.s.kv - w.s.q_len + token;
      span[i] = row_span(a, w.s, pos[i]);
      slope[i] = ok && a.slopes ? a.slopes[head] : 0.f;
#pragma unroll
      for (int v = 0; v < kDims; ++v) o[i][v] = 0.f;
    }
    const int steps = w.count;
    for (int i = 0; i < steps; ++i) {
      const int k0 = block_at(w.t, w.first + i) * kSimtKeys;
      __syncthreads();
      // K and V rows of the tile; rows that no query of the tile sees, or that
      // lie in a bad page, are zeros, whatever the cache holds there
      for (int v = threadIdx.x; v < 2 * kSimtKeys * (D / kVec); v += kSimtThreads) {
        const int which = v / (kSimtKeys * (D / kVec));
        const int rem = v - which * (kSimtKeys * (D / kVec));
        const int r = rem / (D / kVec), c = (rem - r * (D / kVec)) * kVec;
        const int j = k0 + r;
        float x[kVec];
#pragma unroll
        for (int e = 0; e < kVec; ++e) x[e] = 0.f;
        if (j < w.s.kv && (j < w.s.pre || (j >= w.t.lo && j <= w.t.hi))) {
          const int id = page_id(a, w.b, j >> a.page_shift);
          if (id >= 0) {
            const T* src = static_cast<const T*>(which ? a.v_cache : a.k_cache) +
                           int64_t(id) * a.page_stride + int64_t(h) * a.head_stride +
                           int64_t(j & ((1 << a.page_shift) - 1)) * a.row_stride + c;
            const uint4 raw = *reinterpret_cast<const uint4*>(src);
            const T* e4 = reinterpret_cast<const T*>(&raw);
#pragma unroll
            for (int e = 0; e < kVec; ++e) x[e] = to_f32(e4[e]);
          }
        }
        float* dst = which ? Vs + r * D + c : Ks + r * kLd + c;
#pragma unroll
        for (int e = 0; e < kVec; ++e) dst[e] = x[e];
      }
      __syncthreads();
      const int j = k0 + lane;
      float z[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) z[r] = 0.f;
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        const float4 k4 = *reinterpret_cast<const float4*>(Ks + lane * kLd + d);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          const float4 q4 = *reinterpret_cast<const float4*>(Qs + (warp * kRows + r) * D + d);
          z[r] = fmaf(q4.x, k4.x, z[r]);
          z[r] = fmaf(q4.y, k4.y, z[r]);
          z[r] = fmaf(q4.z, k4.z, z[r]);
          z[r] = fmaf(q4.w, k4.w, z[r]);
        }
      }
      float p[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        float x = z[r] * a.scale;
        if (a.cap > 0.f) x = a.cap * tanhf(x / a.cap);
        if (a.slopes) x = fmaf(slope[r], float(j - pos[r]), x);
        x *= log2e;
        const bool see = j < w.s.kv && (j < w.s.pre || (j >= span[r].lo && j <= span[r].hi));
        x = see ? x : -INFINITY;
        float mx = x;
#pragma unroll
        for (int off = 16; off; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float mn = fmaxf(m[r], mx);
        const float ms = mn == -INFINITY ? 0.f : mn;  // nothing seen so far
        const float corr = exp2f(m[r] - ms);
        p[r] = exp2f(x - ms);
        l[r] = l[r] * corr + p[r];
        m[r] = mn;
#pragma unroll
        for (int v = 0; v < kDims; ++v) o[r][v] *= corr;
      }
#pragma unroll 4
      for (int k = 0; k < kSimtKeys; ++k) {
        float vv[kDims];
#pragma unroll
        for (int v = 0; v < kDims; v += 2)
          *reinterpret_cast<float2*>(&vv[v]) =
              *reinterpret_cast<const float2*>(Vs + k * D + lane * kDims + v);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          const float pk = __shfl_sync(0xffffffffu, p[r], k);
#pragma unroll
          for (int v = 0; v < kDims; ++v) o[r][v] = fmaf(pk, vv[v], o[r][v]);
        }
      }
    }
    const bool whole = w.whole();
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      float L = l[r];
#pragma unroll
      for (int off = 16; off; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
      int token, head;
      const int row = warp * kRows + r;
      if (!row_place(a, w.s, w.qt, w.hm, row, &token, &head)) continue;
      if (whole) {
        const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
        T* dst = static_cast<T*>(a.out) + int64_t(w.s.q0 + token) * a.o_ts + int64_t(head) * a.o_hs;
#pragma unroll
        for (int v = 0; v < kDims; ++v) dst[lane * kDims + v] = from_f32<T>(o[r][v] * inv);
        if (a.lse && lane == 0)
          a.lse[int64_t(w.s.q0 + token) * a.Hq + head] =
              L > 0.f || L != L ? (m[r] + log2f(L)) * 0.6931471805599453f : -INFINITY;
      } else {
        const int64_t at = int64_t(w.slot()) * R + row;
        float* dst = a.part_o + at * D + lane * kDims;
#pragma unroll
        for (int v = 0; v < kDims; ++v) dst[v] = o[r][v];
        if (lane == 0) a.part_ml[at] = make_float2(m[r], L);
      }
    }
  }
}

template <typename T, int D, int R>
static cudaError_t launch_simt(PagedArgs a, cudaStream_t s) {
  a.R = R;
  a.TK = kSimtKeys;
  a.mt = (a.G + R - 1) / R;
  a.tq = a.cu_q ? (a.mt == 1 ? R / a.G : 1) : 1;
  a.min_steps = 4;
  a.extra = 1;
  const size_t plan = kPlanScratch;
  size_t smem = sizeof(float) * (R * D + kSimtKeys * (D + 4) + kSimtKeys * D);
  if (smem < plan) smem = plan;
  auto* k = paged_simt_kernel<T, D, R>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  const int grid = paged_grid(2);
  e = launch_kernel(k, dim3(grid), dim3(kSimtThreads), smem, s, false, a);
  if (e != cudaSuccess) return e;
  return launch_paged_join(a, D, sizeof(T) == 2, grid, s);
}

cudaError_t launch_paged_simt(PagedArgs a, int D, cudaStream_t s) {
  return D == 128 ? launch_simt<float, 128, 16>(a, s) : launch_simt<float, 64, 16>(a, s);
}

}  // namespace fkv
