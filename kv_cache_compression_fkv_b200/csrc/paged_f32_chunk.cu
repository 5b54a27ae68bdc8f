// Attention of a ragged batch of query tokens over the paged cache in fp32 (the
// library's accuracy mode), on the CUDA cores: fp32 products and sums throughout.
//
// Bound by the FMA pipe.  A CTA takes 64 (token, head) rows, each of its four warps
// 16 of them against whole 32-key blocks of K and V, which arrive by asynchronous
// copies one step ahead.  Scores: a lane owns 4 rows x 4 keys (rows 4 rg .., keys
// kg + 8 i), so 4 + 4 reads of 16 bytes feed 64 FMAs (32 packed ones); the blocks are swizzled so
// that each read is one wavefront (8 keys side by side, or 4 rows broadcast).
// P V: 4 rows x D / 8 dims per lane, 1 + D / 32 reads per key for D / 2 FMAs, the
// probabilities passing through the warp's own corner of shared memory.  A warp
// keeps the maxima, sums and outputs of its rows, so warps share nothing but the
// key blocks.
//
// Measured: 1000 queries over 4000 keys, 16 heads, D = 128: 0.84 ms = 34 TFLOP/s
// (14 with 16 rows per CTA and a lane per key, 29 with unpacked products).
#include "paged_f32.cuh"

namespace fkv {

constexpr int kChunkRows = 64, kWarpRows = 16;

template <int D>
struct ChunkCfg {
  static constexpr int kStage = 2 * kF32Keys * D;            // floats: K, V
  static constexpr int kOffQ = 2 * kStage;                   // [64][D]
  static constexpr int kOffP = kOffQ + kChunkRows * D;       // [warp][32 keys][16 rows]
  static constexpr int kFloats = kOffP + 4 * kF32Keys * kWarpRows;
};

// Place of 16-byte chunk c of K row r, and of query row r.
template <int D>
__device__ __forceinline__ int k_swz(int r, int c) {
  return r * D + ((c ^ (r & 7)) << 2);
}
template <int D>
__device__ __forceinline__ int q_swz(int r, int c) {
  return r * D + ((c ^ ((r >> 2) & 7)) << 2);
}

template <int D>
__global__ void __launch_bounds__(kF32Threads, 2) paged_f32_chunk_kernel(const PagedArgs a) {
  using C = ChunkCfg<D>;
  constexpr int kCols = D / 32;  // 16-byte columns of the output per lane
  extern __shared__ __align__(16) float sm[];
  __shared__ PlanRec rec;
  __shared__ int2 place[kChunkRows];  // token and head of a row of the unit; head -1: no row
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rg = lane & 3, kg = lane >> 2;  // row group; key group, or dim group
  plan_part<kF32Threads>(a, reinterpret_cast<int64_t*>(sm), &rec);
  const float kLog2e = 1.4426950408889634f;
  float* Q = sm + C::kOffQ;
  float* P = sm + C::kOffP + warp * kF32Keys * kWarpRows;

  Walk lw, w;
  lw.begin(a, rec);
  w.begin(a, rec);
  int li = 0, ln = 0, ids[Rows<D>::kCount];
  unsigned want = 0;
  if (!lw.done()) fetch_pages<D>(a, lw, 0, ids, want);
  auto load_next = [&]() {
    if (!lw.done()) {
      float* stage = sm + (ln & 1) * C::kStage;
      load_keys<D>(a, lw, li, ids, want, [&](int r, int c) { return stage + k_swz<D>(r, c); },
                   [&](int r, int c) { return stage + kF32Keys * D + r * D + c * 4; });
      ++ln;
      if (++li == lw.count) {
        li = 0;
        lw.next(a);
      }
      if (!lw.done()) fetch_pages<D>(a, lw, li, ids, want);
    }
    cp_async_commit();
  };

  int n = 0;
  if (!w.done()) load_next();
  for (; !w.done(); w.next(a)) {
    __syncthreads();  // the last unit's queries and places are done with
    if (threadIdx.x < kChunkRows) {
      int token, head;
      const bool valid = row_place(a, w.s, w.qt, w.hm, threadIdx.x, &token, &head);
      place[threadIdx.x] = make_int2(w.s.q0 + token, valid ? head : -1);
    }
    __syncthreads();
#pragma unroll 2
    for (int e = threadIdx.x; e < kChunkRows * (D / 4); e += kF32Threads) {
      const int r = e / (D / 4), c = e % (D / 4);
      const int2 at = place[r];
      const bool read = at.y >= 0;
      const float* src = static_cast<const float*>(a.q);
      if (read) src += int64_t(at.x) * a.q_ts + int64_t(at.y) * a.q_hs + c * 4;
      cp_async16(Q + q_swz<D>(r, c), src, read);
    }
    cp_async_commit();
    const int p0 = w.s.kv - w.s.q_len + w.qt * a.tq;  // position of the first token
    const int all_hi = a.causal ? p0 : w.s.kv - 1;
    const int all_lo = a.window > 0 ? p0 + a.tq - a.window : 0;
    bool live = false;  // some row of this warp is there
    int pos[4];
    float slope[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int2 at = place[warp * kWarpRows + rg * 4 + r];
      const bool valid = at.y >= 0;
      pos[r] = w.s.kv - w.s.q_len + at.x - w.s.q0;
      slope[r] = a.slopes && valid ? a.slopes[at.y] : 0.f;
      live |= valid;
    }
    live = __any_sync(0xffffffffu, live);
    float m[4], l[4];
    float2 o[4][kCols][2];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int c = 0; c < kCols; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e) o[r][c][e] = make_float2(0.f, 0.f);
    }
    for (int i = 0; i < w.count; ++i, ++n) {
      cp_async_wait<0>();
      __syncthreads();  // step n (and the queries) are here for all; step n - 1 is done with
      load_next();
      if (!live) continue;
      const float* K = sm + (n & 1) * C::kStage;
      const float* V = K + kF32Keys * D;
      const int k0 = block_at(w.t, w.first + i) * kF32Keys;
      float2 zz[4][4];  // sums over even and odd dims
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int k = 0; k < 4; ++k) zz[r][k] = make_float2(0.f, 0.f);
#pragma unroll 2
      for (int c = 0; c < D / 4; ++c) {
        float4 q4[4], k4[4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
          q4[r] = *reinterpret_cast<const float4*>(Q + q_swz<D>(warp * kWarpRows + rg * 4 + r, c));
#pragma unroll
        for (int k = 0; k < 4; ++k)
          k4[k] = *reinterpret_cast<const float4*>(K + k_swz<D>(kg + 8 * k, c));
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            zz[r][k] = fma2(make_float2(q4[r].x, q4[r].y), make_float2(k4[k].x, k4[k].y), zz[r][k]);
            zz[r][k] = fma2(make_float2(q4[r].z, q4[r].w), make_float2(k4[k].z, k4[k].w), zz[r][k]);
          }
      }
      const bool full = k0 + 31 < w.s.pre || (k0 >= all_lo && k0 + 31 <= all_hi);
      // options by the block, so that the code of those a call lacks is never fetched
      float z[4][4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int k = 0; k < 4; ++k) z[r][k] = (zz[r][k].x + zz[r][k].y) * a.scale;
      if (a.cap > 0.f) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int k = 0; k < 4; ++k) z[r][k] = a.cap * tanhf(z[r][k] / a.cap);
      }
      if (a.slopes) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int k = 0; k < 4; ++k) z[r][k] = fmaf(slope[r], float(k0 + kg + 8 * k - pos[r]), z[r][k]);
      }
      if (!full) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const RowSpan rs = row_span(a, w.s, pos[r]);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int j = k0 + kg + 8 * k;
            if (!(j < w.s.kv && (j < w.s.pre || (j >= rs.lo && j <= rs.hi)))) z[r][k] = -INFINITY;
          }
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float mx = -INFINITY;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          z[r][k] *= kLog2e;
          mx = fmaxf(mx, z[r][k]);
        }
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float mn = fmaxf(m[r], mx);
        const float ms = mn == -INFINITY ? 0.f : mn;  // nothing seen so far
        const float corr = exp2_fast(m[r] - ms);
        l[r] *= corr;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          z[r][k] = exp2_fast(z[r][k] - ms);
          l[r] += z[r][k];
        }
        if (mn > m[r]) {  // the same in the lanes of a row
#pragma unroll
          for (int c = 0; c < kCols; ++c)
#pragma unroll
            for (int e = 0; e < 2; ++e) o[r][c][e] = mul2(o[r][c][e], make_float2(corr, corr));
          m[r] = mn;
        }
      }
      __syncwarp();  // the last block's probabilities are read
#pragma unroll
      for (int k = 0; k < 4; ++k)
        *reinterpret_cast<float4*>(P + (kg + 8 * k) * kWarpRows + rg * 4) =
            make_float4(z[0][k], z[1][k], z[2][k], z[3][k]);
      __syncwarp();
#pragma unroll 2
      for (int k = 0; k < kF32Keys; ++k) {
        const float4 p = *reinterpret_cast<const float4*>(P + k * kWarpRows + rg * 4);
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const float4 v = *reinterpret_cast<const float4*>(V + k * D + c * 32 + kg * 4);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float2 pr = r == 0 ? make_float2(p.x, p.x) : r == 1 ? make_float2(p.y, p.y)
                            : r == 2 ? make_float2(p.z, p.z) : make_float2(p.w, p.w);
            o[r][c][0] = fma2(pr, make_float2(v.x, v.y), o[r][c][0]);
            o[r][c][1] = fma2(pr, make_float2(v.z, v.w), o[r][c][1]);
          }
        }
      }
    }
    if (!live) continue;
    // the rows leave through the warp's own queries, which are done with: a rolled
    // loop of whole rows (straight-line code for every row took longer to fetch
    // than to run)
    const bool whole = w.whole();
    __syncwarp();
    float* O = Q + warp * kWarpRows * D;
    float2* ml = reinterpret_cast<float2*>(P);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], off);
#pragma unroll
      for (int c = 0; c < kCols; ++c)
        *reinterpret_cast<float4*>(O + (rg * 4 + r) * D + (c * 8 + (kg ^ rg)) * 4) =
            make_float4(o[r][c][0].x, o[r][c][0].y, o[r][c][1].x, o[r][c][1].y);
      if (kg == 0) ml[rg * 4 + r] = make_float2(m[r], l[r]);
    }
    __syncwarp();
    if (lane < kWarpRows) {
      const int row = warp * kWarpRows + lane;
      const int2 to = place[row];
      const float2 v = ml[lane];
      const bool some = v.y > 0.f || v.y != v.y;
      if (to.y >= 0) {
        if (!whole) a.part_ml[int64_t(w.slot()) * kChunkRows + row] = v;
        else if (a.lse)
          a.lse[int64_t(to.x) * a.Hq + to.y] = some ? (v.x + log2f(v.y)) * 0.6931471805599453f : -INFINITY;
      }
      ml[lane].x = !whole ? 1.f : (some ? 1.f / v.y : 0.f);
    }
    __syncwarp();
    constexpr int kChunks = D / 4;
#pragma unroll 2
    for (int e = lane; e < kWarpRows * kChunks; e += 32) {
      const int r = e / kChunks, c = e % kChunks, row = warp * kWarpRows + r;
      const int2 to = place[row];
      const float f = ml[r].x;
      const float4 x = *reinterpret_cast<const float4*>(O + r * D + (c ^ (r >> 2)) * 4);
      float* dst = whole ? static_cast<float*>(a.out) + int64_t(to.x) * a.o_ts + int64_t(to.y) * a.o_hs
                         : a.part_o + (int64_t(w.slot()) * kChunkRows + row) * D;
      if (to.y >= 0)
        *reinterpret_cast<float4*>(dst + c * 4) = make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
    }
  }
  cp_async_wait<0>();
}

template <int D>
static cudaError_t launch_chunk(PagedArgs a, cudaStream_t s) {
  using C = ChunkCfg<D>;
  a.R = kChunkRows;
  a.tk_shift = 5;
  a.mt = (a.G + kChunkRows - 1) / kChunkRows;
  a.tq = a.mt == 1 ? kChunkRows / a.G : 1;
  // as for single tokens: 26 us from 3 blocks up for 4 short pieces, 49 from 8
  a.min_steps = 3;
  a.extra = 2;
  // Units cut by themselves (own_steps 1 / 2): five pieces with a window 19.3 / 27.9 us
  // (on the line 27.0)
  a.own_steps = 1;
  a.slack = 3;
  size_t smem = sizeof(float) * C::kFloats;
  static_assert(2 * (sizeof(float) * C::kFloats + 1024 + 1024) <= 233472 &&
                    2 * (kPlanScratch + 1024 + 1024) <= 233472,
                "two CTAs per SM");
  if (smem < kPlanScratch) smem = kPlanScratch;
  auto* k = paged_f32_chunk_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  const int grid = paged_grid(2);
  a.own_units = grid / (a.Hkv * a.mt);
  e = launch_kernel(k, dim3(grid), dim3(kF32Threads), smem, s, false, a);
  if (e != cudaSuccess) return e;
  return launch_paged_join(a, D, false, false, grid, s);
}

cudaError_t launch_paged_attend_f32(const PagedArgs& a, int D, cudaStream_t s) {
  return D == 128 ? launch_chunk<128>(a, s) : launch_chunk<64>(a, s);
}

}  // namespace fkv
