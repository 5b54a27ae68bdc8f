// Attention of one new token per sequence over the paged cache in fp32 (the
// library's accuracy mode), on the CUDA cores: fp32 products and sums throughout.
//
// The four warps of a CTA stream 32-key blocks of K and V through a ring filled
// with 16-byte asynchronous copies (rows that no query sees, or of a bad page, are
// filled with zeros, whatever the cache holds there).  Each warp takes 8 keys of
// every block: four lanes share a key and split its dims for the scores of all R
// rows, then lane (key, row) holds one score, so the softmax step is three
// shuffles; for P V a lane owns D / 32 output dims.  Every warp keeps the running
// maximum, sum and output of the R rows for its keys, so the warps meet once per
// block (for the ring) and join at the end of a unit.
// Bound by the instructions beside the loads: R = 1, 4 and 16 for up to as many
// query heads per KV head, since rows that are not there cost as much as others
// (16 sequences, windows of 1024 keys, one head per KV head: 42 us with R = 1, 51
// with R = 4; the bytes take 21).
#include "paged_f32.cuh"

namespace fkv {

template <int D, int R>
struct F32Cfg {
  static constexpr int kK = kF32Keys * D, kV = kF32Keys * D;
  static constexpr int kStages = 2;
  static constexpr int kPerSm = R == 16 ? 2 : (D == 128 ? 3 : 4);  // resident CTAs
  // keys of P V in straight-line code: the first pass through an instruction is
  // slow, and with many rows 4 take as long as 8 once it is there (one block of 131
  // keys, R = 16: 34 us a call with whole loops, 31 with 4; long caches 113 and 110)
  static constexpr int kAhead = R == 1 ? 8 : 4;
  static constexpr int kP = R == 1 ? 4 : R;                // floats per key of P
  static constexpr int kQ = R * D;                         // one slot per stage
  static constexpr int kStage = kK + kV + kQ;              // floats
  static constexpr int kOffP = kStages * kStage;           // [32 keys][kP]
  static constexpr int kOffO = kOffP + kF32Keys * kP;      // [2][R][D]
  static constexpr int kOffMl = kOffO + 2 * R * D;         // [4][R] float2
  static constexpr int kOffRow = kOffMl + 4 * R * 2;       // [R] (factor, head)
  static constexpr int kFloats = kOffRow + 2 * (R == 1 ? 2 : R);
};

// Place of 16-byte chunk c of K row r: odd rows swap the halves of each 128
// bytes, so that the eight lanes of a read (two keys, four chunks) meet no bank twice.
template <int D>
__device__ __forceinline__ int k_at(int r, int c) {
  return r * D + ((c ^ ((r & 1) << 2)) << 2);
}

// Starts the copies of step i of a unit into a stage, and of the unit's queries
// with its first step.
template <int D, int R>
__device__ __forceinline__ void load_step(const PagedArgs& a, const Walk& w, int i, float* stage,
                                          const int (&ids)[Rows<D>::kCount], unsigned want) {
  using C = F32Cfg<D, R>;
  load_keys<D>(a, w, i, ids, want, [&](int r, int c) { return stage + k_at<D>(r, c); },
               [&](int r, int c) { return stage + C::kK + r * D + c * 4; });
  if (i == 0) {
    constexpr int kPass = Rows<D>::kPass;
    const int row0 = int(threadIdx.x) / Rows<D>::kChunks, c = int(threadIdx.x) % Rows<D>::kChunks * 4;
    float* Q = stage + C::kK + C::kV;
#pragma unroll
    for (int p = 0; p < (R + kPass - 1) / kPass; ++p) {
      const int r = row0 + p * kPass;
      if (r < R) {
        int token, head;
        const bool read = row_place(a, w.s, w.qt, w.hm, r, &token, &head);
        const float* src = static_cast<const float*>(a.q);
        if (read) src += int64_t(w.s.q0 + token) * a.q_ts + int64_t(head) * a.q_hs + c;
        cp_async16(Q + r * D + c, src, read);
      }
    }
  }
}

template <int D, int R>
__global__ void __launch_bounds__(kF32Threads, F32Cfg<D, R>::kPerSm) paged_f32_kernel(const PagedArgs a) {
  using C = F32Cfg<D, R>;
  constexpr int kDims = D / 32;  // output dims per lane
  constexpr int kGroups = R == 1 ? 1 : R / 4;
  extern __shared__ __align__(16) float sm[];
  __shared__ PlanRec rec;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  plan_part<kF32Threads>(a, reinterpret_cast<int64_t*>(sm), &rec);
  const float kLog2e = 1.4426950408889634f;
  float* P = sm + C::kOffP;
  float* O = sm + C::kOffO;
  float2* ML = reinterpret_cast<float2*>(sm + C::kOffMl);
  float2* Row = reinterpret_cast<float2*>(sm + C::kOffRow);
  // this lane's key inside a block, and its dims quarter (scores) or row in each
  // group of four (softmax)
  const int key = warp * 8 + (lane >> 2), sub = lane & 3;

  // the loads run kStages - 1 steps ahead, over the ends of units
  Walk lw, w;
  lw.begin(a, rec);
  w.begin(a, rec);
  int li = 0, ln = 0, ids[Rows<D>::kCount];
  unsigned want = 0;
  if (!lw.done()) fetch_pages<D>(a, lw, 0, ids, want);
  auto load_next = [&]() {
    if (!lw.done()) {
      load_step<D, R>(a, lw, li, sm + (ln % C::kStages) * C::kStage, ids, want);
      ++ln;
      if (++li == lw.count) {
        li = 0;
        lw.next(a);
      }
      if (!lw.done()) fetch_pages<D>(a, lw, li, ids, want);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < C::kStages - 1; ++s) load_next();

  int n = 0;
  for (; !w.done(); w.next(a)) {
    const int h = w.hm / a.mt, m0 = (w.hm - h * a.mt) * R;
    const int p0 = w.s.kv - w.s.q_len + w.qt * a.tq;  // position of the first token
    const int all_hi = a.causal ? p0 : w.s.kv - 1;
    const int all_lo = a.window > 0 ? p0 + a.tq - a.window : 0;
    // rows 4 g + sub: position, span and slope
    int pos[kGroups];
    float slope[kGroups];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const int r = R == 1 ? 0 : 4 * g + sub;
      const int i = m0 + r;
      pos[g] = p0;
      slope[g] = a.slopes && i < a.G ? a.slopes[h * a.G + i] : 0.f;
    }
    float m[kGroups], l[kGroups], o[R][kDims];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      m[g] = -INFINITY;
      l[g] = 0.f;
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int d = 0; d < kDims; ++d) o[r][d] = 0.f;
    // the queries stay in the stage of the unit's first step: keep a copy
    float* Qs = O;  // free between joins: [R][D] of its 2 R D floats
    for (int i = 0; i < w.count; ++i, ++n) {
      cp_async_wait<C::kStages - 2>();
      __syncthreads();  // step n is here for all; step n - 1 is done with
      float* stage = sm + (n % C::kStages) * C::kStage;
      load_next();
      const float* Q = i == 0 ? stage + C::kK + C::kV : Qs;
      const int k0 = block_at(w.t, w.first + i) * kF32Keys, j = k0 + key;
      float z[R];
#pragma unroll
      for (int r = 0; r < R; ++r) z[r] = 0.f;
#pragma unroll 4
      for (int c = 0; c < D / 16; ++c) {
        const int d = (4 * c + sub) * 4;
        const float4 k4 = *reinterpret_cast<const float4*>(stage + k_at<D>(key, 4 * c + sub));
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float4 q4 = *reinterpret_cast<const float4*>(Q + r * D + d);
          z[r] = fmaf(q4.x, k4.x, z[r]);
          z[r] = fmaf(q4.y, k4.y, z[r]);
          z[r] = fmaf(q4.z, k4.z, z[r]);
          z[r] = fmaf(q4.w, k4.w, z[r]);
        }
      }
      const bool full = k0 + 31 < w.s.pre || (k0 >= all_lo && k0 + 31 <= all_hi);
      float corr[kGroups];
      bool grew = false;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        float x;
        if constexpr (R == 1) {
          x = z[0] + __shfl_xor_sync(0xffffffffu, z[0], 1);
          x += __shfl_xor_sync(0xffffffffu, x, 2);
        } else {
          // four dot products over four lanes: lane `sub` ends with row 4 g + sub
          float u = sub & 1 ? z[4 * g] : z[4 * g + 1], v = sub & 1 ? z[4 * g + 2] : z[4 * g + 3];
          u = __shfl_xor_sync(0xffffffffu, u, 1);
          v = __shfl_xor_sync(0xffffffffu, v, 1);
          const float s01 = (sub & 1 ? z[4 * g + 1] : z[4 * g]) + u;
          const float s23 = (sub & 1 ? z[4 * g + 3] : z[4 * g + 2]) + v;
          const float t = __shfl_xor_sync(0xffffffffu, sub & 2 ? s01 : s23, 2);
          x = (sub & 2 ? s23 : s01) + t;
        }
        x *= a.scale;
        if (a.cap > 0.f) x = a.cap * tanhf(x / a.cap);
        if (a.slopes) x = fmaf(slope[g], float(j - pos[g]), x);
        x *= kLog2e;
        if (!full) {
          const RowSpan rs = row_span(a, w.s, pos[g]);
          if (!(j < w.s.kv && (j < w.s.pre || (j >= rs.lo && j <= rs.hi)))) x = -INFINITY;
        }
        float mx = x;
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float mn = fmaxf(m[g], mx);
        const float ms = mn == -INFINITY ? 0.f : mn;  // nothing seen so far
        corr[g] = exp2_fast(m[g] - ms);
        grew |= mn > m[g];
        const float p = exp2_fast(x - ms);
        l[g] = l[g] * corr[g] + p;
        m[g] = mn;
        if (R > 1 || sub == 0) P[key * C::kP + (R == 1 ? 0 : 4 * g + sub)] = p;
      }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float f = __shfl_sync(0xffffffffu, corr[r / 4], r & 3);
#pragma unroll
          for (int d = 0; d < kDims; ++d) o[r][d] *= f;
        }
      }
      __syncwarp();
      const float* V = stage + C::kK + lane * kDims;
#pragma unroll(C::kAhead)
      for (int k = 0; k < 8; ++k) {
        float vv[kDims];
#pragma unroll
        for (int d = 0; d < kDims; d += 2)
          *reinterpret_cast<float2*>(&vv[d]) =
              *reinterpret_cast<const float2*>(V + (warp * 8 + k) * D + d);
        if constexpr (R == 1) {
          const float p = P[(warp * 8 + k) * C::kP];
#pragma unroll
          for (int d = 0; d < kDims; ++d) o[0][d] = fmaf(p, vv[d], o[0][d]);
        }
#pragma unroll
        for (int g = 0; g < R / 4; ++g) {
          const float4 p = *reinterpret_cast<const float4*>(P + (warp * 8 + k) * C::kP + 4 * g);
#pragma unroll
          for (int d = 0; d < kDims; ++d) {
            o[4 * g][d] = fmaf(p.x, vv[d], o[4 * g][d]);
            o[4 * g + 1][d] = fmaf(p.y, vv[d], o[4 * g + 1][d]);
            o[4 * g + 2][d] = fmaf(p.z, vv[d], o[4 * g + 2][d]);
            o[4 * g + 3][d] = fmaf(p.w, vv[d], o[4 * g + 3][d]);
          }
        }
      }
      if (i == 0 && w.count > 1) {
        // before the stage is loaded again, which is after the next barrier at
        // the earliest; read after that barrier too
#pragma unroll
        for (int e = threadIdx.x * 4; e < R * D; e += kF32Threads * 4)
          *reinterpret_cast<float4*>(Qs + e) = *reinterpret_cast<const float4*>(Q + e);
      }
      __syncwarp();  // P is read by all lanes before the next block's is written
    }
    // ---- join the warps: each scales its sums to the rows' common maximum, then
    // warps 2, 3 leave theirs in the two slots, warps 0, 1 add their own, and the
    // rows are written by all threads in a rolled loop (straight-line code for every
    // row took longer to fetch than to run)
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) l[g] += __shfl_xor_sync(0xffffffffu, l[g], off);
      if (lane < (R == 1 ? 1 : 4)) ML[warp * R + 4 * g + lane] = make_float2(m[g], l[g]);
    }
    __syncthreads();  // and the queries' copy is read
    float f[kGroups];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const int r = R == 1 ? 0 : 4 * g + sub;
      const float mx = fmaxf(fmaxf(ML[r].x, ML[R + r].x), fmaxf(ML[2 * R + r].x, ML[3 * R + r].x));
      f[g] = exp2_fast(m[g] - (mx == -INFINITY ? 0.f : mx));
    }
    float* mine = O + (warp & 1) * R * D + lane * kDims;
#pragma unroll
    for (int half = 1; half >= 0; --half) {
      if (warp >> 1 == half) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float fr = __shfl_sync(0xffffffffu, f[r / 4], r & 3);
#pragma unroll
          for (int d = 0; d < kDims; d += 2) {
            float2* at = reinterpret_cast<float2*>(mine + r * D + d);
            float2 x = make_float2(o[r][d] * fr, o[r][d + 1] * fr);
            if (half == 0) {
              const float2 y = *at;
              x.x += y.x;
              x.y += y.y;
            }
            *at = x;
          }
        }
      }
      __syncthreads();
    }
    const bool whole = w.whole();
    if (threadIdx.x < R) {
      const int r = threadIdx.x;
      int token, head;
      if (row_place(a, w.s, w.qt, w.hm, r, &token, &head)) {
        const int64_t tok = int64_t(w.s.q0) + token;
        float M = ML[r].x, L = 0.f;
#pragma unroll
        for (int i = 1; i < 4; ++i) M = fmaxf(M, ML[i * R + r].x);
        const float Ms = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int i = 0; i < 4; ++i) L = fmaf(ML[i * R + r].y, exp2_fast(ML[i * R + r].x - Ms), L);
        const bool some = L > 0.f || L != L;
        if (!whole) a.part_ml[int64_t(w.slot()) * R + r] = make_float2(M, L);
        else if (a.lse) a.lse[tok * a.Hq + head] = some ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
        Row[r] = make_float2(!whole ? 1.f : (some ? 1.f / L : 0.f), __int_as_float(head));
      } else {
        Row[r].y = __int_as_float(-1);
      }
    }
    __syncthreads();
#pragma unroll 1
    for (int e = threadIdx.x; e < R * (D / 4); e += kF32Threads) {
      const int r = e / (D / 4), d = e % (D / 4) * 4, head = __float_as_int(Row[r].y);
      const float fr = Row[r].x;
      const float4 x = *reinterpret_cast<const float4*>(O + r * D + d);
      const float4 y = *reinterpret_cast<const float4*>(O + R * D + r * D + d);
      float* dst = whole ? static_cast<float*>(a.out) + int64_t(w.s.q0) * a.o_ts + int64_t(head) * a.o_hs
                         : a.part_o + (int64_t(w.slot()) * R + r) * D;
      if (head >= 0)
        *reinterpret_cast<float4*>(dst + d) =
            make_float4((x.x + y.x) * fr, (x.y + y.y) * fr, (x.z + y.z) * fr, (x.w + y.w) * fr);
    }
    __syncthreads();  // the joined sums are read before the next unit copies its queries there
  }
  cp_async_wait<0>();
}

template <int D, int R>
static cudaError_t launch_f32(PagedArgs a, cudaStream_t s) {
  using C = F32Cfg<D, R>;
  a.R = R;
  a.tk_shift = 5;
  a.mt = (a.G + R - 1) / R;
  a.tq = 1;
  // the whole of a unit of one block: parts from 3, 4, 8 up take 10.6, 14.1 and 17.4
  // us for 6 sequences of 3 keys
  a.min_steps = 3;
  a.extra = 2;
  // Units cut by themselves (own_steps 1 / 2 / 3): a sequence of 131 keys, 2 KV heads
  // for 32: 13.9 / 19.5 / 22.4 us (on the line 20.7); with slack 4 the windows of 16
  // sequences take 47 us instead of 43.
  a.own_steps = 1;
  a.slack = 3;
  size_t smem = sizeof(float) * C::kFloats;
  if (smem < kPlanScratch) smem = kPlanScratch;
  static_assert(C::kPerSm * (sizeof(float) * C::kFloats + 1024 + 64) <= 233472 &&
                    C::kPerSm * (kPlanScratch + 1024 + 64) <= 233472,
                "resident CTAs per SM");
  auto* k = paged_f32_kernel<D, R>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  const int grid = paged_grid(C::kPerSm);
  a.own_units = grid / (a.Hkv * a.mt);
  e = launch_kernel(k, dim3(grid), dim3(kF32Threads), smem, s, false, a);
  if (e != cudaSuccess) return e;
  return launch_paged_join(a, D, false, false, grid, s);
}

cudaError_t launch_paged_decode_f32(const PagedArgs& a, int D, cudaStream_t s) {
  if (a.G == 1) return D == 128 ? launch_f32<128, 1>(a, s) : launch_f32<64, 1>(a, s);
  if (a.G <= 4) return D == 128 ? launch_f32<128, 4>(a, s) : launch_f32<64, 4>(a, s);
  return D == 128 ? launch_f32<128, 16>(a, s) : launch_f32<64, 16>(a, s);
}

}  // namespace fkv
