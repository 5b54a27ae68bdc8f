// Attention of one new token per sequence over the paged cache (bf16).
//
//   out_h = sum_j softmax_j(z_hj) v_j,  z_hj = scale q_h . k_j (capped, biased)
//
// Bound by memory: each visible key and value is read once from HBM for all
// query heads that share it.  A warp-level MMA (m16n8k16) takes up to 16 such
// heads as its rows: with the 128-row tcgen05 tile of the chunk kernel seven
// eighths or more of every softmax would be spent on empty rows, and the tensor
// work here (2 x 16 rows per key) is far below what the warp MMA sustains.
//
// A CTA streams 64-key blocks of K and V through a ring in shared memory, filled
// by one producer warp with TMA boxes of page rows (128-byte swizzle); two CTAs
// per SM keep about 200 KB of loads in flight.  Each of the four consumer warps
// takes 16 keys of every block and keeps its own running maximum, sum and
// 16 x D output in registers, so the warps do not meet inside the loop; they are
// merged through shared memory at the end of a unit, in the ring stage that the
// unit read last.  Probabilities enter P V as two bf16 terms (p and its rounding
// error): the products are then as exact as fp32 weights, and the second MMA is
// hidden behind the loads.
//
// Measured (8 KV heads, 32 query heads; on the GPU, calls back to back in a graph;
// calls from Python in brackets): 64 sequences of 17 .. 8191 keys, 725 MB, 122 us =
// 0.91 of the copy bandwidth (124 to 131); one of 200001 keys, 819 MB, 135 us = 0.93
// with its join (134); one of 131 keys 9.4 us (10.3), of which the division of the
// work takes 1.8, the first blocks 2.2 and the merge and store 1.2.
#include "paged_sm100.cuh"

namespace fkv {
namespace sm100 {

constexpr int kDecThreads = 160;  // four consumer warps, one producer warp
constexpr int kDecKeys = 1 << 6;
constexpr int kDecRows = 16;

template <int D>
struct DecCfg {
  static constexpr int kHalves = D / 64;
  static constexpr uint32_t kOperand = kDecKeys * D * 2;  // bytes of the K (or V) block
  static constexpr uint32_t kStage = 2 * kOperand;
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr uint32_t kQ = kDecRows * D * 2;
  static constexpr uint32_t kOffQ = kStages * kStage;
  static constexpr uint32_t kOffBar = kOffQ + 2 * kQ;
};

struct DecBars {
  uint64_t full[6], empty[6], q_full[2], q_empty[2];
  uint64_t read, wrote;    // merge: every warp has read the last block / written its sums
  // join: every warp has stored its partial / knows who joins / gathered the sums
  uint64_t stored, last, gathered;
  float2 ml[4][kDecRows];  // (max, sum) of each warp
  PlanRec rec;
  int joins;  // this CTA wrote the last partial of the unit
  int abort;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Byte offset of 16-byte chunk `chunk` of row `row` in a [D / 64][rows][64] bf16
// block in the 128-byte swizzle that TMA writes.
template <int kRows>
__device__ __forceinline__ uint32_t sw_off(int row, int chunk) {
  return uint32_t(chunk >> 3) * (kRows * 128) + uint32_t(row) * 128 +
         uint32_t(((chunk & 7) ^ (row & 7)) << 4);
}
// The four consumer warps meet (bounded, unlike a named barrier).
__device__ __forceinline__ bool consumers_meet(uint64_t* bar, uint32_t parity, int lane,
                                               volatile int* abort) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
  return warp_wait(bar, parity, abort);
}

// The last CTA of a unit joins its `parts` (at most kJoinHere) partials, in CTA
// order: the four consumer warps take four columns of a row per thread.  s_ml:
// scratch of parts * 16 float2.
template <int D>
__device__ __forceinline__ bool join_here(const PagedArgs& a, const Walk& w, int cut, int parts,
                                          int head0, int rows, float2* s_ml, uint64_t* gathered,
                                          uint32_t parity, volatile int* abort) {
  const int tid = threadIdx.x;  // 0 .. 127
  auto slot_row = [&](int i) {  // first row of partial i
    return int64_t(i == 0 ? 2 * cut - 1 : 2 * (cut - 1 + i)) * kDecRows;
  };
  for (int k = tid; k < parts * kDecRows; k += 128)
    if ((k & 15) < rows) s_ml[k] = __ldcg(a.part_ml + slot_row(k >> 4) + (k & 15));
  if (!consumers_meet(gathered, parity, tid & 31, abort)) return false;
  for (int e = tid * 4; e < rows * D; e += 512) {
    const int row = e / D, col = e % D;
    float M = -INFINITY, L = 0.f;
    for (int i = 0; i < parts; ++i) M = fmaxf(M, s_ml[i * kDecRows + row].x);
    const float Ms = M == -INFINITY ? 0.f : M;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kJoinHere; ++i) {
      if (i >= parts) break;
      const float4 v = __ldcg(reinterpret_cast<const float4*>(a.part_o + (slot_row(i) + row) * D + col));
      const float2 ml = s_ml[i * kDecRows + row];
      const float f = ex2(ml.x - Ms);
      L = fmaf(ml.y, f, L);
      y.x = fmaf(v.x, f, y.x);
      y.y = fmaf(v.y, f, y.y);
      y.z = fmaf(v.z, f, y.z);
      y.w = fmaf(v.w, f, y.w);
    }
    const bool some = L > 0.f || L != L;
    const float inv = some ? 1.f / L : 0.f;
    const int head = head0 + row;
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + int64_t(w.s.q0) * a.o_ts +
                              int64_t(head) * a.o_hs + col) =
        make_uint2(pack_bf16(y.x * inv, y.y * inv), pack_bf16(y.z * inv, y.w * inv));
    if (a.lse && col == 0)
      a.lse[int64_t(w.s.q0) * a.Hq + head] = some ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
  }
  return true;
}

template <int D>
__global__ void __launch_bounds__(kDecThreads, 2)
paged_decode_kernel(const __grid_constant__ CUtensorMap tm_q,
                    const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const PagedArgs a) {
  using C = DecCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align1024(smem_raw);
  DecBars* bars = reinterpret_cast<DecBars*>(sm + C::kOffBar);
  volatile int* abort = &bars->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 4);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->q_full[s], 1);
      mbar_init(&bars->q_empty[s], 4);
    }
    mbar_init(&bars->read, 4);
    mbar_init(&bars->wrote, 4);
    mbar_init(&bars->stored, 4);
    mbar_init(&bars->last, 4);
    mbar_init(&bars->gathered, 4);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (threadIdx.x == 128) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  // the ring is free scratch until the first load; the fence orders that use
  // before the copies of the async proxy
  plan_part<kDecThreads>(a, reinterpret_cast<int64_t*>(sm), &bars->rec);
  if (a.B > 32) {
    fence_proxy_async_smem();
    __syncthreads();
  }
  Walk w;
  w.begin(a, bars->rec);
  if (warp == 4) {
    // ------------------------------------------------------------ producer
    const int box_rows = a.page_shift < 6 ? 1 << a.page_shift : 64;
    const int per_page = 2 * C::kHalves;
    const int my_page = lane / per_page;                   // page of the block
    const int my_half = lane % C::kHalves;
    const bool my_v = (lane / C::kHalves) & 1;
    const bool boxed = my_page * box_rows < kDecKeys;
    const CUtensorMap* map = my_v ? &tm_v : &tm_k;
    uint32_t n = 0, u = 0;
    bool ok = true;
    for (; ok && !w.done(); w.next(a), ++u) {
      const int h = w.hm / a.mt, m = w.hm - h * a.mt;
      if (!(ok = warp_wait(&bars->q_empty[u & 1], ((u >> 1) & 1) ^ 1, abort))) break;
      if (lane == 0) {
        mbar_expect_tx(&bars->q_full[u & 1], C::kQ);
        for (int half = 0; half < C::kHalves; ++half)
          tma_load_3d(sm + C::kOffQ + (u & 1) * C::kQ + half * (kDecRows * 128), &tm_q,
                      &bars->q_full[u & 1], half * 64, h * a.G + m * kDecRows, w.s.q0);
      }
      const int steps = w.count;
      // this lane's page of step i (a bad id reads as zeros: a page past the end)
      auto page_of = [&](int i) {
        const int key = block_at(w.t, w.first + i) * kDecKeys + my_page * box_rows;
        if (!boxed || !box_seen(w.s, w.t, key, box_rows)) return -1;
        const int id = page_id(a, w.b, key >> a.page_shift);
        return id < 0 ? (a.num_pages > 0 ? a.num_pages : 1) : id;
      };
      int id = page_of(0);
      for (int i = 0; i < steps; ++i, ++n) {
        const int next = i + 1 < steps ? page_of(i + 1) : 0;
        const uint32_t s = n % C::kStages, use = n / C::kStages;
        if (!(ok = warp_wait(&bars->empty[s], (use & 1) ^ 1, abort))) break;
        const unsigned loads = __ballot_sync(0xffffffffu, id >= 0);
        if (lane == 0) {
          if (loads) mbar_expect_tx(&bars->full[s], __popc(loads) * uint32_t(box_rows) * 128);
          else mbar_arrive(&bars->full[s]);
        }
        __syncwarp();
        if (id >= 0) {
          const int key = block_at(w.t, w.first + i) * kDecKeys + my_page * box_rows;
          tma_load_4d(sm + s * C::kStage + (my_v ? C::kOperand : 0) +
                          uint32_t(my_half) * (kDecKeys * 128) + uint32_t(my_page * box_rows) * 128,
                      map, &bars->full[s], my_half * 64, key & ((1 << a.page_shift) - 1), h, id);
        }
        id = next;
      }
    }
    // this CTA's copies complete before its shared memory is given back
    for (uint32_t i = n > C::kStages ? n - C::kStages : 0; i < n; ++i)
      drain_wait(&bars->full[i % C::kStages], (i / C::kStages) & 1);
    for (uint32_t i = u > 2 ? u - 2 : 0; i < u; ++i) drain_wait(&bars->q_full[i & 1], (i >> 1) & 1);
  } else {
    // ------------------------------------------------------------ consumers
    const float kLog2e = 1.4426950408889634f;
    const float sl2 = a.scale * kLog2e;
    const int quad = lane >> 2, col = (lane & 3) * 2;
    uint32_t n = 0, u = 0, joined = 0, gathers = 0;
    bool ok = true;
    for (; ok && !w.done(); w.next(a), ++u) {
      const int h = w.hm / a.mt, m0 = (w.hm - h * a.mt) * kDecRows;
      const int p = w.s.kv - 1;
      if (!(ok = warp_wait(&bars->q_full[u & 1], (u >> 1) & 1, abort))) break;
      uint32_t qf[D / 16][4];
      const uint32_t q_addr = smem_u32(sm + C::kOffQ + (u & 1) * C::kQ);
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        ldsm4(qf[k], q_addr + sw_off<kDecRows>(lane & 15, 2 * k + (lane >> 4)));
      float slope[2] = {0.f, 0.f};
      if (a.slopes) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int g = m0 + quad + 8 * r;
          slope[r] = g < a.G ? a.slopes[h * a.G + g] * kLog2e : 0.f;
        }
      }
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
      float o[D / 8][4];
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
      const int steps = w.count;
      uint32_t s = 0;
      for (int i = 0; i < steps; ++i, ++n) {
        s = n % C::kStages;
        if (!(ok = warp_wait(&bars->full[s], (n / C::kStages) & 1, abort))) break;
        const uint32_t k_addr = smem_u32(sm + s * C::kStage), v_addr = k_addr + C::kOperand;
        const int k0 = block_at(w.t, w.first + i) * kDecKeys + warp * 16;  // this warp's keys
        float x[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[t][e] = 0.f;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t kf[4];
          ldsm4(kf, k_addr + sw_off<kDecKeys>(warp * 16 + (lane >> 4) * 8 + (lane & 7),
                                              2 * k + ((lane >> 3) & 1)));
          mma16816(x[0], qf[k], kf[0], kf[1]);
          mma16816(x[1], qf[k], kf[2], kf[3]);
        }
        // x[t][e]: key k0 + 8 t + col + (e & 1), head row quad + 8 (e >> 1)
        const bool all = (k0 >= w.t.lo && k0 + 15 <= w.t.hi) || k0 + 15 < w.s.pre;
        uint32_t vmask[2] = {0xffffffffu, 0xffffffffu};  // keys that are seen, 16 bits each
        if (!all) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            vmask[t] = 0;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int j = k0 + 8 * t + col + e;
              if (j < w.s.pre || (j >= w.t.lo && j <= w.t.hi)) vmask[t] |= 0xffffu << (16 * e);
            }
          }
        }
        auto seen = [&](int t, int e) { return (vmask[t] >> (16 * (e & 1)) & 1u) != 0; };
        if (a.cap > 0.f) {
          const float inner = a.scale / a.cap, outer = a.cap * kLog2e;
          float most = 0.f;  // without the NaN, which come out of both forms as such
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              // (what is not seen may be anything and must not decide the form)
              x[t][e] = all || seen(t, e) ? x[t][e] * inner : 0.f;
              most = fmaxf(most, fabsf(x[t][e]));
            }
          const bool small = !__any_sync(0xffffffffu, most >= kTanhSmall);
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              const float2 y = make_float2(x[t][e], x[t][e + 1]);
              float2 v;
              if (small) {
                v = mul2(tanh_small(y), make_float2(outer, outer));
              } else {
                float2 num, den;
                float r;
                tanh_parts(y, num, den);
                asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(den.x * den.y));
                r *= outer;
                v = make_float2(num.x * (r * den.y), num.y * (r * den.x));
              }
              x[t][e] = v.x;
              x[t][e + 1] = v.y;
            }
        } else {
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[t][e] *= sl2;
        }
        if (a.slopes) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[t][e] = fmaf(slope[e >> 1], float(k0 + 8 * t + col + (e & 1) - p), x[t][e]);
        }
        if (!all) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!seen(t, e)) x[t][e] = -INFINITY;
        }
        float mn[2], ms[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float v = fmaxf(fmaxf(x[0][2 * r], x[0][2 * r + 1]), fmaxf(x[1][2 * r], x[1][2 * r + 1]));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
          mn[r] = fmaxf(m[r], v);
          ms[r] = mn[r] == -INFINITY ? 0.f : mn[r];  // nothing seen so far
        }
        if (__any_sync(0xffffffffu, mn[0] > m[0] || mn[1] > m[1])) {
          const float c0 = ex2(m[0] - ms[0]), c1 = ex2(m[1] - ms[1]);
          l[0] *= c0;
          l[1] *= c1;
#pragma unroll
          for (int d = 0; d < D / 8; ++d) {
            o[d][0] *= c0;
            o[d][1] *= c0;
            o[d][2] *= c1;
            o[d][3] *= c1;
          }
          m[0] = mn[0];
          m[1] = mn[1];
        }
        uint32_t hi[4], lo[4];  // P as two bf16 terms, in the A layout
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float p0 = ex2(x[t][2 * r] - ms[r]), p1 = ex2(x[t][2 * r + 1] - ms[r]);
            l[r] += p0 + p1;
            const uint32_t b = pack_bf16(p0, p1);
            hi[2 * t + r] = b;
            lo[2 * t + r] = pack_bf16(p0 - __uint_as_float(b << 16),
                                      p1 - __uint_as_float(b & 0xffff0000u));
          }
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
          uint32_t vf[4];
          ldsm4_t(vf, v_addr + sw_off<kDecKeys>(warp * 16 + ((lane >> 3) & 1) * 8 + (lane & 7),
                                                2 * d + (lane >> 4)));
          if (!all) {  // masked rows may hold anything: 0 * NaN is not 0
            vf[0] &= vmask[0];
            vf[1] &= vmask[1];
            vf[2] &= vmask[0];
            vf[3] &= vmask[1];
          }
          mma16816(o[2 * d], hi, vf[0], vf[1]);
          mma16816(o[2 * d], lo, vf[0], vf[1]);
          mma16816(o[2 * d + 1], hi, vf[2], vf[3]);
          mma16816(o[2 * d + 1], lo, vf[2], vf[3]);
        }
        if (i + 1 < steps) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->empty[s]);
        }
      }
      if (!ok) break;
      // The queries are given back here and not behind their loads above: an arrive
      // does not wait for fragments that are still on their way to registers, and the
      // copy of the next unit but one, issued at once, then overtook them (runs of
      // one-block units came out wrong now and then).  Behind the blocks all of them
      // have been used; the next unit's queries lie in the other slot meanwhile.
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->q_empty[u & 1]);
      // ---- merge the warps in the stage read last (still held)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      }
      if (!(ok = consumers_meet(&bars->read, u & 1, lane, abort))) break;
      float* xo = reinterpret_cast<float*>(sm + s * C::kStage);  // [warp][row][D], pairs swizzled
#pragma unroll
      for (int d = 0; d < D / 8; ++d)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = quad + 8 * r;
          const int c2 = (d * 4 + (lane & 3)) ^ ((row & 7) * 4);
          *reinterpret_cast<float2*>(xo + (warp * kDecRows + row) * D + 2 * c2) =
              make_float2(o[d][2 * r], o[d][2 * r + 1]);
        }
      if ((lane & 3) == 0) {
        bars->ml[warp][quad] = make_float2(m[0], l[0]);
        bars->ml[warp][quad + 8] = make_float2(m[1], l[1]);
      }
      if (!(ok = consumers_meet(&bars->wrote, u & 1, lane, abort))) break;
      const int row = threadIdx.x >> 3, part = threadIdx.x & 7;  // D / 8 columns each
      float M = -INFINITY;
#pragma unroll
      for (int i = 0; i < 4; ++i) M = fmaxf(M, bars->ml[i][row].x);
      const float Ms = M == -INFINITY ? 0.f : M;
      float L = 0.f, y[D / 8];
#pragma unroll
      for (int c = 0; c < D / 8; ++c) y[c] = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 ml = bars->ml[i][row];
        const float f = ex2(ml.x - Ms);
        L += ml.y * f;
#pragma unroll
        for (int c = 0; c < D / 8; c += 8) {
          const int c2 = ((part * (D / 8) + c) / 2) ^ ((row & 7) * 4);
          const float4* src = reinterpret_cast<const float4*>(xo + (i * kDecRows + row) * D + 2 * c2);
          const float4 v0 = src[0], v1 = src[1];
          y[c] = fmaf(v0.x, f, y[c]);
          y[c + 1] = fmaf(v0.y, f, y[c + 1]);
          y[c + 2] = fmaf(v0.z, f, y[c + 2]);
          y[c + 3] = fmaf(v0.w, f, y[c + 3]);
          y[c + 4] = fmaf(v1.x, f, y[c + 4]);
          y[c + 5] = fmaf(v1.y, f, y[c + 5]);
          y[c + 6] = fmaf(v1.z, f, y[c + 6]);
          y[c + 7] = fmaf(v1.w, f, y[c + 7]);
        }
      }
      const int g = m0 + row, head = h * a.G + g;
      if (!w.whole()) {
        if (g < a.G) {
          const int64_t at = int64_t(w.slot()) * kDecRows + row;
          float* dst = a.part_o + at * D + part * (D / 8);
#pragma unroll
          for (int c = 0; c < D / 8; c += 4)
            *reinterpret_cast<float4*>(dst + c) = make_float4(y[c], y[c + 1], y[c + 2], y[c + 3]);
          if (part == 0) a.part_ml[at] = make_float2(M, L);
        }
        if (a.join_here) {
          // the CTA that arrives last joins the partials, in CTA order
          int parts;
          const int cut = w.cut_at(bars->rec.per, bars->rec.extra, &parts);
          __threadfence();
          if (!(ok = consumers_meet(&bars->stored, joined & 1, lane, abort))) break;
          if (threadIdx.x == 0) {
            const int before = atomicAdd(&a.arrived[cut], 1);
            __threadfence();
            bars->joins = before == parts - 1;
            if (bars->joins) a.arrived[cut] = 0;  // as the next call finds it
          }
          if (!(ok = consumers_meet(&bars->last, joined & 1, lane, abort))) break;
          ++joined;
          if (bars->joins) {
            if (!(ok = join_here<D>(a, w, cut, parts, h * a.G + m0, min(a.G - m0, kDecRows),
                                    reinterpret_cast<float2*>(xo), &bars->gathered, gathers++ & 1,
                                    abort)))
              break;
          }
        }
      }
      if (w.whole() && g < a.G) {
        const bool some = L > 0.f || L != L;
        const float inv = some ? 1.f / L : 0.f;
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + int64_t(w.s.q0) * a.o_ts +
                             int64_t(head) * a.o_hs + part * (D / 8);
#pragma unroll
        for (int c = 0; c < D / 8; c += 8)
          *reinterpret_cast<uint4*>(dst + c) =
              make_uint4(pack_bf16(y[c] * inv, y[c + 1] * inv), pack_bf16(y[c + 2] * inv, y[c + 3] * inv),
                         pack_bf16(y[c + 4] * inv, y[c + 5] * inv), pack_bf16(y[c + 6] * inv, y[c + 7] * inv));
        if (a.lse && part == 0)
          a.lse[int64_t(w.s.q0) * a.Hq + head] = some ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
      }
      fence_proxy_async_smem();  // the stage was used as scratch: before its next copy
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->empty[s]);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && bars->abort) report(a.status, FKV_ERR_TIMEOUT, blockIdx.x);
}

}  // namespace sm100

template <int D>
static cudaError_t launch_decode(PagedArgs a, cudaStream_t s) {
  using namespace sm100;
  using C = DecCfg<D>;
  a.R = kDecRows;
  a.tk_shift = 6;
  a.mt = (a.G + kDecRows - 1) / kDecRows;
  a.tq = 1;
  a.min_steps = 4;
  a.extra = 1;
  // Units cut by themselves (own_steps 1 / 2 / 3): one sequence of 131 keys, 8 heads
  // 10.3 / 10.7 / 9.3 us on the GPU (on the line 9.2), of 1000 keys 14.3 / 12.0 / 13.0
  // (14.0), 16 sequences of 100 to 1000 keys 17.0 / 16.9 / 16.9 (16.7); with slack 6
  // the last take a sixth longer.
  a.own_steps = 3;
  a.slack = 3;
  CUtensorMap tq, tk, tv;
  if (!paged_tmaps(a, D, kDecKeys, kDecRows, 1, &tq, &tk, &tv)) return cudaErrorNotSupported;
  const size_t smem = 1024 + C::kOffBar + sizeof(DecBars);
  static_assert(C::kStages * C::kStage >= kPlanScratch, "the division's prefix sums fit in the ring");
  static_assert(2 * (1024 + C::kOffBar + sizeof(DecBars) + 1024 + 256) <= 233472,
                "two CTAs per SM");
  auto* k = paged_decode_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  const int grid = paged_grid(2);
  a.own_units = grid / (a.Hkv * a.mt);
  a.join_here = few_parts(a, grid);
  e = launch_kernel(k, dim3(grid), dim3(kDecThreads), smem, s, false, tq, tk, tv, a);
  if (e != cudaSuccess) return e;
  return a.join_here ? cudaSuccess : launch_paged_join(a, D, true, false, grid, s);
}

cudaError_t launch_paged_decode(const PagedArgs& a, int D, cudaStream_t s) {
  return D == 128 ? launch_decode<128>(a, s) : launch_decode<64>(a, s);
}

}  // namespace fkv
