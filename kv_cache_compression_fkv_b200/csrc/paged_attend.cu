// Attention of a ragged batch of query tokens over the paged cache (bf16), on
// the tensor cores.
//
//   out_i = sum_j softmax_j(z_ij) v_j over the keys that query i sees,
//   z_ij = scale q_i . k_j, capped by a tanh and biased by distance on request
//
// Bound by the tensor pipe and the exponentials beside it, as the chunk step's
// attention (attend_sm100.cu), whose pipeline it shares: a 128-row query tile,
// 128-key blocks split between two streams that interleave on the tensor core,
// each with its own softmax warpgroup, logits S_h (overwritten by P_h) and fp32
// output O_h in tensor memory, lazy rescaling, and a merge at the end of a unit.
// What differs:
//   - the 128 rows are (token, head) pairs: the query heads of one KV head share
//     its key blocks, one TMA box [tokens][heads][64 dims] brings them;
//   - key blocks are gathered page by page, one TMA box per page and 64 dims,
//     issued by the lanes of a producer warp at once (one warp for K, one for V);
//   - a CTA's work is an equal part of the batch's key blocks (paged_common.cuh),
//     so causal tiles of different cost, few long or many short sequences all
//     fill the GPU, and a unit that is cut leaves its partial softmax;
//   - blocks that every row sees in full take the unmasked path; in the others
//     each row masks its own columns, and value rows that no row of the tile sees
//     are zeroed in shared memory (P is 0 there, but 0 * NaN is not 0);
//   - a softmax warp whose rows are all empty (few query tokens) skips its work.
// P is rounded to bf16 once, and one pair of exponentials in eight is a polynomial
// good to 9e-5, as in the chunk step's attention: both are the price of the rate.
// Over the whole chunk below the result is off by 0.0023 at most, of which the output's
// own rounding is 0.0017; a second bf16 term of P, as single tokens have it, would
// double the P V products.  The sum of a row takes P before its rounding; sums and
// outputs are fp32.
// The logit's scale and maximum are one FMA, so the largest exponent of a row is the
// rounding of its maximum: normalised away for scores up to 2^30, an overflow from
// 2^31 on (the bound is the entry point's).
//
// Measured (on the GPU, under the power cap; calls from Python in brackets): the 480P
// chunk over 32760 keys, 942 GFLOP, 0.85 to 0.89 ms = 1060 to 1115 TFLOP/s (0.98 ms,
// 962: 0.58 of the burst GEMM, 0.69 of the sustained one); two causal prompts, 637
// GFLOP, 0.70 to 0.80 ms (0.78); 12 short pieces of capped and biased scores 28 us
// (29), most of it one or two blocks' latency per CTA.  Per block and stream the
// softmax takes 2.1k cycles and waits 2k for its next logits.
#include "paged_sm100.cuh"

namespace fkv {
namespace sm100 {

constexpr int kPaThreads = 384;
// Register split as in attend_sm100.cu: 384 * 168 >= 256 * 224 + 128 * 56.
constexpr int kPaSoftmaxRegs = 224;
constexpr int kPaControlRegs = 56;
static_assert(384 * 168 >= 256 * kPaSoftmaxRegs + 128 * kPaControlRegs,
              "register split exceeds the launch allocation");
constexpr int kPaK = 8, kPaV = 10, kPaMma = 9;  // warps: K and Q, V, MMA issuer
constexpr float kPaRescale = 8.0f;              // P stays <= 2^8 between rescales
constexpr int kPaPolyEvery = 8;                 // one exponential pair in 8 on the FMA pipe

template <int D>
struct PaCfg {
  static constexpr int kHalves = D / 64;
  static constexpr uint32_t kTile = 128 * D * 2;
  static constexpr int kKStages = D == 128 ? 3 : 6;
  static constexpr int kVStages = D == 128 ? 3 : 6;
  static constexpr uint32_t kOffK = kTile;
  static constexpr uint32_t kOffV = kOffK + kKStages * kTile;
  static constexpr uint32_t kOffBar = kOffV + kVStages * kTile;
};

struct PaBars {
  uint64_t q_full, q_empty;
  uint64_t k_full[6], k_empty[6], v_full[6], v_empty[6];
  uint64_t s_full[2], p_full[2];
  uint64_t o_ready, o_free, mma_done, x_full, x_read;
  uint32_t tmem_base;
  int abort;
  PlanRec rec;
  float2 xml[2][128];
};

// The blocks of a part of a unit: stream 0 takes the first nb0, stream 1 the rest.
struct Streams {
  int nb0, nb1;
  __device__ __forceinline__ explicit Streams(int n) : nb0((n + 1) / 2), nb1(n / 2) {}
  __device__ __forceinline__ int count(int h) const { return h ? nb1 : nb0; }
  __device__ __forceinline__ int step(int h, int j) const { return h ? nb0 + j : j; }
  // position in the load and MMA order: s0 b0, s1 b0, s0 b1, s1 b1, ...
  __device__ __forceinline__ int pos(int h, int j) const { return j < nb1 ? 2 * j + h : nb1 + j; }
};

// The lowest n bits (none below 0, all from 32 on).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u);
}

// x <- outer tanh(inner x) of 32 logits.  Four quotients share one reciprocal (the
// denominators are at most 176 each).  2000 causal queries over 8000 keys, 16 heads:
// 143 us without a cap, 242 with one of 50, where nearly all warps take the short
// form, 297 with one of 5, where most take the quotient.
// `there`: the columns that the lane's row sees, one bit each (none, if the row is not
// there); the others hold anything and must not decide which form the warp takes.
__device__ __forceinline__ void cap_logits(uint32_t (&x)[32], float inner, float outer, uint32_t there) {
  float most = 0.f;  // a NaN is left out of it, and comes out of both forms as one
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    const float2 y = mul2(make_float2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])),
                          make_float2(inner, inner));
    most = fmax3(most, there >> i & 1u ? fabsf(y.x) : 0.f, there >> i & 2u ? fabsf(y.y) : 0.f);
    x[i] = __float_as_uint(y.x);
    x[i + 1] = __float_as_uint(y.y);
  }
  auto pair = [&](int i) { return make_float2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])); };
  auto put = [&](int i, float2 v) {
    x[i] = __float_as_uint(v.x);
    x[i + 1] = __float_as_uint(v.y);
  };
  if (!__any_sync(0xffffffffu, most >= kTanhSmall)) {
#pragma unroll
    for (int i = 0; i < 32; i += 2) put(i, mul2(tanh_small(pair(i)), make_float2(outer, outer)));
    return;
  }
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    float2 n[2], d[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) tanh_parts(pair(i + 2 * e), n[e], d[e]);
    const float p0 = d[0].x * d[0].y, p1 = d[1].x * d[1].y;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(p0 * p1));
    r *= outer;
    const float r0 = r * p1, r1 = r * p0;
    put(i, mul2(n[0], mul2(make_float2(r0, r0), make_float2(d[0].y, d[0].x))));
    put(i + 2, mul2(n[1], mul2(make_float2(r1, r1), make_float2(d[1].y, d[1].x))));
  }
}

// One operand of the key blocks, loaded by a whole warp.
template <int D, int kStages>
__device__ __forceinline__ bool load_blocks(const PagedArgs& a, const Walk& w, const CUtensorMap* map,
                                            uint8_t* ring, uint64_t* full, uint64_t* empty,
                                            uint32_t& n, volatile int* abort) {
  using C = PaCfg<D>;
  const int lane = threadIdx.x & 31;
  const int box_rows = a.page_shift < 7 ? 1 << a.page_shift : 128;
  const int my_page = lane / C::kHalves, my_half = lane % C::kHalves;
  const bool boxed = my_page * box_rows < 128;
  const int h = w.hm / a.mt;
  const Streams st(w.count);
  auto key_of = [&](int i) {  // i: load order
    const int hh = i < 2 * st.nb1 ? i & 1 : 0, j = i < 2 * st.nb1 ? i >> 1 : i - st.nb1;
    return block_at(w.t, w.first + st.step(hh, j)) * 128 + my_page * box_rows;
  };
  auto page_of = [&](int key) {
    if (!boxed || !box_seen(w.s, w.t, key, box_rows)) return -1;
    const int id = page_id(a, w.b, key >> a.page_shift);
    return id < 0 ? (a.num_pages > 0 ? a.num_pages : 1) : id;  // bad: a page of zeros
  };
  const int steps = st.nb0 + st.nb1;
  int key = key_of(0), id = page_of(key);
  for (int i = 0; i < steps; ++i, ++n) {
    const int next_key = i + 1 < steps ? key_of(i + 1) : 0;
    const int next = i + 1 < steps ? page_of(next_key) : -1;
    const uint32_t s = n % kStages, use = n / kStages;
    if (!warp_wait(&empty[s], (use & 1) ^ 1, abort)) return false;
    const unsigned loads = __ballot_sync(0xffffffffu, id >= 0);
    if (lane == 0) {
      if (loads) mbar_expect_tx(&full[s], __popc(loads) * uint32_t(box_rows) * 128);
      else mbar_arrive(&full[s]);
    }
    __syncwarp();
    if (id >= 0)
      tma_load_4d(ring + s * C::kTile + uint32_t(my_half) * kRegionBytes +
                      uint32_t(my_page * box_rows) * 128,
                  map, &full[s], my_half * 64, key & ((1 << a.page_shift) - 1), h, id);
    key = next_key;
    id = next;
  }
  return true;
}

template <int D>
__global__ void __launch_bounds__(kPaThreads, 1)
paged_attend_kernel(const __grid_constant__ CUtensorMap tm_q,
                    const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const PagedArgs a) {
  using C = PaCfg<D>;
  constexpr int kKS = C::kKStages, kVS = C::kVStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (smem_u32(smem_raw) & 1023u) {  // uniform: every thread sees the same base
    if (threadIdx.x == 0) {
      report(a.status, FKV_ERR_UNSUPPORTED, blockIdx.x);
      a.rec[blockIdx.x] = PlanRec{};  // nothing to join
    }
    return;
  }
  uint8_t* sm = smem_raw;
  PaBars* bars = reinterpret_cast<PaBars*>(sm + C::kOffBar);
  volatile int* abort = &bars->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, 1);
    for (int s = 0; s < kKS; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->k_empty[s], 1);
    }
    for (int s = 0; s < kVS; ++s) {
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->v_empty[s], 1);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(&bars->s_full[h], 1);
      mbar_init(&bars->p_full[h], 128);
    }
    mbar_init(&bars->o_ready, 1);
    mbar_init(&bars->o_free, 256);
    mbar_init(&bars->mma_done, 1);
    mbar_init(&bars->x_full, 256);
    mbar_init(&bars->x_read, 256);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == kPaMma) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  // the tiles are free scratch until the first load
  plan_part<kPaThreads>(a, reinterpret_cast<int64_t*>(sm), &bars->rec);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  Walk w;
  if (warp >= 8) {
    regs_decrease<kPaControlRegs>();
    w.begin(a, bars->rec);
    if (warp == kPaK) {
      // ---------------------------------------------------------- Q and K
      const uint32_t q_bytes = uint32_t(a.mt == 1 ? a.tq * a.G : 128) * 128 * C::kHalves;
      uint32_t n = 0, u = 0;
      for (; !w.done(); w.next(a)) {
        if (!warp_wait(&bars->q_empty, (u & 1) ^ 1, abort)) break;
        if (lane == 0) {
          const int h = w.hm / a.mt, m = w.hm - h * a.mt;
          mbar_expect_tx(&bars->q_full, q_bytes);
          for (int half = 0; half < C::kHalves; ++half)
            tma_load_3d(sm + half * kRegionBytes, &tm_q, &bars->q_full, half * 64,
                        h * a.G + m * 128, w.s.q0 + w.qt * a.tq);
        }
        ++u;
        if (!load_blocks<D, kKS>(a, w, &tm_k, sm + C::kOffK, bars->k_full, bars->k_empty, n, abort)) break;
      }
      for (uint32_t i = n > kKS ? n - kKS : 0; i < n; ++i)
        drain_wait(&bars->k_full[i % kKS], (i / kKS) & 1);
      if (u > 0) drain_wait(&bars->q_full, (u - 1) & 1);
    } else if (warp == kPaV) {
      // ---------------------------------------------------------- V
      uint32_t n = 0;
      for (; !w.done(); w.next(a))
        if (!load_blocks<D, kVS>(a, w, &tm_v, sm + C::kOffV, bars->v_full, bars->v_empty, n, abort)) break;
      for (uint32_t i = n > kVS ? n - kVS : 0; i < n; ++i)
        drain_wait(&bars->v_full[i % kVS], (i / kVS) & 1);
    } else if (warp == kPaMma && lane == 0) {
      // ---------------------------------------------------------- MMA issuer
      constexpr uint32_t kIdQK = idesc_bf16(128, 128, false);
      constexpr uint32_t kIdPV = idesc_bf16(128, D, true);
      constexpr uint32_t kStageDesc = C::kTile >> 4;
      uint32_t uc = 0, ks = 0, kph = 0, vs = 0, vph = 0;
      uint32_t p_use[2] = {0, 0};
      bool ok = true, kf_ok = false, vf_ok = false;
      const uint64_t dq = kmajor_desc(smem_u32(sm), 0);
      const uint64_t dk0 = kmajor_desc(smem_u32(sm + C::kOffK), 0);
      const uint64_t dv0 = mnmajor_desc(smem_u32(sm + C::kOffV), 0);
      for (; ok && !w.done(); w.next(a), ++uc) {
        const Streams st(w.count);
        bool o_free_seen = false;
        // O_h += P_h V for the stream's next block.  K and V stages are used in load
        // order, so the stage of the group that follows is known: its barrier is
        // tested inside this group's MMAs (kf_ok / vf_ok, as in attend_sm100.cu) and
        // waited on only when the test saw it pending.
        auto issue_pv = [&](int h, bool first) -> bool {
          if (!o_free_seen) {
            if (!mbar_wait(&bars->o_free, (uc & 1) ^ 1, abort)) return false;
            o_free_seen = true;
          }
          if (!vf_ok && !mbar_wait(&bars->v_full[vs], vph, abort)) return false;
          vf_ok = false;
          if (!mbar_wait(&bars->p_full[h], p_use[h] & 1, abort)) return false;
          ++p_use[h];
          tc_fence_after();
          kf_ok = mma8_ts_probe(tmem + 256u + 128u * h, tmem + 128u * h, dv0 + uint64_t(vs * kStageDesc),
                                kIdPV, first ? 0u : 1u, &bars->k_full[ks], kph) != 0;
          if (++vs == kVS) { vs = 0; vph ^= 1; }
          return true;
        };
        // S_h = Q K^T for the stream's next block.
        auto issue_s = [&](int h) -> bool {
          if (!kf_ok && !mbar_wait(&bars->k_full[ks], kph, abort)) return false;
          kf_ok = false;
          const uint64_t dk = dk0 + uint64_t(ks * kStageDesc);
          if constexpr (D == 128) {
            vf_ok = mma8_ss_probe(tmem + 128u * h, dq, dk, kIdQK, 0u, &bars->v_full[vs], vph) != 0;
          } else {
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              mma_ss(tmem + 128u * h, dq + uint64_t(k * 2), dk + uint64_t(k * 2), kIdQK, k > 0 ? 1u : 0u);
          }
          mma_commit(&bars->s_full[h]);
          if (++ks == kKS) { ks = 0; kph ^= 1; }
          return true;
        };
        if (!(ok = mbar_wait(&bars->q_full, uc & 1, abort))) break;
        for (int j = 0; ok && j < st.nb0; ++j) {
          if (j > 0 && !(ok = issue_pv(0, j == 1))) break;
          if (!(ok = issue_s(0))) break;
          if (j < st.nb1) {
            if (j > 0 && !(ok = issue_pv(1, j == 1))) break;
            if (!(ok = issue_s(1))) break;
          } else if (j == st.nb1 && j > 0) {
            if (!(ok = issue_pv(1, j == 1))) break;
          }
        }
        if (!ok) break;
        mma_commit(&bars->q_empty);
        if (!(ok = issue_pv(0, st.nb0 == 1))) break;
        if (st.nb1 == st.nb0 && st.nb1 > 0 && !(ok = issue_pv(1, st.nb1 == 1))) break;
        mma_commit(&bars->o_ready);
      }
      mma_commit(&bars->mma_done);  // every MMA completes before TMEM is released
      drain_wait(&bars->mma_done, 0);
    }
  } else {
    regs_increase<kPaSoftmaxRegs>();
    w.begin(a, bars->rec);
    // ------------------------------------------------------------ softmax
    const int h = warp >> 2;                 // stream
    const int row = threadIdx.x & 127;       // query row = TMEM lane
    const uint32_t lane_addr = uint32_t((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_addr + 128u * h, tO = tmem + lane_addr + 256u;
    const float sl2 = a.scale * 1.4426950408889634f;
    const bool plain = a.cap == 0.f && !a.slopes;
    uint32_t use = 0, base = 0, uc = 0;
    bool ok = true;
    for (; ok && !w.done(); w.next(a), ++uc) {
      const Streams st(w.count);
      const int mine = st.count(h);
      int token, head;
      const bool valid = row_place(a, w.s, w.qt, w.hm, row, &token, &head);
      const bool live = __any_sync(0xffffffffu, valid);
      const int pos = w.s.kv - w.s.q_len + token;
      const RowSpan rs = row_span(a, w.s, pos);
      // positions of the tile's first and last token: what every row sees
      const int p_first = w.s.kv - w.s.q_len + w.qt * a.tq;
      const int all_hi = a.causal ? p_first : w.s.kv - 1;
      const int all_lo = a.window > 0 ? p_first + a.tq - a.window : 0;
      const float slope = a.slopes && valid ? a.slopes[head] / a.scale : 0.f;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < mine; ++j, ++use) {
        const int k0 = block_at(w.t, w.first + st.step(h, j)) * 128;
        if (!(ok = warp_wait(&bars->s_full[h], use & 1, abort))) break;
        tc_fence_after();
        if (row == 0) {
          // S_h(j) is complete, and every MMA issued before it: the K stage it
          // read and the V stage of this stream's previous PV are free
          mbar_arrive(&bars->k_empty[(base + uint32_t(st.pos(h, j))) % kKS]);
          if (j > 0) mbar_arrive(&bars->v_empty[(base + uint32_t(st.pos(h, j - 1))) % kVS]);
        }
        const bool full = k0 + 127 < w.s.pre || (k0 >= all_lo && k0 + 127 <= all_hi);
        if (live) {
          if (!plain || !full) {
            // Cap, distance and mask, 32 columns at a time in a loop and back to
            // tensor memory: unrolled over all 128 in registers, the first pass
            // through that code waited 5k to 12k cycles for its instructions.
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t x[32];
              tmem_ld32(tS + c * 32, x);
              tmem_ld_wait();
              const int k = k0 + 32 * c;
              // columns that this row sees, one bit each
              const uint32_t seen =
                  full ? 0xffffffffu
                       : low_bits(w.s.pre - k) | (low_bits(rs.hi + 1 - k) & ~low_bits(rs.lo - k));
              if (a.cap > 0.f) cap_logits(x, a.scale / a.cap, a.cap / a.scale, valid ? seen : 0u);
              if (a.slopes) {
                const float off = slope * float(k - pos);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  x[i] = __float_as_uint(__uint_as_float(x[i]) + fmaf(slope, float(i), off));
              }
              if (!full) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (!(seen >> i & 1u)) x[i] = 0xff800000u;  // -inf
              }
              tmem_st32(tS + c * 32, x);
            }
            tmem_st_wait();
          }
          uint32_t sr[128];
#define SV(i) __uint_as_float(sr[i])
#pragma unroll
          for (int c = 0; c < 4; ++c)
            tmem_ld32(tS + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[c * 32]));
          tmem_ld_wait();
          float mx[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) mx[k] = fmaxf(SV(k), SV(k + 8));
#pragma unroll
          for (int i = 16; i < 128; i += 16)
#pragma unroll
            for (int k = 0; k < 8; ++k) mx[k] = fmax3(mx[k], SV(i + k), SV(i + k + 8));
          const float bmax = fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]),
                                   fmaxf(mx[6], mx[7]));
          const float m_new = fmaxf(m, bmax * sl2);
          if (j == 0) {
            m = m_new;
          } else if (__any_sync(0xffffffffu, valid && m_new > m + kPaRescale)) {
            // (rows that are not there hold anything and must not decide)
            // the PV before S_h(j) is complete, so O_h may be rescaled
            const float alpha = m_new == -INFINITY ? 1.f : ex2(m - m_new);
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              tmem_ld16(tO + 128u * h + c * 16, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st16(tO + 128u * h + c * 16, o);
            }
            tmem_st_wait();
            l *= alpha;
            m = m_new;
          }
          float2 acc[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[k] = make_float2(0.f, 0.f);
          const float ms = m == -INFINITY ? 0.f : m;  // a row that has seen nothing yet
          const float2 sl2x2 = make_float2(sl2, sl2), negm2 = make_float2(-ms, -ms);
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            uint32_t pk[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int c = 64 * hh + 2 * i;
              const float2 e = ffma2(make_float2(SV(c), SV(c + 1)), sl2x2, negm2);
              const float2 p = i % kPaPolyEvery == kPaPolyEvery - 1 ? exp2_poly2(e)
                                                                    : make_float2(ex2(e.x), ex2(e.y));
              acc[i & 3] = fadd2(acc[i & 3], p);
              pk[i] = pack_bf16(p.x, p.y);
            }
            tmem_st32(tS + 32 * hh, pk);
          }
#undef SV
          const float2 s2 = fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3]));
          l += s2.x + s2.y;
          tmem_st_wait();
        }
        if (!full) {
          const int key = k0 + row;
          const bool seen = key < w.s.pre || (key >= w.t.lo && key <= w.t.hi);
          if (__any_sync(0xffffffffu, !seen)) {
            const uint32_t at = base + uint32_t(st.pos(h, j)), s = at % kVS;
            if (!(ok = warp_wait(&bars->v_full[s], (at / kVS) & 1, abort))) break;
            if (!seen) {
              const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll
              for (int half = 0; half < C::kHalves; ++half) {
                uint4* v = reinterpret_cast<uint4*>(sm + C::kOffV + s * C::kTile +
                                                    half * kRegionBytes + row * 128);
#pragma unroll
                for (int c = 0; c < 8; ++c) v[c] = z;
              }
            }
            fence_proxy_async_smem();
          }
        }
        tc_fence_before();
        mbar_arrive(&bars->p_full[h]);
      }
      if (!ok) break;
      const uint32_t last_v = mine > 0 ? (base + uint32_t(st.pos(h, mine - 1))) % kVS : 0u;
      base += uint32_t(st.nb0 + st.nb1);
      // ---- merge the two streams; this thread takes D / 2 columns of its row
      if (!(ok = warp_wait(&bars->o_ready, uc & 1, abort))) break;
      tc_fence_after();
      if (row == 0 && mine > 0) mbar_arrive(&bars->v_empty[last_v]);
      if (!(ok = warp_wait(&bars->x_read, (uc & 1) ^ 1, abort))) break;
      bars->xml[h][row] = make_float2(m, l);
      mbar_arrive(&bars->x_full);
      if (!(ok = warp_wait(&bars->x_full, uc & 1, abort))) break;
      const float2 other = bars->xml[h ^ 1][row];
      mbar_arrive(&bars->x_read);
      if (live) {
        const bool two = st.nb1 > 0;
        const float m0 = h ? other.x : m, l0 = h ? other.y : l;
        const float m1 = two ? (h ? m : other.x) : -INFINITY, l1 = two ? (h ? l : other.y) : 0.f;
        const float M = fmaxf(m0, m1), Ms = M == -INFINITY ? 0.f : M;
        float c0 = ex2(m0 - Ms), c1 = ex2(m1 - Ms);
        const float L = l0 * c0 + l1 * c1;
        const bool whole = w.whole();
        if (whole) {
          const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
          c0 *= inv;
          c1 *= inv;
        }
        const int64_t tok = int64_t(w.s.q0) + token;
        const int64_t at = int64_t(w.slot()) * 128 + row;
        if (valid && h == 0) {
          if (!whole) a.part_ml[at] = make_float2(M, L);
          else if (a.lse)
            a.lse[tok * a.Hq + head] =
                L > 0.f || L != L ? (Ms + log2f(L)) * 0.6931471805599453f : -INFINITY;
        }
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + tok * a.o_ts +
                             int64_t(head) * a.o_hs + h * (D / 2);
        // partials by columns of four, rows side by side: a warp's stores are whole lines
        float4* part = reinterpret_cast<float4*>(a.part_o) + int64_t(w.slot()) * (128 * D / 4) +
                       h * (D / 8) * 128 + row;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint32_t r0[32], r1[32];
          tmem_ld32(tO + h * (D / 2) + c * 32, r0);
          if (two) tmem_ld32(tO + 128u + h * (D / 2) + c * 32, r1);
          tmem_ld_wait();
          float x[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            x[i] = __uint_as_float(r0[i]) * c0;
            if (two) x[i] = fmaf(__uint_as_float(r1[i]), c1, x[i]);
          }
          if (valid && whole) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              *reinterpret_cast<uint4*>(dst + c * 32 + k * 8) =
                  make_uint4(pack_bf16(x[8 * k], x[8 * k + 1]), pack_bf16(x[8 * k + 2], x[8 * k + 3]),
                             pack_bf16(x[8 * k + 4], x[8 * k + 5]), pack_bf16(x[8 * k + 6], x[8 * k + 7]));
          } else if (valid) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              part[(c * 8 + k) * 128] =
                  make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&bars->o_free);
    }
  }

  __syncthreads();
  if (warp == kPaMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && bars->abort) report(a.status, FKV_ERR_TIMEOUT, blockIdx.x);
}

}  // namespace sm100

template <int D>
static cudaError_t launch_attend(PagedArgs a, cudaStream_t s) {
  using namespace sm100;
  using C = PaCfg<D>;
  a.R = 128;
  a.tk_shift = 7;
  a.mt = (a.G + 127) / 128;
  a.tq = a.mt == 1 ? 128 / a.G : 1;
  // Of parts of the line from 4, 8, 16 blocks up: 31, 33 and 46 us for the 30 mixed
  // pieces of a batch.
  a.min_steps = 4;
  // What a unit costs besides its blocks, in blocks: the causal prompts of a batch
  // (short units in the first parts) took 866 / 807 / 760 / 755 us at 4 / 5 / 6 / 8.
  a.extra = 6;
  // Units cut by themselves (own_steps 1 / 2 / 3 / 4): 128 queries over 900 keys, 16
  // heads: 26.0 / 22.6 / 21.5 / 24.0 us (on the line 22.4); the mixed pieces 28.2,
  // with slack 3 as slow as on the line.
  a.own_steps = 3;
  a.slack = 6;
  CUtensorMap tq, tk, tv;
  if (!paged_tmaps(a, D, 128, a.mt == 1 ? a.G : 128, a.tq, &tq, &tk, &tv))
    return cudaErrorNotSupported;
  const size_t smem = C::kOffBar + sizeof(PaBars);
  static_assert(C::kOffBar + sizeof(PaBars) <= 232448, "above the per-CTA limit");
  static_assert(C::kOffBar >= kPlanScratch, "the division's prefix sums fit in the tiles");
  auto* k = paged_attend_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  const int grid = paged_grid(1);
  a.own_units = grid / (a.Hkv * a.mt);
  e = launch_kernel(k, dim3(grid), dim3(kPaThreads), smem, s, false, tq, tk, tv, a);
  if (e != cudaSuccess) return e;
  return launch_paged_join(a, D, true, true, grid, s);
}

cudaError_t launch_paged_attend(const PagedArgs& a, int D, cudaStream_t s) {
  return D == 128 ? launch_attend<128>(a, s) : launch_attend<64>(a, s);
}

}  // namespace fkv
