// Shared pieces of the paged-cache attention kernels: the resolved arguments,
// what a tile of query rows can see, the division of the work over CTAs, and
// the partial results that a split leaves behind.
//
// Work.  A unit is one tile of query rows of one sequence against one KV head:
// the G = Hq / Hkv query heads that share the KV head are packed with `tq`
// tokens into the tile's R rows (row r = token r / G, head r % G; with G > R one
// token and a slice of R heads).  A unit costs as many steps as the key blocks
// of TK keys that any of its rows can see; blocks that no row sees are never
// loaded.  The units of the batch, ordered (sequence, query tile, head), laid
// end to end make one line that is cut into equal parts, one per CTA, whatever
// the lengths are; on it a unit of n steps is n + `extra` long, `extra` (at its
// head) standing for the time that a unit takes besides its steps.  The cut is
// made on the GPU from cu_q, kv_len and prefix_len, so a captured call stays
// valid when the lengths change.
//
// With no more units than CTAs the cuts go elsewhere when that makes the longest
// part little longer: every unit into equal parts of its own, one per CTA, so that
// no CTA has a piece of two units (which is two passes through the code before and
// behind the steps, most of the time of a short call).
//
// Join.  A unit whose steps are cut by a part boundary is finished from the
// partial softmaxes (maximum, sum, unnormalised output, all fp32) of the CTAs
// that share it.  A CTA leaves at most two: of a unit that began in an earlier
// part (slot 0), and of the unit that goes on in the next (slot 1).  They are
// merged in CTA order, so results do not depend on timing.  Who merges: the CTA
// that writes a unit's last partial, where the kernel can and no unit has many;
// paged_join_kernel otherwise.
#pragma once

#include <cuda.h>

#include "fkv_internal.cuh"
#include "paged_plan.h"

namespace fkv {

constexpr int kMaxPagedSeqs = 4096;  // prefix sums of the division fit in shared memory
constexpr int kMaxPagedSms = 148;    // partial slots are sized for this many SMs
constexpr int kMaxPagedCtas = 4 * kMaxPagedSms;

// Most partials that the last CTA of a unit merges itself.  Measured (decode, 8 KV
// heads, one sequence): 131 keys, no unit cut, but that is the GPU's to know: 8.6 us
// a call with the merge inside, 11.7 with a join kernel behind; 1000 keys, units cut
// in 6: 14.3 inside, 13.2 with the kernel; 200k keys, in 37: 140 and 133.
constexpr int kJoinHere = 4;

struct PagedArgs : TileRule {
  const int32_t* page_table;
  const int32_t* kv_len;
  const int32_t* cu_q;
  const int32_t* prefix_len;
  const float* slopes;
  int64_t table_stride;
  int B, Hq;
  int page_shift, num_pages, max_pages, num_tokens;
  int min_steps;  // smallest part worth a CTA
  int extra;      // what a unit costs besides its steps, in steps
  int own_steps;  // smallest part of a unit that is cut by itself
  int own_units;  // most units per head for that: CTAs / (Hkv mt)
  int slack;      // steps that such parts may be longer than those of the line
  int join_here;  // cut units are joined by the kernel itself
  float scale, cap;
  // rows
  const void* q;
  void* out;
  float* lse;
  int64_t q_ts, q_hs, o_ts, o_hs;
  // caches (element strides)
  const void* k_cache;
  const void* v_cache;
  int64_t page_stride, head_stride, row_stride;
  // workspace
  int32_t* status;
  struct PlanRec* rec;  // [kMaxPagedCtas]
  int* arrived;         // [kMaxPagedCtas] partials written, per first cut boundary
  float2* part_ml;      // [slot][R] (max in base 2, sum)
  float* part_o;        // [slot][R][D] unnormalised outputs
};

// Where a CTA's part of the line begins.
struct PlanRec {
  int b, qt, hm, j;  // sequence, query tile, head unit, place inside the unit
  int n;             // length of that unit
  int per;           // length of a part
  int count;         // length of this part (0: none)
  int extra;         // of the units in it (0: units are cut by themselves)
  Seq s;             // the sequence
};

__device__ __forceinline__ Seq load_seq(const PagedArgs& a, int b) {
  Seq s;
  if (a.cu_q) {
    s.q0 = a.cu_q[b];
    const int e = a.cu_q[b + 1];
    s.q_len = e - s.q0;
    if (s.q0 < 0 || e < s.q0 || e > a.num_tokens) {
      report(a.status, FKV_ERR_DEVICE_ARG, b);
      s.q0 = 0;
      s.q_len = 0;
    }
  } else {
    s.q0 = b;
    s.q_len = 1;
  }
  const int cap = a.max_pages << a.page_shift;
  const int kv = a.kv_len[b];
  s.kv = kv < 0 ? 0 : (kv > cap ? cap : kv);
  if (s.kv != kv) report(a.status, FKV_ERR_DEVICE_ARG, b);
  const int pre = a.prefix_len ? a.prefix_len[b] : 0;
  s.pre = pre < 0 ? 0 : (pre > s.kv ? s.kv : pre);
  return s;
}

__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <class T>
__device__ __forceinline__ T warp_scan(T v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}
__device__ __forceinline__ Seq seq_of_lane(const Seq& s, int src) {
  Seq r;
  r.q0 = __shfl_sync(0xffffffffu, s.q0, src);
  r.q_len = __shfl_sync(0xffffffffu, s.q_len, src);
  r.kv = __shfl_sync(0xffffffffu, s.kv, src);
  r.pre = __shfl_sync(0xffffffffu, s.pre, src);
  return r;
}

// Steps of each lane's sequence (of one head unit), or its parts of up to P > 1
// steps; *longest: of its units.  Sequences of many query tiles are counted by the
// whole warp.
__device__ __forceinline__ int64_t seq_steps(const PagedArgs& a, const Seq& s, int lane, int P, int* longest) {
  const int nq = query_tiles(a, s);
  const bool wide = nq > 8;
  int64_t w = 0;
  *longest = 0;
  if (!wide)
    for (int qt = 0; qt < nq; ++qt) {
      const int n = parts_of(tile_span(a, s, qt).n, P);
      w += n;
      if (n > *longest) *longest = n;
    }
  unsigned todo = __ballot_sync(0xffffffffu, wide);
  while (todo) {
    const int src = __ffs(todo) - 1;
    todo &= todo - 1;
    const Seq t = seq_of_lane(s, src);
    const int tiles = query_tiles(a, t);
    int64_t sum = 0;
    int most = 0;
    for (int qt = lane; qt < tiles; qt += 32) {
      const int n = parts_of(tile_span(a, t, qt).n, P);
      sum += n;
      if (n > most) most = n;
    }
    sum = warp_sum(sum);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == src) {
      w = sum;
      *longest = most;
    }
  }
  return w;
}

// Place `rest` of sequence r.s: query tile, head unit and place in the unit (by
// the whole warp; r is the same in every lane).  P = 0: the place on the line;
// else the number of a part of up to P steps.
__device__ __forceinline__ void find_in_seq(const PagedArgs& a, PlanRec& r, int64_t rest, int P, int lane) {
  const int hm_n = a.Hkv * a.mt, nq = query_tiles(a, r.s);
  for (int q0 = 0; q0 < nq; q0 += 32) {
    const int qt = q0 + lane;
    const int n = qt < nq ? tile_span(a, r.s, qt).n + r.extra : 0;
    const int u = P ? parts_of(n, P) : n;
    const int64_t len = int64_t(u) * hm_n, inc = warp_scan(len, lane);
    const unsigned past = __ballot_sync(0xffffffffu, inc > rest);
    if (past) {
      const int src = __ffs(past) - 1;
      const int64_t in = __shfl_sync(0xffffffffu, rest - (inc - len), src);
      const int of = __shfl_sync(0xffffffffu, u, src);
      r.n = __shfl_sync(0xffffffffu, n, src);
      r.qt = q0 + src;
      r.hm = int(in / of);
      r.j = int(in - int64_t(r.hm) * of);
      if (P) {
        r.j *= P;
        r.per = P;
        r.count = r.n - r.j < P ? r.n - r.j : P;
      }
      return;
    }
    rest -= __shfl_sync(0xffffffffu, inc, 31);
  }
}

// Length of a part of a line of `total`.
__device__ __forceinline__ int64_t line_part(const PagedArgs& a, int64_t total) {
  const int64_t per = (total + gridDim.x - 1) / gridDim.x;
  return per < a.min_steps ? a.min_steps : per;
}
// Part of this CTA of the line.
__device__ __forceinline__ PlanRec part_of(const PagedArgs& a, int64_t total, int64_t per, int64_t* start) {
  *start = per * blockIdx.x;
  const int64_t count = total - *start < per ? total - *start : per;
  PlanRec r = {};
  r.per = int(per);
  r.count = count > 0 ? int(count) : 0;
  r.extra = a.extra;
  return r;
}

// The division: every thread of the CTA calls it; `scratch` is shared memory
// (free again afterwards), `rec` the shared result.  Ends with a __syncthreads.
// Up to 32 sequences are divided by one warp in registers; more by the CTA, with
// their prefix sums in the scratch.
constexpr size_t kPlanScratch = sizeof(int64_t) * (32 + kMaxPagedSeqs + 1);
template <int kThreads>
__device__ __forceinline__ void plan_part(const PagedArgs& a, int64_t* scratch, PlanRec* rec) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hm_n = a.Hkv * a.mt;
  const Seq none = {0, 0, 0, 0};
  if (a.B <= 32) {
    if (warp == 0) {
      const Seq s = lane < a.B ? load_seq(a, lane) : none;
      const int nq = query_tiles(a, s);
      int longest;
      int64_t w = seq_steps(a, s, lane, 0, &longest);
      longest = __reduce_max_sync(0xffffffffu, longest);
      // capped: 32 sequences of 2^30 tokens would not fit an int
      const int units = __reduce_add_sync(0xffffffffu, nq < kMaxPagedCtas ? nq : kMaxPagedCtas);
      int P = own_part(units, a.own_units, longest, a.own_steps, a.join_here ? kJoinHere : 0);
      int64_t inc = 0, start = blockIdx.x;
      PlanRec r = {};
      const bool own = P && P + a.extra <= a.min_steps + a.slack;  // whatever the line's are
      if (!own) {
        w = (w + int64_t(nq) * a.extra) * hm_n;
        inc = warp_scan(w, lane);
        const int64_t total = __shfl_sync(0xffffffffu, inc, 31), per = line_part(a, total);
        if (P + a.extra > per + a.slack) P = 0;
        if (!P) r = part_of(a, total, per, &start);
      }
      if (P) {
        w = hm_n * (P >= longest ? nq : int(seq_steps(a, s, lane, P, &longest)));
        inc = warp_scan(int(w), lane);
        r.count = start < __shfl_sync(0xffffffffu, inc, 31);
      }
      if (r.count > 0) {
        const int src = __ffs(__ballot_sync(0xffffffffu, inc > start)) - 1;
        r.b = src;
        r.s = seq_of_lane(s, src);
        find_in_seq(a, r, start - __shfl_sync(0xffffffffu, inc - w, src), P, lane);
      }
      if (lane == 0) {
        *rec = r;
        a.rec[blockIdx.x] = r;
      }
    }
    __syncthreads();
    return;
  }
  int64_t* warp_tot = scratch;     // [kThreads / 32]
  int64_t* cum = scratch + 32;     // [B + 1] length of the sequences before b
  int64_t carry = 0;
  if (tid == 0) cum[0] = 0;
  for (int base = 0; base < a.B; base += kThreads) {
    const int b = base + tid;
    const Seq s = b < a.B ? load_seq(a, b) : none;
    int longest;
    const int64_t inc = warp_scan(
        (seq_steps(a, s, lane, 0, &longest) + int64_t(query_tiles(a, s)) * a.extra) * hm_n, lane);
    if (lane == 31) warp_tot[warp] = inc;
    __syncthreads();
    int64_t before = carry, all = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) before += warp_tot[i];
      all += warp_tot[i];
    }
    if (b < a.B) cum[b + 1] = before + inc;
    carry += all;
    __syncthreads();
  }
  if (warp == 0) {
    int64_t start;
    PlanRec r = part_of(a, carry, line_part(a, carry), &start);
    if (r.count > 0) {
      int lo = 0, hi = a.B - 1;  // the sequence with cum[b] <= start < cum[b + 1]
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (cum[mid + 1] > start) hi = mid;
        else lo = mid + 1;
      }
      r.b = lo;
      r.s = load_seq(a, lo);
      find_in_seq(a, r, start - cum[lo], 0, lane);
    }
    if (lane == 0) {
      *rec = r;
      a.rec[blockIdx.x] = r;
    }
  }
  __syncthreads();
}

// Walks the units of a part that have steps in it.  All roles of a CTA walk alike.
struct Walk {
  Seq s;
  Span t;
  int b, qt, hm;
  int at, left;      // place inside the unit, what is left of the part
  int first, count;  // steps of the unit in this part: first .. first + count - 1
  int64_t from;      // where the unit begins on the line

  __device__ __forceinline__ void begin(const PagedArgs& a, const PlanRec& r) {
    from = int64_t(r.per) * blockIdx.x - r.j;
    b = r.b;
    qt = r.qt;
    hm = r.hm;
    at = r.j;
    left = r.count;
    if (left > 0) {
      s = r.s;
      t = tile_span(a, s, qt);
      cut(r.extra);
      if (count == 0) next(a);
    }
  }
  __device__ __forceinline__ bool done() const { return left <= 0; }
  __device__ __forceinline__ bool whole() const { return first == 0 && count == t.n; }
  __device__ __forceinline__ int slot() const { return 2 * int(blockIdx.x) + (first > 0 ? 0 : 1); }
  // (A part of a unit that is cut by itself is the CTA's only one: `left` is at most
  // what is left of the unit.)
  __device__ __forceinline__ void next(const PagedArgs& a) {
    do {
      left -= t.n + a.extra - at;
      if (left <= 0) return;
      from += t.n + a.extra;
      at = 0;
      if (++hm >= a.Hkv * a.mt) {
        hm = 0;
        if (++qt >= query_tiles(a, s)) {
          qt = 0;
          do {
            s = load_seq(a, ++b);
          } while (s.q_len == 0);
        }
        t = tile_span(a, s, qt);
      }
      cut(a.extra);
    } while (count == 0);
  }
  // The first part boundary that cuts the unit's steps, and the CTAs that share
  // them.
  __device__ __forceinline__ int cut_at(int per, int extra, int* parts) const {
    const int c = int((from + extra) / per) + 1;
    *parts = int((from + t.n + extra - 1) / per) - c + 2;
    return c;
  }
  __device__ __forceinline__ void cut(int extra) {
    const int end = t.n + extra - at < left ? t.n + extra : at + left;
    first = at > extra ? at - extra : 0;
    count = end > extra ? end - extra - first : 0;
  }
};

// Whether any row of a tile sees any of `rows` keys from `key` on.  Pages without
// such a key may be gone (behind a window), and a copy of them is not worth its
// bytes: their scores are masked and their values set to zero whatever the tile
// holds.
__device__ __forceinline__ bool box_seen(const Seq& s, const Span& t, int key, int rows) {
  return key < s.pre || (key <= t.hi && key + rows > t.lo);
}

// Page id of a sequence's p-th page; -1 (reported) when out of range.
__device__ __forceinline__ int page_id(const PagedArgs& a, int b, int p) {
  const int id = a.page_table[int64_t(b) * a.table_stride + p];
  if (id >= 0 && id < a.num_pages) return id;
  report(a.status, FKV_ERR_DEVICE_ARG, b);
  return -1;
}

// Two fp32 lanes per instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)),
        "l"(*reinterpret_cast<uint64_t*>(&c)));
  return *reinterpret_cast<float2*>(&r);
}

// tanh(y) = num / den on pairs, num = y P(y^2), den = Q(y^2), |y| cut off at 8: within
// 9 roundings relative to tanh(y), however small y is (coefficients from fit_tanh.py
// beside this file).  (1 - 2 / (e^2y + 1) takes fewer instructions, but is within
// 1e-7 of 1 and not of y: times a cap far above the scores that is all of them.)
// A NaN comes out in its own num and leaves den finite.
// Where all of a warp's |y| are below 1/2 (caps of 30 to 50 over ordinary scores)
// tanh_small does with half the instructions: y + y^3 p(y^2), within 2 roundings.
constexpr float kTanhMost = 8.f, kTanhSmall = 0.5f;
__device__ __forceinline__ float2 tanh_small(float2 y) {
  constexpr float S[4] = {-3.333314359e-01f, 1.332587898e-01f, -5.304549262e-02f, 1.724149100e-02f};
  auto both = [](float c) { return make_float2(c, c); };
  const float2 u = mul2(y, y);
  float2 p = fma2(both(S[3]), u, both(S[2]));
#pragma unroll
  for (int i = 1; i >= 0; --i) p = fma2(p, u, both(S[i]));
  return fma2(mul2(y, u), p, y);
}
__device__ __forceinline__ float cut_off(float y) {  // keeps a NaN
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(y) : "f"(-kTanhMost));
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(y) : "f"(kTanhMost));
  return y;
}
__device__ __forceinline__ void tanh_parts(float2 y, float2& num, float2& den) {
  constexpr float P[5] = {9.999998212e-01f, 1.271007806e-01f, 2.694026800e-03f, 7.143671155e-06f,
                          -6.107998107e-09f};
  constexpr float Q[4] = {1.000000000e+00f, 4.604324698e-01f, 2.284044214e-02f, 1.964301337e-04f};
  auto both = [](float c) { return make_float2(c, c); };
  y.x = cut_off(y.x);
  y.y = cut_off(y.y);
  float2 u = mul2(y, y);
  u.x = fminf(u.x, kTanhMost * kTanhMost);  // drops a NaN
  u.y = fminf(u.y, kTanhMost * kTanhMost);
  float2 p = fma2(both(P[4]), u, both(P[3]));
#pragma unroll
  for (int i = 2; i >= 0; --i) p = fma2(p, u, both(P[i]));
  num = mul2(p, y);
  den = fma2(both(Q[3]), u, both(Q[2]));
#pragma unroll
  for (int i = 1; i >= 0; --i) den = fma2(den, u, both(Q[i]));
}

// Whether no unit can be cut into more than kJoinHere parts.  A unit is at most as
// long as the page table allows, a part at least min_steps; and the units of a
// sequence are alike, so one has at most 1 / (head units) of the line.
inline bool few_parts(const PagedArgs& a, int grid) {
  const int64_t keys = int64_t(a.max_pages) << a.page_shift;
  const int64_t longest = ((keys + (1 << a.tk_shift) - 1) >> a.tk_shift) + a.extra;
  return longest / a.min_steps + 2 <= kJoinHere || grid / (a.Hkv * a.mt) + 2 <= kJoinHere;
}

struct PagedWs {
  size_t rec, arrived, ml, o, total;
};
inline PagedWs paged_ws_layout() {
  // two slots per CTA; slots x rows is largest for the 128-row tiles, which have
  // one CTA per SM (16-row tiles have up to four)
  PagedWs w;
  const size_t rows = size_t(kMaxPagedSms) * 2 * 128;
  w.rec = 256;
  w.arrived = w.rec + sizeof(PlanRec) * kMaxPagedCtas;
  w.ml = w.arrived + sizeof(int) * kMaxPagedCtas;
  w.ml = (w.ml + 255) & ~size_t(255);
  w.o = w.ml + rows * sizeof(float2);
  w.total = w.o + rows * 128 * sizeof(float);
  return w;
}

// grid of a kernel with `per_sm` resident CTAs and R rows: every slot fits.
inline int paged_grid(int per_sm) {
  const int sms = num_sms();
  return per_sm * (sms < kMaxPagedSms ? sms : kMaxPagedSms);
}

// Arguments of the norm / rotation / append kernel (paged_rows.cu).
struct RowsArgs {
  int tokens, nq, nk, nv;  // heads per token (nv: value rows, append only)
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  void* k_out;             // rows of keys; unused by an append
  int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, qo_ts, qo_hs, ko_ts, ko_hs;
  // norm and rotation
  int norm, half, pairs, axis1, axis2;  // first pair of axis 1 and of axis 2
  float eps;
  const float* q_weight;
  const float* k_weight;
  const float* omega;
  const int32_t* positions;  // NULL: the cache position
  int64_t axis_stride;
  // append
  int append, B, page_shift, num_pages, max_pages;
  const int32_t* cu_q;
  const int32_t* kv_len;
  const int32_t* page_table;
  int64_t table_stride, page_stride, head_stride, row_stride;
  void* k_cache;
  void* v_cache;
  int32_t* status;
};

cudaError_t launch_rows(const RowsArgs& a, bool bf16, int D, cudaStream_t s);
// Tensor maps of a bf16 call's queries [tokens][Hq][D] (box: q_tokens x q_heads rows of
// 64 dims) and caches (box: the rows of a page, at most `keys`, of 64 dims), all in the
// 128-byte swizzle.
bool paged_tmaps(const PagedArgs& a, int D, int keys, int q_heads, int q_tokens, CUtensorMap* q,
                 CUtensorMap* k, CUtensorMap* v);
cudaError_t launch_paged_decode(const PagedArgs& a, int D, cudaStream_t s);
cudaError_t launch_paged_attend(const PagedArgs& a, int D, cudaStream_t s);
// columns: the partial outputs lie as [slot][D / 4][R][4] (the chunk kernel's),
// else as [slot][R][D].
cudaError_t launch_paged_join(const PagedArgs& a, int D, bool bf16, bool columns, int grid,
                              cudaStream_t s);
cudaError_t launch_paged_decode_f32(const PagedArgs& a, int D, cudaStream_t s);
cudaError_t launch_paged_attend_f32(const PagedArgs& a, int D, cudaStream_t s);

}  // namespace fkv
