// Which keys a tile of query rows sees, and which query each row is: plain
// arithmetic, compiled for the GPU by the paged-cache kernels and for the host
// by its test.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define FKV_HD __host__ __device__ __forceinline__
#else
#define FKV_HD inline
#endif

namespace fkv {

// One sequence of a ragged batch: its first query row and their number, its
// cached keys, and how many of the first of them every query sees.
struct Seq {
  int q0, q_len, kv, pre;
};

struct TileRule {
  int G, Hkv;          // query heads per KV head, KV heads
  int R, tk_shift, tq, mt;  // rows per tile, log2 of keys per step, tokens per tile, head slices
  int window, causal;
};

FKV_HD int query_tiles(const TileRule& g, const Seq& s) { return (s.q_len + g.tq - 1) / g.tq; }

// The keys that a tile of queries can see: [0, pre) and [lo, hi] (union over
// its rows), and the key blocks that hold them: blocks [0, nA), then
// [from, from + n - nA).
struct Span {
  int lo, hi, nA, from, n;
};

FKV_HD Span tile_span(const TileRule& g, const Seq& s, int qt) {
  const int first = s.kv - s.q_len + qt * g.tq;
  const int left = s.q_len - qt * g.tq;
  const int last = first + (left < g.tq ? left : g.tq) - 1;
  Span t;
  t.hi = g.causal ? last : s.kv - 1;
  t.lo = g.window > 0 && first - g.window + 1 > 0 ? first - g.window + 1 : 0;
  t.nA = (s.pre + (1 << g.tk_shift) - 1) >> g.tk_shift;
  t.from = t.lo >> g.tk_shift;
  if (t.from < t.nA) t.from = t.nA;
  const int end = t.hi < t.lo ? 0 : (t.hi >> g.tk_shift) + 1;
  t.n = t.nA + (end > t.from ? end - t.from : 0);
  if (t.n == 0) t.n = 1;  // rows that see nothing are still written: one masked step
  return t;
}

FKV_HD int block_at(const Span& t, int j) { return j < t.nA ? j : t.from + (j - t.nA); }

// Division rounded down, 0 <= n < 2^22, k > 0: a quotient in floats is off by less
// than one (half the code of an integer division, of which a short call runs more
// than of anything else).
constexpr int kDivMax = 1 << 22;
FKV_HD int div_down(int n, int k) {
#ifdef __CUDA_ARCH__
  int q = int(__fdividef(float(n), float(k)));
#else
  int q = int(float(n) / float(k));
#endif
  const int r = n - q * k;
  if (r < 0) --q;
  if (r >= k) ++q;
  return q;
}
// Parts of up to P steps of a unit of n steps (P = 0: its steps).
FKV_HD int parts_of(int n, int P) { return P ? div_down(n + P - 1, P) : n; }

// Length of the parts when every unit is cut by itself, into equal parts of at
// least `least` steps and at most `most` parts (0: any), one per CTA; `slots` CTAs
// per head for `units` units of at most `longest` steps.  0 when there are more
// units than CTAs, or none, or a unit is out of div_down's range.
FKV_HD int own_part(int units, int slots, int longest, int least, int most) {
  if (units == 0 || units > slots || longest >= kDivMax / 2) return 0;
  if (longest <= least) return longest;
  int k = div_down(slots, units);
  if (most && k > most) k = most;
  const int p = parts_of(longest, k);
  if (p <= least) return least;
  return parts_of(longest, parts_of(longest, p));
}

// Keys of a row at position p besides the prefix: lo <= j <= hi.
struct RowSpan {
  int lo, hi;
};
FKV_HD RowSpan row_span(const TileRule& g, const Seq& s, int p) {
  RowSpan r;
  r.hi = g.causal ? p : s.kv - 1;
  r.lo = g.window > 0 ? p - g.window + 1 : 0;
  return r;
}

// Row r of a tile: the token inside the sequence and the query head.
FKV_HD bool row_place(const TileRule& g, const Seq& s, int qt, int hm, int r, int* token, int* head) {
  const int h = hm / g.mt, m = hm - h * g.mt;
  int t = 0, i = m * g.R + r;
  if (g.mt == 1) {
    t = r / g.G;
    i = r - t * g.G;
  }
  *token = qt * g.tq + t;
  *head = h * g.G + i;
  return t < g.tq && i < g.G && *token < s.q_len;
}

}  // namespace fkv
