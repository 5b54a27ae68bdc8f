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
