// Host side of the paged-cache entry points: argument checks (all before the
// first launch) and kernel arguments.
#include <math.h>
#include <stdio.h>

#include "paged_common.cuh"

namespace fkv {
namespace {

int32_t launch_status(cudaError_t e) {
  if (e == cudaSuccess) return FKV_OK;
  fprintf(stderr, "fkv: CUDA error %d (%s)\n", int(e), cudaGetErrorString(e));
  return FKV_ERR_CUDA;
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Positions, windows and token counts stay below 2^30, so that their sums and
// differences stay inside 32 bits.
const int64_t kMaxPositions = int64_t(1) << 30;
const int64_t kMaxStride = int64_t(1) << 37;  // elements; tensor maps end at 2^40 bytes

// Row strides as the kernels use them: 0 where the dimension has one entry.
struct Strides {
  int64_t ts, hs;
};

// Checks rows [tokens][heads][D]; an unused array (no tokens or heads) passes.
int32_t check_rows(const fkv_rows_t* r, int64_t tokens, int64_t heads, int D, int elem, bool output,
                   Strides* out) {
  *out = Strides{0, 0};
  if (tokens == 0 || heads == 0) return FKV_OK;
  if (!r || !r->ptr || !aligned(r->ptr, 16)) return FKV_ERR_INVALID_ARG;
  if (tokens > 1) out->ts = r->token_stride;
  if (heads > 1) out->hs = r->head_stride;
  const int64_t strides[] = {out->ts, out->hs};
  for (int64_t s : strides) {
    if (s < 0 || s > kMaxStride) return FKV_ERR_SHAPE;
    if ((s * elem) % 16 != 0) return FKV_ERR_INVALID_ARG;
  }
  if (output) {  // rows of an output are apart from one another
    const int64_t ext_t = heads > 1 ? out->hs * (heads - 1) + D : D;
    const int64_t ext_h = tokens > 1 ? out->ts * (tokens - 1) + D : D;
    const bool tokens_apart = tokens == 1 || out->ts >= ext_t;
    const bool heads_apart = heads == 1 || out->hs >= ext_h;
    const bool each = (tokens == 1 || out->ts >= D) && (heads == 1 || out->hs >= D);
    if (!each || !(tokens_apart || heads_apart)) return FKV_ERR_SHAPE;
  }
  return FKV_OK;
}

int32_t check_type(int32_t dtype, int32_t D) {
  if (dtype != FKV_DTYPE_BF16 && dtype != FKV_DTYPE_FP32) return FKV_ERR_INVALID_ARG;
  if (D < 1) return FKV_ERR_SHAPE;
  if (D != 64 && D != 128) return FKV_ERR_UNSUPPORTED;
  return FKV_OK;
}

int32_t check_rope(const fkv_rope_t* r, int D, int64_t tokens, bool cache_positions, RowsArgs* a) {
  if (r->style != FKV_ROPE_ADJACENT && r->style != FKV_ROPE_HALF) return FKV_ERR_INVALID_ARG;
  if (r->n_axes < 1 || r->n_axes > 3) return FKV_ERR_SHAPE;
  int64_t n = 0;
  int64_t first[4] = {0, 0, 0, 0};
  for (int i = 0; i < r->n_axes; ++i) {
    if (r->axis_pairs[i] < 0) return FKV_ERR_SHAPE;
    n += r->axis_pairs[i];
    first[i + 1] = n;
  }
  for (int i = r->n_axes; i < 3; ++i) first[i + 1] = n;
  if (2 * n > D) return FKV_ERR_SHAPE;
  if (r->style == FKV_ROPE_HALF && n % 8 != 0) return FKV_ERR_UNSUPPORTED;
  if (r->norm && !(r->eps >= 0.f && r->eps <= 3.0e38f)) return FKV_ERR_INVALID_ARG;
  if (n > 0 && tokens > 0) {
    if (!r->omega) return FKV_ERR_INVALID_ARG;
    if (!r->positions && !(cache_positions && r->n_axes == 1)) return FKV_ERR_INVALID_ARG;
    if (r->positions && r->n_axes > 1 && (r->axis_stride < tokens || r->axis_stride > kMaxStride))
      return FKV_ERR_SHAPE;
  }
  if (!aligned(r->q_weight, 4) || !aligned(r->k_weight, 4) || !aligned(r->omega, 4) ||
      !aligned(r->positions, 4))
    return FKV_ERR_INVALID_ARG;
  a->norm = r->norm != 0;
  a->half = r->style == FKV_ROPE_HALF;
  a->pairs = int(n);
  a->axis1 = int(first[1]);
  a->axis2 = int(first[2]);
  a->eps = r->eps;
  a->q_weight = r->q_weight;
  a->k_weight = r->k_weight;
  a->omega = r->omega;
  a->positions = r->positions;
  a->axis_stride = r->n_axes > 1 ? r->axis_stride : 0;
  return FKV_OK;
}

// Checks the cache and batch of a call with `tokens` rows and fills the kernel
// arguments they decide.
int32_t check_paged(const fkv_paged_t* c, int64_t tokens, PagedArgs* a) {
  if (!c) return FKV_ERR_INVALID_ARG;
  int32_t st = check_type(c->dtype, c->head_dim);
  if (st != FKV_OK) return st;
  if (c->flags & ~FKV_PAGED_CAUSAL) return FKV_ERR_INVALID_ARG;
  if (c->num_seqs < 0 || c->num_seqs > kMaxPagedSeqs || c->num_pages < 0 || c->max_pages < 0 ||
      c->num_kv_heads < 1 || c->num_q_heads < 1 || c->window < 0 || tokens < 0 ||
      tokens > kMaxPositions)
    return FKV_ERR_SHAPE;
  if (c->num_q_heads % c->num_kv_heads != 0 || c->num_q_heads > 65535) return FKV_ERR_SHAPE;
  if (c->page_size < 1) return FKV_ERR_SHAPE;
  if (c->page_size < 8 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)) != 0)
    return FKV_ERR_UNSUPPORTED;
  if (int64_t(c->max_pages) * c->page_size > kMaxPositions) return FKV_ERR_SHAPE;
  // the kernels form scale / softcap, softcap / scale and slope / scale
  if (!(c->scale >= 1e-12f && c->scale <= 1e12f)) return FKV_ERR_INVALID_ARG;
  if (c->softcap != 0.f && !(c->softcap >= 1e-12f && c->softcap <= 1e12f))
    return FKV_ERR_INVALID_ARG;
  const int elem = c->dtype == FKV_DTYPE_BF16 ? 2 : 4;
  const int64_t strides[] = {c->page_stride, c->head_stride, c->row_stride};
  const int64_t counts[] = {c->num_pages, c->num_kv_heads, c->page_size};
  int64_t eff[3];
  for (int i = 0; i < 3; ++i) {
    eff[i] = counts[i] > 1 ? strides[i] : c->head_dim;
    if (eff[i] < c->head_dim || eff[i] > kMaxStride) return FKV_ERR_SHAPE;
    if ((eff[i] * elem) % 16 != 0) return FKV_ERR_INVALID_ARG;
  }
  if (c->num_seqs > 1 && (c->table_stride < c->max_pages || c->table_stride > kMaxStride))
    return FKV_ERR_SHAPE;
  if (c->num_pages > 0 && (!c->k_cache || !c->v_cache)) return FKV_ERR_INVALID_ARG;
  if (!aligned(c->k_cache, 16) || !aligned(c->v_cache, 16)) return FKV_ERR_INVALID_ARG;
  if (c->num_seqs > 0 && (!c->kv_len || (!c->page_table && c->max_pages > 0)))
    return FKV_ERR_INVALID_ARG;
  if (!aligned(c->kv_len, 4) || !aligned(c->page_table, 4) || !aligned(c->cu_q, 4) ||
      !aligned(c->prefix_len, 4) || !aligned(c->alibi_slopes, 4))
    return FKV_ERR_INVALID_ARG;
  int shift = 0;
  while ((1 << shift) < c->page_size) ++shift;
  *a = PagedArgs{};
  a->page_table = c->page_table;
  a->kv_len = c->kv_len;
  a->cu_q = c->cu_q;
  a->prefix_len = c->prefix_len;
  a->slopes = c->alibi_slopes;
  a->table_stride = c->num_seqs > 1 ? c->table_stride : 0;
  a->B = c->num_seqs;
  a->Hq = c->num_q_heads;
  a->Hkv = c->num_kv_heads;
  a->G = c->num_q_heads / c->num_kv_heads;
  a->page_shift = shift;
  a->num_pages = c->num_pages;
  a->max_pages = c->max_pages;
  a->num_tokens = int(tokens);
  a->window = c->window < kMaxPositions ? c->window : int(kMaxPositions);
  a->causal = (c->flags & FKV_PAGED_CAUSAL) != 0;
  a->scale = c->scale;
  a->cap = c->softcap;
  a->k_cache = c->k_cache;
  a->v_cache = c->v_cache;
  a->page_stride = eff[0];
  a->head_stride = eff[1];
  a->row_stride = eff[2];
  return FKV_OK;
}

int32_t check_paged_ws(void* ws, PagedArgs* a) {
  if (!ws || !aligned(ws, 256)) return FKV_ERR_WORKSPACE;
  const PagedWs w = paged_ws_layout();
  char* base = static_cast<char*>(ws);
  a->status = reinterpret_cast<int32_t*>(base);
  a->rec = reinterpret_cast<PlanRec*>(base + w.rec);
  a->arrived = reinterpret_cast<int*>(base + w.arrived);
  a->part_ml = reinterpret_cast<float2*>(base + w.ml);
  a->part_o = reinterpret_cast<float*>(base + w.o);
  return FKV_OK;
}

int32_t attention(const fkv_paged_t* c, int64_t tokens, bool single, const fkv_rows_t* q,
                  const fkv_rows_t* out, float* lse, void* ws, void* stream) {
  PagedArgs a;
  int32_t st = check_paged(c, tokens, &a);
  if (st != FKV_OK) return st;
  const int elem = c->dtype == FKV_DTYPE_BF16 ? 2 : 4;
  Strides sq, so;
  if ((st = check_rows(q, tokens, a.Hq, c->head_dim, elem, false, &sq)) != FKV_OK) return st;
  if ((st = check_rows(out, tokens, a.Hq, c->head_dim, elem, true, &so)) != FKV_OK) return st;
  if (!aligned(lse, 4)) return FKV_ERR_INVALID_ARG;
  // tensor maps have no zero strides
  if (tokens > 0 && ((a.Hq > 1 && sq.hs == 0) || (tokens > 1 && sq.ts == 0))) return FKV_ERR_SHAPE;
  if (!single && !c->cu_q && tokens != c->num_seqs) return FKV_ERR_SHAPE;
  if ((st = check_paged_ws(ws, &a)) != FKV_OK) return st;
  if (tokens == 0 || c->num_seqs == 0) return FKV_OK;
  if (single) a.cu_q = nullptr;
  a.q = q->ptr;
  a.out = out->ptr;
  a.lse = lse;
  a.q_ts = sq.ts;
  a.q_hs = sq.hs;
  a.o_ts = so.ts;
  a.o_hs = so.hs;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool f32 = c->dtype == FKV_DTYPE_FP32;
  auto* launch = single ? (f32 ? launch_paged_decode_f32 : launch_paged_decode)
                        : (f32 ? launch_paged_attend_f32 : launch_paged_attend);
  return launch_status(launch(a, c->head_dim, s));
}

}  // namespace
}  // namespace fkv

using namespace fkv;

extern "C" {

int32_t fkv_paged_workspace_size(size_t* bytes) {
  if (!bytes) return FKV_ERR_INVALID_ARG;
  *bytes = paged_ws_layout().total;
  return FKV_OK;
}

int32_t fkv_qk_norm_rope(const fkv_rope_t* r, int32_t dtype, int32_t head_dim, int32_t num_tokens,
                         int32_t num_q_heads, int32_t num_kv_heads, const fkv_rows_t* q,
                         const fkv_rows_t* k, const fkv_rows_t* q_out, const fkv_rows_t* k_out,
                         void* stream) {
  if (!r) return FKV_ERR_INVALID_ARG;
  int32_t st = check_type(dtype, head_dim);
  if (st != FKV_OK) return st;
  if (num_tokens < 0 || num_tokens > kMaxPositions || num_q_heads < 0 || num_kv_heads < 0 || num_q_heads > 65535 ||
      num_kv_heads > 65535)
    return FKV_ERR_SHAPE;
  RowsArgs a = {};
  if ((st = check_rope(r, head_dim, num_tokens, false, &a)) != FKV_OK) return st;
  const int elem = dtype == FKV_DTYPE_BF16 ? 2 : 4;
  Strides sq, sk, sqo, sko;
  if ((st = check_rows(q, num_tokens, num_q_heads, head_dim, elem, false, &sq)) != FKV_OK ||
      (st = check_rows(k, num_tokens, num_kv_heads, head_dim, elem, false, &sk)) != FKV_OK ||
      (st = check_rows(q_out, num_tokens, num_q_heads, head_dim, elem, true, &sqo)) != FKV_OK ||
      (st = check_rows(k_out, num_tokens, num_kv_heads, head_dim, elem, true, &sko)) != FKV_OK)
    return st;
  a.tokens = num_tokens;
  a.nq = num_q_heads;
  a.nk = num_kv_heads;
  a.q = q ? q->ptr : nullptr;
  a.k = k ? k->ptr : nullptr;
  a.q_out = q_out ? q_out->ptr : nullptr;
  a.k_out = k_out ? k_out->ptr : nullptr;
  a.q_ts = sq.ts, a.q_hs = sq.hs, a.k_ts = sk.ts, a.k_hs = sk.hs;
  a.qo_ts = sqo.ts, a.qo_hs = sqo.hs, a.ko_ts = sko.ts, a.ko_hs = sko.hs;
  return launch_status(launch_rows(a, dtype == FKV_DTYPE_BF16, head_dim,
                                   static_cast<cudaStream_t>(stream)));
}

int32_t fkv_paged_append(const fkv_paged_t* c, const fkv_rope_t* r, int32_t num_tokens,
                         const fkv_rows_t* q, const fkv_rows_t* k, const fkv_rows_t* v,
                         const fkv_rows_t* q_out, void* ws, void* stream) {
  PagedArgs p;
  int32_t st = check_paged(c, num_tokens, &p);
  if (st != FKV_OK) return st;
  RowsArgs a = {};
  if (r && (st = check_rope(r, c->head_dim, num_tokens, true, &a)) != FKV_OK) return st;
  if ((q != nullptr) != (q_out != nullptr)) return FKV_ERR_INVALID_ARG;
  if (!c->cu_q && num_tokens != c->num_seqs) return FKV_ERR_SHAPE;
  const int elem = c->dtype == FKV_DTYPE_BF16 ? 2 : 4;
  const int nq = q ? p.Hq : 0;
  Strides sq, sk, sv, sqo;
  if ((st = check_rows(q, num_tokens, nq, c->head_dim, elem, false, &sq)) != FKV_OK ||
      (st = check_rows(k, num_tokens, p.Hkv, c->head_dim, elem, false, &sk)) != FKV_OK ||
      (st = check_rows(v, num_tokens, p.Hkv, c->head_dim, elem, false, &sv)) != FKV_OK ||
      (st = check_rows(q_out, num_tokens, nq, c->head_dim, elem, true, &sqo)) != FKV_OK)
    return st;
  if ((st = check_paged_ws(ws, &p)) != FKV_OK) return st;
  if (num_tokens == 0 || c->num_seqs == 0) return FKV_OK;
  a.tokens = num_tokens;
  a.nq = nq;
  a.nk = a.nv = p.Hkv;
  a.q = q ? q->ptr : nullptr;
  a.q_out = q_out ? q_out->ptr : nullptr;
  a.k = k->ptr;
  a.v = v->ptr;
  a.q_ts = sq.ts, a.q_hs = sq.hs, a.k_ts = sk.ts, a.k_hs = sk.hs, a.v_ts = sv.ts, a.v_hs = sv.hs;
  a.qo_ts = sqo.ts, a.qo_hs = sqo.hs;
  a.append = 1;
  a.B = p.B;
  a.page_shift = p.page_shift;
  a.num_pages = p.num_pages;
  a.max_pages = p.max_pages;
  a.cu_q = p.cu_q;
  a.kv_len = p.kv_len;
  a.page_table = p.page_table;
  a.table_stride = p.table_stride;
  a.page_stride = p.page_stride;
  a.head_stride = p.head_stride;
  a.row_stride = p.row_stride;
  a.k_cache = c->k_cache;
  a.v_cache = c->v_cache;
  a.status = p.status;
  return launch_status(launch_rows(a, c->dtype == FKV_DTYPE_BF16, c->head_dim,
                                   static_cast<cudaStream_t>(stream)));
}

int32_t fkv_paged_decode(const fkv_paged_t* c, const fkv_rows_t* q, const fkv_rows_t* out,
                         float* lse, void* ws, void* stream) {
  return attention(c, c ? c->num_seqs : 0, true, q, out, lse, ws, stream);
}

int32_t fkv_paged_attend(const fkv_paged_t* c, int32_t num_tokens, const fkv_rows_t* q,
                         const fkv_rows_t* out, float* lse, void* ws, void* stream) {
  return attention(c, num_tokens, false, q, out, lse, ws, stream);
}

}  // extern "C"
