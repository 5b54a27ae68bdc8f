// Per-head RMS norm and rotation of query and key rows, and the append of keys
// and values to a paged cache, in one pass over the rows.
//
//   y = x / sqrt(mean(x^2) + eps) * w
//   (y_a, y_b) -> (y_a cos - y_b sin, y_a sin + y_b cos) for the pairs (a, b)
//
// Bound by memory: every row is read once and written once in 16-byte vectors
// (a row of D elements takes D * sizeof(T) / 16 lanes; the sum of squares and
// the partner values of the half-split pairs travel by shuffles inside them).
// The angles depend on the token alone, so a CTA takes one token and a slice of
// its heads and evaluates the token's cosines once.  Angles: omega * position
// is formed and reduced to a fraction of a turn in fp64 (fp32 would lose 1e-2
// radians at position 10^5), the sine and cosine of the fraction in fp32.
#include "paged_common.cuh"

namespace fkv {

constexpr int kRowThreads = 256;

// The sequence of token t: the last b with cu_q[b] <= t, found 32 ways at a
// time by the warp (two rounds of loads for 1024 sequences).
__device__ __forceinline__ int find_seq(const int32_t* cu_q, int B, int t, int lane) {
  int lo = 0, len = B;
  while (len > 1) {
    const int step = (len + 31) >> 5;
    const bool ok = lane * step < len && cu_q[lo + lane * step] <= t;
    const int c = __popc(__ballot_sync(0xffffffffu, ok));
    if (c == 0) return 0;
    lo += (c - 1) * step;
    const int left = len - (c - 1) * step;
    len = left < step ? left : step;
  }
  return lo;
}

__device__ __forceinline__ void unpack(const uint4& raw, float (&x)[8]) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(const uint4& raw, float (&x)[4]) {
  x[0] = __uint_as_float(raw.x);
  x[1] = __uint_as_float(raw.y);
  x[2] = __uint_as_float(raw.z);
  x[3] = __uint_as_float(raw.w);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint4 repack(const float (&x)[8]) {
  return make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}
__device__ __forceinline__ uint4 repack(const float (&x)[4]) {
  return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                    __float_as_uint(x[3]));
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

// One new token of an append: where its key and value go.
struct Place {
  int64_t page_off;  // element offset of its cache row (head 0); -1: dropped
  int pos;           // cache position
  int live;          // 0: a padded row
};

__device__ __forceinline__ Place find_place(const RowsArgs& a, int t, int lane) {
  Place p = {-1, 0, 0};
  int b = t, i = 0, q_len = 1;
  if (a.cu_q) {
    b = find_seq(a.cu_q, a.B, t, lane);
    const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1];
    if (q0 < 0 || q1 < q0 || q1 > a.tokens) {
      if (lane == 0) report(a.status, FKV_ERR_DEVICE_ARG, b);
      return p;
    }
    i = t - q0;
    q_len = q1 - q0;
    if (i < 0 || i >= q_len) return p;
  }
  p.live = 1;
  const int cap = a.max_pages << a.page_shift;
  int kv = a.kv_len[b];
  bool bad = kv < 0 || kv > cap;
  if (bad) kv = kv < 0 ? 0 : cap;
  p.pos = kv - q_len + i;
  int id = -1;
  if (p.pos >= 0) id = a.page_table[int64_t(b) * a.table_stride + (p.pos >> a.page_shift)];
  if (id >= 0 && id < a.num_pages)
    p.page_off = int64_t(id) * a.page_stride + int64_t(p.pos & ((1 << a.page_shift) - 1)) * a.row_stride;
  else
    bad = true;
  if (bad && lane == 0) report(a.status, FKV_ERR_DEVICE_ARG, b);
  return p;
}

// A CTA takes kTok tokens and a slice of their rows.  Half as many threads as a
// row has vectors share it: with half-split pairs a thread holds both halves of
// its pairs (dims i .. and n + i ..), so the turn needs no exchange, one read of
// the cosines serves two vectors, and the row's sum of squares one shuffle less.
template <typename T, int D, int kTok>
__global__ void __launch_bounds__(kRowThreads) rows_kernel(const RowsArgs a, int slice_rows) {
  constexpr int kVec = 16 / int(sizeof(T));  // elements per vector
  constexpr int kChunks = D / kVec;          // vectors per row
  constexpr int kTpr = kChunks / 2;          // threads per row
  constexpr int kPass = kRowThreads / kTpr;  // rows per pass of the CTA
  __shared__ __align__(16) float s_cos[kTok][D / 2], s_sin[kTok][D / 2];
  __shared__ __align__(16) float s_w[2][D];
  __shared__ Place s_place[kTok];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t0 = int(blockIdx.x) * kTok;
  const int n_tok = kTok == 1 ? 1 : min(kTok, a.tokens - t0);
  const int n_rows = a.nq + a.nk + a.nv;
  const int first = int(blockIdx.y) * slice_rows;
  const int rows = min(slice_rows, n_rows - first);  // of each token
  const int total = rows * n_tok;
  const int i = tid % kTpr;
  // this thread's two vectors: the halves of its pairs, or neighbours
  const int half_chunks = a.half ? a.pairs / kVec : 0;
  const bool split = i < half_chunks;
  const int ca = split ? i : 2 * i, cb = split ? i + half_chunks : 2 * i + 1;

  auto source = [&](int t, int row) -> const T* {
    if (row < a.nq) return static_cast<const T*>(a.q) + int64_t(t) * a.q_ts + int64_t(row) * a.q_hs;
    row -= a.nq;
    if (row < a.nk) return static_cast<const T*>(a.k) + int64_t(t) * a.k_ts + int64_t(row) * a.k_hs;
    return static_cast<const T*>(a.v) + int64_t(t) * a.v_ts + int64_t(row - a.nk) * a.v_hs;
  };
  int item = tid / kTpr;  // (token, row) pair, rows innermost
  int tok = item / rows, row = item - tok * rows;
  uint4 ra, rb;
  auto load = [&]() {
    if (item < total) {
      const T* src = source(t0 + tok, first + row);
      ra = __ldcs(reinterpret_cast<const uint4*>(src + ca * kVec));
      rb = __ldcs(reinterpret_cast<const uint4*>(src + cb * kVec));
    }
  };
  load();

  if (a.append) {
    for (int k = warp; k < n_tok; k += kRowThreads / 32) {
      const Place p = find_place(a, t0 + k, lane);
      if (lane == 0) s_place[k] = p;
    }
  }
  if (a.norm)
    for (int k = tid; k < 2 * D; k += kRowThreads) {
      const float* w = k < D ? a.q_weight : a.k_weight;
      s_w[k >= D][k & (D - 1)] = w ? w[k & (D - 1)] : 1.f;
    }
  if (a.append) __syncthreads();
  for (int k = tid; k < n_tok * a.pairs; k += kRowThreads) {
    const int tk = kTok == 1 ? 0 : k / a.pairs, j = k - tk * a.pairs;
    const int axis = (j >= a.axis1) + (j >= a.axis2);
    const int p = a.positions ? a.positions[axis * a.axis_stride + t0 + tk] : s_place[tk].pos;
    const double turns = double(p) * (double(a.omega[j]) * 0.15915494309189535);
    sincospif(2.f * float(turns - rint(turns)), &s_sin[tk][j], &s_cos[tk][j]);
  }
  __syncthreads();

  const unsigned group = ((kTpr == 32 ? 0u : 1u << kTpr) - 1u) << (lane & ~(kTpr - 1));
  while (item < total) {  // the threads of a row stay together
    const uint4 xa = ra, xb = rb;
    const int t = tok, r = first + row;
    item += kPass;
    row += kPass;
    while (row >= rows) {
      row -= rows;
      ++tok;
    }
    load();
    const bool is_q = r < a.nq, is_v = r >= a.nq + a.nk;
    T* dst;
    if (a.append && !s_place[t].live) continue;
    if (is_q) {
      dst = static_cast<T*>(a.q_out) + int64_t(t0 + t) * a.qo_ts + int64_t(r) * a.qo_hs;
    } else if (!a.append) {
      dst = static_cast<T*>(a.k_out) + int64_t(t0 + t) * a.ko_ts + int64_t(r - a.nq) * a.ko_hs;
    } else {
      const int64_t off = s_place[t].page_off;
      if (off < 0) continue;
      dst = (is_v ? static_cast<T*>(a.v_cache) : static_cast<T*>(a.k_cache)) + off +
            int64_t(is_v ? r - a.nq - a.nk : r - a.nq) * a.head_stride;
    }
    uint4 ya = xa, yb = xb;
    if (!is_v) {
      float x[2][kVec];
      unpack(xa, x[0]);
      unpack(xb, x[1]);
      float2(&x2)[2][kVec / 2] = reinterpret_cast<float2(&)[2][kVec / 2]>(x);
      if (a.norm) {
        float2 s2 = mul2(x2[0][0], x2[0][0]);
#pragma unroll
        for (int e = 1; e < kVec; ++e)
          s2 = fma2(x2[e / (kVec / 2)][e % (kVec / 2)], x2[e / (kVec / 2)][e % (kVec / 2)], s2);
        float ss = s2.x + s2.y;
#pragma unroll
        for (int o = kTpr / 2; o; o >>= 1) ss += __shfl_xor_sync(group, ss, o);
        const float n = rsqrtf(fmaf(ss, 1.f / D, a.eps));
        const float2 n2 = make_float2(n, n);
        const float* w = s_w[is_q ? 0 : 1];
#pragma unroll
        for (int e = 0; e < kVec / 2; ++e) {
          x2[0][e] = mul2(x2[0][e], mul2(n2, *reinterpret_cast<const float2*>(w + ca * kVec + 2 * e)));
          x2[1][e] = mul2(x2[1][e], mul2(n2, *reinterpret_cast<const float2*>(w + cb * kVec + 2 * e)));
        }
      }
      if (split) {  // pairs (ca + e, cb + e)
#pragma unroll
        for (int e = 0; e < kVec / 2; ++e) {
          const float2 c = *reinterpret_cast<const float2*>(&s_cos[t][ca * kVec + 2 * e]);
          const float2 s = *reinterpret_cast<const float2*>(&s_sin[t][ca * kVec + 2 * e]);
          const float2 lo = x2[0][e], hi = x2[1][e];
          x2[0][e] = fma2(lo, c, mul2(hi, make_float2(-s.x, -s.y)));
          x2[1][e] = fma2(hi, c, mul2(lo, s));
        }
      } else if (!a.half) {  // adjacent pairs
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const int p0 = (v ? cb : ca) * (kVec / 2);
#pragma unroll
          for (int e = 0; e < kVec / 2; ++e)
            if (p0 + e < a.pairs) {
              const float c = s_cos[t][p0 + e], s = s_sin[t][p0 + e];
              const float lo = x[v][2 * e], hi = x[v][2 * e + 1];
              x[v][2 * e] = lo * c - hi * s;
              x[v][2 * e + 1] = lo * s + hi * c;
            }
        }
      }
      ya = repack(x[0]);
      yb = repack(x[1]);
    }
    *reinterpret_cast<uint4*>(dst + ca * kVec) = ya;
    *reinterpret_cast<uint4*>(dst + cb * kVec) = yb;
  }
}

template <typename T, int D>
static cudaError_t launch_rows_of(const RowsArgs& a, cudaStream_t s) {
  constexpr int kPass = kRowThreads / (D * int(sizeof(T)) / 32);
  const int n_rows = a.nq + a.nk + a.nv;
  // Many tokens: four per CTA, which share one search of their places and one
  // round of cosines.  Few tokens: one pass of rows per CTA, for latency.
  if (a.tokens >= 4 * 2 * num_sms())
    return launch_kernel(rows_kernel<T, D, 4>, dim3(unsigned((a.tokens + 3) / 4)), dim3(kRowThreads), 0,
                         s, false, a, n_rows);
  const int slices = (n_rows + kPass - 1) / kPass;
  return launch_kernel(rows_kernel<T, D, 1>, dim3(unsigned(a.tokens), unsigned(slices)),
                       dim3(kRowThreads), 0, s, false, a, kPass);
}

cudaError_t launch_rows(const RowsArgs& a, bool bf16, int D, cudaStream_t s) {
  if (a.tokens == 0 || a.nq + a.nk + a.nv == 0) return cudaSuccess;
  if (bf16) return D == 128 ? launch_rows_of<__nv_bfloat16, 128>(a, s) : launch_rows_of<__nv_bfloat16, 64>(a, s);
  return D == 128 ? launch_rows_of<float, 128>(a, s) : launch_rows_of<float, 64>(a, s);
}

}  // namespace fkv
