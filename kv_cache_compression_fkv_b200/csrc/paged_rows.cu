// Per-head RMS norm and rotation of query and key rows, and the append of keys
// and values to a paged cache, in one pass over the rows.
//
//   y = x / sqrt(mean(x^2) + eps) * w
//   (y_a, y_b) -> (y_a cos - y_b sin, y_a sin + y_b cos) for the pairs (a, b)
//
// Bound by memory: every row is read and written once, in 16-byte vectors.  The
// angles depend on the token alone, so a warp takes one token and a run of its
// rows, evaluates the token's cosines once and keeps them, and the weights, in
// registers; a CTA of two such warps shares nothing.  Angles: omega * position is
// formed and reduced to a fraction of a turn in fp64 (fp32 would lose 1e-2 radians
// at position 10^5), the sine and cosine of the fraction in fp32.
//
// Measured: 14002 prompt tokens of 32 + 8 + 8 heads, 344 MB, 69 us on the GPU = 0.76 of
// the copy bandwidth, 71 a call (ncu: 23% of the warps resident, 2.1 instructions a
// cycle); a 480P chunk, 57.5 MB, 15 us on the GPU with a cold L2, 16.5 a call, of which
// the launch and the first loads take 5.  Slower or
// equal: CTAs over four tokens with the cosines in shared memory (19 / 76 us; its
// reads met in the banks), the rows staged by asynchronous copies (18 / 73), more
// resident warps by fewer registers (21 / 82: spills).
#include "paged_common.cuh"

namespace fkv {

constexpr int kRowThreads = 64;

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

// One new token of an append: where its key and value go.
struct Place {
  int64_t page_off;  // element offset of its cache row (head 0); -1: dropped
  int pos;           // cache position
  int live;          // 0: a padded row
};

// Reports bad offsets and lengths, of sequences without a token too: the warp of
// token t looks after sequences t, t + tokens, ...
__device__ __forceinline__ void check_seqs(const RowsArgs& a, int t, int lane) {
  const int cap = a.max_pages << a.page_shift;
  for (int64_t b = t + int64_t(lane) * a.tokens; b < a.B; b += int64_t(32) * a.tokens) {
    const int kv = a.kv_len[b];
    bool bad = kv < 0 || kv > cap;
    if (a.cu_q) {
      const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1];
      bad |= q0 < 0 || q1 < q0 || q1 > a.tokens;
    }
    if (bad) report(a.status, FKV_ERR_DEVICE_ARG, int(b));
  }
}

// First sequence with good offsets around token t, by a scan; -1: none.  Only for
// tokens whose search among bad offsets went astray.
__device__ __noinline__ int scan_seq(const int32_t* cu_q, int B, int tokens, int t, int lane) {
  for (int b0 = 0; b0 < B; b0 += 32) {
    const int b = b0 + lane;
    const bool in = b < B && cu_q[b] >= 0 && cu_q[b] <= t && t < cu_q[b + 1] && cu_q[b + 1] <= tokens;
    const unsigned found = __ballot_sync(0xffffffffu, in);
    if (found) return b0 + __ffs(found) - 1;
  }
  return -1;
}

__device__ __forceinline__ Place find_place(const RowsArgs& a, int t, int lane) {
  Place p = {-1, 0, 0};
  int b = t, i = 0, q_len = 1;
  if (a.cu_q) {
    b = find_seq(a.cu_q, a.B, t, lane);
    int q0 = a.cu_q[b], q1 = a.cu_q[b + 1];
    if (t < q0 || t >= q1 || q0 < 0 || q1 > a.tokens) {
      // behind the last offset (a padded row), or the offsets are not ascending
      if (b == a.B - 1 && q0 >= 0 && q0 <= q1 && q1 <= t) return p;
      b = scan_seq(a.cu_q, a.B, a.tokens, t, lane);
      if (b < 0) return p;
      q0 = a.cu_q[b];
      q1 = a.cu_q[b + 1];
    }
    i = t - q0;
    q_len = q1 - q0;
  }
  p.live = 1;
  const int cap = a.max_pages << a.page_shift;
  int kv = a.kv_len[b];
  kv = kv < 0 ? 0 : (kv > cap ? cap : kv);
  p.pos = kv - q_len + i;
  int id = -1;
  if (p.pos >= 0) id = a.page_table[int64_t(b) * a.table_stride + (p.pos >> a.page_shift)];
  if (id >= 0 && id < a.num_pages)
    p.page_off = int64_t(id) * a.page_stride + int64_t(p.pos & ((1 << a.page_shift) - 1)) * a.row_stride;
  else if (lane == 0)
    report(a.status, FKV_ERR_DEVICE_ARG, b);
  return p;
}

// A warp takes one token and a run of its rows: the place, the cosines (two
// pairs a lane) and the weights are then the warp's own, held in registers over
// its rows, and no warp waits for another.  Half as many threads as a row has
// vectors share it; with half-split pairs a thread holds both halves of its pairs
// (dims i .. and n + i ..), so the turn needs no exchange.
template <typename T, int D>
struct RowTurn {
  static constexpr int kVec = 16 / int(sizeof(T));  // elements per vector
  static constexpr int kTpr = D / kVec / 2;         // threads per row
  static constexpr int kStep = 32 / kTpr;           // rows per step of the warp
  int da, db;       // first dims of this thread's two vectors
  bool split;       // its pairs are (da + e, db + e)
  int adjacent;     // its adjacent pairs that turn: bit e
  float2 cs[kVec];  // (cosine, sine) of its pairs
  float2 w[kVec];   // weights of da .., db ..

  __device__ __forceinline__ void weights(const float* src) {
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      const int d = (e < kVec / 2 ? da : db) + 2 * (e % (kVec / 2));
      w[e] = src ? make_float2(src[d], src[d + 1]) : make_float2(1.f, 1.f);
    }
  }
  __device__ __forceinline__ void row(uint4 (&y)[2], bool norm, float eps, unsigned group) const {
    float x[2][kVec];
    unpack(y[0], x[0]);
    unpack(y[1], x[1]);
    if (norm) {
      float2(&x2)[kVec] = reinterpret_cast<float2(&)[kVec]>(x);
      float2 s2 = mul2(x2[0], x2[0]);
#pragma unroll
      for (int e = 1; e < kVec; ++e) s2 = fma2(x2[e], x2[e], s2);
      float ss = s2.x + s2.y;
#pragma unroll
      for (int o = kTpr / 2; o; o >>= 1) ss += __shfl_xor_sync(group, ss, o);
      const float n = rsqrtf(fmaf(ss, 1.f / D, eps));
#pragma unroll
      for (int e = 0; e < kVec; ++e) x2[e] = mul2(x2[e], mul2(make_float2(n, n), w[e]));
    }
    if (split) {
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const float lo = x[0][e], hi = x[1][e];
        x[0][e] = lo * cs[e].x - hi * cs[e].y;
        x[1][e] = lo * cs[e].y + hi * cs[e].x;
      }
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e)
        if (adjacent & (1 << e)) {
          float& lo = x[e / (kVec / 2)][2 * (e % (kVec / 2))];
          float& hi = x[e / (kVec / 2)][2 * (e % (kVec / 2)) + 1];
          const float l = lo, h = hi;
          lo = l * cs[e].x - h * cs[e].y;
          hi = l * cs[e].y + h * cs[e].x;
        }
    }
    y[0] = repack(x[0]);
    y[1] = repack(x[1]);
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(kRowThreads) rows_kernel(const RowsArgs a, int run_rows) {
  using R = RowTurn<T, D>;
  constexpr int kVec = R::kVec, kStep = R::kStep, kTpr = R::kTpr;
  __shared__ float2 s_cs[kRowThreads / 32][D / 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = int(blockIdx.x) * (kRowThreads / 32) + warp;
  if (t >= a.tokens) return;
  const int first = int(blockIdx.y) * run_rows, end = first + run_rows;
  const int i = lane % kTpr;
  const int half_chunks = a.half ? a.pairs / kVec : 0;
  R turn;
  turn.split = i < half_chunks;
  turn.da = (turn.split ? i : 2 * i) * kVec;
  turn.db = (turn.split ? i + half_chunks : 2 * i + 1) * kVec;
  turn.adjacent = 0;
  Place place = {-1, 0, 1};
  if (a.append) {
    if (blockIdx.y == 0) check_seqs(a, t, lane);
    place = find_place(a, t, lane);
    if (!place.live) return;
  }
  if (first < a.nq + a.nk && a.pairs > 0) {
    for (int j = lane; j < a.pairs; j += 32) {
      const int axis = (j >= a.axis1) + (j >= a.axis2);
      const int p = a.positions ? a.positions[axis * a.axis_stride + t] : place.pos;
      const double turns = double(p) * (double(a.omega[j]) * 0.15915494309189535);
      float2 r;
      sincospif(2.f * float(turns - rint(turns)), &r.y, &r.x);
      s_cs[warp][j] = r;
    }
    __syncwarp();
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      const int j = a.half ? turn.da + e : ((e < kVec / 2 ? turn.da : turn.db) >> 1) + e % (kVec / 2);
      turn.cs[e] = j < a.pairs ? s_cs[warp][j] : make_float2(1.f, 0.f);
      if (!a.half && j < a.pairs) turn.adjacent |= 1 << e;
    }
  }
  const unsigned group = ((kTpr == 32 ? 0u : 1u << kTpr) - 1u) << (lane & ~(kTpr - 1));
  // Rows [from, to) of one array, two steps of loads in flight.
  auto pass = [&](const T* src, int64_t src_hs, T* dst, int64_t dst_hs, int from, int to, bool rotate) {
    int r = from + lane / kTpr;
    src += int64_t(r) * src_hs;
    dst += int64_t(r) * dst_hs;
    const int64_t src_step = kStep * src_hs, dst_step = kStep * dst_hs;
    uint4 raw[2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (r + u * kStep < to) {
        raw[u][0] = __ldcs(reinterpret_cast<const uint4*>(src + turn.da));
        raw[u][1] = __ldcs(reinterpret_cast<const uint4*>(src + turn.db));
      }
      src += src_step;
    }
    while (r < to) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (r >= to) break;  // the threads of a row leave together
        uint4 y[2] = {raw[u][0], raw[u][1]};
        if (r + 2 * kStep < to) {
          raw[u][0] = __ldcs(reinterpret_cast<const uint4*>(src + turn.da));
          raw[u][1] = __ldcs(reinterpret_cast<const uint4*>(src + turn.db));
        }
        if (rotate) turn.row(y, a.norm, a.eps, group);
        *reinterpret_cast<uint4*>(dst + turn.da) = y[0];
        *reinterpret_cast<uint4*>(dst + turn.db) = y[1];
        r += kStep;
        src += src_step;
        dst += dst_step;
      }
    }
  };
  if (first < a.nq) {
    if (a.norm) turn.weights(a.q_weight);
    pass(static_cast<const T*>(a.q) + int64_t(t) * a.q_ts, a.q_hs,
         static_cast<T*>(a.q_out) + int64_t(t) * a.qo_ts, a.qo_hs, first, min(end, a.nq), true);
  }
  if (a.append && place.page_off < 0) return;
  const int k0 = max(first - a.nq, 0), k1 = min(end - a.nq, a.nk);
  if (k0 < k1) {
    if (a.norm) turn.weights(a.k_weight);
    T* dst = a.append ? static_cast<T*>(a.k_cache) + place.page_off
                      : static_cast<T*>(a.k_out) + int64_t(t) * a.ko_ts;
    pass(static_cast<const T*>(a.k) + int64_t(t) * a.k_ts, a.k_hs, dst,
         a.append ? a.head_stride : a.ko_hs, k0, k1, true);
  }
  const int v0 = max(first - a.nq - a.nk, 0), v1 = min(end - a.nq - a.nk, a.nv);
  if (v0 < v1)
    pass(static_cast<const T*>(a.v) + int64_t(t) * a.v_ts, a.v_hs,
         static_cast<T*>(a.v_cache) + place.page_off, a.head_stride, v0, v1, false);
}

template <typename T, int D>
static cudaError_t launch_rows_of(const RowsArgs& a, cudaStream_t s) {
  constexpr int kStep = 32 / (D * int(sizeof(T)) / 32);
  constexpr int kWarps = kRowThreads / 32;
  const int n_rows = a.nq + a.nk + a.nv;
  // Runs as long as the token's rows, or shorter where there are few tokens, down
  // to one step each, so that about 16 warps per SM share the rows.
  const int64_t want = int64_t(16) * num_sms();
  int64_t runs = (want + a.tokens - 1) / a.tokens;
  const int64_t most = (n_rows + kStep - 1) / kStep;
  if (runs > most) runs = most;
  int run_rows = int((n_rows + runs - 1) / runs);
  run_rows = (run_rows + kStep - 1) / kStep * kStep;
  runs = (n_rows + run_rows - 1) / run_rows;
  const dim3 grid(unsigned((a.tokens + kWarps - 1) / kWarps), unsigned(runs));
  return launch_kernel(rows_kernel<T, D>, grid, dim3(kRowThreads), 0, s, false, a, run_rows);
}

cudaError_t launch_rows(const RowsArgs& a, bool bf16, int D, cudaStream_t s) {
  if (a.tokens == 0 || a.nq + a.nk + a.nv == 0) return cudaSuccess;
  if (bf16) return D == 128 ? launch_rows_of<__nv_bfloat16, 128>(a, s) : launch_rows_of<__nv_bfloat16, 64>(a, s);
  return D == 128 ? launch_rows_of<float, 128>(a, s) : launch_rows_of<float, 64>(a, s);
}

}  // namespace fkv
