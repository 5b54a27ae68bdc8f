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

constexpr int kRowUnroll = 4;  // vectors that a thread has in flight

// grid (tokens, slices of rows_per_cta rows); rows_per_cta * D / vector <=
// kRowUnroll * blockDim.x, so every load of the CTA is issued before the
// token's place and cosines are worked out.
template <typename T, int D>
__global__ void __launch_bounds__(kRowThreads) rows_kernel(const RowsArgs a, int rows_per_cta) {
  constexpr int kVec = 16 / int(sizeof(T));  // elements per vector
  constexpr int kLanes = D / kVec;           // lanes per row
  __shared__ float2 cs[D / 2];
  const int t = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31;
  const int c = tid % kLanes, d0 = c * kVec;
  const int pass = blockDim.x / kLanes;      // rows per pass of the CTA
  const int n_rows = a.nq + a.nk + a.nv;
  const int row0 = int(blockIdx.y) * rows_per_cta + tid / kLanes;
  const int row1 = min(int(blockIdx.y + 1) * rows_per_cta, n_rows);
  uint4 raw[kRowUnroll];
#pragma unroll
  for (int u = 0; u < kRowUnroll; ++u) {
    const int row = row0 + u * pass;
    if (row < row1) {
      const T* src;
      if (row < a.nq) src = static_cast<const T*>(a.q) + int64_t(t) * a.q_ts + int64_t(row) * a.q_hs;
      else if (row < a.nq + a.nk)
        src = static_cast<const T*>(a.k) + int64_t(t) * a.k_ts + int64_t(row - a.nq) * a.k_hs;
      else
        src = static_cast<const T*>(a.v) + int64_t(t) * a.v_ts + int64_t(row - a.nq - a.nk) * a.v_hs;
      raw[u] = __ldcs(reinterpret_cast<const uint4*>(src + d0));
    }
  }
  float wq[kVec], wk[kVec];
#pragma unroll
  for (int u = 0; u < kVec; ++u) wq[u] = wk[u] = 1.f;
  if (a.norm) {
#pragma unroll
    for (int u = 0; u < kVec; ++u) {
      if (a.q_weight) wq[u] = a.q_weight[d0 + u];
      if (a.k_weight) wk[u] = a.k_weight[d0 + u];
    }
  }
  int64_t page_off = -1;  // element offset of the token's cache row (head 0)
  int pos = 0;
  if (a.append) {
    int b = t, i = 0, q_len = 1;
    if (a.cu_q) {
      b = find_seq(a.cu_q, a.B, t, lane);
      const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1];
      if (q0 < 0 || q1 < q0 || q1 > a.tokens) {
        if (tid == 0) report(a.status, FKV_ERR_DEVICE_ARG, b);
        return;
      }
      i = t - q0;
      q_len = q1 - q0;
      if (i < 0 || i >= q_len) return;  // a padded row
    }
    const int cap = a.max_pages << a.page_shift;
    int kv = a.kv_len[b];
    if (kv < 0 || kv > cap) {
      if (tid == 0) report(a.status, FKV_ERR_DEVICE_ARG, b);
      kv = kv < 0 ? 0 : cap;
    }
    pos = kv - q_len + i;
    int id = -1;
    if (pos >= 0) id = a.page_table[int64_t(b) * a.table_stride + (pos >> a.page_shift)];
    if (id >= 0 && id < a.num_pages)
      page_off = int64_t(id) * a.page_stride +
                 int64_t(pos & ((1 << a.page_shift) - 1)) * a.row_stride;
    else if (tid == 0)
      report(a.status, FKV_ERR_DEVICE_ARG, b);
  }
  for (int i = tid; i < a.pairs; i += blockDim.x) {
    const int axis = (i >= a.axis1) + (i >= a.axis2);
    const int p = a.positions ? a.positions[axis * a.axis_stride + t] : pos;
    const double turns = double(p) * (double(a.omega[i]) * 0.15915494309189535);
    float sn, cn;
    sincospif(2.f * float(turns - rint(turns)), &sn, &cn);
    cs[i] = make_float2(cn, sn);
  }
  __syncthreads();
  const unsigned group = kLanes == 32 ? 0xffffffffu : ((1u << kLanes) - 1u) << (lane & ~(kLanes - 1));
#pragma unroll
  for (int u = 0; u < kRowUnroll; ++u) {
    const int row = row0 + u * pass;
    if (row >= row1) break;  // the lanes of a row leave together
    const bool is_q = row < a.nq, is_v = row >= a.nq + a.nk;
    T* dst;
    if (is_q) dst = static_cast<T*>(a.q_out) + int64_t(t) * a.qo_ts + int64_t(row) * a.qo_hs;
    else if (!a.append) dst = static_cast<T*>(a.k_out) + int64_t(t) * a.ko_ts + int64_t(row - a.nq) * a.ko_hs;
    else {
      if (page_off < 0) continue;
      dst = is_v ? static_cast<T*>(a.v_cache) + page_off + int64_t(row - a.nq - a.nk) * a.head_stride
                 : static_cast<T*>(a.k_cache) + page_off + int64_t(row - a.nq) * a.head_stride;
    }
    if (is_v) {
      *reinterpret_cast<uint4*>(dst + d0) = raw[u];
      continue;
    }
    float x[kVec];
    unpack(raw[u], x);
    if (a.norm) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < kVec; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
      for (int o = kLanes / 2; o; o >>= 1) ss += __shfl_xor_sync(group, ss, o);
      const float r = rsqrtf(fmaf(ss, 1.f / D, a.eps));
#pragma unroll
      for (int e = 0; e < kVec; ++e) x[e] *= r * (is_q ? wq[e] : wk[e]);
    }
    if (a.half) {
      // dims below n pair with dims n further (n a multiple of the vector)
      const bool lo = d0 < a.pairs, turn = d0 < 2 * a.pairs;
      const int other = (c + (lo ? 1 : -1) * (a.pairs / kVec)) & (kLanes - 1);
      float y[kVec];
#pragma unroll
      for (int e = 0; e < kVec; ++e)
        y[e] = __shfl_sync(group, x[e], (lane & ~(kLanes - 1)) | other);
      if (turn) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          const float2 r = cs[(lo ? d0 : d0 - a.pairs) + e];
          x[e] = lo ? x[e] * r.x - y[e] * r.y : y[e] * r.y + x[e] * r.x;
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < kVec; e += 2) {
        const int i = (d0 + e) >> 1;
        if (i < a.pairs) {
          const float2 r = cs[i];
          const float x0 = x[e], x1 = x[e + 1];
          x[e] = x0 * r.x - x1 * r.y;
          x[e + 1] = x0 * r.y + x1 * r.x;
        }
      }
    }
    *reinterpret_cast<uint4*>(dst + d0) = repack(x);
  }
}

cudaError_t launch_rows(const RowsArgs& a, bool bf16, int D, cudaStream_t s) {
  const int n_rows = a.nq + a.nk + a.nv;
  if (a.tokens == 0 || n_rows == 0) return cudaSuccess;
  const int lanes = D * (bf16 ? 2 : 4) / 16;
  const int most = kRowUnroll * kRowThreads / lanes;  // rows that one CTA takes
  const int slices = (n_rows + most - 1) / most;
  const int rows_per_cta = (n_rows + slices - 1) / slices;
  // 128 threads where they hold the rows in flight: more CTAs per SM, and fewer
  // threads that wait for the token's cosines
  const int threads = rows_per_cta * lanes <= kRowUnroll * 128 ? 128 : kRowThreads;
  const dim3 grid(unsigned(a.tokens), unsigned(slices));
  auto* k = bf16 ? (D == 128 ? rows_kernel<__nv_bfloat16, 128> : rows_kernel<__nv_bfloat16, 64>)
                 : (D == 128 ? rows_kernel<float, 128> : rows_kernel<float, 64>);
  return launch_kernel(k, grid, dim3(unsigned(threads)), 0, s, false, a, rows_per_cta);
}

}  // namespace fkv
