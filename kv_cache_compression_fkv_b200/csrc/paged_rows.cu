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

template <typename T, int D>
__global__ void __launch_bounds__(kRowThreads) rows_kernel(const RowsArgs a, int rows_per_cta) {
  constexpr int kVec = 16 / int(sizeof(T));   // elements per vector
  constexpr int kLanes = D / kVec;            // lanes per row
  constexpr int kPass = kRowThreads / kLanes; // rows per pass of the CTA
  __shared__ float2 cs[D / 2];
  const int t = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31;
  const int n_rows = a.nq + a.nk + a.nv;
  const int row0 = int(blockIdx.y) * rows_per_cta;
  const int row1 = row0 + rows_per_cta < n_rows ? row0 + rows_per_cta : n_rows;
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
    } else if (t >= a.B) {
      return;
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
  for (int i = tid; i < a.pairs; i += kRowThreads) {
    const int axis = (i >= a.axis1) + (i >= a.axis2);
    const int p = a.positions ? a.positions[axis * a.axis_stride + t] : pos;
    const double turns = double(p) * (double(a.omega[i]) * 0.15915494309189535);
    float sn, cn;
    sincospif(2.f * float(turns - rint(turns)), &sn, &cn);
    cs[i] = make_float2(cn, sn);
  }
  __syncthreads();
  const int c = tid % kLanes, d0 = c * kVec;
  const unsigned group = kLanes == 32 ? 0xffffffffu : ((1u << kLanes) - 1u) << (lane & ~(kLanes - 1));
  for (int base = row0; base < row1; base += kPass) {
    const int row = base + tid / kLanes;
    if (row >= row1) break;  // whole row groups leave together
    const bool is_q = row < a.nq, is_v = row >= a.nq + a.nk;
    const int h = is_q ? row : (is_v ? row - a.nq - a.nk : row - a.nq);
    const T* src = is_q ? static_cast<const T*>(a.q) + int64_t(t) * a.q_ts + int64_t(h) * a.q_hs
                 : is_v ? static_cast<const T*>(a.v) + int64_t(t) * a.v_ts + int64_t(h) * a.v_hs
                        : static_cast<const T*>(a.k) + int64_t(t) * a.k_ts + int64_t(h) * a.k_hs;
    T* dst;
    if (is_q) dst = static_cast<T*>(a.q_out) + int64_t(t) * a.qo_ts + int64_t(h) * a.qo_hs;
    else if (!a.append) dst = static_cast<T*>(a.k_out) + int64_t(t) * a.ko_ts + int64_t(h) * a.ko_hs;
    else {
      if (page_off < 0) continue;
      dst = static_cast<T*>(is_v ? a.v_cache : a.k_cache) + page_off + int64_t(h) * a.head_stride;
    }
    uint4 raw = *reinterpret_cast<const uint4*>(src + d0);
    if (!is_v) {
      float x[kVec];
      const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
      for (int u = 0; u < kVec; ++u) x[u] = to_f32(e[u]);
      if (a.norm) {
        float ss = 0.f;
#pragma unroll
        for (int u = 0; u < kVec; ++u) ss = fmaf(x[u], x[u], ss);
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1) ss += __shfl_xor_sync(group, ss, o);
        const float r = 1.f / sqrtf(ss * (1.f / D) + a.eps);
        const float* w = is_q ? a.q_weight : a.k_weight;
#pragma unroll
        for (int u = 0; u < kVec; ++u) x[u] *= r;
        if (w) {
#pragma unroll
          for (int u = 0; u < kVec; ++u) x[u] *= w[d0 + u];
        }
      }
      if (a.half) {
        // dims below n pair with dims n further (n a multiple of the vector)
        const bool lo = d0 < a.pairs, turn = d0 < 2 * a.pairs;
        const int other = (c + (lo ? 1 : -1) * (a.pairs / kVec)) & (kLanes - 1);
        float y[kVec];
#pragma unroll
        for (int u = 0; u < kVec; ++u)
          y[u] = __shfl_sync(group, x[u], (lane & ~(kLanes - 1)) | other);
        if (turn) {
#pragma unroll
          for (int u = 0; u < kVec; ++u) {
            const float2 r = cs[(lo ? d0 : d0 - a.pairs) + u];
            x[u] = lo ? x[u] * r.x - y[u] * r.y : y[u] * r.y + x[u] * r.x;
          }
        }
      } else {
#pragma unroll
        for (int u = 0; u < kVec; u += 2) {
          const int i = (d0 + u) >> 1;
          if (i < a.pairs) {
            const float2 r = cs[i];
            const float x0 = x[u], x1 = x[u + 1];
            x[u] = x0 * r.x - x1 * r.y;
            x[u + 1] = x0 * r.y + x1 * r.x;
          }
        }
      }
      T* z = reinterpret_cast<T*>(&raw);
#pragma unroll
      for (int u = 0; u < kVec; ++u) z[u] = from_f32<T>(x[u]);
    }
    *reinterpret_cast<uint4*>(dst + d0) = raw;
  }
}

cudaError_t launch_rows(const RowsArgs& a, bool bf16, int D, cudaStream_t s) {
  const int n_rows = a.nq + a.nk + a.nv;
  if (a.tokens == 0 || n_rows == 0) return cudaSuccess;
  const int rows_per_cta = n_rows;
  const dim3 grid(unsigned(a.tokens), unsigned((n_rows + rows_per_cta - 1) / rows_per_cta));
  auto* k = bf16 ? (D == 128 ? rows_kernel<__nv_bfloat16, 128> : rows_kernel<__nv_bfloat16, 64>)
                 : (D == 128 ? rows_kernel<float, 128> : rows_kernel<float, 64>);
  return launch_kernel(k, grid, dim3(kRowThreads), 0, s, false, a, rows_per_cta);
}

}  // namespace fkv
