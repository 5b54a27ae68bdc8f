// Pieces shared by the two fp32 kernels of the paged cache: asynchronous copies
// of 32-key blocks, with the pages of a block looked up one step ahead.
#pragma once

#include "paged_common.cuh"

namespace fkv {

constexpr int kF32Threads = 128;
constexpr int kF32Keys = 1 << 5;

// 16-byte asynchronous copies; read == false fills with zeros and reads nothing.
__device__ __forceinline__ void cp_async16(float* dst, const void* src, bool read) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src), "r"(read ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The rows that a thread copies of a step: 16 bytes at column `col` of rows
// row0, row0 + kPass, ...
template <int D>
struct Rows {
  static constexpr int kChunks = D / 4;                 // 16-byte chunks per row
  static constexpr int kPass = kF32Threads / kChunks;   // rows per pass
  static constexpr int kCount = kF32Keys / kPass;
};

// Table entries of the pages that hold this thread's rows of step i of a unit,
// fetched one step ahead of their use (-1: the row is not wanted).
template <int D>
__device__ __forceinline__ void fetch_pages(const PagedArgs& a, const Walk& w, int i,
                                            int (&ids)[Rows<D>::kCount], unsigned& want) {
  const int block = block_at(w.t, w.first + i) * kF32Keys;
  const int k0 = block + int(threadIdx.x) / Rows<D>::kChunks;
  const int32_t* table = a.page_table + int64_t(w.b) * a.table_stride;
  const bool one = (1 << a.page_shift) >= kF32Keys;  // the block lies in one page
  int id = -1;
  if (one && block < w.s.kv) id = table[block >> a.page_shift];
  want = 0;
#pragma unroll
  for (int p = 0; p < Rows<D>::kCount; ++p) {
    const int j = k0 + p * Rows<D>::kPass;
    const bool read = j < w.s.kv && (j < w.s.pre || (j >= w.t.lo && j <= w.t.hi));
    ids[p] = -1;
    if (read) {
      ids[p] = one ? id : table[j >> a.page_shift];
      want |= 1u << p;
    }
  }
}

// Starts the copies of step i of a unit: K chunk c of row r to k_to(r, c), V chunk
// to v_to(r, c) (16-byte chunks); rows that are not wanted, or lie in a bad page
// (reported), are filled with zeros.
template <int D, class KTo, class VTo>
__device__ __forceinline__ void load_keys(const PagedArgs& a, const Walk& w, int i,
                                          const int (&ids)[Rows<D>::kCount], unsigned want,
                                          KTo&& k_to, VTo&& v_to) {
  constexpr int kPass = Rows<D>::kPass;
  const int row0 = int(threadIdx.x) / Rows<D>::kChunks, c = int(threadIdx.x) % Rows<D>::kChunks;
  const int k0 = block_at(w.t, w.first + i) * kF32Keys + row0;
  const int64_t head = int64_t(w.hm / a.mt) * a.head_stride + c * 4;
  const float* kc = static_cast<const float*>(a.k_cache) + head;
  const float* vc = static_cast<const float*>(a.v_cache) + head;
  const float* none = static_cast<const float*>(a.q);  // an address to name when nothing is read
#pragma unroll
  for (int p = 0; p < Rows<D>::kCount; ++p) {
    const int r = row0 + p * kPass, j = k0 + p * kPass, id = ids[p];
    const bool read = id >= 0 && id < a.num_pages;
    if (!read && (want >> p & 1u)) report(a.status, FKV_ERR_DEVICE_ARG, w.b);
    const int64_t off =
        int64_t(id) * a.page_stride + int64_t(j & ((1 << a.page_shift) - 1)) * a.row_stride;
    cp_async16(k_to(r, c), read ? kc + off : none, read);
    cp_async16(v_to(r, c), read ? vc + off : none, read);
  }
}

}  // namespace fkv
