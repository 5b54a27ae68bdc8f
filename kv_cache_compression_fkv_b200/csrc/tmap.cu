// Host-side creation of TMA tensor maps.  cuTensorMapEncodeTiled is a driver
// function; it is fetched through the runtime's driver entry-point query so
// that the library does not link libcuda and still loads on a machine
// without a GPU driver.
#include <cudaTypedefs.h>

#include <mutex>

#include "fkv_internal.cuh"
#include "paged_common.cuh"
#include "sm100_common.cuh"

namespace fkv {

static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

bool make_tmap_bf16(CUtensorMap* map, const void* base, uint64_t rows, uint64_t slabs,
                    uint64_t row_stride_bytes, uint64_t slab_stride_bytes) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
  if (!fn || !base || rows == 0 || slabs == 0) return false;
  if ((reinterpret_cast<uintptr_t>(base) & 15u) || (row_stride_bytes & 15u) ||
      (slab_stride_bytes & 15u))
    return false;
  cuuint64_t dims[3] = {128, rows, slabs};
  cuuint64_t strides[2] = {row_stride_bytes, slab_stride_bytes};
  cuuint32_t box[3] = {64, 128, 1};
  cuuint32_t elem_strides[3] = {1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides,
                  box, elem_strides, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

bool make_tmap_u8(CUtensorMap* map, const void* base, uint64_t rows, uint64_t slabs,
                  uint64_t row_stride_bytes, uint64_t slab_stride_bytes) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
  if (!fn || !base || rows == 0 || slabs == 0) return false;
  if ((reinterpret_cast<uintptr_t>(base) & 15u) || (row_stride_bytes & 15u) ||
      (slab_stride_bytes & 15u))
    return false;
  cuuint64_t dims[3] = {128, rows, slabs};
  cuuint64_t strides[2] = {row_stride_bytes, slab_stride_bytes};
  cuuint32_t box[3] = {128, 128, 1};
  cuuint32_t elem_strides[3] = {1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides,
                  box, elem_strides, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// Map of bf16 rows in columns of 64, in the 128-byte swizzle.
static bool encode_rows(CUtensorMap* map, const void* base, uint32_t rank, const cuuint64_t* dims,
                        const cuuint64_t* strides, const cuuint32_t* box) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims,
                  strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool paged_tmaps(const PagedArgs& a, int D, int keys, int q_heads, int q_tokens, CUtensorMap* q,
                 CUtensorMap* k, CUtensorMap* v) {
  const cuuint64_t row = cuuint64_t(D) * 2;  // bytes; also the stride of a dimension of one entry
  const cuuint64_t q_dims[3] = {cuuint64_t(D), cuuint64_t(a.Hq), cuuint64_t(a.num_tokens)};
  const cuuint64_t q_strides[2] = {a.Hq > 1 ? cuuint64_t(a.q_hs) * 2 : row,
                                   a.num_tokens > 1 ? cuuint64_t(a.q_ts) * 2 : row};
  const cuuint32_t q_box[3] = {64, cuuint32_t(q_heads), cuuint32_t(q_tokens)};
  if (!encode_rows(q, a.q, 3, q_dims, q_strides, q_box)) return false;
  // A cache without pages gets a map of one page that no copy reads (every page
  // id is then out of range, and reads as the zeros outside the map).
  const bool none = a.num_pages == 0;
  const int rows = 1 << a.page_shift;
  const cuuint64_t dims[4] = {cuuint64_t(D), cuuint64_t(rows), cuuint64_t(a.Hkv),
                              cuuint64_t(none ? 1 : a.num_pages)};
  const cuuint64_t strides[3] = {cuuint64_t(a.row_stride) * 2, cuuint64_t(a.head_stride) * 2,
                                 cuuint64_t(a.page_stride) * 2};
  const cuuint32_t box[4] = {64, cuuint32_t(rows < keys ? rows : keys), 1, 1};
  return encode_rows(k, none ? a.q : a.k_cache, 4, dims, strides, box) &&
         encode_rows(v, none ? a.q : a.v_cache, 4, dims, strides, box);
}

int num_sms() {
  static int cached[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  if (!cached[dev]) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
      n = 148;
    cached[dev] = n;
  }
  return cached[dev];
}

}  // namespace fkv
