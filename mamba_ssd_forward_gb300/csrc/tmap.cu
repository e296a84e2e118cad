// TMA tensor-map construction, the library-wide device error word and the
// per-device SM count.
#include <atomic>
#include <mutex>

#include "ssd_internal.cuh"
#include "tmap.cuh"

namespace ssd {

namespace {

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                 const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                 const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_fn() {
  static EncodeTiled fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiled>(p);
  });
  return fn;
}

bool make_tmap(CUtensorMap *map, const void *base, bool bf16, int rank, const uint64_t *dims,
               const uint64_t *strides, const uint32_t *box, CUtensorMapSwizzle swizzle) {
  EncodeTiled fn = encode_fn();
  if (!fn || rank < 1 || rank > 5) return false;
  cuuint64_t gd[5], gs[4];
  cuuint32_t bx[5], es[5];
  for (int i = 0; i < rank; ++i) {
    gd[i] = dims[i];
    bx[i] = box[i];
    es[i] = 1;
  }
  for (int i = 0; i + 1 < rank; ++i) gs[i] = strides[i];
  const CUresult r =
      fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
         (cuuint32_t)rank, const_cast<void *>(base), gd, gs, bx, es,
         CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

}  // namespace

bool make_tmap_sw128(CUtensorMap *map, const void *base, bool bf16, int rank,
                     const uint64_t *dims, const uint64_t *strides, const uint32_t *box) {
  return make_tmap(map, base, bf16, rank, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}
bool make_tmap_sw64(CUtensorMap *map, const void *base, bool bf16, int rank, const uint64_t *dims,
                    const uint64_t *strides, const uint32_t *box) {
  return make_tmap(map, base, bf16, rank, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_64B);
}

// Device error word: kernels that give up a bounded wait record a code here
// when the call has no workspace of its own.
__device__ int g_device_error = 0;

cudaError_t read_and_clear_error(int *word, cudaStream_t st, int *code) {
  int zero = 0;
  cudaError_t e = cudaMemcpyAsync(code, word, sizeof(int), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaMemcpyAsync(word, &zero, sizeof(int), cudaMemcpyHostToDevice, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  return e;
}

int *device_error_word() {
  void *p = nullptr;
  if (cudaGetSymbolAddress(&p, g_device_error) != cudaSuccess) return nullptr;
  return static_cast<int *>(p);
}

int sm_count() {
  constexpr int kMaxDev = 256;
  static std::atomic<int> cache[kMaxDev];  // 0 = not looked up yet
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return 148;
  int n = cache[dev].load(std::memory_order_relaxed);
  if (n > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    n = 148;
  cache[dev].store(n, std::memory_order_relaxed);  // every thread stores the same value
  return n;
}

}  // namespace ssd
