// Global gradient norm over many tensors, and clipping:
//   norm = sqrt(sum of every g^2),   dst = src min(1, max_norm / (norm + eps))
//
// Two bandwidth passes over the same blocks of kBlock elements: the sums of
// squares, one partial per block, and the scaling.  The tensors' addresses
// travel as kernel parameters, kTensors to a launch, so no table is copied to
// the device.  Each scaling block adds the partials itself, in one order.
#include <cmath>

#include "layer.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 512;
constexpr int64_t kBlock = 32768;  // elements of one tensor per thread block
constexpr int kTensors = 96;       // tensors per launch

struct Table {
  const void *src[kTensors];
  void *dst[kTensors];
  int64_t n[kTensors];
  int first[kTensors + 1];  // first block of each tensor, within the launch
  unsigned char bf16[kTensors];
  int count;
};

__device__ __forceinline__ int tensor_of(const Table &t, int blk) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.first[mid] <= blk) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ float block_total(float v, float *scratch) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if (threadIdx.x % 32 == 0) scratch[threadIdx.x / 32] = v;
  __syncthreads();
  float s = scratch[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) s += scratch[w];
  return s;
}

template <typename IO>
__device__ __forceinline__ float squares(const IO *p, int64_t n) {
  float s = 0.f;
  for (int64_t i = threadIdx.x; i < n; i += kThreads) {
    const float v = ld_io(p + i);
    s = fmaf(v, v, s);
  }
  return s;
}

__global__ void __launch_bounds__(kThreads)
squares_kernel(const __grid_constant__ Table t, float *__restrict__ part, int *err) {
  __shared__ float scratch[kThreads / 32];
  const int k = tensor_of(t, blockIdx.x);
  const int64_t at = (int64_t)(blockIdx.x - t.first[k]) * kBlock;
  if (!SSD_IN_BOUNDS(at >= 0 && at < t.n[k], err, 50)) return;
  const int64_t n = t.n[k] - at < kBlock ? t.n[k] - at : kBlock;
  const float s = t.bf16[k] ? squares(static_cast<const __nv_bfloat16 *>(t.src[k]) + at, n)
                            : squares(static_cast<const float *>(t.src[k]) + at, n);
  const float total = block_total(s, scratch);
  if (threadIdx.x == 0) part[blockIdx.x] = total;
}

template <typename IO>
__device__ __forceinline__ void scale(const IO *src, IO *dst, int64_t n, float k) {
  for (int64_t i = threadIdx.x; i < n; i += kThreads) st_io(dst + i, ld_io(src + i) * k);
}

// part: the partials of every launch, `parts` of them
__global__ void __launch_bounds__(kThreads)
scale_kernel(const __grid_constant__ Table t, const float *__restrict__ part, int64_t parts,
             float max_norm, float eps, float *__restrict__ norm, bool write_norm, int *err) {
  __shared__ float scratch[kThreads / 32];
  float s = 0.f;
  for (int64_t i = threadIdx.x; i < parts; i += kThreads) s += part[i];
  const float root = sqrtf(block_total(s, scratch));
  if (write_norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = root;
  if (t.count == 0) return;
  const float k = max_norm / (root + eps);
  const float factor = k > 1.f ? 1.f : k;  // a NaN stays one
  const int j = tensor_of(t, blockIdx.x);
  const int64_t at = (int64_t)(blockIdx.x - t.first[j]) * kBlock;
  if (!SSD_IN_BOUNDS(at >= 0 && at < t.n[j], err, 51)) return;
  const int64_t n = t.n[j] - at < kBlock ? t.n[j] - at : kBlock;
  if (t.bf16[j])
    scale(static_cast<const __nv_bfloat16 *>(t.src[j]) + at,
          static_cast<__nv_bfloat16 *>(t.dst[j]) + at, n, factor);
  else
    scale(static_cast<const float *>(t.src[j]) + at, static_cast<float *>(t.dst[j]) + at, n,
          factor);
}

int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }

// Calls f(table, blocks) for each launch's worth of tensors; a tensor whose
// blocks would overflow a launch's grid is cut.
template <typename F>
cudaError_t for_each_table(const ssd_grad *g, int n, F f) {
  constexpr int64_t kMost = 1 << 20;  // blocks per launch
  Table t{};
  int64_t blocks = 0;
  cudaError_t e = cudaSuccess;
  auto flush = [&]() {
    if (t.count == 0 || e != cudaSuccess) return;
    t.first[t.count] = (int)blocks;
    e = f(t, blocks);
    t.count = 0;
    blocks = 0;
  };
  for (int i = 0; i < n; ++i) {
    const bool bf = g[i].dtype == SSD_BF16;
    const size_t es = bf ? 2 : 4;
    for (int64_t at = 0; at < g[i].n;) {
      if (t.count == kTensors || blocks == kMost) flush();
      const int64_t room = (kMost - blocks) * kBlock;
      const int64_t take = g[i].n - at < room ? g[i].n - at : room;
      t.src[t.count] = static_cast<const char *>(g[i].src) + at * es;
      t.dst[t.count] = static_cast<char *>(g[i].dst) + at * es;
      t.n[t.count] = take;
      t.bf16[t.count] = bf;
      t.first[t.count++] = (int)blocks;
      blocks += blocks_of(take);
      at += take;
    }
  }
  flush();
  return e;
}

int64_t total_blocks(const ssd_grad *g, int n) {
  int64_t blocks = 0;
  for (int i = 0; i < n; ++i) blocks += blocks_of(g[i].n);
  return blocks;
}

}  // namespace

size_t clip_grad_workspace(const ssd_grad *g, int n) {
  return sizeof(float) * (size_t)(total_blocks(g, n) + 1);
}

cudaError_t launch_clip_grad(const ssd_grad *g, int n, float max_norm, float eps, float *norm,
                             void *ws, int *err, cudaStream_t st) {
  float *part = static_cast<float *>(ws);
  const int64_t parts = total_blocks(g, n);
  int64_t at = 0;
  cudaError_t e = for_each_table(g, n, [&](const Table &t, int64_t blocks) {
    squares_kernel<<<(unsigned)blocks, kThreads, 0, st>>>(t, part + at, err);
    at += blocks;
    return cudaGetLastError();
  });
  if (e != cudaSuccess) return e;
  if (parts == 0) {  // nothing to scale: the norm of no elements is zero
    scale_kernel<<<1, kThreads, 0, st>>>(Table{}, part, 0, max_norm, eps, norm, true, err);
    return cudaGetLastError();
  }
  bool first = true;
  return for_each_table(g, n, [&](const Table &t, int64_t blocks) {
    scale_kernel<<<(unsigned)blocks, kThreads, 0, st>>>(t, part, parts, max_norm, eps, norm, first,
                                                       err);
    first = false;
    return cudaGetLastError();
  });
}

}  // namespace ssd
