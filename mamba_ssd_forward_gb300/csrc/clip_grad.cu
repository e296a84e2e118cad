// Global gradient norm over many tensors, and clipping:
//   norm = sqrt(sum of every g^2),   dst = src min(1, max_norm / (norm + eps))
//
// Two bandwidth passes over the tensors in chunks of equal size: the sums of
// squares, one partial sum a block, and the scaling, whose blocks first add the
// partial sums, all in the same order.  The tensors' addresses travel as kernel
// parameters, kTensors to a launch, so no table is copied to the device.  The
// second pass walks backwards and stores past the cache, so it finds the end
// of what the first one read in L2 (129 MB).  Measured: 80 million fp32
// elements, 322 MB read and written, 152 us (the scaling alone
// 94 us, 6.8 TB/s).
#include <cmath>

#include "layer.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 512;
constexpr int kPerSm = 3;      // blocks
constexpr int kTensors = 96;   // tensors per launch
constexpr int kUnroll = 4;     // vectors of 16 bytes a thread has in flight

struct Table {
  const void *src[kTensors];
  void *dst[kTensors];
  int64_t n[kTensors];
  int first[kTensors + 1];  // first chunk of each tensor, within the launch
  unsigned char bf16[kTensors], wide[kTensors];  // wide: src and dst on 16 bytes
  int count, chunk;                              // chunk: bytes
};

__device__ __forceinline__ int tensor_of(const Table &t, int chunk) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.first[mid] <= chunk) lo = mid; else hi = mid - 1;
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

// 16 bytes as they are in memory, and an element of them.
__device__ __forceinline__ float element(const uint4 &q, int e, float) {
  const uint32_t w = e == 0 ? q.x : e == 1 ? q.y : e == 2 ? q.z : q.w;
  return __uint_as_float(w);
}
__device__ __forceinline__ float element(const uint4 &q, int e, __nv_bfloat16) {
  const uint32_t w = e / 2 == 0 ? q.x : e / 2 == 1 ? q.y : e / 2 == 2 ? q.z : q.w;
  return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
}

template <typename IO>
__device__ __forceinline__ float squares(const IO *p, int n, bool wide) {
  constexpr int V = 16 / (int)sizeof(IO);
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  int done = 0;
  if (wide) {
    const int nv = n / V;
    done = nv * V;
    for (int i = threadIdx.x; i < nv; i += kThreads * kUnroll) {
      uint4 q[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        q[k] = make_uint4(0, 0, 0, 0);
        if (i + k * kThreads < nv)
          q[k] = *reinterpret_cast<const uint4 *>(p + (i + k * kThreads) * V);
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float v = element(q[k], e, IO(0.f));
          s[e % 4] = fmaf(v, v, s[e % 4]);
        }
    }
  }
#pragma unroll 8
  for (int i = done + threadIdx.x; i < n; i += kThreads) {
    const float v = ld_io(p + i);
    s[0] = fmaf(v, v, s[0]);
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

__device__ __forceinline__ void store_past(float *p, const float (&v)[4]) {
  __stcs(reinterpret_cast<float4 *>(p), make_float4(v[0], v[1], v[2], v[3]));
}
__device__ __forceinline__ void store_past(__nv_bfloat16 *p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
}

__global__ void __launch_bounds__(kThreads, kPerSm)
squares_kernel(const __grid_constant__ Table t, float *__restrict__ part, int *err) {
  __shared__ float scratch[kThreads / 32];
  float s = 0.f;
  for (int c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
    const int k = tensor_of(t, c);
    const int64_t per = t.chunk / (t.bf16[k] ? 2 : 4), at = (c - t.first[k]) * per;
    if (!SSD_IN_BOUNDS(at >= 0 && at < t.n[k], err, 50)) continue;
    const int n = (int)(t.n[k] - at < per ? t.n[k] - at : per);
    s += t.bf16[k] ? squares(static_cast<const __nv_bfloat16 *>(t.src[k]) + at, n, t.wide[k])
                   : squares(static_cast<const float *>(t.src[k]) + at, n, t.wide[k]);
  }
  const float total = block_total(s, scratch);
  if (threadIdx.x == 0) part[blockIdx.x] = total;
}

// The factor from the partial sums of every launch, `parts` of them, added in
// the same order by every block.
struct Scale {
  const float *part;
  int parts;
  float max_norm, eps;
  float *norm;  // written by the first launch's first block
};
__device__ __forceinline__ float factor_of(const Scale &sc, float *scratch) {
  float s = 0.f;
  for (int i = threadIdx.x; i < sc.parts; i += kThreads) s += sc.part[i];
  const float root = sqrtf(block_total(s, scratch));
  if (sc.norm && blockIdx.x == 0 && threadIdx.x == 0) *sc.norm = root;
  const float k = sc.max_norm / (root + sc.eps);
  return k > 1.f ? 1.f : k;  // a NaN stays one
}

// One chunk of kUnroll vectors a thread, loaded before the factor is known.
// src and dst may be the same: a thread has read what it writes.
template <typename IO>
__device__ __forceinline__ void scale(const IO *src, IO *dst, int n, bool wide, const Scale &sc,
                                      float *scratch) {
  constexpr int V = 16 / (int)sizeof(IO);
  const int nv = wide ? n / V : 0;
  uint4 q[kUnroll];
#pragma unroll
  for (int k = 0; k < kUnroll; ++k)
    if (threadIdx.x + k * kThreads < nv)
      q[k] = *reinterpret_cast<const uint4 *>(src + (threadIdx.x + k * kThreads) * V);
  const float f = factor_of(sc, scratch);
#pragma unroll
  for (int k = 0; k < kUnroll; ++k)
    if (threadIdx.x + k * kThreads < nv) {
      float v[V];
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = element(q[k], e, IO(0.f)) * f;
      store_past(dst + (threadIdx.x + k * kThreads) * V, v);
    }
#pragma unroll 8
  for (int i = nv * V + threadIdx.x; i < n; i += kThreads) st_io(dst + i, ld_io(src + i) * f);
}

__global__ void __launch_bounds__(kThreads, kPerSm)
scale_kernel(const __grid_constant__ Table t, const __grid_constant__ Scale sc, int *err) {
  __shared__ float scratch[kThreads / 32];
  if (t.count == 0) {
    factor_of(sc, scratch);
    return;
  }
  const int c = (int)(gridDim.x - 1 - blockIdx.x), j = tensor_of(t, c);
  const int64_t per = t.chunk / (t.bf16[j] ? 2 : 4), at = (c - t.first[j]) * per;
  if (!SSD_IN_BOUNDS(at >= 0 && at < t.n[j], err, 51)) return;
  const int n = (int)(t.n[j] - at < per ? t.n[j] - at : per);
  if (t.bf16[j])
    scale(static_cast<const __nv_bfloat16 *>(t.src[j]) + at,
          static_cast<__nv_bfloat16 *>(t.dst[j]) + at, n, t.wide[j], sc, scratch);
  else
    scale(static_cast<const float *>(t.src[j]) + at, static_cast<float *>(t.dst[j]) + at, n,
          t.wide[j], sc, scratch);
}

int grid_most() { return sm_count() * kPerSm; }

// Bytes per chunk of the first pass: some four chunks a block, 8 to 128 KB.
int chunk_of(const ssd_grad *g, int n) {
  int64_t total = 0;
  for (int i = 0; i < n; ++i) total += g[i].n * (g[i].dtype == SSD_BF16 ? 2 : 4);
  int chunk = 131072;
  while (chunk > 8192 && total / chunk < 4 * (int64_t)grid_most()) chunk /= 2;
  return chunk;
}
constexpr int kScaleChunk = kThreads * kUnroll * 16;  // of the second

// Calls f(table, chunks) for each launch's worth of tensors; a tensor whose
// chunks would overflow a launch's count is cut.
template <typename F>
cudaError_t for_each_table(const ssd_grad *g, int n, int chunk, F f) {
  constexpr int64_t kMost = 1 << 30;  // chunks per launch
  Table t{};
  t.chunk = chunk;
  int64_t chunks = 0;
  cudaError_t e = cudaSuccess;
  auto flush = [&]() {
    if (t.count == 0 || e != cudaSuccess) return;
    t.first[t.count] = (int)chunks;
    e = f(t, (int)chunks);
    t.count = 0;
    chunks = 0;
  };
  for (int i = 0; i < n; ++i) {
    const bool bf = g[i].dtype == SSD_BF16;
    const size_t es = bf ? 2 : 4;
    for (int64_t at = 0; at < g[i].n;) {
      if (t.count == kTensors || chunks == kMost) flush();
      const int64_t per = chunk / (int64_t)es, room = (kMost - chunks) * per;
      const int64_t take = g[i].n - at < room ? g[i].n - at : room;
      t.src[t.count] = static_cast<const char *>(g[i].src) + at * es;
      t.dst[t.count] = static_cast<char *>(g[i].dst) + at * es;
      t.n[t.count] = take;
      t.bf16[t.count] = bf;
      t.wide[t.count] = ptr_aligned(t.src[t.count], 16) && ptr_aligned(t.dst[t.count], 16);
      t.first[t.count++] = (int)chunks;
      chunks += (take + per - 1) / per;
      at += take;
    }
  }
  flush();
  return e;
}

}  // namespace

// A launch of the first pass has at most grid_most() partial sums.  Every
// kTensors tensors end a launch, and so may 2^30 chunks of 2^11 elements.
size_t clip_grad_workspace(const ssd_grad *g, int n) {
  int64_t launches = (n + kTensors - 1) / kTensors + 1;
  for (int i = 0; i < n; ++i) launches += g[i].n >> 41;
  return sizeof(float) * (size_t)(launches * grid_most());
}

cudaError_t launch_clip_grad(const ssd_grad *g, int n, float max_norm, float eps, float *norm,
                             void *ws, int *err, cudaStream_t st) {
  float *part = static_cast<float *>(ws);
  Scale sc{part, 0, max_norm, eps, norm};
  const cudaError_t e = for_each_table(g, n, chunk_of(g, n), [&](const Table &t, int chunks) {
    const int blocks = chunks < grid_most() ? chunks : grid_most();
    squares_kernel<<<blocks, kThreads, 0, st>>>(t, part + sc.parts, err);
    sc.parts += blocks;
    return cudaGetLastError();
  });
  if (e != cudaSuccess) return e;
  if (sc.parts == 0) {  // nothing to scale: the norm of no elements is zero
    scale_kernel<<<1, kThreads, 0, st>>>(Table{}, sc, err);
    return cudaGetLastError();
  }
  return for_each_table(g, n, kScaleChunk, [&](const Table &t, int chunks) {
    scale_kernel<<<chunks, kThreads, 0, st>>>(t, sc, err);
    sc.norm = nullptr;
    return cudaGetLastError();
  });
}

}  // namespace ssd
