// Shared by the operators around the scan (causal_conv.cu, selective_scan*.cu,
// gated_norm.cu, clip_grad.cu) and their entry points (layer_api.cu).
#pragma once

#include "ssd_internal.cuh"
#include "ssd_layer.h"

namespace ssd {

// A [batch, seqlen, channels] view of element type T, channels dense.
template <typename T>
struct SeqView {
  T *p;
  int64_t bs, ts;
  __device__ __forceinline__ T *at(int64_t b, int64_t t) const { return p + b * bs + t * ts; }
};
template <typename T>
inline SeqView<T> view_of(const ssd_seq *s) {
  return s ? SeqView<T>{static_cast<T *>(s->data), s->batch_stride, s->token_stride}
           : SeqView<T>{nullptr, 0, 0};
}

// Whether base and strides allow loads of `bytes` bytes along the channels.
inline bool view_aligned(const ssd_seq *s, size_t elem, size_t bytes) {
  if (!s || !s->data) return true;
  return ((reinterpret_cast<uintptr_t>(s->data) | (uintptr_t)(s->batch_stride * (int64_t)elem) |
           (uintptr_t)(s->token_stride * (int64_t)elem)) & (bytes - 1)) == 0;
}
inline bool ptr_aligned(const void *p, size_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

// V consecutive elements as fp32; V = 1 needs no alignment, else V elements'.
template <int V, typename T>
__device__ __forceinline__ void load_vec(const T *p, float (&v)[V]) {
  if constexpr (V == 1) {
    v[0] = ld_io(p);
  } else if constexpr (V == 2 && sizeof(T) == 4) {
    const float2 f = *reinterpret_cast<const float2 *>(p);
    v[0] = f.x, v[1] = f.y;
  } else if constexpr (V == 2) {
    const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
    v[0] = __uint_as_float(w << 16), v[1] = __uint_as_float(w & 0xffff0000u);
  } else if constexpr (sizeof(T) == 4) {
    static_assert(V % 4 == 0, "");
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 f = *reinterpret_cast<const float4 *>(p + i);
      v[i] = f.x, v[i + 1] = f.y, v[i + 2] = f.z, v[i + 3] = f.w;
    }
  } else {
    static_assert(V == 4 || V == 8, "");
    uint32_t w[V / 2];
    if constexpr (V == 8) {
      const uint4 u = *reinterpret_cast<const uint4 *>(p);
      w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    } else {
      const uint2 u = *reinterpret_cast<const uint2 *>(p);
      w[0] = u.x, w[1] = u.y;
    }
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {  // a bf16 is the upper half of its fp32
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}
template <int V, typename T>
__device__ __forceinline__ void store_vec(T *p, const float (&v)[V]) {
  if constexpr (V == 1) {
    st_io(p, v[0]);
  } else if constexpr (V == 2 && sizeof(T) == 4) {
    *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
  } else if constexpr (V == 2) {
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(v[0], v[1]);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V; i += 4)
      *reinterpret_cast<float4 *>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else {
    uint32_t w[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    if constexpr (V == 8)
      *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else
      *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
  }
}

// Asynchronous copies of 16, 8 or 4 bytes to shared memory.
__device__ __forceinline__ void copy4(void *dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy8(void *dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void copies_issued() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All groups but the newest `left` have landed.
template <int left>
__device__ __forceinline__ void copies_landed() {
  asm volatile("cp.async.wait_group %0;" ::"n"(left) : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 1 / (1 + exp(-v)): exact limits at both ends (0 and 1); a few ulp between.
__device__ __forceinline__ float sigmoid(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2(-kLog2e * v)));
  return r;
}
__device__ __forceinline__ float silu(float v) { return v * sigmoid(v); }
// d silu(v) / dv = sig (1 + v (1 - sig))
__device__ __forceinline__ float dsilu(float v) {
  const float s = sigmoid(v);
  return s * fmaf(v, 1.f - s, 1.f);
}

// Tokens of sequence b: lengths[b] clamped to [0, L], or L.
__device__ __forceinline__ int64_t tokens_of(const int32_t *lengths, int64_t b, int64_t L) {
  if (!lengths) return L;
  const int64_t n = lengths[b];
  return n < 0 ? 0 : n > L ? L : n;
}

// Column sums of up to four partial arrays in one launch, rows added in a
// fixed order: dst[i] = sum_{r < rows} src[r * n + i].
struct ColSum {
  struct Seg {
    const float *src;
    float *dst;
    int64_t rows, n;
  } seg[4];
  int nseg;
};
cudaError_t launch_colsum(const ColSum &a, int *err, cudaStream_t st);

// Validated arguments of each operator, as the entry points received them.
struct ConvArgs {
  int64_t b, L, D;
  int W, silu;
  const ssd_seq *x, *gy, *y, *dx;
  const float *weight, *bias;
  const void *state, *gfinal;
  const int32_t *lengths;
  void *final_state, *dstate;
  float *dweight, *dbias;
};
cudaError_t launch_causal_conv(const ConvArgs &a, ssd_dtype io, int *err, cudaStream_t st);
cudaError_t launch_causal_conv_step(const ConvArgs &a, ssd_dtype io, int *err, cudaStream_t st);
size_t causal_conv_backward_workspace(const ConvArgs &a, ssd_dtype io);
cudaError_t launch_causal_conv_backward(const ConvArgs &a, ssd_dtype io, void *ws, int *err,
                                        cudaStream_t st);

struct ScanArgs {
  int64_t b, L, D, N, G;
  int softplus;
  const ssd_seq *u, *dt, *B, *C, *z, *y, *gy;
  const float *A, *Dskip, *dt_bias, *h0, *gfinal;
  const int32_t *lengths;
  float *final_state;
  const ssd_scan_grads *out;
};
size_t selective_scan_workspace(const ScanArgs &a, ssd_dtype io);
cudaError_t launch_selective_scan(const ScanArgs &a, ssd_dtype io, void *ws, int *err,
                                  cudaStream_t st);
// final_state holds the state, read and written in place
cudaError_t launch_selective_scan_step(const ScanArgs &a, ssd_dtype io, int *err,
                                       cudaStream_t st);
size_t selective_scan_backward_workspace(const ScanArgs &a, ssd_dtype io);
cudaError_t launch_selective_scan_backward(const ScanArgs &a, ssd_dtype io, void *ws, int *err,
                                           cudaStream_t st);

struct NormArgs {
  int64_t b, L, D, G;
  float eps;
  int gate, center;
  const ssd_seq *x, *z, *y, *gy, *dx, *dz;
  const float *weight, *bias;
  float *dweight, *dbias;
};
cudaError_t launch_gated_norm(const NormArgs &a, ssd_dtype io, int *err, cudaStream_t st);
size_t gated_norm_backward_workspace(const NormArgs &a, ssd_dtype io);
cudaError_t launch_gated_norm_backward(const NormArgs &a, ssd_dtype io, void *ws, int *err,
                                       cudaStream_t st);

size_t clip_grad_workspace(const ssd_grad *grads, int n);
cudaError_t launch_clip_grad(const ssd_grad *grads, int n, float max_norm, float eps, float *norm,
                             void *ws, int *err, cudaStream_t st);

}  // namespace ssd
