// Group norm per token with a SiLU gate, channels last.  Over each group of
// D / G channels of a token:
//   r = x silu(z) or x;  r -= mean(r) (centred);  n = r / sqrt(mean(r^2) + eps)
//   v = n weight + bias;  y = v silu(z) or v
//
// A bandwidth kernel: x and z read once, y written once.  The product x silu(z)
// is rounded by itself (no fused multiply-add with the mean), so r - mean(r)
// is exactly zero where all of a group's r are equal.
#include <type_traits>

#include "layer.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Sum of v over the block, in every thread; a fixed order.
__device__ __forceinline__ float block_sum(float v, float *scratch) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if (threadIdx.x % 32 == 0) scratch[threadIdx.x / 32] = v;
  __syncthreads();
  float s = scratch[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) s += scratch[w];
  __syncthreads();
  return s;
}

template <typename IO, int V>
__global__ void __launch_bounds__(kThreads)
norm_kernel(SeqView<const IO> x, const float *__restrict__ weight, const float *__restrict__ bias,
            SeqView<const IO> z, SeqView<IO> y, int64_t L, int group, float eps, int gate,
            bool center, int64_t nb, int *err) {
  __shared__ float scratch[kWarps];
  const int64_t b = blockIdx.x / L, t = blockIdx.x % L;
  const int64_t c0 = (int64_t)blockIdx.y * group;
  if (!SSD_IN_BOUNDS(b < nb && t < L, err, 40)) return;
  const IO *xr = x.at(b, t) + c0;
  const IO *zr = gate ? z.at(b, t) + c0 : nullptr;
  IO *yr = y.at(b, t) + c0;
  auto value = [&](int i, float (&r)[V]) {
    load_vec<V>(xr + i, r);
    if (gate == SSD_GATE_INPUT) {
      float g[V];
      load_vec<V>(zr + i, g);
#pragma unroll
      for (int k = 0; k < V; ++k) r[k] = __fmul_rn(r[k], silu(g[k]));
    }
  };
  float mean = 0.f, r[V];
  if (center) {
    float s = 0.f;
    for (int i = threadIdx.x * V; i < group; i += kThreads * V) {
      value(i, r);
#pragma unroll
      for (int k = 0; k < V; ++k) s += r[k];
    }
    mean = block_sum(s, scratch) / (float)group;
  }
  float s = 0.f;
  for (int i = threadIdx.x * V; i < group; i += kThreads * V) {
    value(i, r);
#pragma unroll
    for (int k = 0; k < V; ++k) s = fmaf(r[k] - mean, r[k] - mean, s);
  }
  const float rstd = rsqrtf(block_sum(s, scratch) / (float)group + eps);
  for (int i = threadIdx.x * V; i < group; i += kThreads * V) {
    value(i, r);
    float g[V];
    if (gate == SSD_GATE_OUTPUT) load_vec<V>(zr + i, g);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      float v = (r[k] - mean) * rstd * weight[c0 + i + k];
      if (bias) v += bias[c0 + i + k];
      r[k] = gate == SSD_GATE_OUTPUT ? v * silu(g[k]) : v;
    }
    store_vec<V>(yr + i, r);
  }
}

// What the gradients of one group of one token need.
struct Stat {
  float mean, rstd, qn, q;  // mean(r), 1 / root, mean(q n), mean(q)
};

// r, n and dL/dv of V channels.
template <int V, typename IO>
__device__ __forceinline__ void parts(const IO *xr, const IO *zr, const IO *gr, int64_t i,
                                      int gate, float (&x)[V], float (&z)[V], float (&gy)[V],
                                      float (&r)[V], float (&gv)[V]) {
  load_vec<V>(xr + i, x);
  load_vec<V>(gr + i, gy);
  if (gate) load_vec<V>(zr + i, z);
#pragma unroll
  for (int k = 0; k < V; ++k) {
    r[k] = gate == SSD_GATE_INPUT ? __fmul_rn(x[k], silu(z[k])) : x[k];
    gv[k] = gate == SSD_GATE_OUTPUT ? gy[k] * silu(z[k]) : gy[k];
  }
}

template <typename IO, int V>
__global__ void __launch_bounds__(kThreads)
norm_stat_kernel(SeqView<const IO> x, const float *__restrict__ weight, SeqView<const IO> z,
                 SeqView<const IO> gy, Stat *__restrict__ stat, int64_t L, int group, float eps,
                 int gate, bool center, int64_t nb, int *err) {
  __shared__ float scratch[kWarps];
  const int64_t b = blockIdx.x / L, t = blockIdx.x % L;
  const int64_t c0 = (int64_t)blockIdx.y * group;
  if (!SSD_IN_BOUNDS(b < nb && t < L, err, 41)) return;
  const IO *xr = x.at(b, t) + c0, *gr = gy.at(b, t) + c0;
  const IO *zr = gate ? z.at(b, t) + c0 : nullptr;
  float xv[V], zv[V], gyv[V], r[V], gv[V];
  Stat st{};
  if (center) {
    float s = 0.f;
    for (int i = threadIdx.x * V; i < group; i += kThreads * V) {
      parts<V>(xr, zr, gr, i, gate, xv, zv, gyv, r, gv);
#pragma unroll
      for (int k = 0; k < V; ++k) s += r[k];
    }
    st.mean = block_sum(s, scratch) / (float)group;
  }
  float s = 0.f, qr = 0.f, q = 0.f;
  for (int i = threadIdx.x * V; i < group; i += kThreads * V) {
    parts<V>(xr, zr, gr, i, gate, xv, zv, gyv, r, gv);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const float d = r[k] - st.mean, w = gv[k] * weight[c0 + i + k];
      s = fmaf(d, d, s);
      qr = fmaf(w, d, qr);
      q += w;
    }
  }
  st.rstd = rsqrtf(block_sum(s, scratch) / (float)group + eps);
  st.qn = block_sum(qr, scratch) * st.rstd / (float)group;
  st.q = center ? block_sum(q, scratch) / (float)group : 0.f;
  if (threadIdx.x == 0) stat[(int64_t)blockIdx.x * gridDim.y + blockIdx.y] = st;
}

// A thread owns V columns and walks a slice of the rows, so dweight and dbias
// need no exchange within the slice.
template <typename IO, int V>
__global__ void __launch_bounds__(kThreads)
norm_grad_kernel(SeqView<const IO> x, const float *__restrict__ weight,
                 const float *__restrict__ bias, SeqView<const IO> z, SeqView<const IO> gy,
                 const Stat *__restrict__ stat, SeqView<IO> dx, SeqView<IO> dz,
                 float *__restrict__ part_w, float *__restrict__ part_b, int64_t L, int64_t D,
                 int64_t rows, int64_t per, int group, int gate, int *err) {
  const int64_t c = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * V;
  if (c >= D) return;
  if (!SSD_IN_BOUNDS(c + V <= D, err, 42)) return;
  const int64_t r0 = blockIdx.y * per, r1 = r0 + per < rows ? r0 + per : rows;
  const int64_t G = D / group, grp = c / group;
  float w[V], bi[V], dw[V], db[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    w[k] = weight[c + k];
    bi[k] = bias ? bias[c + k] : 0.f;
    dw[k] = db[k] = 0.f;
  }
  for (int64_t row = r0; row < r1; ++row) {
    const int64_t b = row / L, t = row % L;
    const Stat st = stat[row * G + grp];
    float xv[V], zv[V], gyv[V], r[V], gv[V], ox[V], oz[V];
    parts<V>(x.at(b, t), gate ? z.at(b, t) : nullptr, gy.at(b, t), c, gate, xv, zv, gyv, r, gv);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const float n = (r[k] - st.mean) * st.rstd;
      dw[k] = fmaf(gv[k], n, dw[k]);
      db[k] += gv[k];
      const float gr = st.rstd * (gv[k] * w[k] - n * st.qn - st.q);
      ox[k] = gate == SSD_GATE_INPUT ? gr * silu(zv[k]) : gr;
      if (gate)
        oz[k] = (gate == SSD_GATE_INPUT ? gr * xv[k] : gyv[k] * fmaf(n, w[k], bi[k])) *
                dsilu(zv[k]);
    }
    store_vec<V>(dx.at(b, t) + c, ox);
    if (gate) store_vec<V>(dz.at(b, t) + c, oz);
  }
#pragma unroll
  for (int k = 0; k < V; ++k) {
    part_w[blockIdx.y * D + c + k] = dw[k];
    part_b[blockIdx.y * D + c + k] = db[k];
  }
}

template <typename T>
struct tag {
  using type = T;
};
template <typename F>
cudaError_t dispatch(ssd_dtype io, bool vec, F f) {
  auto by_vec = [&](auto io_c) {
    return vec ? f(io_c, std::integral_constant<int, 4>{})
               : f(io_c, std::integral_constant<int, 1>{});
  };
  return io == SSD_BF16 ? by_vec(tag<__nv_bfloat16>{}) : by_vec(tag<float>{});
}

bool vectored(const NormArgs &a, ssd_dtype io) {
  const size_t e = io == SSD_BF16 ? 2 : 4, bytes = 4 * e;
  return (a.D / a.G) % 4 == 0 && view_aligned(a.x, e, bytes) && view_aligned(a.z, e, bytes) &&
         view_aligned(a.y, e, bytes) && view_aligned(a.gy, e, bytes) &&
         view_aligned(a.dx, e, bytes) && view_aligned(a.dz, e, bytes);
}

// Row slices of the gradient kernel and the rows of each.
int64_t slice_rows(const NormArgs &a) {
  const int64_t rows = a.b * a.L;
  const int64_t per = (rows + 255) / 256;
  return per < 4 ? 4 : per;
}
int64_t slices(const NormArgs &a) { return (a.b * a.L + slice_rows(a) - 1) / slice_rows(a); }

}  // namespace

cudaError_t launch_gated_norm(const NormArgs &a, ssd_dtype io, int *err, cudaStream_t st) {
  return dispatch(io, vectored(a, io), [&](auto io_c, auto v_c) {
    using IO = typename decltype(io_c)::type;
    const dim3 grid((unsigned)(a.b * a.L), (unsigned)a.G);
    norm_kernel<IO, decltype(v_c)::value><<<grid, kThreads, 0, st>>>(
        view_of<const IO>(a.x), a.weight, a.bias, view_of<const IO>(a.z), view_of<IO>(a.y), a.L,
        (int)(a.D / a.G), a.eps, a.gate, a.center, a.b, err);
    return cudaGetLastError();
  });
}

size_t gated_norm_backward_workspace(const NormArgs &a, ssd_dtype) {
  return sizeof(Stat) * (size_t)(a.b * a.L * a.G) + 2 * sizeof(float) * (size_t)(slices(a) * a.D);
}

cudaError_t launch_gated_norm_backward(const NormArgs &a, ssd_dtype io, void *ws, int *err,
                                       cudaStream_t st) {
  Stat *stat = static_cast<Stat *>(ws);
  float *part_w = reinterpret_cast<float *>(stat + a.b * a.L * a.G);
  float *part_b = part_w + slices(a) * a.D;
  const cudaError_t e = dispatch(io, vectored(a, io), [&](auto io_c, auto v_c) {
    using IO = typename decltype(io_c)::type;
    constexpr int V = decltype(v_c)::value;
    const int group = (int)(a.D / a.G);
    norm_stat_kernel<IO, V><<<dim3((unsigned)(a.b * a.L), (unsigned)a.G), kThreads, 0, st>>>(
        view_of<const IO>(a.x), a.weight, view_of<const IO>(a.z), view_of<const IO>(a.gy), stat,
        a.L, group, a.eps, a.gate, a.center, a.b, err);
    const cudaError_t e1 = cudaGetLastError();
    if (e1 != cudaSuccess) return e1;
    const dim3 grid((unsigned)((a.D / V + kThreads - 1) / kThreads), (unsigned)slices(a));
    norm_grad_kernel<IO, V><<<grid, kThreads, 0, st>>>(
        view_of<const IO>(a.x), a.weight, a.bias, view_of<const IO>(a.z),
        view_of<const IO>(a.gy), stat, view_of<IO>(a.dx), view_of<IO>(a.dz), part_w, part_b, a.L,
        a.D, a.b * a.L, slice_rows(a), group, a.gate, err);
    return cudaGetLastError();
  });
  if (e != cudaSuccess) return e;
  ColSum s{};
  s.nseg = 2;
  s.seg[0] = {part_w, a.dweight, slices(a), a.D};
  s.seg[1] = {part_b, a.dbias, slices(a), a.D};
  return launch_colsum(s, err, st);
}

}  // namespace ssd
