// The residual's addition and the root-mean-square norm in front of a block:
//   t = x + r,  y = t rstd w,  rstd = 1 / sqrt(mean(t^2) + eps)
// y in the I/O type or in e4m3 with scales, t kept in the residual stream's type.
// Its gradients from t:  n = t rstd,  g = gy w,
//   dt = rstd (g - n mean(g n)) + gt,  dw = sum over tokens of gy n
//
// Bandwidth kernels: everything is read once and written once.  A token belongs
// to a team (a warp, or a block where a warp's registers do not hold the token),
// whose threads keep V consecutive channels a vector, K vectors each, in
// registers between the sum and the output.
#include <cuda_fp8.h>

#include "model.cuh"

namespace ssd {
namespace {

constexpr float kTop8 = 448.f;  // the largest e4m3 value
// The smallest scale: 1 / scale stays finite.
constexpr float kLeastScale = 1.17549435e-38f;

template <typename IO>
constexpr int vec_of() { return sizeof(IO) == 2 ? 8 : 4; }

// V channels from c on of a row of D; the missing ones are zero.
template <int V, typename T>
__device__ __forceinline__ void load_row(const T *p, int c, int D, bool wide, float (&v)[V]) {
  if (wide) {
    load_vec<V>(p + c, v);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = c + e < D ? ld_io(p + c + e) : 0.f;
  }
}
template <int V, typename T>
__device__ __forceinline__ void store_row(T *p, int c, int D, bool wide, const float (&v)[V]) {
  if (wide) {
    store_vec<V>(p + c, v);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (c + e < D) st_io(p + c + e, v[e]);
  }
}
template <int V>
__device__ __forceinline__ void store_e4m3(uint8_t *p, int c, int D, bool wide,
                                           const float (&v)[V]) {
  uint32_t w[V / 4];
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i], v[4 * i + 1]),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2], v[4 * i + 3]),
                                                 __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | hi << 16;
  }
  if (wide) {
    if constexpr (V == 8) *reinterpret_cast<uint2 *>(p + c) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t *>(p + c) = w[0];
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (c + e < D) p[c + e] = (uint8_t)(w[e / 4] >> (8 * (e % 4)));
  }
}

// Sums (or maxima) of M values over a warp or, `warps` > 1, over the block, in
// every thread; a fixed order.  Calls in turn use the halves of `scratch`.
template <int M, bool kMax = false>
__device__ __forceinline__ void team_all(float (&v)[M], float (*scratch)[M][32], int warps,
                                         int turn) {
  auto join = [](float a, float b) { return kMax ? fmaxf(a, b) : a + b; };
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
#pragma unroll
    for (int m = 0; m < M; ++m) v[m] = join(v[m], __shfl_xor_sync(0xffffffffu, v[m], off));
  if (warps == 1) return;
  const int lane = threadIdx.x % 32;
  if (lane == 0)
#pragma unroll
    for (int m = 0; m < M; ++m) scratch[turn][m][threadIdx.x / 32] = v[m];
  __syncthreads();
#pragma unroll
  for (int m = 0; m < M; ++m) v[m] = lane < warps ? scratch[turn][m][lane] : 0.f;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
#pragma unroll
    for (int m = 0; m < M; ++m) v[m] = join(v[m], __shfl_xor_sync(0xffffffffu, v[m], off));
}

struct Quant {
  uint8_t *q;
  int64_t bs, ts;  // of q
  float *scales;
  int block, parts;  // channels to a scale (0: the token), scales to a token
};

template <typename IO, typename ST, int K, bool kQuant>
__global__ void __launch_bounds__(1024)
add_norm_kernel(SeqView<const IO> x, SeqView<const ST> residual, const float *__restrict__ weight,
                SeqView<IO> y, SeqView<ST> total, Quant qu, int64_t L, int64_t rows, int D,
                float eps, int warps, bool wide, int *err) {
  constexpr int V = vec_of<IO>();
  __shared__ float scratch[2][1][32];
  const int team = 32 * warps;  // a warp, or the block
  const int64_t row = warps == 1 ? (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32
                                 : blockIdx.x;
  if (row >= rows) return;
  const int tid = warps == 1 ? threadIdx.x % 32 : threadIdx.x;
  const int64_t b = row / L, at = row % L;
  if (!SSD_IN_BOUNDS((int64_t)team * K * V >= D, err, 90)) return;
  const IO *xr = x.at(b, at);
  const ST *rr = residual.p ? residual.at(b, at) : nullptr;
  float t[K][V], s[1] = {0.f};
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (tid + k * team) * V;
    if (c < D) {
      load_row<V>(xr, c, D, wide, t[k]);
      if (rr) {
        float r[V];
        load_row<V>(rr, c, D, wide, r);
#pragma unroll
        for (int e = 0; e < V; ++e) t[k][e] += r[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) t[k][e] = 0.f;
    }
  }
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) s[0] = fmaf(t[k][e], t[k][e], s[0]);
  team_all(s, scratch, warps, 0);
  const float rstd = rsqrtf(s[0] / (float)D + eps);
  float top[1] = {0.f};
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (tid + k * team) * V;
    if (c < D) {
      if (total.p) store_row<V>(total.at(b, at), c, D, wide, t[k]);
      float w[V];
      load_row<V>(weight, c, D, wide, w);
#pragma unroll
      for (int e = 0; e < V; ++e) t[k][e] = t[k][e] * rstd * w[e];
      if constexpr (!kQuant) store_row<V>(y.at(b, at), c, D, wide, t[k]);
    }
    if constexpr (kQuant) {
      if (qu.block == 0) {
#pragma unroll
        for (int e = 0; e < V; ++e) top[0] = fmaxf(top[0], fabsf(t[k][e]));
      }
    }
  }
  if constexpr (kQuant) {
    uint8_t *q = qu.q + b * qu.bs + at * qu.ts;
    float *scales = qu.scales + row * qu.parts;
    if (qu.block == 0) team_all<1, true>(top, scratch, warps, 1);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (tid + k * team) * V;
      float m = top[0];
      if (qu.block) {  // block / V neighbouring lanes hold it
        m = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) m = fmaxf(m, fabsf(t[k][e]));
        for (int off = qu.block / V / 2; off > 0; off >>= 1)
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
      }
      if (c >= D) continue;
      const bool small = m < kTop8 * kLeastScale;
      const float scale = m == 0.f ? 0.f : small ? kLeastScale : m / kTop8;
      const float up = m == 0.f ? 0.f : small ? 1.f / kLeastScale : kTop8 / m;
      float v[V];
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = t[k][e] * up;
      store_e4m3<V>(q, c, D, wide, v);
      if (qu.block ? c % qu.block == 0 : c == 0) scales[qu.block ? c / qu.block : 0] = scale;
    }
  }
}

template <typename IO, typename ST, int K>
__global__ void __launch_bounds__(512)
add_norm_grad_kernel(SeqView<const ST> total, const float *__restrict__ weight,
                     SeqView<const IO> gy, SeqView<const ST> gtotal, SeqView<IO> dx,
                     SeqView<ST> dres, float *__restrict__ part, int64_t L, int64_t rows, int D,
                     float eps, int warps, bool wide, int *err) {
  constexpr int V = vec_of<IO>();
  __shared__ float scratch[2][2][32];
  const int team = 32 * warps, per = warps == 1 ? blockDim.x / 32 : 1;  // teams to a block
  const int64_t first = (int64_t)blockIdx.x * per + (warps == 1 ? threadIdx.x / 32 : 0);
  const int tid = warps == 1 ? threadIdx.x % 32 : threadIdx.x;
  if (!SSD_IN_BOUNDS((int64_t)team * K * V >= D, err, 91)) return;
  float dw[K][V];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) dw[k][e] = 0.f;
  int turn = 0;
  for (int64_t row = first; row < rows; row += (int64_t)gridDim.x * per, turn ^= 1) {
    const int64_t b = row / L, at = row % L;
    float t[K][V], g[K][V], s[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (tid + k * team) * V;
      if (c < D) {
        load_row<V>(total.at(b, at), c, D, wide, t[k]);
        load_row<V>(gy.at(b, at), c, D, wide, g[k]);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) t[k][e] = g[k][e] = 0.f;
      }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (tid + k * team) * V;
      if (c >= D) continue;
      float w[V];
      load_row<V>(weight, c, D, wide, w);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        s[0] = fmaf(t[k][e], t[k][e], s[0]);
        s[1] = fmaf(g[k][e] * w[e], t[k][e], s[1]);
      }
    }
    team_all(s, scratch, warps, turn);
    const float rstd = rsqrtf(s[0] / (float)D + eps), mean = s[1] * rstd / (float)D;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (tid + k * team) * V;
      if (c >= D) continue;
      float w[V], o[V];
      load_row<V>(weight, c, D, wide, w);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float n = t[k][e] * rstd;
        dw[k][e] = fmaf(g[k][e], n, dw[k][e]);
        o[e] = rstd * (g[k][e] * w[e] - n * mean);
      }
      if (gtotal.p) {
        float gt[V];
        load_row<V>(gtotal.at(b, at), c, D, wide, gt);
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] += gt[e];
      }
      if (dx.p) store_row<V>(dx.at(b, at), c, D, wide, o);
      if (dres.p) store_row<V>(dres.at(b, at), c, D, wide, o);
    }
  }
  if (!part) return;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (tid + k * team) * V;
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (c + e < D) part[first * D + c + e] = dw[k][e];
  }
}

// How a token is shared out: vectors to a thread, warps to its team, threads to a
// block.
struct Shares {
  int K, warps, threads;
};
Shares shares_of(int64_t D, int V, int most_threads) {
  const int64_t vecs = (D + V - 1) / V;
  Shares s{1, 1, 128};
  if (vecs <= 32) return s;
  int64_t threads = (vecs + 31) / 32 * 32;
  while (threads > most_threads) {
    s.K *= 2;
    threads = ((vecs + s.K - 1) / s.K + 31) / 32 * 32;
  }
  s.warps = (int)threads / 32, s.threads = (int)threads;
  return s;
}

template <typename F>
cudaError_t with_vectors(int K, F f) {
  switch (K) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 4: return f(std::integral_constant<int, 4>());
    case 8: return f(std::integral_constant<int, 8>());
    case 16: return f(std::integral_constant<int, 16>());
  }
  return cudaErrorInvalidValue;
}

constexpr int kFwdThreads = 512, kGradThreads = 512;

template <typename IO, typename ST>
cudaError_t forward(const AddNormArgs &a, int *err, cudaStream_t st) {
  constexpr int V = vec_of<IO>();
  const Shares s = shares_of(a.D, V, kFwdThreads);
  const int64_t rows = a.b * a.L, per = s.warps == 1 ? s.threads / 32 : 1;
  const bool quant = a.scales != nullptr;
  const bool wide = a.D % V == 0 && ptr_aligned(a.weight, 16) && view_aligned(a.x, sizeof(IO), 16) &&
                    view_aligned(a.residual, sizeof(ST), 16) &&
                    view_aligned(a.total, sizeof(ST), 16) &&
                    (quant ? view_aligned(a.y, 1, V) : view_aligned(a.y, sizeof(IO), 16));
  Quant q{};
  if (quant) {
    q.q = static_cast<uint8_t *>(a.y->data), q.bs = a.y->batch_stride, q.ts = a.y->token_stride;
    q.scales = a.scales, q.block = (int)a.block;
    q.parts = a.block ? (int)((a.D + a.block - 1) / a.block) : 1;
  }
  const unsigned grid = (unsigned)((rows + per - 1) / per);
  return with_vectors(s.K, [&](auto k) {
    constexpr int K = decltype(k)::value;
    if (quant)
      add_norm_kernel<IO, ST, K, true><<<grid, s.threads, 0, st>>>(
          view_of<const IO>(a.x), view_of<const ST>(a.residual), a.weight, SeqView<IO>{},
          view_of<ST>(a.total), q, a.L, rows, (int)a.D, a.eps, s.warps, wide, err);
    else
      add_norm_kernel<IO, ST, K, false><<<grid, s.threads, 0, st>>>(
          view_of<const IO>(a.x), view_of<const ST>(a.residual), a.weight, view_of<IO>(a.y),
          view_of<ST>(a.total), q, a.L, rows, (int)a.D, a.eps, s.warps, wide, err);
    return cudaGetLastError();
  });
}

// Teams that walk the tokens: as many as run at once, each with its share of dw.
int64_t grad_blocks(const AddNormArgs &a, const Shares &s) {
  const int64_t rows = a.b * a.L, per = s.warps == 1 ? s.threads / 32 : 1;
  const int64_t most = (int64_t)sm_count() * (1024 / s.threads);
  const int64_t all = (rows + per - 1) / per;
  return all < most ? all : most;
}

template <typename IO, typename ST>
cudaError_t backward(const AddNormArgs &a, void *ws, int *err, cudaStream_t st) {
  constexpr int V = vec_of<IO>();
  const Shares s = shares_of(a.D, V, kGradThreads);
  const int64_t rows = a.b * a.L, per = s.warps == 1 ? s.threads / 32 : 1;
  const int64_t blocks = grad_blocks(a, s);
  const bool wide = a.D % V == 0 && ptr_aligned(a.weight, 16) &&
                    view_aligned(a.total, sizeof(ST), 16) && view_aligned(a.gy, sizeof(IO), 16) &&
                    view_aligned(a.gtotal, sizeof(ST), 16) && view_aligned(a.dx, sizeof(IO), 16) &&
                    view_aligned(a.dresidual, sizeof(ST), 16);
  float *part = a.dweight ? static_cast<float *>(ws) : nullptr;
  const cudaError_t e = with_vectors(s.K, [&](auto k) {
    constexpr int K = decltype(k)::value;
    add_norm_grad_kernel<IO, ST, K><<<(unsigned)blocks, s.threads, 0, st>>>(
        view_of<const ST>(a.total), a.weight, view_of<const IO>(a.gy),
        view_of<const ST>(a.gtotal), view_of<IO>(a.dx), view_of<ST>(a.dresidual), part, a.L, rows,
        (int)a.D, a.eps, s.warps, wide, err);
    return cudaGetLastError();
  });
  if (e != cudaSuccess || !part) return e;
  ColSum c{};
  c.nseg = 1;
  c.seg[0] = {part, a.dweight, blocks * per, a.D};
  return launch_colsum(c, err, st);
}

}  // namespace

size_t add_norm_backward_workspace(const AddNormArgs &a, ssd_dtype io, ssd_dtype) {
  const Shares s = shares_of(a.D, io == SSD_BF16 ? 8 : 4, kGradThreads);
  const int64_t per = s.warps == 1 ? s.threads / 32 : 1;
  return sizeof(float) * (size_t)(grad_blocks(a, s) * per * a.D);
}
cudaError_t launch_add_norm(const AddNormArgs &a, ssd_dtype io, ssd_dtype stream, int *err,
                            cudaStream_t st) {
  if (io == SSD_F32) return forward<float, float>(a, err, st);
  return stream == SSD_F32 ? forward<__nv_bfloat16, float>(a, err, st)
                           : forward<__nv_bfloat16, __nv_bfloat16>(a, err, st);
}
cudaError_t launch_add_norm_backward(const AddNormArgs &a, ssd_dtype io, ssd_dtype stream, void *ws,
                                     int *err, cudaStream_t st) {
  if (io == SSD_F32) return backward<float, float>(a, ws, err, st);
  return stream == SSD_F32 ? backward<__nv_bfloat16, float>(a, ws, err, st)
                           : backward<__nv_bfloat16, __nv_bfloat16>(a, ws, err, st);
}

}  // namespace ssd
