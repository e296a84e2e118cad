// Short causal convolution along the tokens, per channel, with SiLU:
//   v_t = bias + sum_{k<W} w_k x_{t-W+1+k},   y_t = silu(v_t)
// where the W - 1 tokens before the first are the rows of a state.
//
// A bandwidth kernel: x read once, y written once; 2W + 4 operations per
// element.  A thread takes V neighbouring channels and a run of tokens, with
// the last W - 1 inputs in registers, so x is read once but for the W - 1
// tokens in front of each run (which the neighbouring run brought into L2).
#include <type_traits>

#include "layer.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;  // rows loaded before the arithmetic of the first

template <int V>
__device__ __forceinline__ void zero(float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = 0.f;
}

// The convolution's parameters of channels c .. c + V - 1.
template <int W, int V>
struct Taps {
  float w[W][V], bias[V];
  __device__ __forceinline__ void load(const float *weight, const float *b, int64_t c, int64_t D,
                                       int *err) {
    if (!SSD_IN_BOUNDS(c + V <= D, err, 30)) return;
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
      for (int k = 0; k < W; ++k) w[k][i] = weight[(c + i) * W + k];
      bias[i] = b ? b[c + i] : 0.f;
    }
  }
};

// Row p of the inputs, p in [-(W-1), len): a row of the state below zero.
template <int W, int V, typename IO>
__device__ __forceinline__ void input_row(const SeqView<const IO> &x, const IO *state, int64_t b,
                                          int64_t p, int64_t c, int64_t D, int64_t L, int *err,
                                          float (&v)[V]) {
  zero(v);
  if (!SSD_IN_BOUNDS(p >= -(W - 1) && p < L && c + V <= D, err, 31)) return;
  if (p >= 0)
    load_vec<V>(x.at(b, p) + c, v);
  else if (state)
    load_vec<V>(state + (b * (W - 1) + (p + W - 1)) * D + c, v);
}

template <typename IO, int W, int V>
__global__ void __launch_bounds__(kThreads)
conv_kernel(SeqView<const IO> x, const float *__restrict__ weight, const float *__restrict__ bias,
            const IO *__restrict__ state, const int32_t *__restrict__ lengths, SeqView<IO> y,
            IO *__restrict__ final_state, int64_t L, int64_t D, int run, bool act, int *err) {
  const int64_t nv = D / V;
  const int64_t idx = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t c = idx % nv * V;
  const int64_t t0 = idx / nv * run;
  const int64_t b = blockIdx.y;
  if (t0 >= L) return;
  const int64_t len = tokens_of(lengths, b, L);
  const int64_t t1 = t0 + run < L ? t0 + run : L;
  const int64_t te = t1 < len ? t1 : len;
  if (t0 < te) {
    Taps<W, V> p;
    p.load(weight, bias, c, D, err);
    float win[W - 1][V];
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      input_row<W, V>(x, state, b, t0 - (W - 1) + j, c, D, L, err, win[j]);
    for (int64_t t = t0; t < te; t += kAhead) {
      float in[kAhead][V];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (t + u < te) input_row<W, V>(x, state, b, t + u, c, D, L, err, in[u]);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (t + u >= te) break;
        float out[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float v = p.bias[i];
#pragma unroll
          for (int k = 0; k < W - 1; ++k) v = fmaf(p.w[k][i], win[k][i], v);
          v = fmaf(p.w[W - 1][i], in[u][i], v);
          out[i] = act ? silu(v) : v;
#pragma unroll
          for (int k = 0; k < W - 2; ++k) win[k][i] = win[k + 1][i];
          win[W - 2][i] = in[u][i];
        }
        if (SSD_IN_BOUNDS(t + u >= 0 && t + u < L, err, 32)) store_vec<V>(y.at(b, t + u) + c, out);
      }
    }
  }
  float none[V];
  zero(none);
  for (int64_t t = te > t0 ? te : t0; t < t1; ++t) store_vec<V>(y.at(b, t) + c, none);
  if (t0 == 0 && final_state) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      float v[V];
      input_row<W, V>(x, state, b, len - (W - 1) + j, c, D, L, err, v);
      store_vec<V>(final_state + (b * (W - 1) + j) * D + c, v);
    }
  }
}

template <typename IO, int W, int V>
__global__ void __launch_bounds__(kThreads)
conv_step_kernel(SeqView<const IO> x, const float *__restrict__ weight,
                 const float *__restrict__ bias, IO *__restrict__ state, SeqView<IO> y, int64_t nb,
                 int64_t D, bool act, int *err) {
  const int64_t nv = D / V;
  const int64_t idx = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t c = idx % nv * V, b = idx / nv;
  if (b >= nb) return;
  if (!SSD_IN_BOUNDS(c + V <= D, err, 33)) return;
  float win[W][V], out[V];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) load_vec<V>(state + (b * (W - 1) + j) * D + c, win[j]);
  load_vec<V>(x.at(b, 0) + c, win[W - 1]);
  Taps<W, V> p;
  p.load(weight, bias, c, D, err);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float v = p.bias[i];
#pragma unroll
    for (int k = 0; k < W; ++k) v = fmaf(p.w[k][i], win[k][i], v);
    out[i] = act ? silu(v) : v;
  }
  store_vec<V>(y.at(b, 0) + c, out);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) store_vec<V>(state + (b * (W - 1) + j) * D + c, win[j + 1]);
}

// Backward.  With g_t = gy_t silu'(v_t) (v recomputed from the window),
//   dx_p = sum_k w_k g_{p+W-1-k},  dw_k = sum_t g_t x_{t-W+1+k},  dbias = sum_t g_t,
// dx at p < 0 being the state's gradient.  A block is 32 channel vectors by
// kRuns runs of tokens; a thread walks its run and the W - 1 tokens after it
// (whose g its last dx need), holding the W pending dx and the sums of dw and
// dbias in registers.  The block adds its runs' sums in order and writes one
// partial row; a column sum finishes.  x and gy read once, dx written once.
constexpr int kRuns = 8;

template <typename IO, int W, int V>
__global__ void __launch_bounds__(32 * kRuns)
conv_bwd_kernel(SeqView<const IO> x, const float *__restrict__ weight,
                const float *__restrict__ bias, const IO *__restrict__ state,
                SeqView<const IO> gy, const IO *__restrict__ gfinal,
                const int32_t *__restrict__ lengths, SeqView<IO> dx, IO *__restrict__ dstate,
                float *__restrict__ part_w, float *__restrict__ part_b, int64_t L, int64_t D,
                int run, bool act, int *err) {
  __shared__ float sums[kRuns][32 * V * (W + 1)];
  const int lane = threadIdx.x % 32, slot = threadIdx.x / 32;
  const int64_t c = ((int64_t)blockIdx.x * 32 + lane) * V;
  const int64_t b = blockIdx.z;
  const int64_t t0 = ((int64_t)blockIdx.y * kRuns + slot) * run;
  const int64_t len = tokens_of(lengths, b, L);
  float dw[W][V], db[V];
#pragma unroll
  for (int k = 0; k < W; ++k) zero(dw[k]);
  zero(db);
  if (c < D && t0 < L) {
    Taps<W, V> p;
    p.load(weight, bias, c, D, err);
    const int64_t t1 = t0 + run < L ? t0 + run : L;
    const int64_t p0 = t0 == 0 ? -(W - 1) : t0;  // the first run owns the state's rows too
    float win[W - 1][V], pend[W][V];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      zero(win[j]);
      if (t0 < len) input_row<W, V>(x, state, b, t0 - (W - 1) + j, c, D, L, err, win[j]);
    }
#pragma unroll
    for (int k = 0; k < W; ++k) zero(pend[k]);
    for (int64_t t = t0; t < t1 + W - 1; ++t) {
      if (t < len) {
        float in[V], g[V];
        input_row<W, V>(x, state, b, t, c, D, L, err, in);
        zero(g);
        if (SSD_IN_BOUNDS(t >= 0 && t < L, err, 34)) load_vec<V>(gy.at(b, t) + c, g);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float v = p.bias[i];
#pragma unroll
          for (int k = 0; k < W - 1; ++k) v = fmaf(p.w[k][i], win[k][i], v);
          v = fmaf(p.w[W - 1][i], in[i], v);
          if (act) g[i] *= dsilu(v);
#pragma unroll
          for (int k = 0; k < W; ++k) pend[k][i] = fmaf(p.w[k][i], g[i], pend[k][i]);
          if (t < t1) {
#pragma unroll
            for (int k = 0; k < W - 1; ++k) dw[k][i] = fmaf(g[i], win[k][i], dw[k][i]);
            dw[W - 1][i] = fmaf(g[i], in[i], dw[W - 1][i]);
            db[i] += g[i];
          }
#pragma unroll
          for (int k = 0; k < W - 2; ++k) win[k][i] = win[k + 1][i];
          win[W - 2][i] = in[i];
        }
      }
      const int64_t q = t - (W - 1);  // complete now
      if (q >= p0 && q < t1) {
        if (gfinal && q < len && q >= len - (W - 1)) {
          float f[V];
          load_vec<V>(gfinal + (b * (W - 1) + (q - len + W - 1)) * D + c, f);
#pragma unroll
          for (int i = 0; i < V; ++i) pend[0][i] += f[i];
        }
        if (q >= 0) {
          if (dx.p) store_vec<V>(dx.at(b, q) + c, pend[0]);
        } else if (dstate) {
          store_vec<V>(dstate + (b * (W - 1) + (q + W - 1)) * D + c, pend[0]);
        }
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k) pend[k][i] = pend[k + 1][i];
        pend[W - 1][i] = 0.f;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int k = 0; k < W; ++k) sums[slot][(lane * V + i) * W + k] = dw[k][i];
    sums[slot][32 * V * W + lane * V + i] = db[i];
  }
  __syncthreads();
  const int64_t row = b * gridDim.y + blockIdx.y;
  const int64_t c0 = (int64_t)blockIdx.x * 32 * V;
  for (int j = threadIdx.x; j < 32 * V * (W + 1); j += 32 * kRuns) {
    float s = sums[0][j];
#pragma unroll
    for (int r = 1; r < kRuns; ++r) s += sums[r][j];
    if (j < 32 * V * W) {
      const int64_t k = c0 * W + j;
      if (k < D * W) part_w[row * D * W + k] = s;
    } else {
      const int64_t k = c0 + (j - 32 * V * W);
      if (k < D) part_b[row * D + k] = s;
    }
  }
}

template <typename T>
struct tag {
  using type = T;
};

// (I/O type, width, channels per thread): vectors of 4 channels where every
// row starts on a vector boundary, else single channels.
template <typename F>
cudaError_t dispatch(ssd_dtype io, int W, bool vec, F f) {
  auto by_vec = [&](auto io_c, auto w_c) {
    return vec ? f(io_c, w_c, std::integral_constant<int, 4>{})
               : f(io_c, w_c, std::integral_constant<int, 1>{});
  };
  auto by_w = [&](auto io_c) {
    if (W == 2) return by_vec(io_c, std::integral_constant<int, 2>{});
    if (W == 3) return by_vec(io_c, std::integral_constant<int, 3>{});
    return by_vec(io_c, std::integral_constant<int, 4>{});
  };
  return io == SSD_BF16 ? by_w(tag<__nv_bfloat16>{}) : by_w(tag<float>{});
}

bool vectored(const ConvArgs &a, ssd_dtype io) {
  const size_t e = io == SSD_BF16 ? 2 : 4, bytes = 4 * e;
  return a.D % 4 == 0 && view_aligned(a.x, e, bytes) && view_aligned(a.y, e, bytes) &&
         view_aligned(a.gy, e, bytes) && view_aligned(a.dx, e, bytes) &&
         ptr_aligned(a.state, bytes) && ptr_aligned(a.gfinal, bytes) &&
         ptr_aligned(a.final_state, bytes) && ptr_aligned(a.dstate, bytes);
}

// Tokens per run of the backward: short runs when long ones would leave SMs
// idle, longer ones where the grid's second dimension would overflow.
int bwd_run(const ConvArgs &a) {
  const int64_t run = a.b * a.L * a.D >= (int64_t)1 << 22 ? 32 : 8;
  const int64_t least = (a.L + 65535 * kRuns - 1) / (65535 * kRuns);
  return (int)(run > least ? run : least);
}
int64_t bwd_rows(const ConvArgs &a) {
  const int64_t per = (int64_t)bwd_run(a) * kRuns;
  return (a.L + per - 1) / per;
}

}  // namespace

cudaError_t launch_causal_conv(const ConvArgs &a, ssd_dtype io, int *err, cudaStream_t st) {
  const bool vec = vectored(a, io);
  return dispatch(io, a.W, vec, [&](auto io_c, auto w_c, auto v_c) {
    using IO = typename decltype(io_c)::type;
    constexpr int V = decltype(v_c)::value;
    const int run = 16;
    const int64_t items = (a.D / V) * ((a.L + run - 1) / run);
    const dim3 grid((unsigned)((items + kThreads - 1) / kThreads), (unsigned)a.b);
    conv_kernel<IO, decltype(w_c)::value, V><<<grid, kThreads, 0, st>>>(
        view_of<const IO>(a.x), a.weight, a.bias, static_cast<const IO *>(a.state), a.lengths,
        view_of<IO>(a.y), static_cast<IO *>(a.final_state), a.L, a.D, run, a.silu, err);
    return cudaGetLastError();
  });
}

cudaError_t launch_causal_conv_step(const ConvArgs &a, ssd_dtype io, int *err, cudaStream_t st) {
  const bool vec = vectored(a, io);
  return dispatch(io, a.W, vec, [&](auto io_c, auto w_c, auto v_c) {
    using IO = typename decltype(io_c)::type;
    constexpr int V = decltype(v_c)::value;
    const int64_t items = a.b * (a.D / V);
    conv_step_kernel<IO, decltype(w_c)::value, V>
        <<<(unsigned)((items + kThreads - 1) / kThreads), kThreads, 0, st>>>(
            view_of<const IO>(a.x), a.weight, a.bias, static_cast<IO *>(a.final_state),
            view_of<IO>(a.y), a.b, a.D, a.silu, err);
    return cudaGetLastError();
  });
}

size_t causal_conv_backward_workspace(const ConvArgs &a, ssd_dtype) {
  return sizeof(float) * (size_t)(a.b * bwd_rows(a) * a.D * (a.W + 1));
}

cudaError_t launch_causal_conv_backward(const ConvArgs &a, ssd_dtype io, void *ws, int *err,
                                        cudaStream_t st) {
  const bool vec = vectored(a, io);
  const int64_t rows = a.b * bwd_rows(a);
  float *part_w = static_cast<float *>(ws), *part_b = part_w + rows * a.D * a.W;
  const cudaError_t e = dispatch(io, a.W, vec, [&](auto io_c, auto w_c, auto v_c) {
    using IO = typename decltype(io_c)::type;
    constexpr int V = decltype(v_c)::value;
    const dim3 grid((unsigned)((a.D + 32 * V - 1) / (32 * V)), (unsigned)bwd_rows(a),
                    (unsigned)a.b);
    conv_bwd_kernel<IO, decltype(w_c)::value, V><<<grid, 32 * kRuns, 0, st>>>(
        view_of<const IO>(a.x), a.weight, a.bias, static_cast<const IO *>(a.state),
        view_of<const IO>(a.gy), static_cast<const IO *>(a.gfinal), a.lengths,
        view_of<IO>(a.dx), static_cast<IO *>(a.dstate), part_w, part_b, a.L, a.D, bwd_run(a),
        a.silu, err);
    return cudaGetLastError();
  });
  if (e != cudaSuccess) return e;
  ColSum s{};
  s.nseg = 2;
  s.seg[0] = {part_w, a.dweight, rows, a.D * a.W};
  s.seg[1] = {part_b, a.dbias, rows, a.D};
  return launch_colsum(s, err, st);
}

}  // namespace ssd
