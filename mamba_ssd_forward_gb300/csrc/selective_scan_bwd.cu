// Gradients of the selective scan.  With e_t = exp(s_t A), o_t = gy_t silu(z_t)
// and the adjoint state G_t = o_t C_t + e_{t+1} G_{t+1}:
//   du = s sum_n G B + D o          ds = sum_n G (u B + A e h_{t-1})
//   dA = sum_t s G e h_{t-1}        dB = sum_d G s u,   dC = sum_d o h
//   dz = gy (sum_n h C + D u) silu'(z),   ddt = ds softplus'
//
// Three steps: the states at every kSpan-th token; then span by span from the
// end, the states of the span again and the adjoint backwards over it; then
// the sums over channel tiles (dB, dC) and over sequences (dA, dD, ddt_bias).
#include "scan_common.cuh"

namespace ssd {
namespace {

using namespace scan;

constexpr int kThreads = 128;
constexpr int kSpan = 16;

template <typename IO, int NL>
__global__ void __launch_bounds__(kThreads)
states_kernel(In<IO> in, float *__restrict__ states, int64_t spans, int *err) {
  const int64_t ch = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / NL;
  const int n0 = threadIdx.x % NL * 4, N = in.N;
  const int64_t b = blockIdx.y;
  if (ch >= in.D) return;
  const int64_t d = ch, g = d / in.per_group;
  if (!SSD_IN_BOUNDS(b < in.nb, err, 71)) return;
  const int64_t len = tokens_of(in.lengths, b, in.L);
  float A[4], h[4] = {0.f, 0.f, 0.f, 0.f};
  load4_tail(in.A + d * N, n0, N, A);
#pragma unroll
  for (int i = 0; i < 4; ++i) A[i] *= kLog2e;
  if (in.h0) load4_tail(in.h0 + (b * in.D + d) * N, n0, N, h);
  const float bias = in.dt_bias ? in.dt_bias[d] : 0.f;
  for (int64_t t = 0; t < len; ++t) {
    if (t % kSpan == 0)
      store4_tail(states + ((b * spans + t / kSpan) * in.D + d) * N, n0, N, h);
    float B[4];
    load4_tail(in.B.at(b, t) + g * N, n0, N, B);
    const float u = ld_io(in.u.at(b, t) + d);
    const float s = step_of(ld_io(in.dt.at(b, t) + d) + bias, in.softplus);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      h[i] = fmaf(ex2(s * A[i]), h[i], n0 + i < N ? s * u * B[i] : 0.f);
  }
}

template <typename IO>
struct Out {
  SeqView<IO> du, ddt, dz;
  float *partB, *partC;            // [tile, b, L, G, N]
  float *partA, *partD, *partBias; // [b, D, N], [b, D], [b, D]
  float *dh0;
};

// grid: (tile of channels, group, sequence); a tile's channels share a group.
template <typename IO, int NL>
__global__ void __launch_bounds__(kThreads)
adjoint_kernel(In<IO> in, SeqView<const IO> gy, const float *__restrict__ gfinal,
               const float *__restrict__ states, int64_t spans, Out<IO> out, int *err) {
  constexpr int kWarps = kThreads / 32;
  __shared__ float sumB[kWarps][4 * NL], sumC[kWarps][4 * NL];
  const int64_t chan = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / NL;
  const int lane = threadIdx.x % NL, n0 = lane * 4, N = in.N;
  const int64_t g = blockIdx.y, G = gridDim.y, b = blockIdx.z;
  const bool live = chan < in.per_group;
  const int64_t d = g * in.per_group + (live ? chan : in.per_group - 1);
  if (!SSD_IN_BOUNDS(b < in.nb && d < in.D, err, 72)) return;
  const int64_t len = tokens_of(in.lengths, b, in.L);
  float A[4], dA[4] = {0.f, 0.f, 0.f, 0.f}, ad[4] = {0.f, 0.f, 0.f, 0.f};
  load4_tail(in.A + d * N, n0, N, A);
  if (gfinal) load4_tail(gfinal + (b * in.D + d) * N, n0, N, ad);
  const float bias = in.dt_bias ? in.dt_bias[d] : 0.f, skip = in.Dskip ? in.Dskip[d] : 0.f;
  float dD = 0.f, dbias = 0.f;
  for (int64_t sp = (len + kSpan - 1) / kSpan - 1; sp >= 0; --sp) {
    const int64_t t0 = sp * kSpan;
    const int n = (int)(len - t0 < kSpan ? len - t0 : kSpan);
    float h[4], before[kSpan][4];
    load4_tail(states + ((b * spans + sp) * in.D + d) * N, n0, N, h);
#pragma unroll
    for (int j = 0; j < kSpan; ++j) {
      if (j >= n) break;
      float B[4];
      load4_tail(in.B.at(b, t0 + j) + g * N, n0, N, B);
      const float u = ld_io(in.u.at(b, t0 + j) + d);
      const float s = step_of(ld_io(in.dt.at(b, t0 + j) + d) + bias, in.softplus);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        before[j][i] = h[i];
        h[i] = fmaf(ex2(s * A[i] * kLog2e), h[i], n0 + i < N ? s * u * B[i] : 0.f);
      }
    }
#pragma unroll
    for (int j = kSpan - 1; j >= 0; --j) {
      if (j >= n) continue;
      const int64_t t = t0 + j;
      float B[4], C[4], pB[4], pC[4];
      load4_tail(in.B.at(b, t) + g * N, n0, N, B);
      load4_tail(in.C.at(b, t) + g * N, n0, N, C);
      const float u = ld_io(in.u.at(b, t) + d);
      const float raw = ld_io(in.dt.at(b, t) + d) + bias;
      const float s = step_of(raw, in.softplus);
      const float gyv = ld_io(gy.at(b, t) + d);
      const float zv = in.z.p ? ld_io(in.z.at(b, t) + d) : 0.f;
      const float o = in.z.p ? gyv * silu(zv) : gyv;
      float yv = 0.f, gB = 0.f, gah = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float e = ex2(s * A[i] * kLog2e);
        const float ht = fmaf(e, before[j][i], n0 + i < N ? s * u * B[i] : 0.f);
        ad[i] = n0 + i < N ? fmaf(o, C[i], ad[i]) : 0.f;
        yv = fmaf(ht, C[i], yv);
        pC[i] = live ? o * ht : 0.f;
        pB[i] = live && n0 + i < N ? ad[i] * s * u : 0.f;
        gB = fmaf(ad[i], B[i], gB);
        ad[i] *= e;
        const float p = ad[i] * before[j][i];
        dA[i] = fmaf(s, p, dA[i]);
        gah = fmaf(A[i], p, gah);
      }
      yv = fmaf(skip, u, sum_lanes<NL>(yv));
      gB = sum_lanes<NL>(gB);
      gah = sum_lanes<NL>(gah);
      float ds = fmaf(u, gB, gah);
      if (in.softplus) ds *= sigmoid(raw);
      dD = fmaf(o, u, dD);
      dbias += ds;
      if (lane == 0 && live) {
        st_io(out.du.at(b, t) + d, fmaf(s, gB, skip * o));
        st_io(out.ddt.at(b, t) + d, ds);
        if (out.dz.p) st_io(out.dz.at(b, t) + d, gyv * yv * dsilu(zv));
      }
      // over the tile's channels: lanes with the same states, then warps
#pragma unroll
      for (int off = NL; off < 32; off <<= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          pB[i] += __shfl_xor_sync(0xffffffffu, pB[i], off);
          pC[i] += __shfl_xor_sync(0xffffffffu, pC[i], off);
        }
      if (threadIdx.x % 32 < NL)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sumB[threadIdx.x / 32][n0 + i] = pB[i];
          sumC[threadIdx.x / 32][n0 + i] = pC[i];
        }
      __syncthreads();
      if ((int)threadIdx.x < N) {
        float vB = sumB[0][threadIdx.x], vC = sumC[0][threadIdx.x];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) vB += sumB[w][threadIdx.x], vC += sumC[w][threadIdx.x];
        const int64_t o4 = ((((int64_t)blockIdx.x * in.nb + b) * in.L + t) * G + g) * N + threadIdx.x;
        out.partB[o4] = vB;
        out.partC[o4] = vC;
      }
      __syncthreads();
    }
  }
  if (!live) return;
  if (out.dh0) store4_tail(out.dh0 + (b * in.D + d) * N, n0, N, ad);
  store4_tail(out.partA + (b * in.D + d) * N, n0, N, dA);
  if (lane == 0) {
    out.partD[b * in.D + d] = dD;
    out.partBias[b * in.D + d] = dbias;
    for (int64_t t = len; t < in.L; ++t) {
      st_io(out.du.at(b, t) + d, 0.f);
      st_io(out.ddt.at(b, t) + d, 0.f);
      if (out.dz.p) st_io(out.dz.at(b, t) + d, 0.f);
    }
  }
}

// dB and dC: the tiles' parts in order; zero past a sequence's end.
template <typename IO>
__global__ void __launch_bounds__(256)
sum_tiles_kernel(const float *__restrict__ partB, const float *__restrict__ partC, int tiles,
                 SeqView<IO> dB, SeqView<IO> dC, const int32_t *__restrict__ lengths, int64_t nb,
                 int64_t L, int64_t GN, int *err) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, n = nb * L * GN;
  if (i >= n) return;
  const int64_t c = i % GN, t = i / GN % L, b = i / GN / L;
  if (!SSD_IN_BOUNDS(b < nb && t < L, err, 73)) return;
  float vB = 0.f, vC = 0.f;
  if (t < tokens_of(lengths, b, L))
    for (int k = 0; k < tiles; ++k) vB += partB[k * n + i], vC += partC[k * n + i];
  st_io(dB.at(b, t) + c, vB);
  st_io(dC.at(b, t) + c, vC);
}

struct Layout {
  int64_t spans, tiles;
  size_t states, partB, partC, partA, partD, partBias, total;  // in floats
};
Layout layout_of(const ScanArgs &a) {
  Layout l;
  const int64_t per = kThreads / lanes_of(a.N);
  l.spans = (a.L + kSpan - 1) / kSpan;
  l.tiles = (a.D / a.G + per - 1) / per;
  size_t at = 0;
  auto take = [&](int64_t n) {
    const size_t r = at;
    at += (size_t)((n + 63) / 64 * 64);
    return r;
  };
  l.states = take(a.b * l.spans * a.D * a.N);
  l.partB = take(l.tiles * a.b * a.L * a.G * a.N);
  l.partC = take(l.tiles * a.b * a.L * a.G * a.N);
  l.partA = take(a.b * a.D * a.N);
  l.partD = take(a.b * a.D);
  l.partBias = take(a.b * a.D);
  l.total = at;
  return l;
}

}  // namespace

size_t selective_scan_backward_workspace(const ScanArgs &a, ssd_dtype) {
  return sizeof(float) * layout_of(a).total;
}

cudaError_t launch_selective_scan_backward(const ScanArgs &a, ssd_dtype io, void *ws, int *err,
                                           cudaStream_t st) {
  const Layout l = layout_of(a);
  float *f = static_cast<float *>(ws);
  const cudaError_t e = dispatch(io, a.N, [&](auto io_c, auto nl_c) {
    using IO = typename decltype(io_c)::type;
    constexpr int NL = decltype(nl_c)::value;
    const In<IO> in = in_of<IO>(a);
    const dim3 all((unsigned)((a.D * NL + kThreads - 1) / kThreads), (unsigned)a.b);
    states_kernel<IO, NL><<<all, kThreads, 0, st>>>(in, f + l.states, l.spans, err);
    cudaError_t e1 = cudaGetLastError();
    if (e1 != cudaSuccess) return e1;
    Out<IO> out;
    out.du = view_of<IO>(&a.out->du), out.ddt = view_of<IO>(&a.out->ddt);
    out.dz = view_of<IO>(&a.out->dz);
    out.partB = f + l.partB, out.partC = f + l.partC, out.partA = f + l.partA;
    out.partD = f + l.partD, out.partBias = f + l.partBias, out.dh0 = a.out->dh0;
    const dim3 grid((unsigned)l.tiles, (unsigned)a.G, (unsigned)a.b);
    adjoint_kernel<IO, NL><<<grid, kThreads, 0, st>>>(in, view_of<const IO>(a.gy), a.gfinal,
                                                      f + l.states, l.spans, out, err);
    e1 = cudaGetLastError();
    if (e1 != cudaSuccess) return e1;
    const int64_t n = a.b * a.L * a.G * a.N;
    sum_tiles_kernel<IO><<<(unsigned)((n + 255) / 256), 256, 0, st>>>(
        f + l.partB, f + l.partC, (int)l.tiles, view_of<IO>(&a.out->dB),
        view_of<IO>(&a.out->dC), a.lengths, a.b, a.L, a.G * a.N, err);
    return cudaGetLastError();
  });
  if (e != cudaSuccess) return e;
  ColSum s{};
  s.nseg = 3;
  s.seg[0] = {f + l.partA, a.out->dA, a.b, a.D * a.N};
  s.seg[1] = {f + l.partD, a.out->dD, a.b, a.D};
  s.seg[2] = {f + l.partBias, a.out->ddt_bias, a.b, a.D};
  return launch_colsum(s, err, st);
}

}  // namespace ssd
