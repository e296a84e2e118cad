// Shared by the selective scan's kernels.  A channel's N states lie on NL
// neighbouring lanes (a power of two), four to a lane; states N and up of the
// last lanes are kept at zero.
#pragma once

#include <cfloat>
#include <type_traits>

#include "layer.cuh"

namespace ssd {
namespace scan {

constexpr float kLn2 = 0.6931471805599453f;

// The step of a token: v = dt + bias, or log(1 + exp(v)) as
// max(v, 0) + t q(t) with t = exp(-|v|) in (0, 1], which neither overflows nor
// loses small values.  q is the degree-8 polynomial of least relative error
// for log(1 + t) / t on [0, 1] (exchange algorithm; 3e-8, and 1.7e-7 with the
// roundings of fp32).
__device__ __forceinline__ float step_of(float v, bool softplus) {
  if (!softplus) return v;
  const float t = ex2(-kLog2e * fabsf(v));
  float q = 0.0052326940931379795f;
  q = fmaf(q, t, -0.02950523979961872f);
  q = fmaf(q, t, 0.07822595536708832f);
  q = fmaf(q, t, -0.13663245737552643f);
  q = fmaf(q, t, 0.19106006622314453f);
  q = fmaf(q, t, -0.2484298199415207f);
  q = fmaf(q, t, 0.3331909775733948f);
  q = fmaf(q, t, -0.4999949336051941f);
  q = fmaf(q, t, 0.9999999403953552f);
  return fmaf(t, q, fmaxf(v, 0.f));
}

// A in units of log2, finite: A = -inf is a decay of zero, but the places that
// hold no token take steps of zero, and there the decay has to be one.
__device__ __forceinline__ float log2_decay(float a) {
  a *= kLog2e;
  return a < -FLT_MAX ? -FLT_MAX : a;
}

// The slope of softplus where its value is s: 1 - exp(-s), by its series where
// the difference would cancel (the term left out is below 1e-8 of it).
__device__ __forceinline__ float slope_of_step(float s) {
  float q = -1.f / 40320.f;
  q = fmaf(q, s, 1.f / 5040.f);
  q = fmaf(q, s, -1.f / 720.f);
  q = fmaf(q, s, 1.f / 120.f);
  q = fmaf(q, s, -1.f / 24.f);
  q = fmaf(q, s, 1.f / 6.f);
  q = fmaf(q, s, -0.5f);
  q = fmaf(q, s, 1.f);
  return s < 0.5f ? q * s : 1.f - ex2(-kLog2e * s);
}

// Pairs of fp32 in 64-bit registers: one instruction for two products.
typedef unsigned long long pair;
__device__ __forceinline__ pair pack(float a, float b) {
  pair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(a), "f"(b));
  return p;
}
__device__ __forceinline__ void unpack(pair p, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ pair mul2(pair a, pair b) {
  pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ pair fma2(pair a, pair b, pair c) {
  pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ pair ex2_2(pair x) {
  float a, b;
  unpack(x, a, b);
  return pack(ex2(a), ex2(b));
}
__device__ __forceinline__ float sum2(pair p) {
  float a, b;
  unpack(p, a, b);
  return a + b;
}

__device__ __forceinline__ pair add2(pair a, pair b) {
  pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ pair both(float v) { return pack(v, v); }

// The four states of a lane: loads of a row of N floats or I/O elements from
// index n0 on, zero past N.
template <typename T>
__device__ __forceinline__ void load4_tail(const T *row, int n0, int N, float (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = n0 + i < N ? ld_io(row + n0 + i) : 0.f;
}
__device__ __forceinline__ void store4_tail(float *row, int n0, int N, const float (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n0 + i < N) row[n0 + i] = v[i];
}

// Sum over the NL lanes of a channel, in every lane.
template <int NL>
__device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
  for (int off = NL / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

template <typename T>
struct tag {
  using type = T;
};

// Lanes per channel: the least power of two with four states to a lane.
inline int lanes_of(int64_t N) {
  int nl = 1;
  while (nl * 4 < N) nl *= 2;
  return nl;
}

template <typename F>
cudaError_t dispatch(ssd_dtype io, int64_t N, F f) {
  auto by_lanes = [&](auto io_c) {
    switch (lanes_of(N)) {
      case 1: return f(io_c, std::integral_constant<int, 1>{});
      case 2: return f(io_c, std::integral_constant<int, 2>{});
      case 4: return f(io_c, std::integral_constant<int, 4>{});
      case 8: return f(io_c, std::integral_constant<int, 8>{});
      default: return f(io_c, std::integral_constant<int, 16>{});
    }
  };
  return io == SSD_BF16 ? by_lanes(tag<__nv_bfloat16>{}) : by_lanes(tag<float>{});
}

// Bytes of the pieces in which rows of the inputs can be copied: 16 where
// every row is whole such pieces, else 4 (always for fp32), else single
// elements of 2.
inline int piece_of(const ScanArgs &a, ssd_dtype io) {
  const size_t e = io == SSD_BF16 ? 2 : 4;
  auto fits = [&](size_t n) {
    return a.N * e % n == 0 && (a.D / a.G) * e % n == 0 && view_aligned(a.u, e, n) &&
           view_aligned(a.dt, e, n) && view_aligned(a.z, e, n) && view_aligned(a.gy, e, n) &&
           view_aligned(a.B, e, n) && view_aligned(a.C, e, n);
  };
  return fits(16) ? 16 : fits(4) ? 4 : 2;
}

// The first n of ROWS rows from p on, `cols` of COLS columns, to shared memory
// in pieces of E elements: 4 bytes asynchronously, or single elements at once,
// which leaves zeros elsewhere.  A lane keeps its column.
template <int COLS, int ROWS, int E, typename IO>
__device__ __forceinline__ void copy_pieces(IO *dst, const IO *p, int64_t ts, int n, int cols,
                                            int lane) {
  constexpr bool WORDS = E * sizeof(IO) == 4;
  constexpr int W = COLS / E, LANES = W < 32 ? W : 32, STEP = 32 / LANES;
  constexpr int TURNS = ROWS / STEP > 1 ? ROWS / STEP : 1;
  const int r = lane / LANES;
#pragma unroll
  for (int c = lane % LANES * E; c < COLS; c += 32 * E) {
    const IO *q = p + r * ts + c;
    IO v[TURNS];
#pragma unroll
    for (int k = 0; k < TURNS; ++k) {
      const bool ok = c < cols && r + k * STEP < n;
      if (WORDS) {
        if (ok) copy4(dst + (r + k * STEP) * COLS + c, q + k * STEP * ts);
      } else {
        v[k] = ok ? q[k * STEP * ts] : IO(0.f);
      }
    }
    if (!WORDS)
#pragma unroll
      for (int k = 0; k < TURNS; ++k)
        if (r + k * STEP < ROWS) dst[(r + k * STEP) * COLS + c] = v[k];
  }
}
template <int COLS, int ROWS, typename IO>
__device__ __forceinline__ void copy_small(IO *dst, const IO *p, int64_t ts, int n, int cols,
                                           int lane, bool words) {
  if (words || sizeof(IO) == 4)
    copy_pieces<COLS, ROWS, 4 / (int)sizeof(IO)>(dst, p, ts, n, cols, lane);
  else
    copy_pieces<COLS, ROWS, 1>(dst, p, ts, n, cols, lane);
}

// The inputs of the forward recurrence, as the kernels take them.
template <typename IO>
struct In {
  SeqView<const IO> u, dt, B, C, z;
  const float *A, *Dskip, *dt_bias, *h0;
  const int32_t *lengths;
  int64_t nb, L, D;
  int N, per_group;  // states, channels per group
  bool softplus;
};
template <typename IO>
In<IO> in_of(const ScanArgs &a) {
  In<IO> i;
  i.u = view_of<const IO>(a.u), i.dt = view_of<const IO>(a.dt);
  i.B = view_of<const IO>(a.B), i.C = view_of<const IO>(a.C), i.z = view_of<const IO>(a.z);
  i.A = a.A, i.Dskip = a.Dskip, i.dt_bias = a.dt_bias, i.h0 = a.h0;
  i.lengths = a.lengths;
  i.nb = a.b, i.L = a.L, i.D = a.D, i.N = (int)a.N, i.per_group = (int)(a.D / a.G);
  i.softplus = a.softplus;
  return i;
}

}  // namespace scan
}  // namespace ssd
