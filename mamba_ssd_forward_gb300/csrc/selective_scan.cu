// Selective scan, forward and single token.  Per channel d and state n, with
// the step s_t = softplus(dt_t + bias):
//   h_t = exp(s_t A) h_{t-1} + s_t u_t B_t,   y_t = (sum_n h_t C_t + D u_t) silu(z_t)
#include "scan_common.cuh"

namespace ssd {
namespace {

using namespace scan;

constexpr int kThreads = 128;

// One channel on NL lanes, the tokens in order.  STEP: one token, the state
// read from and written to final_state.
template <typename IO, int NL, bool STEP>
__global__ void __launch_bounds__(kThreads)
scan_kernel(In<IO> in, SeqView<IO> y, float *__restrict__ final_state, int *err) {
  const int64_t ch = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / NL;
  const int lane = threadIdx.x % NL, n0 = lane * 4, N = in.N;
  const int64_t b = blockIdx.y;
  const bool live = ch < in.D;
  const int64_t d = live ? ch : in.D - 1;  // idle lanes repeat the last channel, unstored
  const int64_t g = d / in.per_group;
  if (!SSD_IN_BOUNDS(b < in.nb && g * in.per_group <= d && d < in.D, err, 70)) return;
  const int64_t len = STEP ? 1 : tokens_of(in.lengths, b, in.L);
  float A[4], h[4];
  load4_tail(in.A + d * N, n0, N, A);
#pragma unroll
  for (int i = 0; i < 4; ++i) A[i] *= kLog2e, h[i] = 0.f;
  const float *first = STEP ? final_state : in.h0;
  if (first) load4_tail(first + (b * in.D + d) * N, n0, N, h);
  const float bias = in.dt_bias ? in.dt_bias[d] : 0.f, skip = in.Dskip ? in.Dskip[d] : 0.f;
  for (int64_t t = 0; t < len; ++t) {
    float B[4], C[4], acc = 0.f;
    load4_tail(in.B.at(b, t) + g * N, n0, N, B);
    load4_tail(in.C.at(b, t) + g * N, n0, N, C);
    const float u = ld_io(in.u.at(b, t) + d);
    const float s = step_of(ld_io(in.dt.at(b, t) + d) + bias, in.softplus);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[i] = fmaf(ex2(s * A[i]), h[i], n0 + i < N ? s * u * B[i] : 0.f);
      acc = fmaf(h[i], C[i], acc);
    }
    acc = fmaf(skip, u, sum_lanes<NL>(acc));
    if (in.z.p) acc *= silu(ld_io(in.z.at(b, t) + d));
    if (lane == 0 && live) st_io(y.at(b, t) + d, acc);
  }
  if (!STEP && lane == 0 && live)
    for (int64_t t = len; t < in.L; ++t) st_io(y.at(b, t) + d, 0.f);
  if (final_state && live) store4_tail(final_state + (b * in.D + d) * N, n0, N, h);
}

template <bool STEP>
cudaError_t launch(const ScanArgs &a, ssd_dtype io, int *err, cudaStream_t st) {
  return dispatch(io, a.N, [&](auto io_c, auto nl_c) {
    using IO = typename decltype(io_c)::type;
    constexpr int NL = decltype(nl_c)::value;
    const dim3 grid((unsigned)((a.D * NL + kThreads - 1) / kThreads), (unsigned)a.b);
    scan_kernel<IO, NL, STEP>
        <<<grid, kThreads, 0, st>>>(in_of<IO>(a), view_of<IO>(a.y), a.final_state, err);
    return cudaGetLastError();
  });
}

}  // namespace

size_t selective_scan_workspace(const ScanArgs &, ssd_dtype) { return 0; }

cudaError_t launch_selective_scan(const ScanArgs &a, ssd_dtype io, void *, int *err,
                                  cudaStream_t st) {
  return launch<false>(a, io, err, st);
}

cudaError_t launch_selective_scan_step(const ScanArgs &a, ssd_dtype io, int *err,
                                       cudaStream_t st) {
  return launch<true>(a, io, err, st);
}

}  // namespace ssd
