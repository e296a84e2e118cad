// One token of the selective scan for every sequence: a bandwidth kernel, the
// fp32 state read and written once (8 N bytes per channel against 8 for the
// rest).  A channel's states lie on NL neighbouring lanes, four to a lane.
#include "scan_common.cuh"

namespace ssd {
namespace {

using namespace scan;

constexpr int kThreads = 128;

// VEC: four states at a time (N a multiple of four, rows on such boundaries).
template <typename IO, int NL, bool VEC>
__global__ void __launch_bounds__(kThreads)
step_kernel(In<IO> in, SeqView<IO> y, float *__restrict__ state, int *err) {
  const int64_t ch = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / NL;
  const int lane = threadIdx.x % NL, n0 = lane * 4, N = in.N;
  const int64_t b = blockIdx.y;
  const bool live = ch < in.D;
  const int64_t d = live ? ch : in.D - 1;  // idle lanes repeat the last channel, unstored
  const int64_t g = d / in.per_group;
  if (!SSD_IN_BOUNDS(b < in.nb && g * in.per_group <= d && d < in.D, err, 76)) return;
  float *hs = state + (b * in.D + d) * N;
  float A[4], h[4], B[4], C[4], acc = 0.f;
  auto four = [&](const auto *row, float (&v)[4]) {
    if (!VEC) return load4_tail(row, n0, N, v);
    v[0] = v[1] = v[2] = v[3] = 0.f;
    if (n0 < N) load_vec<4>(row + n0, v);
  };
  four(hs, h);
  four(in.A + d * N, A);
  four(in.B.at(b, 0) + g * N, B);
  four(in.C.at(b, 0) + g * N, C);
  const float u = ld_io(in.u.at(b, 0) + d);
  const float s = step_of(ld_io(in.dt.at(b, 0) + d) + (in.dt_bias ? in.dt_bias[d] : 0.f),
                          in.softplus);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = fmaf(ex2(s * A[i] * kLog2e), h[i], n0 + i < N ? s * u * B[i] : 0.f);
    acc = fmaf(h[i], C[i], acc);
  }
  acc = fmaf(in.Dskip ? in.Dskip[d] : 0.f, u, sum_lanes<NL>(acc));
  if (in.z.p) acc *= silu(ld_io(in.z.at(b, 0) + d));
  if (!live) return;
  if (lane == 0) st_io(y.at(b, 0) + d, acc);
  if (!VEC)
    store4_tail(hs, n0, N, h);
  else if (n0 < N)
    store_vec<4>(hs + n0, h);
}

}  // namespace

cudaError_t launch_selective_scan_step(const ScanArgs &a, ssd_dtype io, int *err,
                                       cudaStream_t st) {
  return dispatch(io, a.N, [&](auto io_c, auto nl_c) {
    using IO = typename decltype(io_c)::type;
    constexpr int NL = decltype(nl_c)::value;
    const dim3 grid((unsigned)((a.D * NL + kThreads - 1) / kThreads), (unsigned)a.b);
    const size_t e = sizeof(IO);
    const bool vec = a.N % 4 == 0 && ptr_aligned(a.final_state, 16) && ptr_aligned(a.A, 16) &&
                     view_aligned(a.B, e, 4 * e) && view_aligned(a.C, e, 4 * e);
    if (vec)
      step_kernel<IO, NL, true>
          <<<grid, kThreads, 0, st>>>(in_of<IO>(a), view_of<IO>(a.y), a.final_state, err);
    else
      step_kernel<IO, NL, false>
          <<<grid, kThreads, 0, st>>>(in_of<IO>(a), view_of<IO>(a.y), a.final_state, err);
    return cudaGetLastError();
  });
}

}  // namespace ssd
