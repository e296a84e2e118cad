// One token of the selective scan for every sequence: a bandwidth kernel, the
// fp32 state read and written once (8 N bytes per channel against 8 for the
// rest).  A channel's states lie on NL neighbouring lanes, four to a lane.
// 64 sequences of 5120 channels, 16 states: 12.5 us with the states (21 MB, read
// and written) in L2, 17 without (2.6 TB/s: a launch and one round trip to
// memory are most of it).
#include "scan_common.cuh"

namespace ssd {
namespace {

using namespace scan;

constexpr int kThreads = 128;
constexpr int kSeqs = 2;

// VEC: four states at a time (N a multiple of four, rows on such boundaries).
// SEQS sequences to a thread, which then reads A once for them and has as many
// states in flight.
template <typename IO, int NL, bool VEC, int SEQS>
__global__ void __launch_bounds__(kThreads)
step_kernel(In<IO> in, SeqView<IO> y, float *__restrict__ state, int *err) {
  const int64_t ch = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / NL;
  const int lane = threadIdx.x % NL, n0 = lane * 4, N = in.N;
  const int64_t b0 = (int64_t)blockIdx.y * SEQS;
  const bool live = ch < in.D;
  const int64_t d = live ? ch : in.D - 1;  // idle lanes repeat the last channel, unstored
  const int64_t g = d / in.per_group;
  if (!SSD_IN_BOUNDS(b0 < in.nb && g * in.per_group <= d && d < in.D, err, 76)) return;
  auto four = [&](const auto *row, float (&v)[4]) {
    if (!VEC) return load4_tail(row, n0, N, v);
    v[0] = v[1] = v[2] = v[3] = 0.f;
    if (n0 < N) load_vec<4>(row + n0, v);
  };
  float A[4], h[SEQS][4], B[SEQS][4], C[SEQS][4], u[SEQS], s[SEQS], z[SEQS];
#pragma unroll
  for (int q = 0; q < SEQS; ++q) {
    const int64_t b = b0 + q < in.nb ? b0 + q : in.nb - 1;
    four(state + (b * in.D + d) * N, h[q]);
    four(in.B.at(b, 0) + g * N, B[q]);
    four(in.C.at(b, 0) + g * N, C[q]);
    u[q] = ld_io(in.u.at(b, 0) + d);
    s[q] = ld_io(in.dt.at(b, 0) + d);
    z[q] = in.z.p ? ld_io(in.z.at(b, 0) + d) : 0.f;
  }
  four(in.A + d * N, A);
  const float bias = in.dt_bias ? in.dt_bias[d] : 0.f, skip = in.Dskip ? in.Dskip[d] : 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) A[i] = log2_decay(A[i]);
#pragma unroll
  for (int q = 0; q < SEQS; ++q) {
    const int64_t b = b0 + q;
    s[q] = step_of(s[q] + bias, in.softplus);
    float acc = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[q][i] = fmaf(ex2(s[q] * A[i]), h[q][i], n0 + i < N ? s[q] * u[q] * B[q][i] : 0.f);
      acc = fmaf(h[q][i], C[q][i], acc);
    }
    acc = fmaf(skip, u[q], sum_lanes<NL>(acc));
    if (in.z.p) acc *= silu(z[q]);
    if (!live || b >= in.nb) continue;
    if (lane == 0) st_io(y.at(b, 0) + d, acc);
    float *hs = state + (b * in.D + d) * N;
    if (!VEC)
      store4_tail(hs, n0, N, h[q]);
    else if (n0 < N)
      store_vec<4>(hs + n0, h[q]);
  }
}

}  // namespace

cudaError_t launch_selective_scan_step(const ScanArgs &a, ssd_dtype io, int *err,
                                       cudaStream_t st) {
  return dispatch(io, a.N, [&](auto io_c, auto nl_c) {
    using IO = typename decltype(io_c)::type;
    constexpr int NL = decltype(nl_c)::value;
    const size_t e = sizeof(IO);
    const bool vec = a.N % 4 == 0 && ptr_aligned(a.final_state, 16) && ptr_aligned(a.A, 16) &&
                     view_aligned(a.B, e, 4 * e) && view_aligned(a.C, e, 4 * e);
    // several sequences to a thread where that still leaves every SM half its threads
    const bool many = a.b * a.D * NL / kSeqs >= (int64_t)sm_count() * 1024;
    auto go = [&](auto vec_c, auto seqs_c) {
      constexpr int SEQS = decltype(seqs_c)::value;
      const dim3 grid((unsigned)((a.D * NL + kThreads - 1) / kThreads),
                      (unsigned)((a.b + SEQS - 1) / SEQS));
      step_kernel<IO, NL, decltype(vec_c)::value, SEQS>
          <<<grid, kThreads, 0, st>>>(in_of<IO>(a), view_of<IO>(a.y), a.final_state, err);
      return cudaGetLastError();
    };
    using one = std::integral_constant<int, 1>;
    using several = std::integral_constant<int, kSeqs>;
    if (vec) return many ? go(std::true_type{}, several{}) : go(std::true_type{}, one{});
    return many ? go(std::false_type{}, several{}) : go(std::false_type{}, one{});
  });
}

}  // namespace ssd
