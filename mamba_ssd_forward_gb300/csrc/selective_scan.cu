// Selective scan, forward.  Per channel d and state n, with the step
// s_t = softplus(dt_t + bias):
//   h_t = exp(s_t A) h_{t-1} + s_t u_t B_t,   y_t = (sum_n h_t C_t + D u_t) silu(z_t)
//
// Every decay is an exponential of its own (they differ by channel, state and
// token), so the work is one exponential and four multiply-adds per (token,
// channel, state), 16 of them to the 8 bytes of a bf16 token and channel:
// bound by the SM's exponentials (32 a clock) and multiply-adds (128 a clock).
//
// A lane holds a channel and up to 16 of its states as fp32 pairs, so the sum
// over the states stays in the lane, each u, dt and z is read by one lane, and
// B and C, equal for the warp's 32 channels, are broadcast from shared memory.
// A warp runs alone, kTile tokens at a time: it stages their B and C and
// prepares what each channel needs of them (s, s u, D u, silu(z)), then runs
// the states; it needs no barrier but its own.
//
// Measured (bf16, 16 states, GB300): 16 sequences of 512 tokens and 5120
// channels, uncut: 248 us, 2.7e12 (token, channel, state) a second; two of
// 2048 tokens, in five segments: 176 us; 16384 tokens of 1536 channels: 205 us.
// A pair multiply-add with three register operands takes three cycles of a
// scheduler, so the body is 107 cycles a token and warp where nothing stalls.
//
// Where the channels give too few warps the tokens are cut into segments, one
// warp each.  A first launch runs every segment but the last from a zero state
// and keeps its end state and its steps' sum (the decay over a segment is
// exp(A sum s)); in the second each segment joins the ends before it, in
// order, into its start state and runs its tokens with the outputs.
#include "scan_common.cuh"

namespace ssd {
namespace {

using namespace scan;

constexpr int kWarps = 4;  // independent warps per block
// Per SM.  Four blocks of 128 registers ran slower when that was measured (218 us
// where three took 194; with what followed three take 176).
constexpr int kBlocks = 3;
constexpr int kTile = 8;    // tokens staged at a time

// A warp's part of the work: sequence, group, channel tile, segment.  The
// first launch cuts each segment but the last into parts.
struct Cut {
  int tiles, segments, parts;  // tiles per group, parts per segment
  int64_t span;                // tokens per part
};

// A warp's copies of kTile tokens' rows of one view into COLS columns of
// shared memory.  VEC: 16 bytes at a time, the lanes taking turns over the
// pieces of the rows; else element by element (2 x 2048 x 1536, N = 16: 64 to 66 us
// against 78 in fp32 and 87 in bf16, whose elements cannot be copied asynchronously).
template <typename IO, int COLS, bool VEC>
struct RowCopy {
  static constexpr int kPer = 16 / (int)sizeof(IO), kPieces = COLS >= kPer ? COLS / kPer : 1;
  const IO *p;  // of the next tile; VEC: of this lane
  int64_t ts;
  int row, col, cols;
  __device__ __forceinline__ RowCopy(const SeqView<const IO> &m, int64_t b, int64_t t,
                                     int64_t first_col, int valid, int lane)
      : ts(m.ts), row(VEC ? lane / kPieces : 0), col(VEC ? lane % kPieces * kPer : lane),
        cols(valid) {
    p = m.at(b, t + row) + first_col + (VEC ? col : 0);
  }
  // the first n tokens of the next tile
  __device__ __forceinline__ void issue(IO *dst, int n) {
    if constexpr (VEC) {
#pragma unroll
      for (int r = 0; r < kTile; r += 32 / kPieces)
        if (col < cols && row + r < n && row + r < kTile)
          copy16(dst + (row + r) * COLS + col, p + r * ts);
    } else {
      copy_pieces<COLS, kTile, 1>(dst, p, ts, n, cols, col);
    }
    p += kTile * ts;
  }
};

// A warp's shared memory.
template <typename IO, int NPT, int NL, bool OUT>
struct __align__(16) Warp {
  static constexpr int T = kTile, TO = OUT ? T : 1, CW = 32 / NL, NP = NPT * NL;
  using Step = typename std::conditional<OUT, float4, float2>::type;
  struct __align__(16) {  // a tile as it is in memory, and the next one
    IO u[T][CW], dt[T][CW], z[TO][CW], B[T][NP], C[TO][NP];
  } raw[2];
  Step step[NL > 1 ? T : 1][CW];  // s, s u and, for the outputs, D u and silu(z)
  float B[T][NP], C[TO][NP];
};

// NPT states to a lane, NL lanes to a channel.  OUT: the outputs too; else
// only the segment's end (ends, sums).
template <typename IO, int NPT, int NL, bool VEC, bool OUT>
__global__ void __launch_bounds__(32 * kWarps, kBlocks)
scan_kernel(In<IO> in, Cut cut, SeqView<IO> y, float *__restrict__ final_state,
            float *__restrict__ ends, float *__restrict__ sums, int64_t units, int *err) {
  constexpr int NP = NPT * NL, TT = kTile;
  constexpr int CW = 32 / NL;  // channels per warp
  using Step = typename Warp<IO, NPT, NL, OUT>::Step;
  extern __shared__ __align__(16) unsigned char smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, nl = lane % NL;
  auto &sm = reinterpret_cast<Warp<IO, NPT, NL, OUT> *>(smem)[warp];
  int64_t unit = (int64_t)blockIdx.x * kWarps + warp;
  if (unit >= units) return;
  // units run over tiles, groups, segments (parts of them but the last in the
  // first launch), sequences
  const int tile = (int)(unit % cut.tiles);
  const int64_t G = in.D / in.per_group;
  const int64_t g = unit / cut.tiles % G;
  const int ends_of = (cut.segments - 1) * cut.parts, segs = OUT ? cut.segments : ends_of;
  const int64_t span = OUT ? cut.span * cut.parts : cut.span;
  const int64_t seg = unit / cut.tiles / G % segs, b = unit / cut.tiles / G / segs;
  auto slot = [&](int64_t j) {  // of part j's end
    return ((b * ends_of + j) * G + g) * cut.tiles + tile;
  };
  const int c = tile * CW + lane / NL;
  const bool live = c < in.per_group, stores = live && nl == 0;
  const int64_t d = g * in.per_group + (live ? c : 0);  // idle lanes repeat channel 0, unstored
  const int N = in.N, n0 = nl * NPT;
  if (!SSD_IN_BOUNDS(b < in.nb && d < in.D, err, 70)) return;
  const int64_t len = tokens_of(in.lengths, b, in.L);
  const int64_t first = seg * span, last = min(first + span, in.L);
  const int64_t t1 = min(last, len);

  pair A[NPT / 2], h[NPT / 2];
#pragma unroll
  for (int i = 0; i < NPT / 2; ++i) {
    const int n = n0 + 2 * i;
    const float *row = in.A + d * N;
    A[i] = pack(n < N ? log2_decay(row[n]) : 0.f, n + 1 < N ? log2_decay(row[n + 1]) : 0.f);
    h[i] = 0;
    if (OUT && in.h0) {
      row = in.h0 + (b * in.D + d) * N;
      h[i] = pack(n < N ? row[n] : 0.f, n + 1 < N ? row[n + 1] : 0.f);
    }
  }
  if (OUT)
#pragma unroll 2
    for (int64_t k = 0; k < seg * cut.parts; ++k) {
      const float *e = ends + slot(k) * NPT * 32 + lane;
      const pair total = both(sums[slot(k) * CW + lane / NL]);
#pragma unroll
      for (int i = 0; i < NPT / 2; ++i)
        h[i] = fma2(ex2_2(mul2(total, A[i])), h[i], pack(e[2 * i * 32], e[(2 * i + 1) * 32]));
    }
  const int cols = min(CW, in.per_group - tile * CW);
  const int64_t c0 = g * in.per_group + tile * CW;
  // the channel whose tokens this lane prepares
  const int mine = lane % CW;
  const float bias = in.dt_bias && mine < cols ? in.dt_bias[c0 + mine] : 0.f;
  const float skip = OUT && in.Dskip && mine < cols ? in.Dskip[c0 + mine] : 0.f;
  RowCopy<IO, CW, VEC> cu(in.u, b, first, c0, cols, lane), cd(in.dt, b, first, c0, cols, lane),
      cz(in.z, b, first, c0, cols, lane);
  RowCopy<IO, NP, VEC> cB(in.B, b, first, g * N, N, lane), cC(in.C, b, first, g * N, N, lane);
  const bool gated = OUT && in.z.p;
  auto issue = [&](int64_t t, auto &raw) {
    const int n = (int)(t1 - t < TT ? t1 - t : TT);
    if (n > 0 && SSD_IN_BOUNDS(t >= 0 && t + n <= in.L, err, 74)) {
      cu.issue(raw.u[0], n);
      cd.issue(raw.dt[0], n);
      cB.issue(raw.B[0], n);
      if (OUT) cC.issue(raw.C[0], n);
      if (gated) cz.issue(raw.z[0], n);
    }
    copies_issued();
  };
  if (N < NP) {  // states past N stay zero
    for (int i = lane; i < TT * NP; i += 32)
      for (int k = 0; k < 2; ++k) {
        sm.raw[k].B[0][i] = IO(0.f);
        if (OUT) sm.raw[k].C[0][i] = IO(0.f);
      }
    __syncwarp();
  }
  IO *py = OUT ? y.at(b, first) + d : nullptr;
  float total = 0.f;
  issue(first, sm.raw[0]);
  for (int64_t t0 = first, turn = 0; t0 < t1; t0 += TT, turn ^= 1) {
    issue(t0 + TT, sm.raw[turn ^ 1]);
    copies_landed<1>();
    __syncwarp();
    const int n = (int)(t1 - t0 < TT ? t1 - t0 : TT);
    const auto &raw = sm.raw[turn];
    // what the tokens need besides the states
    constexpr int EB = TT * NP / 32;
    constexpr int EV = EB % 4 == 0 ? 4 : 1;
#pragma unroll
    for (int i = 0; i < EB; i += EV) {
      const bool here = (lane * EB + i) / NP < n;  // nothing was copied for the tokens after
      auto stage = [&](const IO *from, float *to) {
        float v[EV];
        load_vec<EV>(from + lane * EB + i, v);
#pragma unroll
        for (int e = 0; e < EV; ++e) v[e] = here ? v[e] : 0.f;
        store_vec<EV>(to + lane * EB + i, v);
      };
      stage(&raw.B[0][0], &sm.B[0][0]);
      if (OUT) stage(&raw.C[0][0], &sm.C[0][0]);
    }
    constexpr int EACH = TT * CW / 32;  // tokens of its channel that a lane prepares
    Step own[NL > 1 ? 1 : TT];
#pragma unroll
    for (int i = 0; i < (EACH > 0 ? EACH : 1); ++i) {
      const int k = lane / CW + i * (32 / CW);
      if (EACH == 0 && k >= TT) break;
      const float uk = ld_io(&raw.u[k][mine]);
      const float s = step_of(ld_io(&raw.dt[k][mine]) + bias, in.softplus);
      Step st;
      if constexpr (OUT)
        st = make_float4(s, s * uk, skip * uk, gated ? silu(ld_io(&raw.z[k][mine])) : 1.f);
      else
        st = make_float2(s, s * uk);
      if (k >= n) st.x = st.y = 0.f;  // leaves the state as it is
      if (!OUT) total += st.x;
      if constexpr (NL > 1)
        sm.step[k][mine] = st;
      else
        own[i] = st;  // the lane's own channel: it stays in registers
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < TT; ++k) {
      Step st;
      if constexpr (NL > 1)
        st = sm.step[k][lane / NL];
      else
        st = own[k];
      const pair ss = both(st.x), su = both(st.y);
      pair acc = 0;
      const ulonglong2 *pB = reinterpret_cast<const ulonglong2 *>(&sm.B[k][n0]);
      const ulonglong2 *pC = reinterpret_cast<const ulonglong2 *>(&sm.C[OUT ? k : 0][n0]);
#pragma unroll
      for (int q = 0; q < NPT / 4; ++q) {
        const ulonglong2 B = pB[q];
        h[2 * q] = fma2(ex2_2(mul2(ss, A[2 * q])), h[2 * q], mul2(su, B.x));
        h[2 * q + 1] = fma2(ex2_2(mul2(ss, A[2 * q + 1])), h[2 * q + 1], mul2(su, B.y));
        if (OUT) {
          const ulonglong2 C = pC[q];
          acc = fma2(h[2 * q], C.x, acc);
          acc = fma2(h[2 * q + 1], C.y, acc);
        }
      }
      if constexpr (OUT) {
        const float o = (sum_lanes<NL>(sum2(acc)) + st.z) * st.w;
        if (k < n && stores) st_io(py, o);
        py += y.ts;
      }
    }
    __syncwarp();
  }
  copies_landed<0>();
  if (OUT) {
    if (stores)
      for (int64_t t = max(first, t1); t < last; ++t) st_io(y.at(b, t) + d, 0.f);
    if (final_state && live && seg == cut.segments - 1)
#pragma unroll
      for (int i = 0; i < NPT / 2; ++i) {
        float h0, h1;
        unpack(h[i], h0, h1);
        float *row = final_state + (b * in.D + d) * N + n0 + 2 * i;
        if (n0 + 2 * i < N) row[0] = h0;
        if (n0 + 2 * i + 1 < N) row[1] = h1;
      }
  } else {
    float *e = ends + slot(seg) * NPT * 32 + lane;
#pragma unroll
    for (int i = 0; i < NPT / 2; ++i) {
      float h0, h1;
      unpack(h[i], h0, h1);
      e[2 * i * 32] = h0;
      e[(2 * i + 1) * 32] = h1;
    }
#pragma unroll
    for (int off = 16; off >= CW; off /= 2) total += __shfl_xor_sync(0xffffffffu, total, off);
    if (lane < CW) sums[slot(seg) * CW + lane] = total;
  }
}

// States per lane and lanes per channel.  (Four or eight states to a lane give
// more warps, which would not have to be cut: 16 states on four lanes took 312
// us where segments take 177.)
struct Split {
  int npt, nl;
};
Split split_of(const ScanArgs &a) {
  if (a.N <= 16) return {a.N <= 4 ? 4 : a.N <= 8 ? 8 : 16, 1};
  return {16, a.N <= 32 ? 2 : 4};
}

// Segments: as many as the warps resident at once (three blocks to an SM;
// twice as many took a tenth longer on 16384 tokens of 1536 channels), of 32
// tokens at least (512 tokens of 1536 channels: 28 us, at 64 tokens 34 us), and
// no more than they hold tokens each, since a segment joins all the ends before
// it (32 channels of 100000 tokens: 317 segments 150 us, 1786 400 us).
// Fewer than three are not worth the first launch: 1280 warps of their own run
// uncut.  The first launch has a segment less, and its warps fill their rounds
// badly: it cuts segments further where rounds of shorter parts take less time
// in all (2 x 2048 x 5120: 1280 warps of 1824, 194 us; four parts each, 2.8
// rounds, 177; three or five parts 185, 187).  Every part is one more end to
// join, so there are kEnds at most.
constexpr int kEnds = 16;
constexpr int kPerSm = 12;
Cut cut_of(const ScanArgs &a) {
  Cut c;
  const int cw = 32 / split_of(a).nl;
  c.tiles = (int)((a.D / a.G + cw - 1) / cw);
  const int64_t warps = a.b * a.G * c.tiles, room = (int64_t)sm_count() * kPerSm;
  int64_t s = room / warps;
  s = min(s, (a.L + 31) / 32);
  while (s * s > a.L) --s;
  if (s < 3) s = 1;
  c.parts = 1;
  auto rounds = [&](int64_t p) { return (warps * (s - 1) * p + room - 1) / room; };
  if (s > 1)
    for (int64_t p = 2; p * (s - 1) <= kEnds && 32 * p * s <= a.L; ++p)
      if (rounds(p) * c.parts < rounds(c.parts) * p) c.parts = (int)p;
  c.span = ((a.L + s * c.parts - 1) / (s * c.parts) + 7) / 8 * 8;
  c.segments = (int)((a.L + c.span * c.parts - 1) / (c.span * c.parts));
  return c;
}
int64_t slots_of(const ScanArgs &a, const Cut &c) {
  return a.b * (c.segments - 1) * c.parts * a.G * c.tiles;
}

}  // namespace

size_t selective_scan_workspace(const ScanArgs &a, ssd_dtype) {
  const Cut c = cut_of(a);
  return c.segments == 1 ? 0 : sizeof(float) * 32 * (split_of(a).npt + 1) * slots_of(a, c);
}

cudaError_t launch_selective_scan(const ScanArgs &a, ssd_dtype io, void *ws, int *err,
                                  cudaStream_t st) {
  const Cut c = cut_of(a);
  const int64_t per_seg = a.b * a.G * c.tiles;
  float *ends = static_cast<float *>(ws);
  float *sums = ends + (c.segments == 1 ? 0 : slots_of(a, c) * 32 * split_of(a).npt);
  const int piece = piece_of(a, io);
  auto go = [&](auto io_c, auto npt_c, auto nl_c, auto vec_c) {
    using IO = typename decltype(io_c)::type;
    constexpr int NPT = decltype(npt_c)::value, NL = decltype(nl_c)::value;
    constexpr bool VEC = decltype(vec_c)::value;
    const In<IO> in = in_of<IO>(a);
    constexpr size_t m0 = kWarps * sizeof(Warp<IO, NPT, NL, false>);
    constexpr size_t m1 = kWarps * sizeof(Warp<IO, NPT, NL, true>);
    const cudaError_t e0 = cudaFuncSetAttribute(scan_kernel<IO, NPT, NL, VEC, true>,
                                                cudaFuncAttributeMaxDynamicSharedMemorySize, m1);
    if (e0 != cudaSuccess) return e0;
    const SeqView<IO> y = view_of<IO>(a.y);
    auto blocks = [](int64_t units) { return (unsigned)((units + kWarps - 1) / kWarps); };
    if (c.segments > 1) {
      const int64_t n = per_seg * (c.segments - 1) * c.parts;
      scan_kernel<IO, NPT, NL, VEC, false>
          <<<blocks(n), 32 * kWarps, m0, st>>>(in, c, y, nullptr, ends, sums, n, err);
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
    const int64_t n = per_seg * c.segments;
    scan_kernel<IO, NPT, NL, VEC, true>
        <<<blocks(n), 32 * kWarps, m1, st>>>(in, c, y, a.final_state, ends, sums, n, err);
    return cudaGetLastError();
  };
  auto by_vec = [&](auto io_c, auto npt_c, auto nl_c) {
    return piece == 16 ? go(io_c, npt_c, nl_c, std::true_type{})
                       : go(io_c, npt_c, nl_c, std::false_type{});
  };
  auto by_n = [&](auto io_c) {
    using std::integral_constant;
    const Split p = split_of(a);
    using four = integral_constant<int, 4>;
    using eight = integral_constant<int, 8>;
    using sixteen = integral_constant<int, 16>;
    using one = integral_constant<int, 1>;
    using two = integral_constant<int, 2>;
    if (p.npt == 4) return by_vec(io_c, four{}, one{});
    if (p.npt == 8) return by_vec(io_c, eight{}, one{});
    if (p.nl == 1) return by_vec(io_c, sixteen{}, one{});
    if (p.nl == 2) return by_vec(io_c, sixteen{}, two{});
    return by_vec(io_c, sixteen{}, four{});
  };
  return io == SSD_BF16 ? by_n(tag<__nv_bfloat16>{}) : by_n(tag<float>{});
}

}  // namespace ssd
