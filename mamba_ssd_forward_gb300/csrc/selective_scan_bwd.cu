// Gradients of the selective scan.  With e_t = exp(s_t A), o_t = gy_t silu(z_t)
// and the adjoint state G_t = o_t C_t + q_t, q_{t-1} = e_t G_t:
//   du = s sum_n G B + D o          ds = sum_n (u G B + A q_{t-1} h_{t-1})
//   dA = sum_t s q_{t-1} h_{t-1}    dB = sum_d G s u,   dC = sum_d o h
//   dz = gy (sum_n h C + D u) silu'(z),   ddt = ds softplus'
//
// The states are needed backwards in time, so they are recomputed from the
// state at the start of each segment of SEG (16) tokens:
// 1. ends_kernel: each segment's end from a zero state and its steps' sum; per
//    part of several segments the adjoint that reaches its front, summed
//    forwards as sum_t exp(A (s_1 + .. + s_t)) o_t C_t.
// 2. chain_kernel: those joined in order into every segment's start state and
//    every part's arriving adjoint (and dh0).
// 3. adjoint_kernel: a warp per part, segment by segment from the last: the
//    states at every fourth token, kept in shared memory; then four tokens at
//    a time from the last, their states again (in registers) and the adjoint
//    back over them.
// 4. the sums over channel tiles (dB, dC) and over parts (dA, dD, ddt_bias).
//
// A lane holds four channels, as two fp32 pairs, of four states: the sums over
// the channels (dB, dC) and over the states (du, ds, dz) are then both mostly
// inside the lane, 7 and 6 exchanges a token for 16 states.  Bound by the
// arithmetic: 3.75 exponentials and some 25 multiply-adds per (token, channel,
// state) against 46 bytes per (token, channel).
//
// Measured, bf16, 4 sequences of 1024 tokens, 2048 channels of 16 states: 297
// us in all; ends 59, chain 14, adjoint 202, the sums 21.  A segment's inputs
// are copied to shared memory while the one before is worked on (405 -> 366).
#include "scan_common.cuh"

namespace ssd {
namespace {

using namespace scan;

// Warps of the adjoint to an SM: at 8 a lane has some 240 registers and spills
// next to nothing; at 10, 168 registers with spills, a tenth more time.
constexpr int kMin = 8;
constexpr int kMinEnds = 16;  // 128 registers; 12 warps (162) and 20 (96) were slower

// How a warp lies over channels and states.
template <int NL>
struct Geo {
  static constexpr int CG = 32 / NL, CW = 4 * CG, NP = 4 * NL;
  static constexpr int SEG = 512 / CW < 16 ? 512 / CW : 16;  // tokens per segment
};

// Sums of v[0..V) over LANES lanes, STRIDE apart, spread over them: afterwards
// lane idx holds the sums of V / LANES values from idx V / LANES on, or, with
// fewer values than lanes, that of value idx V / LANES.
template <int STRIDE, int LANES, int V>
__device__ __forceinline__ void spread(float (&v)[V], int lane) {
  int half = V / 2;
#pragma unroll
  for (int off = LANES / 2; off > 0; off /= 2) {
    if (half >= 1) {
      const bool up = lane / STRIDE & off;
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        if (i >= half) break;
        const float send = up ? v[i] : v[half + i], keep = up ? v[half + i] : v[i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, send, off * STRIDE);
      }
      half /= 2;
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], off * STRIDE);
    }
  }
}

// The work's division: channel tiles per group, segments per sequence, parts
// of `per` segments.
struct Parts {
  int tiles;
  int64_t segments, parts;
  int per;
};

// Where a warp stands.
struct Unit {
  int tile;
  int64_t g, part, b, tile_id;  // tile_id: over (sequence, group, tile)
};
__device__ __forceinline__ Unit unit_of(int64_t i, const Parts &p, int64_t G) {
  Unit u;
  u.tile = (int)(i % p.tiles);
  u.g = i / p.tiles % G;
  u.part = i / p.tiles / G % p.parts;
  u.b = i / p.tiles / G / p.parts;
  u.tile_id = (u.b * G + u.g) * p.tiles + u.tile;
  return u;
}

struct Buffers {
  float2 *ends;        // [tile_id][segment][8][32]: ends, then start states
  float *sums;         // [tile_id][segment][CW]: the segment's steps
  float2 *adj;         // [tile_id][part][8][32]: adjoints at the front, then arriving ones
  float *part_sums;    // [tile_id][part][CW]
  float *partB, *partC;              // [tile][b, L, G, N]
  float *partA, *partD, *partBias;   // [b, part, D, N], [b, part, D] twice
};

// s, u and o of a segment, and its B and C with every value twice.
template <int NL>
struct Stage {
  using G = Geo<NL>;
  float s[G::SEG][G::CW], u[G::SEG][G::CW], o[G::SEG][G::CW];
  float2 B[G::SEG][G::NP], C[G::SEG][G::NP];
};

// A segment's inputs as they are in memory, copied one segment ahead.
template <typename IO, int NL>
struct __align__(16) Raw {
  using G = Geo<NL>;
  IO u[G::SEG][G::CW], dt[G::SEG][G::CW], gy[G::SEG][G::CW], z[G::SEG][G::CW];
  IO B[G::SEG][G::NP], C[G::SEG][G::NP];
};

// The first n rows from token t0 on of a view's columns, 16 bytes at a time.
template <int COLS, int ROWS, typename IO>
__device__ __forceinline__ void copy_rows(IO *dst, const SeqView<const IO> &m, int64_t b,
                                          int64_t t0, int n, int64_t first, int cols, int lane) {
  constexpr int kPer = 16 / (int)sizeof(IO), kPieces = COLS >= kPer ? COLS / kPer : 1;
  const int row = lane / kPieces, col = lane % kPieces * kPer;
  const IO *p = m.at(b, t0 + row) + first + col;
#pragma unroll
  for (int r = 0; r < ROWS; r += 32 / kPieces)
    if (col < cols && row + r < n && row + r < ROWS)
      copy16(dst + (row + r) * COLS + col, p + r * m.ts);
}
template <bool VEC, typename IO, int NL>
__device__ __forceinline__ void copy_segment(const In<IO> &in, const SeqView<const IO> &gy,
                                             Raw<IO, NL> &raw, int64_t b, int64_t g, int64_t c0,
                                             int live, int64_t t0, int n, int lane, bool words,
                                             int *err) {
  using Ge = Geo<NL>;
  if constexpr (!VEC) {
    if (n > 0 && SSD_IN_BOUNDS(t0 >= 0 && t0 + n <= in.L, err, 80)) {
      auto rows = [&](IO *dst, const SeqView<const IO> &m) {
        copy_small<Ge::CW, Ge::SEG>(dst, m.at(b, t0) + c0, m.ts, n, live, lane, words);
      };
      rows(raw.u[0], in.u);
      rows(raw.dt[0], in.dt);
      rows(raw.gy[0], gy);
      if (in.z.p) rows(raw.z[0], in.z);
      const int64_t col = g * in.N;
      copy_small<Ge::NP, Ge::SEG>(raw.B[0], in.B.at(b, t0) + col, in.B.ts, n, in.N, lane, words);
      copy_small<Ge::NP, Ge::SEG>(raw.C[0], in.C.at(b, t0) + col, in.C.ts, n, in.N, lane, words);
    }
  } else if (n > 0 && SSD_IN_BOUNDS(t0 >= 0 && t0 + n <= in.L, err, 80)) {
    copy_rows<Ge::CW, Ge::SEG>(raw.u[0], in.u, b, t0, n, c0, live, lane);
    copy_rows<Ge::CW, Ge::SEG>(raw.dt[0], in.dt, b, t0, n, c0, live, lane);
    copy_rows<Ge::CW, Ge::SEG>(raw.gy[0], gy, b, t0, n, c0, live, lane);
    if (in.z.p) copy_rows<Ge::CW, Ge::SEG>(raw.z[0], in.z, b, t0, n, c0, live, lane);
    copy_rows<Ge::NP, Ge::SEG>(raw.B[0], in.B, b, t0, n, g * in.N, in.N, lane);
    copy_rows<Ge::NP, Ge::SEG>(raw.C[0], in.C, b, t0, n, g * in.N, in.N, lane);
  }
  copies_issued();
}

// Four channels of one token of a view, the first `count` of them.  VEC: all
// four, on their boundary.
template <bool VEC, typename IO>
__device__ __forceinline__ void store_four(const SeqView<IO> &m, int64_t b, int64_t t, int64_t c,
                                           int count, const float (&v)[4]) {
  IO *p = m.at(b, t) + c;
  if constexpr (VEC) {
    store_vec<4>(p, v);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < count) st_io(p + e, v[e]);
  }
}

// The columns of a segment that a lane prepares and finishes, four at a time:
// always the same four, over TURNS tokens.
template <int NL>
struct Lanes {
  using Ge = Geo<NL>;
  static constexpr int PR = Ge::CW / 4, TURNS = Ge::SEG * PR / 32;
  static_assert(PR <= 32 && TURNS >= 1, "");
  // a parameter of those columns
  __device__ static __forceinline__ void load(const float *p, int64_t c0, int live, int lane,
                                              float (&v)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = lane % PR * 4 + e;
      v[e] = p && c < live ? p[c0 + c] : 0.f;
    }
  }
};

// Fills a Stage from `raw`, where n tokens of the segment were copied, and gz =
// gy silu'(z) if asked; zero beyond them and beyond the tile's `live` channels,
// which leaves states and adjoints alone.
template <typename IO, int NL>
__device__ __forceinline__ void fill(const In<IO> &in, const Raw<IO, NL> &raw, Stage<NL> &sm,
                                     float (*gz)[Geo<NL>::CW], int live, int n, int lane,
                                     const float (&bias)[4]) {
  using Ge = Geo<NL>;
  using La = Lanes<NL>;
  const int c = lane % La::PR * 4;
#pragma unroll
  for (int i = 0; i < La::TURNS; ++i) {
    const int r = (lane + i * 32) / La::PR;
    float u[4], dt[4], z[4], go[4], s[4], gd[4];
    load_vec<4>(&raw.u[r][c], u);
    load_vec<4>(&raw.dt[r][c], dt);
    load_vec<4>(&raw.gy[r][c], go);
    load_vec<4>(&raw.z[r][c], z);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool ok = r < n && c + e < live;
      s[e] = ok ? step_of(dt[e] + bias[e], in.softplus) : 0.f;
      u[e] = ok ? u[e] : 0.f;
      gd[e] = 0.f;
      if (!ok) go[e] = 0.f;
      if (ok && in.z.p) {
        const float sig = sigmoid(z[e]);
        gd[e] = go[e] * (sig * fmaf(z[e], 1.f - sig, 1.f));
        go[e] *= z[e] * sig;
      }
    }
    store_vec<4>(&sm.s[r][c], s);
    store_vec<4>(&sm.u[r][c], u);
    store_vec<4>(&sm.o[r][c], go);
    if (gz) store_vec<4>(&gz[r][c], gd);
  }
#pragma unroll
  for (int q = lane; q < Ge::SEG * Ge::NP; q += 32) {
    const int r = q / Ge::NP, k = q % Ge::NP;
    const bool ok = r < n && k < in.N;
    const float vB = ok ? ld_io(&raw.B[r][k]) : 0.f, vC = ok ? ld_io(&raw.C[r][k]) : 0.f;
    sm.B[r][k] = make_float2(vB, vB);
    sm.C[r][k] = make_float2(vC, vC);
  }
}

// A lane's pairs of a state row-major over [channels][N], and of A.
__device__ __forceinline__ pair load_pair(const float *p, int64_t d, int c, int live, int n,
                                          int N) {
  if (n >= N) return 0;
  return pack(c < live ? p[(d + c) * N + n] : 0.f,
              c + 1 < live ? p[(d + c + 1) * N + n] : 0.f);
}
__device__ __forceinline__ pair load_decays(const float *A, int64_t d, int c, int live, int n,
                                            int N) {
  float a, b;
  unpack(load_pair(A, d, c, live, n, N), a, b);
  return pack(log2_decay(a), log2_decay(b));
}

// Two pairs (four channels) of a row of a Stage array; four values, each
// twice, of B or C.
__device__ __forceinline__ void four(const float *p, pair (&v)[2]) {
  const ulonglong2 q = *reinterpret_cast<const ulonglong2 *>(p);
  v[0] = q.x, v[1] = q.y;
}
__device__ __forceinline__ void four_twice(const float2 *p, pair (&v)[4]) {
  const ulonglong2 a = reinterpret_cast<const ulonglong2 *>(p)[0];
  const ulonglong2 b = reinterpret_cast<const ulonglong2 *>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
}

template <typename IO, int NL, bool VEC>
__global__ void __launch_bounds__(32, kMinEnds)
ends_kernel(In<IO> in, SeqView<const IO> gy, Parts parts, Buffers buf, bool words, int *err) {
  using Ge = Geo<NL>;
  extern __shared__ __align__(16) unsigned char raw_smem[];
  Stage<NL> &sm = *reinterpret_cast<Stage<NL> *>(raw_smem);
  Raw<IO, NL> &raw = *reinterpret_cast<Raw<IO, NL> *>(raw_smem + sizeof(Stage<NL>));
  const int lane = threadIdx.x, nl = lane % NL, cg = lane / NL;
  const Unit un = unit_of(blockIdx.x, parts, in.D / in.per_group);
  const int64_t c0 = un.g * in.per_group + un.tile * Ge::CW;
  const int live = min(Ge::CW, in.per_group - un.tile * Ge::CW);
  if (!SSD_IN_BOUNDS(un.b < in.nb && c0 + live <= in.D, err, 71)) return;
  const int64_t len = tokens_of(in.lengths, un.b, in.L);
  float bias[4];
  Lanes<NL>::load(in.dt_bias, c0, live, lane, bias);
  pair A[4][2], P[4][2], R[4][2], all[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      A[i][p] = load_decays(in.A, c0, cg * 4 + p * 2, live, nl * 4 + i, in.N);
      P[i][p] = both(1.f);
      R[i][p] = 0;
    }
  const int64_t last = min((un.part + 1) * parts.per, parts.segments);
  auto tokens = [&](int64_t seg) {  // of a segment
    const int64_t t0 = seg * Ge::SEG;
    return (int)(len - t0 < 0 ? 0 : len - t0 < Ge::SEG ? len - t0 : Ge::SEG);
  };
  auto ahead = [&](int64_t seg) {
    copy_segment<VEC>(in, gy, raw, un.b, un.g, c0, live, seg * Ge::SEG,
                         seg < last ? tokens(seg) : 0, lane, words, err);
  };
  ahead(un.part * parts.per);
  for (int64_t seg = un.part * parts.per; seg < last; ++seg) {
    const int n = tokens(seg);
    pair h[4][2], sum[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i][0] = h[i][1] = 0;
    if (n > 0) {
      copies_landed<0>();
      __syncwarp();
      fill<IO, NL>(in, raw, sm, nullptr, live, n, lane, bias);
      __syncwarp();
      ahead(seg + 1);
#pragma unroll 4
      for (int k = 0; k < Ge::SEG; ++k) {
        pair s[2], su[2], o[2], B[4], C[4];
        four(&sm.s[k][cg * 4], s);
        four(&sm.u[k][cg * 4], su);
        su[0] = mul2(su[0], s[0]), su[1] = mul2(su[1], s[1]);
        four(&sm.o[k][cg * 4], o);
        four_twice(&sm.B[k][nl * 4], B);
        four_twice(&sm.C[k][nl * 4], C);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          sum[p] = add2(sum[p], s[p]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const pair e = ex2_2(mul2(s[p], A[i][p]));
            h[i][p] = fma2(e, h[i][p], mul2(su[p], B[i]));
            P[i][p] = mul2(e, P[i][p]);
            R[i][p] = fma2(P[i][p], mul2(o[p], C[i]), R[i][p]);
          }
        }
      }
    }
    const int64_t at = un.tile_id * parts.segments + seg;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int p = 0; p < 2; ++p)
        reinterpret_cast<pair *>(buf.ends)[(at * 8 + i * 2 + p) * 32 + lane] = h[i][p];
    all[0] = add2(all[0], sum[0]), all[1] = add2(all[1], sum[1]);
    if (nl == 0) {
      pair *q = reinterpret_cast<pair *>(buf.sums + at * Ge::CW + cg * 4);
      q[0] = sum[0], q[1] = sum[1];
    }
  }
  const int64_t at = un.tile_id * parts.parts + un.part;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int p = 0; p < 2; ++p)
      reinterpret_cast<pair *>(buf.adj)[(at * 8 + i * 2 + p) * 32 + lane] = R[i][p];
  if (nl == 0) {
    pair *q = reinterpret_cast<pair *>(buf.part_sums + at * Ge::CW + cg * 4);
    q[0] = all[0], q[1] = all[1];
  }
}

// Two blocks per tile, for the states and for the adjoints: thread (i, p, lane)
// as the warps above hold the pairs.
template <int NL>
__global__ void __launch_bounds__(256)
chain_kernel(const float *__restrict__ A, const float *__restrict__ h0,
             const float *__restrict__ gfinal, float *__restrict__ dh0, Parts parts, Buffers buf,
             int64_t nb, int64_t D, int N, int per_group, int *err) {
  using Ge = Geo<NL>;
  constexpr int kBatch = 8;  // entries loaded ahead
  const int lane = threadIdx.x % 32, ip = threadIdx.x / 32, nl = lane % NL, cg = lane / NL;
  const int64_t G = D / per_group, id = blockIdx.x;
  const int tile = (int)(id % parts.tiles);
  const int64_t g = id / parts.tiles % G, b = id / parts.tiles / G;
  const int64_t c0 = g * per_group + tile * Ge::CW;
  const int live = min(Ge::CW, per_group - tile * Ge::CW);
  if (!SSD_IN_BOUNDS(b < nb && c0 + live <= D, err, 78)) return;
  const int c = cg * 4 + ip % 2 * 2, n = nl * 4 + ip / 2;
  const pair a = load_decays(A, c0, c, live, n, N);
  // x = exp(A sum) x + end over `count` entries, in order or backwards; each
  // entry is replaced by the x that arrives there
  auto chain = [&](pair x, pair *v, const float *sum, int64_t count, bool back) {
    pair end[kBatch], s[kBatch];
    auto load = [&](int64_t k) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int64_t at = back ? count - 1 - k - j : k + j;
        end[j] = s[j] = 0;
        if (k + j < count) {
          end[j] = v[at * 256];
          s[j] = *reinterpret_cast<const pair *>(sum + at * Ge::CW);
        }
      }
    };
    load(0);
    for (int64_t k = 0; k < count; k += kBatch) {
      pair e[kBatch], f[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) e[j] = end[j], f[j] = s[j];
      load(k + kBatch);  // the next entries, before these are replaced
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int64_t at = back ? count - 1 - k - j : k + j;
        if (k + j < count) v[at * 256] = x;
        x = fma2(ex2_2(mul2(f[j], a)), x, e[j]);  // past the end: x itself
      }
    }
    return x;
  };
  const int64_t row = b * D;
  if (blockIdx.y == 0) {
    const pair first = h0 ? load_pair(h0 + row * N, c0, c, live, n, N) : 0;
    chain(first, reinterpret_cast<pair *>(buf.ends) + id * parts.segments * 256 + ip * 32 + lane,
          buf.sums + id * parts.segments * Ge::CW + c, parts.segments, false);
    return;
  }
  const pair arriving = gfinal ? load_pair(gfinal + row * N, c0, c, live, n, N) : 0;
  const pair q =
      chain(arriving, reinterpret_cast<pair *>(buf.adj) + id * parts.parts * 256 + ip * 32 + lane,
            buf.part_sums + id * parts.parts * Ge::CW + c, parts.parts, true);
  if (dh0 && n < N) {
    float x, y;
    unpack(q, x, y);
    if (c < live) dh0[(row + c0 + c) * N + n] = x;
    if (c + 1 < live) dh0[(row + c0 + c + 1) * N + n] = y;
  }
}

template <typename IO>
struct Out {
  SeqView<IO> du, ddt, dz;
};

template <typename IO, int NL>
struct AdjointSmem {
  using Ge = Geo<NL>;
  static constexpr int SUB = Ge::SEG / 4;
  Stage<NL> st;
  float gB[Ge::SEG][Ge::CW], gah[Ge::SEG][Ge::CW];
  float dz[Ge::SEG][Ge::CW];  // gy silu'(z), then times the ungated output
  pair start[SUB > 1 ? SUB - 1 : 1][8][32];  // states in front of tokens 4, 8, ..
  Raw<IO, NL> raw;
};

template <typename IO, int NL, bool VEC>
__global__ void __launch_bounds__(32, kMin)
adjoint_kernel(In<IO> in, SeqView<const IO> gy, Parts parts, Buffers buf, Out<IO> out, bool words,
               int *err) {
  using Ge = Geo<NL>;
  constexpr int SUB = Ge::SEG / 4;
  extern __shared__ __align__(16) unsigned char raw_smem[];
  auto &sm = *reinterpret_cast<AdjointSmem<IO, NL> *>(raw_smem);
  Raw<IO, NL> &raw = sm.raw;
  const int lane = threadIdx.x, nl = lane % NL, cg = lane / NL, N = in.N;
  const int64_t G = in.D / in.per_group;
  const Unit un = unit_of(blockIdx.x, parts, G);
  const int64_t c0 = un.g * in.per_group + un.tile * Ge::CW;
  const int live = min(Ge::CW, in.per_group - un.tile * Ge::CW);
  if (!SSD_IN_BOUNDS(un.b < in.nb && c0 + live <= in.D, err, 72)) return;
  const int64_t len = tokens_of(in.lengths, un.b, in.L);
  pair A[4][2], q[4][2], dA[4][2];
  const int64_t mine = un.tile_id * parts.parts + un.part;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      A[i][p] = load_decays(in.A, c0, cg * 4 + p * 2, live, nl * 4 + i, N);
      q[i][p] = reinterpret_cast<const pair *>(buf.adj)[(mine * 8 + i * 2 + p) * 32 + lane];
      dA[i][p] = 0;
    }
  // which sums this lane is left with, and where they go: dB and dC of states
  // (KC of the eight over the channels), the sums of G B and A q h of channels
  // (KN of the eight over the states)
  constexpr int KC = Ge::CG < 8 ? 8 / Ge::CG : 1, DC = Ge::CG > 8 ? Ge::CG / 8 : 1;
  constexpr int KN = NL < 8 ? 8 / NL : 1, DN = NL > 8 ? NL / 8 : 1;
  constexpr int kRow = Ge::SEG * Ge::CW;  // from gB to gah
  const bool keeps_c = cg % DC == 0, keeps_n = nl % DN == 0;
  const int64_t per_token = G * N;
  float *to_part[KC];
#pragma unroll
  for (int j = 0; j < KC; ++j) {
    const int v = cg / DC * KC + j, st = nl * 4 + v % 4;
    to_part[j] = st >= N ? nullptr
                         : (v < 4 ? buf.partB : buf.partC) +
                               ((un.tile * in.nb + un.b) * in.L * G + un.g) * N + st;
  }
  const int vn = nl / DN * KN;
  float *to_sums = &sm.gB[0][0] + vn / 4 * kRow + cg * 4 + vn % 4;
  using La = Lanes<NL>;
  constexpr int PR = La::PR, TURNS = La::TURNS;
  float bias[4], skip[4];
  La::load(in.dt_bias, c0, live, lane, bias);
  La::load(in.Dskip, c0, live, lane, skip);
  float dD[4], dbias[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) dD[e] = dbias[e] = 0.f;
  // the channels whose output this lane is left with
  constexpr int KEEP = NL < 4 ? 4 / NL : 1, DUP = NL > 4 ? NL / 4 : 1;
  const int out_c = cg * 4 + nl / DUP * KEEP;
  float out_skip[KEEP];
#pragma unroll
  for (int j = 0; j < KEEP; ++j)
    out_skip[j] = in.Dskip && out_c + j < live ? in.Dskip[c0 + out_c + j] : 0.f;

  const int64_t last = min((un.part + 1) * parts.per, parts.segments);
  auto tokens = [&](int64_t seg) {  // of a segment
    const int64_t t0 = seg * Ge::SEG;
    return (int)(len - t0 < 0 ? 0 : len - t0 < Ge::SEG ? len - t0 : Ge::SEG);
  };
  auto ahead = [&](int64_t seg) {
    copy_segment<VEC>(in, gy, raw, un.b, un.g, c0, live, seg * Ge::SEG,
                         seg >= un.part * parts.per ? tokens(seg) : 0, lane, words, err);
  };
  ahead(last - 1);
  for (int64_t seg = last - 1; seg >= un.part * parts.per; --seg) {
    const int64_t t0 = seg * Ge::SEG;
    const int n = tokens(seg);
    const pair *from = reinterpret_cast<const pair *>(buf.ends) +
                       (un.tile_id * parts.segments + seg) * 256 + lane;
    pair h[4][2];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i / 2][i % 2] = from[i * 32];
    copies_landed<0>();
    __syncwarp();
    if (n > 0) {
      fill<IO, NL>(in, raw, sm.st, in.z.p ? sm.dz : nullptr, live, n, lane, bias);
      __syncwarp();
      ahead(seg - 1);
      // the states in front of every fourth token
#pragma unroll 1
      for (int sub = 1; sub < SUB; ++sub) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int t = sub * 4 - 4 + k;
          pair s[2], su[2], B[4];
          four(&sm.st.s[t][cg * 4], s);
          four(&sm.st.u[t][cg * 4], su);
          su[0] = mul2(su[0], s[0]), su[1] = mul2(su[1], s[1]);
          four_twice(&sm.st.B[t][nl * 4], B);
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              h[i][p] = fma2(ex2_2(mul2(s[p], A[i][p])), h[i][p], mul2(su[p], B[i]));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sm.start[sub - 1][i][lane] = h[i / 2][i % 2];
      }
#pragma unroll 1
      for (int sub = SUB - 1; sub >= 0; --sub) {
        pair hs[5][4][2];  // before each token, and after the last
#pragma unroll
        for (int i = 0; i < 8; ++i)
          hs[0][i / 2][i % 2] = sub > 0 ? sm.start[sub > 0 ? sub - 1 : 0][i][lane] : from[i * 32];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int t = sub * 4 + k;
          pair s[2], su[2], B[4], C[4];
          four(&sm.st.s[t][cg * 4], s);
          four(&sm.st.u[t][cg * 4], su);
          su[0] = mul2(su[0], s[0]), su[1] = mul2(su[1], s[1]);
          four_twice(&sm.st.B[t][nl * 4], B);
          four_twice(&sm.st.C[t][nl * 4], C);
          float y[4];
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            pair acc = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              hs[k + 1][i][p] =
                  fma2(ex2_2(mul2(s[p], A[i][p])), hs[k][i][p], mul2(su[p], B[i]));
              acc = fma2(hs[k + 1][i][p], C[i], acc);
            }
            unpack(acc, y[2 * p], y[2 * p + 1]);
          }
          spread<1, NL, 4>(y, lane);
          if (in.z.p && nl % DUP == 0)
#pragma unroll
            for (int j = 0; j < KEEP; ++j)
              sm.dz[t][out_c + j] *=
                  fmaf(NL == 1 ? skip[j] : out_skip[j], sm.st.u[t][out_c + j], y[j]);
        }
#pragma unroll
        for (int k = 3; k >= 0; --k) {
          const int t = sub * 4 + k;
          pair s[2], su[2], o[2], B[4], C[4];
          four(&sm.st.s[t][cg * 4], s);
          four(&sm.st.u[t][cg * 4], su);
          su[0] = mul2(su[0], s[0]), su[1] = mul2(su[1], s[1]);
          four(&sm.st.o[t][cg * 4], o);
          four_twice(&sm.st.B[t][nl * 4], B);
          four_twice(&sm.st.C[t][nl * 4], C);
          float over_c[8], over_n[8];  // dB, dC of the states; sums of G B, A q h of the channels
          pair dB[4], dC[4];
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            pair gB = 0, gah = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const pair Gt = fma2(o[p], C[i], q[i][p]);
              dB[i] = p ? fma2(Gt, su[p], dB[i]) : mul2(Gt, su[p]);
              dC[i] = p ? fma2(hs[k + 1][i][p], o[p], dC[i]) : mul2(hs[k + 1][i][p], o[p]);
              gB = fma2(Gt, B[i], gB);
              q[i][p] = mul2(Gt, ex2_2(mul2(s[p], A[i][p])));
              const pair qh = mul2(q[i][p], hs[k][i][p]);
              dA[i][p] = fma2(s[p], qh, dA[i][p]);
              gah = fma2(A[i][p], qh, gah);
            }
            unpack(gB, over_n[2 * p], over_n[2 * p + 1]);
            unpack(gah, over_n[4 + 2 * p], over_n[4 + 2 * p + 1]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) over_c[i] = sum2(dB[i]), over_c[4 + i] = sum2(dC[i]);
          spread<NL, Ge::CG, 8>(over_c, lane);
          spread<1, NL, 8>(over_n, lane);
          if (keeps_c && t < n)
#pragma unroll
            for (int j = 0; j < KC; ++j)
              if (to_part[j]) to_part[j][(t0 + t) * per_token] = over_c[j];
          if (keeps_n)
#pragma unroll
            for (int j = 0; j < KN; ++j) to_sums[t * Ge::CW + j % 4 + j / 4 * kRow] = over_n[j];
        }
      }
      __syncwarp();
    }
    if (n == 0) ahead(seg - 1);
    // what remains is per token and channel
    const int c = lane % PR * 4, cols = live - c;  // this lane's, if any
#pragma unroll NL == 1 ? 1 : TURNS
    for (int i = 0; i < TURNS; ++i) {
      const int r = (lane + i * 32) / PR;
      const int64_t t = t0 + r;
      if (t >= in.L || cols <= 0) continue;
      float s[4], u[4], o[4], gB[4], gah[4], dz[4], du[4], ddt[4];
      load_vec<4>(&sm.st.s[r][c], s);
      load_vec<4>(&sm.st.u[r][c], u);
      load_vec<4>(&sm.st.o[r][c], o);
      load_vec<4>(&sm.gB[r][c], gB);
      load_vec<4>(&sm.gah[r][c], gah);
      load_vec<4>(&sm.dz[r][c], dz);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool ok = r < n;
        du[e] = ok ? fmaf(s[e], gB[e], skip[e] * o[e]) : 0.f;
        const float g = fmaf(u[e], gB[e], gah[e] * kLn2);
        ddt[e] = !ok ? 0.f : in.softplus ? g * slope_of_step(s[e]) : g;
        dz[e] = ok ? dz[e] : 0.f;
        if (ok) dD[e] = fmaf(o[e], u[e], dD[e]);
        dbias[e] += ddt[e];
      }
      store_four<VEC>(out.du, un.b, t, c0 + c, cols, du);
      store_four<VEC>(out.ddt, un.b, t, c0 + c, cols, ddt);
      if (out.dz.p) store_four<VEC>(out.dz, un.b, t, c0 + c, cols, dz);
    }
  }
  const int64_t row = un.b * parts.parts + un.part;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      float x, y;
      unpack(dA[i][p], x, y);
      const int c = cg * 4 + p * 2, st = nl * 4 + i;
      if (st >= N) continue;
      if (c < live) buf.partA[(row * in.D + c0 + c) * N + st] = x;
      if (c + 1 < live) buf.partA[(row * in.D + c0 + c + 1) * N + st] = y;
    }
  // lanes with the same columns hold different tokens
#pragma unroll
  for (int e = 0; e < 4; ++e) {
#pragma unroll
    for (int off = 16; off >= PR; off /= 2) {
      dD[e] += __shfl_xor_sync(0xffffffffu, dD[e], off);
      dbias[e] += __shfl_xor_sync(0xffffffffu, dbias[e], off);
    }
    const int c = lane % PR * 4 + e;
    if (lane < PR && c < live) {
      buf.partD[row * in.D + c0 + c] = dD[e];
      buf.partBias[row * in.D + c0 + c] = dbias[e];
    }
  }
}

// dB and dC: the tiles' parts in order; zero past a sequence's end.  V states
// of a token to a thread.
template <typename IO, int V>
__global__ void __launch_bounds__(128)
sum_tiles_kernel(const float *__restrict__ partB, const float *__restrict__ partC, int tiles,
                 SeqView<IO> dB, SeqView<IO> dC, const int32_t *__restrict__ lengths, int64_t nb,
                 int64_t L, int64_t GN, int *err) {
  const int64_t i = ((int64_t)blockIdx.x * 128 + threadIdx.x) * V, n = nb * L * GN;
  if (i >= n) return;
  const int64_t c = i % GN, t = i / GN % L, b = i / GN / L;
  if (!SSD_IN_BOUNDS(b < nb && t < L && c + V <= GN, err, 73)) return;
  float s[V];
#pragma unroll
  for (int e = 0; e < V; ++e) s[e] = 0.f;
  const float *part = (blockIdx.y ? partC : partB) + i;
  if (t < tokens_of(lengths, b, L)) {
#pragma unroll 8
    for (int k = 0; k < tiles; ++k) {
      float v[V];
      load_vec<V>(part + k * n, v);
#pragma unroll
      for (int e = 0; e < V; ++e) s[e] += v[e];
    }
  }
  IO *o = (blockIdx.y ? dC : dB).at(b, t) + c;
#pragma unroll
  for (int e = 0; e < V; ++e) st_io(o + e, s[e]);
}

// Segments to a part: enough parts for about two rounds of resident warps, at
// most 16 segments (each part writes 2 KB of dA).
Parts parts_of(const ScanArgs &a, int cw, int seg) {
  Parts p;
  p.tiles = (int)((a.D / a.G + cw - 1) / cw);
  p.segments = (a.L + seg - 1) / seg;
  const int64_t all = a.b * a.G * p.tiles * p.segments, want = (int64_t)sm_count() * 24;
  int64_t per = all / want;
  per = per < 1 ? 1 : per > 16 ? 16 : per;
  if (per > p.segments) per = p.segments;
  p.per = (int)per;
  p.parts = (p.segments + per - 1) / per;
  return p;
}

struct Layout {
  Parts parts;
  size_t ends, sums, adj, part_sums, partB, partC, partA, partD, partBias, total;  // in floats
};
template <int NL>
Layout layout_of(const ScanArgs &a) {
  using Ge = Geo<NL>;
  Layout l;
  l.parts = parts_of(a, Ge::CW, Ge::SEG);
  const Parts &p = l.parts;
  const int64_t ids = a.b * a.G * p.tiles;
  size_t at = 0;
  auto take = [&](int64_t n) {
    const size_t r = at;
    at += (size_t)((n + 63) / 64 * 64);
    return r;
  };
  l.ends = take(ids * p.segments * 512);
  l.sums = take(ids * p.segments * Ge::CW);
  l.adj = take(ids * p.parts * 512);
  l.part_sums = take(ids * p.parts * Ge::CW);
  l.partB = take(p.tiles * a.b * a.L * a.G * a.N);
  l.partC = take(p.tiles * a.b * a.L * a.G * a.N);
  l.partA = take(a.b * p.parts * a.D * a.N);
  l.partD = take(a.b * p.parts * a.D);
  l.partBias = take(a.b * p.parts * a.D);
  l.total = at;
  return l;
}

// Whether the outputs' rows are vectors of four.
bool whole_fours(const ScanArgs &a, ssd_dtype io) {
  const size_t e = io == SSD_BF16 ? 2 : 4;
  return view_aligned(&a.out->du, e, 4 * e) && view_aligned(&a.out->ddt, e, 4 * e) &&
         view_aligned(&a.out->dz, e, 4 * e);
}

}  // namespace

size_t selective_scan_backward_workspace(const ScanArgs &a, ssd_dtype) {
  auto of = [&](auto nl) { return sizeof(float) * layout_of<decltype(nl)::value>(a).total; };
  switch (lanes_of(a.N)) {
    case 1: return of(std::integral_constant<int, 1>{});
    case 2: return of(std::integral_constant<int, 2>{});
    case 4: return of(std::integral_constant<int, 4>{});
    case 8: return of(std::integral_constant<int, 8>{});
    default: return of(std::integral_constant<int, 16>{});
  }
}

cudaError_t launch_selective_scan_backward(const ScanArgs &a, ssd_dtype io, void *ws, int *err,
                                           cudaStream_t st) {
  float *f = static_cast<float *>(ws);
  return dispatch(io, a.N, [&](auto io_c, auto nl_c) {
    using IO = typename decltype(io_c)::type;
    constexpr int NL = decltype(nl_c)::value;
    using Ge = Geo<NL>;
    const Layout l = layout_of<NL>(a);
    Buffers buf;
    buf.ends = reinterpret_cast<float2 *>(f + l.ends), buf.sums = f + l.sums;
    buf.adj = reinterpret_cast<float2 *>(f + l.adj), buf.part_sums = f + l.part_sums;
    buf.partB = f + l.partB, buf.partC = f + l.partC, buf.partA = f + l.partA;
    buf.partD = f + l.partD, buf.partBias = f + l.partBias;
    const In<IO> in = in_of<IO>(a);
    const SeqView<const IO> gy = view_of<const IO>(a.gy);
    const Out<IO> out{view_of<IO>(&a.out->du), view_of<IO>(&a.out->ddt), view_of<IO>(&a.out->dz)};
    const int64_t ids = a.b * a.G * l.parts.tiles, units = ids * l.parts.parts;
    const int piece = piece_of(a, io);
    auto run = [&](auto vec_c) {
      constexpr bool VEC = decltype(vec_c)::value;
      constexpr size_t m0 = sizeof(Stage<NL>) + sizeof(Raw<IO, NL>);
      constexpr size_t m1 = sizeof(AdjointSmem<IO, NL>);
      cudaError_t e = cudaFuncSetAttribute(ends_kernel<IO, NL, VEC>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, (int)m0);
      if (e != cudaSuccess) return e;
      ends_kernel<IO, NL, VEC><<<(unsigned)units, 32, m0, st>>>(in, gy, l.parts, buf, piece == 4,
                                                                err);
      e = cudaGetLastError();
      if (e != cudaSuccess) return e;
      chain_kernel<NL><<<dim3((unsigned)ids, 2), 256, 0, st>>>(
          a.A, a.h0, a.gfinal, a.out->dh0, l.parts, buf, a.b, a.D, (int)a.N, in.per_group, err);
      e = cudaGetLastError();
      if (e != cudaSuccess) return e;
      e = cudaFuncSetAttribute(adjoint_kernel<IO, NL, VEC>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)m1);
      if (e != cudaSuccess) return e;
      adjoint_kernel<IO, NL, VEC><<<(unsigned)units, 32, m1, st>>>(in, gy, l.parts, buf, out,
                                                                   piece == 4, err);
      return cudaGetLastError();
    };
    // 16-byte pieces of rows in and vectors of four out, or any rows (N = 16,
    // 2 x 1024 x 1536: 138 us in bf16 and 166 in fp32, at odd offsets 181 and 209)
    cudaError_t e =
        piece == 16 && whole_fours(a, io) ? run(std::true_type{}) : run(std::false_type{});
    if (e != cudaSuccess) return e;
    const int64_t n = a.b * a.L * a.G * a.N;
    auto tiles = [&](auto v_c) {
      constexpr int V = decltype(v_c)::value;
      sum_tiles_kernel<IO, V><<<dim3((unsigned)((n / V + 127) / 128), 2), 128, 0, st>>>(
          buf.partB, buf.partC, l.parts.tiles, view_of<IO>(&a.out->dB), view_of<IO>(&a.out->dC),
          a.lengths, a.b, a.L, a.G * a.N, err);
    };
    if (a.G * a.N % 4 == 0)
      tiles(std::integral_constant<int, 4>{});
    else
      tiles(std::integral_constant<int, 1>{});
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    ColSum s{};
    s.nseg = 3;
    s.seg[0] = {buf.partA, a.out->dA, a.b * l.parts.parts, a.D * a.N};
    s.seg[1] = {buf.partD, a.out->dD, a.b * l.parts.parts, a.D};
    s.seg[2] = {buf.partBias, a.out->ddt_bias, a.b * l.parts.parts, a.D};
    return launch_colsum(s, err, st);
  });
}

}  // namespace ssd
