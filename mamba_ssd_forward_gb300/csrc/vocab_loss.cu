// Softmax cross entropy of hidden states against a large vocabulary, without
// its logits in memory:
//   z = x W^T,  lse_i = log sum_v exp z_iv,  loss_i = lse_i - z_i,target
//   dz = (exp(z - lse) - onehot) g,  dx = dz W,  dW = dz^T x
//
// Forward: one product (gemm.cuh) whose epilogue keeps, for each row and run of
// columns, the largest logit and the sum of exponentials about it; a second
// launch joins the runs.  Backward: in pieces of the vocabulary the logits are
// computed again, their epilogue writes the piece of dz, and one launch adds its
// shares of dx and computes its rows of dW.  Bound by the tensor cores: 2 n V d
// operations forward, 6 n V d backward.  Measured: 8192 tokens x 2560, 50280 words,
// bf16, forward and backward 5170 to 5250 us, 1.61 to 1.63 PFLOP/s (under the power cap);
// forward of 2048 x 768 107 us, 1.5 PFLOP/s; 1021 x 771, 32003 words, fp32, 537 us; forward of
// 5 x 2560, 50280 words, bf16, 58 us, 4.4 TB/s of W.
//
// Tokens without a target are left out before the products: the others' rows of
// x are packed together (so whatever the left out rows hold reaches nothing),
// their number stays on the device.
//
// bf16: the products of the logits are exact, their fp32 sums those of the tensor cores,
// which cut towards zero at 24 bits with each 16 channels (all d in one go: losses measured
// 4e-7 off, 6e-8 where the same products are added with rounding; the fp32 path's segments
// would keep the epilogue from running under the next tile's products).  dz is rounded once
// to bf16, as the operand of both gradient products (up to 2^-8 of each term, as far off
// as the gradients' own rounding); a factor common to all tokens is applied to
// the fp32 sums instead.  fp32: x, W and dz are split into two fp16 planes after
// scaling by powers of two that take the largest value to 2^14..2^15 (values
// below 2^-28 of the largest keep 2^-39 of it), three products each.  Tokens' factors
// of their own may be of very different sizes, so they are no part of dz there: dx takes a
// token's factor after the product, dW from g x in the place of x.
#include <cmath>

#include "gemm.cuh"
#include "model.cuh"

namespace ssd {
namespace {

using gemm::Product;
using gemm::Tile;

constexpr int kBN = 256;
constexpr int kRun = kBN / 2;  // columns of one epilogue warp: a run of the statistics

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// ------------------------------------------------- largest values, and scales

// The power of two (its exponent) that takes values of the size of `top` (a float's
// bits) to 2^14 .. 2^15; 0 for zero.
__device__ __forceinline__ int shift_of(uint32_t top) {
  if (top == 0) return 0;
  const int e = (int)(top >> 23) - 127;
  return 14 - (e < -110 ? -110 : e);
}
// 2^e, held within 2^-126 .. 2^127.  (Not zero below: logits are multiplied by it, and
// the words that fill up a row's last tile are -inf.  A sum of 65536 products of scaled
// operands is at most 2^46, so a logit that is held is 2^-80 at most.)
__device__ __forceinline__ float pow2(int e) {
  e = e < -126 ? -126 : e > 127 ? 127 : e;
  return __uint_as_float((uint32_t)(127 + e) << 23);
}

// kTopG: of g x, for factors that each token has of its own; the sum of the largest two's
// exponents plus kTopBias (0: nothing but zeros).
enum Top { kTopX, kTopW, kTopG, kTops };
constexpr int kTopBias = 512;
// The exponent that takes the products g x below 2^15.
__device__ __forceinline__ int product_shift(uint32_t top) {
  return top == 0 ? 0 : 13 - ((int)top - kTopBias);
}

__device__ __forceinline__ bool counted(int64_t target, int64_t ignore) { return target != ignore; }

// Bits of the largest finite |value| of x's rows with a target and of W, and the size of
// the largest g x.  (A row's infinity or NaN must not cost the other rows their
// scale.)  The order of the maxima has no say.
__device__ __forceinline__ uint32_t size_of(float v) {
  const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}
__global__ void __launch_bounds__(256)
top_kernel(SeqView<const float> x, const int64_t *__restrict__ targets, int64_t ignore, int64_t L,
           int64_t n, const float *__restrict__ w, int64_t ws, int64_t V, int64_t d,
           const float *__restrict__ g, uint32_t *__restrict__ top, int *err) {
  uint32_t most[kTops] = {0, 0, 0};
  const int64_t thread = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, lane = threadIdx.x % 32;
  const int64_t threads = (int64_t)gridDim.x * blockDim.x, warp = thread / 32, warps = threads / 32;
  // W's rows one after the other are one run (row by row, 4 bytes a lane, 32003 x 771
  // took 29 us, so 23)
  const bool run = ws == d && (reinterpret_cast<uintptr_t>(w) & 15) == 0;
  if (run) {
    constexpr int kAtOnce = 8;
    const int64_t all = V * d, vecs = all / 4;
    uint32_t m = 0;
    for (int64_t i = thread; i < vecs; i += kAtOnce * threads) {
      float4 v[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int64_t at = i + k * threads;
        v[k] = at < vecs && SSD_IN_BOUNDS(4 * at + 4 <= V * d, err, 510)
                   ? reinterpret_cast<const float4 *>(w)[at]
                   : make_float4(0, 0, 0, 0);
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
        m = max(max(m, max(size_of(v[k].x), size_of(v[k].y))),
                max(size_of(v[k].z), size_of(v[k].w)));
    }
    if (4 * vecs + thread < all) m = max(m, size_of(w[4 * vecs + thread]));
    most[kTopW] = m;
  }
  for (int64_t r = warp; r < (run ? n : n + V); r += warps) {
    if (r < n && !counted(targets[r], ignore)) continue;
    const float *p = r < n ? x.at(r / L, r % L) : w + (r - n) * ws;
    uint32_t m = 0;
    if (!SSD_IN_BOUNDS(r < n + V, err, 511)) continue;
    for (int64_t c = lane; c < d; c += 8 * 32) {
      uint32_t v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = c + 32 * k < d ? size_of(p[c + 32 * k]) : 0u;
#pragma unroll
      for (int k = 0; k < 8; ++k) m = max(m, v[k]);
    }
    if (r < n) {
      most[kTopX] = max(most[kTopX], m);
      if (const uint32_t f = g ? size_of(g[r]) : 0u; f && m)
        most[kTopG] = max(most[kTopG], (m >> 23) + (f >> 23) - 2 * 127 + kTopBias);
    } else {
      most[kTopW] = max(most[kTopW], m);
    }
  }
#pragma unroll
  for (int k = 0; k < kTops; ++k) {
    const uint32_t m = __reduce_max_sync(0xffffffffu, most[k]);
    if (lane == 0 && m) atomicMax(top + k, m);
  }
}

// --------------------------------------------------------------- packed rows

// One value in the operand type: bf16 as it is, or the planes of an fp32.
__device__ __forceinline__ void split(float v, float scale, __half &hi, __half &lo) {
  const float s = v * scale;
  hi = __float2half_rn(s);
  lo = __float2half_rn(s - __half2float(hi));
}
// A row of `d` values into its place (and, fp32, into the second plane `ps`
// elements on).
__device__ __forceinline__ void pack_row(const __nv_bfloat16 *src, uint16_t *dst, int64_t,
                                         int64_t d, float, int tid, int threads) {
  const uint16_t *s = reinterpret_cast<const uint16_t *>(src);
  const int64_t wide = ((reinterpret_cast<uintptr_t>(src) & 15) == 0) ? d / 8 : 0;
#pragma unroll 4
  for (int64_t i = tid; i < wide; i += threads)
    reinterpret_cast<uint4 *>(dst)[i] = reinterpret_cast<const uint4 *>(s)[i];
  constexpr int kAtOnce = 8;
  for (int64_t i = 8 * wide + tid; i < d; i += kAtOnce * threads) {
    uint16_t v[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) v[k] = i + k * threads < d ? s[i + k * threads] : 0;
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
      if (i + k * threads < d) dst[i + k * threads] = v[k];
  }
}
template <typename F>
__device__ __forceinline__ void pack_planes(const float *src, uint16_t *dst, int64_t ps, int64_t d,
                                            F scaled, int tid, int threads) {
  constexpr int kAtOnce = 8;
  for (int64_t i = tid; i < d; i += kAtOnce * threads) {
    float v[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) v[k] = i + k * threads < d ? src[i + k * threads] : 0.f;
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      __half hi, lo;
      split(scaled(v[k]), 1.f, hi, lo);
      if (i + k * threads < d) {
        dst[i + k * threads] = __half_as_ushort(hi);
        dst[ps + i + k * threads] = __half_as_ushort(lo);
      }
    }
  }
}
__device__ __forceinline__ void pack_row(const float *src, uint16_t *dst, int64_t ps, int64_t d,
                                         float scale, int tid, int threads) {
  pack_planes(src, dst, ps, d, [=](float v) { return v * scale; }, tid, threads);
}
// The same of a row times its token's factor and 2^shift: x 2^k m with g 2^shift = m 2^k,
// 2^k in halves, so that nothing between leaves the number range.
__device__ __forceinline__ void pack_product(const float *src, uint16_t *dst, int64_t ps,
                                             int64_t d, float g, int shift, int tid, int threads) {
  int k = 0;
  float m = g;
  if (g != 0.f && isfinite(g)) m = frexpf(g, &k), k += shift;
  const float a = pow2(k / 2), b = pow2(k - k / 2);
  pack_planes(src, dst, ps, d, [=](float v) { return v * a * b * m; }, tid, threads);
}

// What the later launches know of the rows with a target.
struct Rows {
  int *live;       // their number
  int *token;      // [n] which token each is
  int *target;     // [n] its target, -1 if that is no word
  float *zt;       // [n] its target's logit (forward)
  float *lse, *g;  // [n] (backward)
};

constexpr int kPackTokens = 8, kPackThreads = 256;  // a warp to a token
constexpr int kPackCols = 256;                      // columns to a block at least
constexpr int kGroup = 2048;                        // tokens counted together

// Targets of each group of tokens.
__global__ void __launch_bounds__(kPackThreads)
count_kernel(const int64_t *__restrict__ targets, int64_t ignore, int64_t n,
             int *__restrict__ counts, int *err) {
  __shared__ int sums[kPackThreads / 32];
  const int64_t first = (int64_t)blockIdx.x * kGroup;
  int c = 0;
#pragma unroll
  for (int k = 0; k < kGroup / kPackThreads; ++k) {
    const int64_t i = first + k * kPackThreads + threadIdx.x;
    if (i < n) c += counted(targets[i], ignore);
  }
  c = __reduce_add_sync(0xffffffffu, c);
  if (threadIdx.x % 32 == 0) sums[threadIdx.x / 32] = c;
  __syncthreads();
  if (threadIdx.x || !SSD_IN_BOUNDS(first < n, err, 512)) return;
  for (int w = 1; w < kPackThreads / 32; ++w) c += sums[w];
  counts[blockIdx.x] = c;
}

// A block takes kPackTokens tokens, and of few tokens `cols` columns (a warp takes its
// row load by load: 4 x 2370 bf16 30 us from cold caches as one block, 5 so).  It counts the targets in front of them
// itself (they come from L2), so no launch of its own makes the list; of many
// tokens (counts not NULL) those of whole groups are counted before.
template <typename IO>
__global__ void __launch_bounds__(kPackThreads)
pack_kernel(SeqView<const IO> x, const int64_t *__restrict__ targets, int64_t ignore, int64_t V,
            int64_t L, int64_t n, int64_t d, const float *__restrict__ lse,
            const float *__restrict__ gloss, SeqView<IO> dx, float *__restrict__ loss,
            float *__restrict__ lse_out, const int *__restrict__ counts, Rows rows,
            uint16_t *__restrict__ xp, uint16_t *__restrict__ xg, int64_t ld, int64_t ps,
            int planes, int64_t cols, const uint32_t *__restrict__ top, int *err) {
  __shared__ int sums[kPackThreads / 32], place[kPackTokens], mine_all;
  const int64_t first = (int64_t)blockIdx.x * kPackTokens;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  if (!SSD_IN_BOUNDS(first < n, err, 513)) return;
  int before = 0;
  const int64_t groups = counts ? first / kGroup : 0;
  for (int64_t i = tid; i < groups; i += kPackThreads) before += counts[i];
#pragma unroll 4
  for (int64_t i = groups * kGroup + tid; i < first; i += kPackThreads)
    before += counted(targets[i], ignore);
  before = __reduce_add_sync(0xffffffffu, before);
  if (lane == 0) sums[warp] = before;
  __syncthreads();
  before = 0;
#pragma unroll
  for (int w = 0; w < kPackThreads / 32; ++w) before += sums[w];
  const int here = (int)(n - first < kPackTokens ? n - first : kPackTokens);
  if (warp == 0) {
    const bool mine = lane < here && counted(targets[first + (lane < here ? lane : 0)], ignore);
    const unsigned all = __ballot_sync(0xffffffffu, mine);
    if (lane < kPackTokens) place[lane] = mine ? before + __popc(all & ((1u << lane) - 1)) : -1;
    if (lane == 0) mine_all = __popc(all);
    __syncwarp();
    if (lane < here && blockIdx.y == 0) {
      const int64_t t = first + lane;
      if (mine && SSD_IN_BOUNDS(place[lane] < n, err, 514)) {
        const int64_t word = targets[t];
        const bool real = word >= 0 && word < V;
        rows.token[place[lane]] = (int)t;
        rows.target[place[lane]] = real ? (int)word : -1;
        if (rows.zt) rows.zt[place[lane]] = __int_as_float(0x7fc00000);  // until a tile writes it
        if (rows.lse) {
          rows.lse[place[lane]] = lse[t];
          rows.g[place[lane]] = !real ? __int_as_float(0x7fc00000) : gloss ? gloss[t] : 1.f;
        }
      } else if (!mine) {
        if (loss) loss[t] = 0.f;
        if (lse_out) lse_out[t] = 0.f;
      }
    }
  }
  __syncthreads();
  const float scale = top ? pow2(shift_of(top[kTopX])) : 1.f;
  if (warp < here) {
    const int64_t t = first + warp, b = t / L, at = t % L;
    const int64_t c0 = blockIdx.y * cols, n_cols = d - c0 < cols ? d - c0 : cols;
    const bool fits = SSD_IN_BOUNDS(place[warp] < n && c0 + n_cols <= ld &&
                                        ((int64_t)place[warp] + 1) * ld <= ps, err, 515);
    if (fits && place[warp] >= 0) {
      const int64_t to = (int64_t)place[warp] * ld + c0;
      pack_row(x.at(b, at) + c0, xp + to, ps, n_cols, scale, lane, 32);
      if constexpr (sizeof(IO) == 4) {
        const int64_t word = targets[t];
        if (xg)
          pack_product(x.at(b, at) + c0, xg + to, ps, n_cols,
                       word >= 0 && word < V ? gloss[t] : __int_as_float(0x7fc00000),
                       product_shift(top[kTopG]), lane, 32);
      }
    } else if (fits && dx.p)
      for (int64_t c = lane; c < n_cols; c += 32) st_io(dx.at(b, at) + c0 + c, 0.f);
  }
  if (first + kPackTokens < n || blockIdx.y) return;
  const int64_t live = before + mine_all;
  if (tid == 0) *rows.live = (int)live;
  // backward the rows are k of a product, in stages of kTileK: the last one's other
  // rows are zero (as are those of dz), whatever lay there
  const int64_t end = rows.lse ? (live + gemm::kTileK - 1) / gemm::kTileK * gemm::kTileK : live;
  for (int p = 0; p < planes; ++p)
    for (int64_t i = (live * ld) / 8 + tid; i < end * ld / 8; i += kPackThreads) {
      if (!SSD_IN_BOUNDS(8 * i + 8 <= ps, err, 516)) break;
      reinterpret_cast<uint4 *>(xp + p * ps)[i] = make_uint4(0, 0, 0, 0);
      if (xg) reinterpret_cast<uint4 *>(xg + p * ps)[i] = make_uint4(0, 0, 0, 0);
    }
}

// Rows of W for the products, where TMA cannot take them as they are.
template <typename IO>
__global__ void __launch_bounds__(256)
pack_weight_kernel(const IO *__restrict__ w, int64_t ws, int64_t rows, int64_t d,
                   uint16_t *__restrict__ wp, int64_t ld, int64_t ps,
                   const uint32_t *__restrict__ top, int *err) {
  const int64_t r = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  if (r >= rows || !SSD_IN_BOUNDS(r * ld + d <= ps, err, 517)) return;
  pack_row(w + r * ws, wp + r * ld, ps, d, top ? pow2(shift_of(top[kTopW])) : 1.f,
           threadIdx.x % 32, 32);
}

// ------------------------------------------------------------------ epilogues

// The logits' statistics: the largest logit m and the sum of exp(z - m), each
// exponential off by 2^-21 of itself.  (About m rather than in units of log2 from
// the start, which would cost a multiplication less: logits near the end of the
// number range would overflow.)
struct StatsEpi {
  struct Args {
    float2 *part;  // [runs][ld]
    int64_t ld, n;  // rows of `part`; tokens
    Rows rows;
    const uint32_t *top;
    int V, word0, run0, runs;  // words of this piece; its first word and run; all runs
  };
  const Args &a;
  int *err;
  static constexpr bool kStaged = false;
  static constexpr int kWarps = 8;
  using Pane = gemm::Panes<128>;
  float unit, m, s;  // unit: a logit to the tensor cores' sum
  int row, run, target;
  bool live;
  __device__ __forceinline__ StatsEpi(const Args &args, Pane, int *e) : a(args), err(e) {
    unit = a.top ? pow2(-shift_of(a.top[kTopX]) - shift_of(a.top[kTopW])) : 1.f;
  }
  __device__ __forceinline__ void begin(const Tile &, int r, int col, int M) {
    row = r, live = r < M, run = a.run0 + col / kRun;
    m = -INFINITY, s = 0.f;
    target = live && SSD_IN_BOUNDS(r < a.n, err, 518) ? a.rows.target[r] - a.word0 : -1;
  }
  __device__ __forceinline__ void chunk(float (&v)[gemm::kChunk], int col, int) {
    if (col >= a.V) return;
    const int words = a.V - col;
    const int at = target - col;
    if (at >= 0 && at < gemm::kChunk && at < words) {
      float z = 0.f;
#pragma unroll
      for (int i = 0; i < gemm::kChunk; ++i) z = i == at ? v[i] : z;
      if (SSD_IN_BOUNDS(row < a.n, err, 519)) a.rows.zt[row] = z * unit;
    }
    if (words < gemm::kChunk) {
#pragma unroll
      for (int i = 0; i < gemm::kChunk; ++i) v[i] = i < words ? v[i] : -INFINITY;
    }
    float top = v[0];
#pragma unroll
    for (int i = 1; i < gemm::kChunk; ++i) top = fmaxf(top, v[i]);
    const float next = fmaxf(m, top * unit);
    const float about = next == -INFINITY ? 0.f : next;  // of nothing but -inf the sum is zero
    float q[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < gemm::kChunk; ++i) q[i % 4] += ex2(fmaf(v[i], unit, -about) * kLog2e);
    s = s * ex2((m - about) * kLog2e) + ((q[0] + q[1]) + (q[2] + q[3]));
    m = next;
  }
  __device__ __forceinline__ void end() {
    if (live && SSD_IN_BOUNDS(row < a.ld && run < a.runs, err, 520))
      a.part[(int64_t)run * a.ld + row] = make_float2(m, s);
  }
};

// Eight values as bf16, or as the planes of an fp32.
__device__ __forceinline__ uint4 pack8(const float *v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void split8(const float *v, uint4 &hi, uint4 &lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __half h0, l0, h1, l1;
    split(v[2 * i], 1.f, h0, l0);
    split(v[2 * i + 1], 1.f, h1, l1);
    h[i] = __half_as_ushort(h0) | (uint32_t)__half_as_ushort(h1) << 16;
    l[i] = __half_as_ushort(l0) | (uint32_t)__half_as_ushort(l1) << 16;
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// dz of a piece of the vocabulary.
template <typename IO>
struct DlogitEpi {
  struct Args {
    CUtensorMap dz;
    Rows rows;
    const uint32_t *top;
    int64_t n;  // tokens
    int V, word0, own;  // own: each token has a factor, which is no part of dz
  };
  static constexpr bool kStaged = true, kSplit = sizeof(IO) == 4;
  static constexpr int kWarps = 8;
  using Pane = gemm::Panes<128>;
  const Args &a;
  Pane panes;
  int *err;
  float scale, up, lse, g;
  int row0, target;
  bool live;
  __device__ __forceinline__ DlogitEpi(const Args &args, Pane p, int *e)
      : a(args), panes(p), err(e) {
    scale = up = 1.f;
    if constexpr (kSplit) {
      scale = pow2(-shift_of(a.top[kTopX]) - shift_of(a.top[kTopW]));
      up = pow2(14);
    }
  }
  __device__ __forceinline__ void begin(const Tile &, int r, int, int M) {
    row0 = r - panes.lane, live = r < M && SSD_IN_BOUNDS(r < a.n, err, 521);
    lse = live ? a.rows.lse[r] : 0.f;
    g = live ? (a.own ? up : a.rows.g[r] * up) : 0.f;
    target = live ? a.rows.target[r] - a.word0 : -1;
  }
  __device__ __forceinline__ void chunk(float (&v)[gemm::kChunk], int col, int j) {
    const int words = a.V - col, at = target - col;
#pragma unroll
    for (int i = 0; i < gemm::kChunk; ++i) {
      float p = ex2(fmaf(v[i], scale, -lse) * kLog2e);
      if (i == at) p -= 1.f;
      v[i] = live && i < words ? p * g : 0.f;
    }
    const int first = (j & 1) * 4;  // pieces of the pane's row: 64 columns in two chunks
    if constexpr (kSplit) {
      if (first == 0) panes.reuse<0>();
#pragma unroll
      for (int i = 0; i < 4; ++i)
        split8(v + 8 * i, panes.cell(0, first + i), panes.cell(1, first + i));
      if (first == 0) return;
      panes.written();
      if (gemm::elected()) {
        panes.store(0, &a.dz, col - gemm::kChunk, row0, 0);
        panes.store(1, &a.dz, col - gemm::kChunk, row0, 1);
        ptx::bulk_commit();
      }
    } else {
      const int pane = (j >> 1) & 1;
      if (first == 0) panes.reuse<1>();
#pragma unroll
      for (int i = 0; i < 4; ++i) panes.cell(pane, first + i) = pack8(v + 8 * i);
      if (first == 0) return;
      panes.written();
      if (gemm::elected()) {
        panes.store(pane, &a.dz, col - gemm::kChunk, row0, 0);
        ptx::bulk_commit();
      }
    }
  }
  __device__ __forceinline__ void end() {}
};

// What the sums of the gradient products are short of: the scales of their
// operands, and the factor that all tokens have in common.
struct Factors {
  Rows rows;
  const uint32_t *top;
  const float *gloss;  // one value for all tokens, or NULL
  int own, mean;       // own: each token has a factor, which dz is short of too
  // Three factors, to be applied in turn: the halves of the scales' exponent, so
  // that nothing between leaves the number range, and the common factor.
  __device__ __forceinline__ float3 of(Top other) const {
    float3 f = make_float3(1.f, 1.f, gloss ? *gloss : 1.f);
    if (mean) {
      const int n = *rows.live;
      f.z /= (float)(n > 1 ? n : 1);
    }
    if (top) {
      const int e = -14 - (own && other == kTopX ? product_shift(top[kTopG])
                                                 : shift_of(top[other]));
      f.x = pow2(e / 2), f.y = pow2(e - e / 2);
    }
    return f;
  }
};
__device__ __forceinline__ float scaled(float v, const float3 &f) { return v * f.x * f.y * f.z; }

// The gradients: product 0 adds up dx over the pieces in fp32 (a slab for each
// part of a piece), product 1 is a piece of dW.
template <typename IO>
struct GradEpi {
  struct Args {
    CUtensorMap sum, dw;  // dw: where its rows allow TMA
    IO *out;              // this piece's rows of dW
    Factors f;
    int d, words, first, direct;
  };
  static constexpr bool kStaged = true, kWide = sizeof(IO) == 4;
  static constexpr int kWarps = 8;
  using Pane = gemm::Panes<128>;
  const Args &a;
  Pane panes;
  int *err;
  float3 factor;
  int which, row0, slab, pane;  // pane: the one whose store is the older
  __device__ __forceinline__ GradEpi(const Args &args, Pane p, int *e)
      : a(args), panes(p), err(e), factor(args.f.of(kTopX)), pane(0) {}
  __device__ __forceinline__ void begin(const Tile &o, int r, int, int) {
    which = o.which, row0 = r - panes.lane, slab = o.batch;
  }
  // 32 columns of fp32 into a pane
  __device__ __forceinline__ void put(const float (&v)[gemm::kChunk]) {
    panes.reuse<1>();
#pragma unroll
    for (int i = 0; i < 8; ++i)
      panes.cell(pane, i) =
          make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                     __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3]));
    panes.written();
  }
  __device__ __forceinline__ void chunk(float (&v)[gemm::kChunk], int col, int j) {
    if (which == 0) {
      if (col >= a.d) return;
      put(v);
      if (gemm::elected()) {
        if (a.first) panes.store(pane, &a.sum, col, row0, slab);
        else panes.add(pane, &a.sum, col, row0, slab);
        ptx::bulk_commit();
      }
      pane ^= 1;
      return;
    }
#pragma unroll
    for (int i = 0; i < gemm::kChunk; ++i) v[i] = scaled(v[i], factor);
    if constexpr (kWide) {
      if (col >= a.d || row0 >= a.words) return;
      put(v);
    } else {
      const int first = (j & 1) * 4;  // pieces of the pane's row: 64 columns in two chunks
      if (first) col -= gemm::kChunk;
      if (col >= a.d || row0 >= a.words) return;
      if (first == 0) panes.reuse<1>();
#pragma unroll
      for (int i = 0; i < 4; ++i) panes.cell(pane, first + i) = pack8(v + 8 * i);
      if (first == 0) return;
      panes.written();
    }
    if (!a.direct) copy(col);
    if (gemm::elected()) {
      if (a.direct) panes.store(pane, &a.dw, col, row0, 0);
      // A group for each use of a pane, an empty one where its values are copied: with
      // all but the newest group read, the other pane's store is, also that of the last
      // tile of dx.
      ptx::bulk_commit();
    }
    pane ^= 1;
  }
  // A pane to rows that TMA cannot write: lanes along the columns.
  __device__ __forceinline__ void copy(int col) {
    const int rows = min(32, a.words - row0);
#pragma unroll 4
    for (int r = 0; r < rows; ++r) {
      const uint32_t w = panes.word(pane, r, panes.lane);
      if (!SSD_IN_BOUNDS(row0 + r < a.words && col < a.d, err, 522)) break;
      IO *o = a.out + (int64_t)(row0 + r) * a.d + col;
      if constexpr (kWide) {
        if (col + panes.lane < a.d) o[panes.lane] = __uint_as_float(w);
      } else {
        uint16_t *u = reinterpret_cast<uint16_t *>(o) + 2 * panes.lane;
        if (col + 2 * panes.lane < a.d) u[0] = (uint16_t)w;
        if (col + 2 * panes.lane + 1 < a.d) u[1] = (uint16_t)(w >> 16);
      }
    }
    __syncwarp();
  }
  __device__ __forceinline__ void end() {}
};

// dx of the tokens with a target: its slabs added in their order, scaled, and
// put back in the tokens' places.  A warp takes 128 columns of a row.
template <typename IO>
__global__ void __launch_bounds__(256)
unpack_kernel(const float *__restrict__ sum, int64_t ld, int64_t zs, int slabs, Factors f,
              SeqView<IO> dx, int64_t L, int64_t d, int *err) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const float3 factor = f.of(kTopW);
  const int live = *f.rows.live, lane = threadIdx.x % 32;
  const int64_t r = blockIdx.x;
  if (r >= live) return;
  const int64_t t = f.rows.token[r];
  if (!SSD_IN_BOUNDS(t < gridDim.x && (r + 1) * ld <= zs, err, 523)) return;
  const float g = f.own ? f.rows.g[r] : 1.f;
  // a large factor last, a small one between the halves: nothing on the way is larger
  // than the result or the sum
  const bool last = fabsf(g) >= 1.f;
  const float g0 = last ? 1.f : g, g1 = last ? g : 1.f;
  IO *o = dx.at(t / L, t % L);
  for (int64_t c = (threadIdx.x / 32) * 128 + lane * 4; c < d; c += blockDim.x * 4) {
    float v[4] = {0.f, 0.f, 0.f, 0.f};  // (ld is a multiple of 16)
#pragma unroll 8
    for (int z = 0; z < slabs; ++z) {
      if (!SSD_IN_BOUNDS(c + 4 <= ld, err, 524)) break;
      const float4 q = *reinterpret_cast<const float4 *>(sum + z * zs + r * ld + c);
      v[0] += q.x, v[1] += q.y, v[2] += q.z, v[3] += q.w;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c + e < d) st_io(o + c + e, v[e] * factor.x * g0 * factor.y * factor.z * g1);
  }
}

// ------------------------------------------------------------ joining the runs

// 32 rows (lanes) to a block; its warps take the runs in turn and their results
// are joined in the warps' order.
constexpr int kJoinWarps = 32;
__global__ void __launch_bounds__(32 * kJoinWarps)
join_kernel(const float2 *__restrict__ part, int64_t ld, int64_t n, int runs, Rows rows,
            float *__restrict__ loss, float *__restrict__ lse, int *err) {
  __shared__ float2 each[kJoinWarps][32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t row = (int64_t)blockIdx.x * 32 + lane;
  const bool live = row < *rows.live;
  float m = -INFINITY, s = 0.f;
  auto join = [&](float2 q) {
    const float next = fmaxf(m, q.x), about = next == -INFINITY ? 0.f : next;
    s = s * ex2((m - about) * kLog2e) + q.y * ex2((q.x - about) * kLog2e);
    m = next;
  };
  if (live && SSD_IN_BOUNDS(row < n && row < ld, err, 525)) {
    int r = warp;
    for (; r + 3 * kJoinWarps < runs; r += 4 * kJoinWarps) {  // four loads at a time
      float2 q[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) q[k] = part[(int64_t)(r + k * kJoinWarps) * ld + row];
#pragma unroll
      for (int k = 0; k < 4; ++k) join(q[k]);
    }
    for (; r < runs; r += kJoinWarps) join(part[(int64_t)r * ld + row]);
  }
  each[warp][lane] = make_float2(m, s);
  __syncthreads();
  if (warp || !live) return;
  for (int w = 1; w < kJoinWarps; ++w) join(each[w][lane]);
  const float l = m + logf(s);
  const int t = rows.token[row];
  if (!SSD_IN_BOUNDS(t < n, err, 526)) return;
  lse[t] = l;
  loss[t] = l - rows.zt[row];
}

// The sum of every token's loss (or the mean over those with a target, 0 without
// one), in a fixed order.
__global__ void __launch_bounds__(1024)
total_kernel(const float *__restrict__ loss, int64_t n, const int *__restrict__ live, int mean,
             float *__restrict__ total) {
  __shared__ float sums[32];
  float s = 0.f;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
#pragma unroll 8
  for (int64_t i = threadIdx.x; i < n; i += 1024) s += loss[i];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  if (threadIdx.x % 32 == 0) sums[threadIdx.x / 32] = s;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  s = sums[threadIdx.x];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  if (threadIdx.x == 0) *total = mean ? s / (float)(*live > 1 ? *live : 1) : s;
}

// -------------------------------------------------------------------- the host

// What a call keeps where.  Pieces: words to a piece (forward: all where W can be
// taken as it is, else as many as keep the packed rows near 256 MB; backward: as
// many as keep dz near that, but 2048 at least, which fill the tiles: more than 65536
// tokens, 32768 in fp32, take more).
struct Plan {
  int planes;
  int64_t rows, ld, piece, dz_ld;  // padded rows; elements to a packed row; words; dz's row
  bool direct;                     // W as it is
  uint32_t *top;
  int *counts;  // NULL for few tokens
  Rows r;
  uint16_t *xp, *xg, *wp, *dz;     // xg: x times the tokens' own factors, NULL if there are none
  float2 *stat;
  float *loss, *sum;
  int64_t runs;
  int slabs, part;  // parts of the k of dx (the piece's words), stages in each
  size_t bytes;
};

constexpr int64_t kPieceBytes = 256ll << 20;

Plan plan_of(const LossArgs &a, ssd_dtype io, bool back, void *ws) {
  Plan p{};
  p.planes = io == SSD_F32 ? 2 : 1;
  p.rows = round_up(a.n, gemm::kTileM);
  p.ld = gemm::padded(a.d);
  p.direct = io == SSD_BF16 && ptr_aligned(a.weight->data, 16) &&
             a.weight->token_stride % 8 == 0 && a.weight->token_stride >= a.d;
  const int64_t all = round_up(a.V, kBN);
  const int64_t per = 2 * p.planes * (back ? p.rows : p.ld);  // bytes to a word
  int64_t piece = kPieceBytes / per / kBN * kBN;
  if (piece < 2048) piece = 2048;
  if (!back && p.direct) piece = all;
  const int64_t pieces = (all + piece - 1) / piece;
  p.piece = round_up((all + pieces - 1) / pieces, kBN);
  p.dz_ld = p.piece;
  p.runs = all / kRun;
  Carver c(ws);
  p.top = c.take<uint32_t>(kTops);
  // (a block would count 8192 targets in a few microseconds, 10^6 in 100)
  p.counts = a.n > 4 * kGroup ? c.take<int>((a.n + kGroup - 1) / kGroup) : nullptr;
  p.r.live = c.take<int>(1);
  p.r.token = c.take<int>(a.n);
  p.r.target = c.take<int>(a.n);
  p.xp = c.take<uint16_t>(p.planes * p.rows * p.ld);
  p.wp = c.take<uint16_t>(p.direct ? 0 : p.planes * p.piece * p.ld);
  if (back) {
    p.r.lse = c.take<float>(a.n);
    p.r.g = c.take<float>(a.n);
    if (p.planes == 2 && a.reduction == SSD_REDUCE_NONE)
      p.xg = c.take<uint16_t>(p.planes * p.rows * p.ld);
    if (!a.gloss || !a.dweight) p.xg = nullptr;
    p.dz = c.take<uint16_t>(p.planes * p.rows * p.dz_ld);
    // dx has few tiles and many k where there are few tokens: as many parts as
    // make two of its tiles no longer than a pair's share of all stages
    const int64_t tn = round_up(a.d, kBN) / kBN, pairs = sm_count() / 2;
    const int64_t steps = p.piece / gemm::kTileK, tall = p.rows / gemm::kTileM;
    const int64_t all = tn * (tall * steps + p.piece / gemm::kTileM * (p.rows / gemm::kTileK));
    const int64_t share = all / (2 * pairs) > 32 ? all / (2 * pairs) : 32;
    int64_t slabs = (steps + share - 1) / share;
    slabs = slabs > 8 ? 8 : slabs;
    p.part = (int)((steps + slabs - 1) / slabs);
    p.slabs = (int)((steps + p.part - 1) / p.part);
    p.sum = c.take<float>(p.slabs * p.rows * gemm::padded(a.d));
  } else {
    p.r.zt = c.take<float>(a.n);
    p.loss = c.take<float>(a.n);
    p.stat = c.take<float2>(p.runs * p.rows);
  }
  p.bytes = c.used;
  return p;
}

template <typename IO>
struct Calls {
  static constexpr int kPlanes = sizeof(IO) == 4 ? 2 : 1;
  static constexpr bool kBf16 = sizeof(IO) == 2;
  static constexpr int kSegment = kBf16 ? 0 : gemm::kExact;

  static cudaError_t pack(const LossArgs &a, const Plan &p, bool back, float *loss, float *lse,
                          int *err, cudaStream_t st) {
    const uint32_t *top = kPlanes == 2 ? p.top : nullptr;
    const float *g = back && a.reduction == SSD_REDUCE_NONE ? a.gloss : nullptr;
    if (top) {
      cudaError_t e = cudaMemsetAsync(p.top, 0, kTops * sizeof(uint32_t), st);
      if (e != cudaSuccess) return e;
      if constexpr (kPlanes == 2)
        top_kernel<<<4 * sm_count(), 256, 0, st>>>(
            view_of<const float>(a.x), a.targets, a.ignore, a.L, a.n,
            static_cast<const float *>(a.weight->data), a.weight->token_stride, a.V, a.d, g, p.top,
            err);
      e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
    if (p.counts) {
      count_kernel<<<(unsigned)((a.n + kGroup - 1) / kGroup), kPackThreads, 0, st>>>(
          a.targets, a.ignore, a.n, p.counts, err);
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
    // (the first launch of the call waits for what is on the stream the ordinary way)
    const int64_t blocks = (a.n + kPackTokens - 1) / kPackTokens;
    const int64_t slices = blocks < 2 * sm_count() ? 2 * sm_count() / blocks : 1;
    int64_t cols = round_up((a.d + slices - 1) / slices, 64);
    cols = cols < kPackCols ? kPackCols : cols;
    const dim3 grid((unsigned)blocks, (unsigned)((a.d + cols - 1) / cols));
    if (top || p.counts)
      return launch_after(pack_kernel<IO>, grid, kPackThreads, 0, st, view_of<const IO>(a.x),
                                a.targets, a.ignore, a.V, a.L, a.n, a.d, a.lse_in, g,
                                view_of<IO>(a.dx), loss, lse, p.counts, p.r, p.xp, p.xg, p.ld,
                                p.rows * p.ld, kPlanes, cols, top, err);
    pack_kernel<IO><<<grid, kPackThreads, 0, st>>>(
        view_of<const IO>(a.x), a.targets, a.ignore, a.V, a.L, a.n, a.d, a.lse_in, g,
        view_of<IO>(a.dx), loss, lse, p.counts, p.r, p.xp, p.xg, p.ld, p.rows * p.ld, kPlanes,
        cols, top, err);
    return cudaGetLastError();
  }

  // The words word0 .. of W as an operand array: its address and strides.
  struct Words {
    const void *at;
    int64_t n, ld, zs;
  };
  static cudaError_t words(const LossArgs &a, const Plan &p, int64_t word0, Words *w, int *err,
                           cudaStream_t st) {
    w->n = a.V - word0 < p.piece ? a.V - word0 : p.piece;
    const IO *src = static_cast<const IO *>(a.weight->data) + word0 * a.weight->token_stride;
    if (p.direct) {
      w->at = src, w->ld = a.weight->token_stride, w->zs = w->n * w->ld;
      return cudaSuccess;
    }
    w->at = p.wp, w->ld = p.ld, w->zs = p.piece * p.ld;
    const uint32_t *top = kPlanes == 2 ? p.top : nullptr;
    return launch_after(pack_weight_kernel<IO>, dim3((unsigned)((w->n + 7) / 8)), 256, 0, st,
                              src, a.weight->token_stride, w->n, a.d, p.wp, p.ld, w->zs, top, err);
  }

  static Product product(int64_t M, int64_t N, int64_t K) {
    Product q{};
    q.M = (int)M, q.N = (int)N, q.K = (int)K, q.batch = 1;
    q.pairs = kPlanes == 2 ? 3 : 1;
    q.a_planes = q.b_planes = kPlanes;
    return q;
  }

  // maps and product of the logits of a piece
  static bool logits(const LossArgs &a, const Plan &p, const Words &w, CUtensorMap *maps,
                     Product *q) {
    *q = product(a.n, w.n, a.d);
    q->live_m = p.r.live;
    return gemm::make_map(&maps[0], p.xp, a.d, p.rows, kPlanes, p.ld, p.rows * p.ld, false,
                          gemm::kRows) &&
           gemm::make_map(&maps[1], w.at, a.d, w.n, kPlanes, w.ld, w.zs, false, kBN / 2);
  }

  static cudaError_t forward(const LossArgs &a, void *ws, int *err, cudaStream_t st) {
    const Plan p = plan_of(a, kBf16 ? SSD_BF16 : SSD_F32, false, ws);
    float *loss = a.loss ? a.loss : p.loss;
    cudaError_t e = pack(a, p, false, loss, a.lse, err, st);
    for (int64_t word0 = 0; word0 < a.V && e == cudaSuccess; word0 += p.piece) {
      Words w;
      e = words(a, p, word0, &w, err, st);
      if (e != cudaSuccess) break;
      CUtensorMap maps[2];
      Product q;
      if (!logits(a, p, w, maps, &q)) return cudaErrorInvalidValue;
      const StatsEpi::Args s{p.stat, p.rows, a.n, p.r, kPlanes == 2 ? p.top : nullptr, (int)w.n,
                             (int)word0, (int)(word0 / kRun), (int)p.runs};
      e = gemm::launch<StatsEpi, kBN, kSegment>(maps, &q, 1, kBf16, s, err, st);
    }
    if (e != cudaSuccess) return e;
    e = launch_after(join_kernel, dim3((unsigned)((a.n + 31) / 32)), 32 * kJoinWarps, 0, st,
                           p.stat, p.rows, a.n, (int)p.runs, p.r, loss, a.lse, err);
    if (e != cudaSuccess || !a.total) return e;
    return launch_after(total_kernel, dim3(1), 1024, 0, st, loss, a.n, p.r.live,
                              (int)(a.reduction == SSD_REDUCE_MEAN), a.total);
  }

  static cudaError_t backward(const LossArgs &a, void *ws, int *err, cudaStream_t st) {
    const Plan p = plan_of(a, kBf16 ? SSD_BF16 : SSD_F32, true, ws);
    const bool each = a.reduction == SSD_REDUCE_NONE && a.gloss;  // a factor for each token
    const bool own = each && kPlanes == 2;
    const uint32_t *top = kPlanes == 2 ? p.top : nullptr;
    const int64_t ps = p.rows * p.dz_ld;
    const Factors f{p.r, top, each ? nullptr : a.gloss, own, a.reduction == SSD_REDUCE_MEAN};
    cudaError_t e = pack(a, p, true, nullptr, nullptr, err, st);
    for (int64_t word0 = 0; word0 < a.V && e == cudaSuccess; word0 += p.piece) {
      Words w;
      e = words(a, p, word0, &w, err, st);
      if (e != cudaSuccess) break;
      CUtensorMap maps[4];
      Product q[2];
      if (!logits(a, p, w, maps, q)) return cudaErrorInvalidValue;
      typename DlogitEpi<IO>::Args z{};
      z.rows = p.r, z.top = top, z.n = a.n, z.V = (int)w.n, z.word0 = (int)word0, z.own = own;
      if (!gemm::make_pane_map<128>(&z.dz, p.dz, false, p.dz_ld, p.rows, kPlanes, p.dz_ld, ps))
        return cudaErrorInvalidValue;
      e = gemm::launch<DlogitEpi<IO>, kBN, kSegment>(maps, q, 1, kBf16, z, err, st);
      if (e != cudaSuccess) break;
      // dx [n, d] += dz [n, words] W [words, d];  dW [words, d] = dz^T x
      q[0] = product(a.dx ? a.n : 0, a.d, w.n);
      q[0].b_mn = 1, q[0].batch = q[0].parts = p.slabs, q[0].part = p.part;
      if (a.dx) q[0].live_m = p.r.live;
      q[1] = product(w.n, a.d, a.n);
      q[1].live_k = p.r.live, q[1].a_mn = q[1].b_mn = 1;
      typename GradEpi<IO>::Args g{};
      g.out = static_cast<IO *>(a.dweight) + word0 * a.d;
      g.f = f, g.d = (int)a.d, g.words = (int)w.n, g.first = word0 == 0;
      g.direct = ptr_aligned(a.dweight, 16) && a.d * sizeof(IO) % 16 == 0;
      const int64_t sld = gemm::padded(a.d);
      if (!gemm::make_map(&maps[0], p.dz, p.dz_ld, p.rows, kPlanes, p.dz_ld, ps, false,
                          gemm::kRows) ||
          !gemm::make_map(&maps[1], w.at, a.d, w.n, kPlanes, w.ld, w.zs, true, kBN / 2) ||
          !gemm::make_map(&maps[2], p.dz, p.dz_ld, p.rows, kPlanes, p.dz_ld, ps, true,
                          gemm::kRows) ||
          !gemm::make_map(&maps[3], p.xg ? p.xg : p.xp, a.d, p.rows, kPlanes, p.ld, p.rows * p.ld,
                          true, kBN / 2) ||
          !gemm::make_pane_map<128>(&g.sum, p.sum, true, sld, p.rows, p.slabs, sld, p.rows * sld) ||
          (a.dweight && g.direct &&
           !gemm::make_pane_map<128>(&g.dw, g.out, !kBf16, a.d, w.n, 1, a.d, w.n * a.d)))
        return cudaErrorInvalidValue;
      e = gemm::launch<GradEpi<IO>, kBN, kSegment>(maps, q, a.dweight ? 2 : 1, kBf16, g, err, st);
    }
    if (e != cudaSuccess || !a.dx) return e;
    const int64_t sld = gemm::padded(a.d), warps = (a.d + 127) / 128;
    return launch_after(unpack_kernel<IO>, dim3((unsigned)a.n),
                              (int)(32 * (warps < 8 ? warps : 8)), 0, st, p.sum, sld, p.rows * sld,
                              p.slabs, f, view_of<IO>(a.dx), a.L, a.d, err);
  }
};

}  // namespace

size_t vocab_loss_workspace(const LossArgs &a, ssd_dtype io) {
  return plan_of(a, io, false, nullptr).bytes;
}
size_t vocab_loss_backward_workspace(const LossArgs &a, ssd_dtype io) {
  return plan_of(a, io, true, nullptr).bytes;
}
cudaError_t launch_vocab_loss(const LossArgs &a, ssd_dtype io, void *ws, int *err,
                              cudaStream_t st) {
  return io == SSD_BF16 ? Calls<__nv_bfloat16>::forward(a, ws, err, st)
                        : Calls<float>::forward(a, ws, err, st);
}
cudaError_t launch_vocab_loss_backward(const LossArgs &a, ssd_dtype io, void *ws, int *err,
                                       cudaStream_t st) {
  return io == SSD_BF16 ? Calls<__nv_bfloat16>::backward(a, ws, err, st)
                        : Calls<float>::backward(a, ws, err, st);
}

}  // namespace ssd
