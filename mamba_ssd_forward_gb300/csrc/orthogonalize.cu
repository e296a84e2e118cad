// Newton-Schulz orthogonalisation of matrices G [rows, cols]:
//   X = G / (|G| + eps);  steps times:  A = X X^T,  B = b A + c A A,  X <- a X + B X
// (A = X^T X and X <- a X + X B where there are more rows than columns: the
// smaller Gram matrix.)
//
// Three products a step (gemm.cuh).  A and B are symmetric: their tiles below the
// diagonal are written as the transposes of those above it.  Bound by the tensor
// cores: s^2 l + s^3 + 2 s^2 l operations a step for s = min, l = max of the sides.
// Measured, five steps in bf16: 10576 x 2560 905 to 920 us, 1.23 PFLOP/s; 24 of
// 768 x 1536 490 us, 0.78 PFLOP/s; small ones 5.4 us a launch.
//
// Precision.  A step takes small singular values times a = 3.4, five steps 485:
// it enlarges the rounding of X with them.  bf16 operands would leave the result
// 1 to 3 % off, so operands are fp16 (11 bits), with X scaled by 2^14 and A, B by
// 2^12: the values of no step with the usual coefficients pass 1.3 and 3, fp16 holds 4 and 16,
// and small entries keep their bits.  The first X is G times a power of two,
// exact for bf16; the rest of its norm is applied to the fp32 sums of the first
// step.  The rounding of X counts through a X alone (B X is small where a X is
// what counts), so a X is taken from X in two fp16 planes (22 bits); in the last
// two steps, where the values are near 1 and nothing is enlarged any more, from the
// operand itself (a X and B X then take the same X: measured 2.2e-3 off against
// 2.4e-3, where rounding to bf16 alone is 1.7e-3).  An fp32 result takes two planes of
// everything, three products each.
#include <cmath>

#include "gemm.cuh"
#include "model.cuh"

namespace ssd {
namespace {

using gemm::Product;
using gemm::Tile;

constexpr float kScale = 16384.f, kGramScale = 4096.f;  // of X; of A and B

// ------------------------------------------------------------ norm and first X

constexpr int kNormThreads = 512;

// Eight consecutive elements from c on of a row of `cols`; those past its end are
// zero.  `wide`: rows start on 16 bytes.
template <typename IO>
__device__ __forceinline__ void load8(const IO *p, int64_t c, int64_t cols, bool wide,
                                      float (&v)[8]) {
  if (wide && c + 8 <= cols) {
    load_vec<8>(p + c, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c + e < cols ? ld_io(p + c + e) : 0.f;
  }
}

// A matrix in groups of eight elements; a thread's groups are gridDim.x kNormThreads
// apart, kAtOnce of them loaded together (10576 x 2560 bf16: the squares 18 us, 3.0
// TB/s with cold caches, the first X 26).  Row and column are walked along: with a
// division a group, and one load at a time, the squares took 20.
constexpr int kAtOnce = 4;
template <typename IO, typename F>
__device__ __forceinline__ void each8(SeqView<const IO> g, int64_t rows, int64_t cols, bool wide,
                                      int *err, F f) {
  const uint32_t per = (uint32_t)((cols + 7) / 8), step = gridDim.x * kNormThreads;
  const uint32_t rs = step / per, cs = step % per;  // to a thread's next group
  const uint32_t i = blockIdx.x * kNormThreads + threadIdx.x;
  uint32_t r = i / per, c = i % per;
  while (r < rows) {
    float v[kAtOnce][8];
    uint32_t rr[kAtOnce], cc[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      rr[k] = r, cc[k] = c * 8;
      if (r < rows && SSD_IN_BOUNDS(cc[k] < cols, err, 530))
        load8(g.at(blockIdx.y, r), cc[k], cols, wide, v[k]);
      r += rs, c += cs;
      if (c >= per) c -= per, ++r;
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
      if (rr[k] < rows) f(v[k], rr[k], cc[k]);
  }
}

// Sums of squares, one a block, in units of 2^(2 e).  e is 0 where the plain sum is within
// kLeastPlain .. kMostPlain: no square has left fp32, and what fell out below is 2^-46 of
// the sum a value.  Else the block walks its values again, for the largest and then times
// 2^-e, which takes that to 1 .. 2.
struct __align__(8) BlockSum {
  float s;
  int e;
};
constexpr float kLeastPlain = 0x1p-80f, kMostPlain = 0x1p120f;
constexpr int kNoNumber = 1000;  // of an infinite or NaN sum, next to which no other counts
template <typename IO>
__global__ void __launch_bounds__(kNormThreads)
squares_kernel(SeqView<const IO> g, int64_t rows, int64_t cols, bool wide,
               BlockSum *__restrict__ part, int *err) {
  constexpr int kWarps = kNormThreads / 32;
  __shared__ float warps[kWarps];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  ptx::griddep_launch_dependents();
  // the warps' values, in their order, in every thread
  auto all = [&](float t, auto join) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) t = join(t, __shfl_xor_sync(0xffffffffu, t, off));
    __syncthreads();
    if (lane == 0) warps[warp] = t;
    __syncthreads();
    t = warps[0];
    for (int w = 1; w < kWarps; ++w) t = join(t, warps[w]);
    return t;
  };
  auto sum = [&](auto scaled) {
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    each8(g, rows, cols, wide, err, [&](const float (&v)[8], int64_t, int64_t) {
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e % 4] = fmaf(scaled(v[e]), scaled(v[e]), s[e % 4]);
    });
    return all((s[0] + s[1]) + (s[2] + s[3]), [](float a, float b) { return a + b; });
  };
  float t = sum([](float v) { return v; });
  int e = 0;
  if (t < kLeastPlain || t > kMostPlain) {
    float top = 0.f;
    each8(g, rows, cols, wide, err, [&](const float (&v)[8], int64_t, int64_t) {
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[i]));
    });
    top = all(top, [](float a, float b) { return fmaxf(a, b); });
    if (top > 0.f && isfinite(top)) {  // (of a NaN as well: it is in t)
      e = ilogbf(top);
      const float a = ldexpf(1.f, -e / 2), b = ldexpf(1.f, -e - -e / 2);
      t = sum([=](float v) { return v * a * b; });
    }
  }
  if (!isfinite(t)) e = kNoNumber;
  if (threadIdx.x == 0) part[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = {t, e};
}

// Eight values as fp16, and what that leaves of them if it is asked for.
__device__ __forceinline__ uint4 pack8(float *v, bool more) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&h);
    if (more) v[2 * i] -= __low2float(h), v[2 * i + 1] -= __high2float(h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// kScale / (|G| + eps) as rest 2^q with rest in [1, 2), from the blocks' sums; for a |G| that
// is no number rest is NaN, and with it the result.  (|G| may leave fp32's range.)
__device__ __forceinline__ float scale_of(const BlockSum *__restrict__ part, int parts, float eps,
                                          int *q) {
  const int lane = threadIdx.x % 32;
  // 2^(2 e) for e <= 0, zero where fp32 ends
  auto less = [](int e) { return e < -63 ? 0.f : __uint_as_float((uint32_t)(127 + 2 * e) << 23); };
  int unit = -kNoNumber;  // the largest of the sums'
  float s = 0.f;          // in the same order in every block
#pragma unroll 4
  for (int i = lane; i < parts; i += 32) {
    const BlockSum b = part[i];
    const int next = b.s != 0.f ? max(unit, b.e) : unit;
    s = s * less(unit - next) + (b.s != 0.f ? b.s * less(b.e - next) : 0.f);
    unit = next;
  }
  const int mine = unit;
  unit = __reduce_max_sync(0xffffffffu, unit);
  s *= less(mine - unit);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  *q = 0;
  if (!isfinite(s)) return __int_as_float(0x7fc00000);
  const float norm = sqrtf(s);
  int en, ee, ew;
  frexpf(norm, &en);
  frexpf(eps, &ee);
  const int top = norm > 0.f ? max(en + unit, ee) : ee;  // norm + eps is 2^(top - 1) at least
  const float whole = kScale / ((norm > 0.f ? ldexpf(norm, unit - top) : 0.f) + ldexpf(eps, -top));
  const float rest = 2.f * frexpf(whole, &ew);
  *q = ew - 1 - top;
  return rest;
}

// The first X: G times the power of two below kScale / (|G| + eps), in one plane
// or two; rest[z]: what is left of that factor, in [1, 2).
template <typename IO>
__global__ void __launch_bounds__(kNormThreads)
start_kernel(SeqView<const IO> g, int64_t rows, int64_t cols, bool wide,
             const BlockSum *__restrict__ part, int parts, float eps, __half *__restrict__ x,
             int64_t ld, int planes, float *__restrict__ rest, int *err) {
  const int64_t z = blockIdx.y;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  __shared__ float factors[2];
  if (threadIdx.x < 32) {  // (every warp for itself: 27 us in place of 26 at 10576 x 2560)
    int q;
    const float left = scale_of(part + z * parts, parts, eps, &q);
    // 2^q in two: it may leave fp32's range where G times it does not
    const int most = max(-126, min(127, q));
    if (threadIdx.x == 0) {
      factors[0] = ldexpf(1.f, most), factors[1] = ldexpf(1.f, q - most);
      if (blockIdx.x == 0) rest[z] = left;
    }
  }
  __syncthreads();
  const float up = factors[0], more = factors[1];
  __half *hi = x + z * 2 * rows * ld, *lo = hi + rows * ld;
  each8(g, rows, cols, wide, err, [&](float (&v)[8], int64_t r, int64_t c) {
    if (!SSD_IN_BOUNDS(r < rows && c + 8 <= ld, err, 531)) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= up;
    if (more != 1.f)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= more;
    *reinterpret_cast<uint4 *>(hi + r * ld + c) = pack8(v, planes == 2);
    if (planes == 2) *reinterpret_cast<uint4 *>(lo + r * ld + c) = pack8(v, false);
  });
}

// ------------------------------------------------------------------ epilogue

// D = (alpha sum + beta C) rest^power, as fp16 planes or, the last X, as the
// result.  C comes through the panes that D leaves by.
enum Kind { kOne, kTwo, kBf16, kF32 };  // one plane, two, the result

template <Kind kind>
struct StepEpi {
  static constexpr bool kPlanes = kind == kOne || kind == kTwo;
  static constexpr int kCount = kind == kTwo ? 2 : 1;  // planes of D
  struct Args {
    CUtensorMap c, d;  // planes of C; of D, or a bf16 result where TMA can write it
    float alpha, beta;
    const float *rest;  // of the first step, else NULL
    int power;
    int c_planes, c_stored;  // planes of C to add (0: no C), and in its array
    int d_stored;            // of D
    int count;               // matrices
    int share;               // columns of the tile that a warp takes
    int symmetric;           // there are mirrored tiles
    __half *out;             // D again, for the mirrored tiles of two planes
    int64_t ld, ps, zs;
    SeqView<__nv_bfloat16> bf16;
    SeqView<float> f32;
    int N, wide;  // columns; wide: rows of the result start on 16 bytes
  };
  // Sixteen warps: with few k to a tile the epilogue is what a tile takes longest
  // for, and the last tile's is not covered by anything.
  static constexpr int kWarps = 16;
  static constexpr bool kStaged = true;
  using Pane = gemm::Panes<64>;
  const Args &a;
  Pane panes;
  int *err;
  float alpha, beta;
  // A chunk's planes, or its plane and its mirror image, have both panes; else each
  // chunk has its own.
  int row, row0, col0, M, mirror, pair;
  int64_t batch;
  __device__ __forceinline__ StepEpi(const Args &args, Pane p, int *e)
      : a(args), panes(p), err(e),
        pair(args.c_planes == 2 || kind == kTwo || args.symmetric) {}
  __device__ __forceinline__ void begin(const Tile &o, int r, int col, int rows) {
    row = r, row0 = r - panes.lane, col0 = col, M = rows, mirror = o.mirror, batch = o.batch;
    float f = 1.f;
    if (a.rest && SSD_IN_BOUNDS(batch < a.count, err, 532)) {
      f = a.rest[batch];
      if (a.power == 2) f *= f;
    }
    alpha = a.alpha * f, beta = a.beta * f;
    panes.template reuse<0>();
    // C of the first chunks, while the products run
    fetch(0);
    if (!pair) fetch(1);
  }
  // whether any of the warp's 32 rows x 32 columns of chunk j is there
  __device__ __forceinline__ bool some(int j) const {
    return row0 < M && col0 + gemm::kChunk * j < a.N && gemm::kChunk * j < a.share;
  }
  __device__ __forceinline__ int slot(int j) const { return pair ? 0 : j & 1; }
  __device__ __forceinline__ void fetch(int j) const {
    if (a.c_planes && some(j))
      panes.fetch(slot(j), slot(j), a.c_planes, &a.c, col0 + gemm::kChunk * j, row0,
                  (int)batch * a.c_stored);
  }
  __device__ __forceinline__ void chunk(float (&v)[gemm::kChunk], int col, int j) {
    if (!some(j)) return;
    const int pane = slot(j);
    if (!a.c_planes) {
#pragma unroll
      for (int i = 0; i < gemm::kChunk; ++i) v[i] *= alpha;
    } else {
      panes.fetched(slot(j));
      const bool two = a.c_planes == 2;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 q = panes.cell(pane, i), u = two ? panes.cell(pane + 1, i) : q;
        const uint32_t w[4] = {q.x, q.y, q.z, q.w}, x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float2 f = __half22float2(*reinterpret_cast<const __half2 *>(w + k));
          if (two) {  // (exact: 22 bits)
            const float2 g = __half22float2(*reinterpret_cast<const __half2 *>(x + k));
            f.x += g.x, f.y += g.y;
          }
          v[8 * i + 2 * k] = fmaf(beta, f.x, alpha * v[8 * i + 2 * k]);
          v[8 * i + 2 * k + 1] = fmaf(beta, f.y, alpha * v[8 * i + 2 * k + 1]);
        }
      }
    }
    if constexpr (kind == kF32) {
      if (row < M && SSD_IN_BOUNDS(batch < a.count && col < a.N, err, 533)) {
        float *o = a.f32.at(batch, row) + col;
        if (a.wide && col + gemm::kChunk <= a.N) {
#pragma unroll
          for (int i = 0; i < gemm::kChunk; i += 4) {
            const float q[4] = {v[i], v[i + 1], v[i + 2], v[i + 3]};
            store_vec<4>(o + i, q);
          }
        } else {
#pragma unroll
          for (int i = 0; i < gemm::kChunk; ++i)
            if (col + i < a.N) o[i] = v[i];
        }
      }
      panes.written();  // (C is read)
      if (pair) fetch(j + 1);
      return;
    }
#pragma unroll
    for (int p = 0; p < kCount; ++p) {
      uint32_t w[gemm::kChunk / 2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 q = kind == kBf16 ? pack_bf16(v + 8 * i) : pack8(v + 8 * i, p + 1 < kCount);
        panes.cell(pane + p, i) = q;
        w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
      }
      if (kind == kOne && mirror) {
        // the image, rows of the columns, into the pane beside
        uint8_t *m = panes.at + (pane + 1) * Pane::kBytes + (panes.lane & 7) * 2;
#pragma unroll
        for (int i = 0; i < gemm::kChunk; ++i)
          *reinterpret_cast<uint16_t *>(m + Pane::swizzled(i, panes.lane >> 3)) =
              (uint16_t)(i & 1 ? w[i / 2] >> 16 : w[i / 2]);
      }
      if (kind == kTwo && mirror && row < M && SSD_IN_BOUNDS(batch < a.count && row < a.N, err, 534)) {
        // (there is no pane left for it: the lanes' rows lie side by side)
        uint16_t *m = reinterpret_cast<uint16_t *>(a.out + batch * a.zs + p * a.ps) +
                      (int64_t)col * a.ld + row;
#pragma unroll
        for (int i = 0; i < gemm::kChunk; ++i)
          if (col + i < a.N) m[i * a.ld] = (uint16_t)(i & 1 ? w[i / 2] >> 16 : w[i / 2]);
      }
    }
    panes.written();
    if (!kPlanes && !a.wide) {
      copy(pane, col);
    } else if (gemm::elected()) {
#pragma unroll
      for (int p = 0; p < kCount; ++p)
        panes.store(pane + p, &a.d, col, row0, (int)batch * a.d_stored + p);
      if (kind == kOne && mirror) panes.store(pane + 1, &a.d, row0, col, (int)batch * a.d_stored);
      ptx::bulk_commit();
    }
    __syncwarp();
    if (pair && some(j + 1)) {  // the panes are free once the store has read them
      panes.template reuse<0>();
      fetch(j + 1);
    }
  }
  static __device__ __forceinline__ uint4 pack_bf16(const float *v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // The pane to rows that TMA cannot write: 16 lanes along a row's columns.
  __device__ __forceinline__ void copy(int pane, int col) {
    const int rows = min(32, M - row0), w = panes.lane & 15;
    if (!SSD_IN_BOUNDS(batch < a.count && row0 < M && col < a.N, err, 535)) return;
#pragma unroll 4
    for (int r = panes.lane >> 4; r < rows; r += 2) {
      const uint32_t q = panes.word(pane, r, w);
      uint16_t *u = reinterpret_cast<uint16_t *>(a.bf16.at(batch, row0 + r) + col) + 2 * w;
      if (col + 2 * w < a.N) u[0] = (uint16_t)q;
      if (col + 2 * w + 1 < a.N) u[1] = (uint16_t)(q >> 16);
    }
    panes.written();  // (it is read)
  }
  __device__ __forceinline__ void end() {}
};

// ------------------------------------------------------ A in parts of its sums

// A = X X^T of long, narrow X is few tiles of many stages, which would be summed one
// after the other by few pairs: its k is cut into parts, which as many pairs sum into
// fp32 slabs, and a launch adds these in their order.
struct SlabEpi {
  struct Args {
    CUtensorMap d;  // [matrix, part][side][side]
    int N;
  };
  static constexpr int kWarps = 16;
  static constexpr bool kStaged = true;
  using Pane = gemm::Panes<128>;
  const Args &a;
  Pane panes;
  int row0, M, batch;
  __device__ __forceinline__ SlabEpi(const Args &args, Pane p, int *) : a(args), panes(p) {}
  __device__ __forceinline__ void begin(const Tile &o, int r, int, int rows) {
    row0 = r - panes.lane, M = rows, batch = o.batch;
  }
  __device__ __forceinline__ void chunk(float (&v)[gemm::kChunk], int col, int) {
    if (row0 >= M || col >= a.N) return;
    panes.reuse<0>();
#pragma unroll
    for (int i = 0; i < 8; ++i)
      panes.cell(0, i) = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                                    __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3]));
    panes.written();
    if (gemm::elected()) {
      panes.store(0, &a.d, col, row0, batch);
      ptx::bulk_commit();
    }
  }
  __device__ __forceinline__ void end() {}
};

// The sum of a matrix's slabs, times alpha rest^2, in fp16 planes; a thread takes eight
// columns.  (Columns from `side` on are nobody's.)
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads)
join_parts_kernel(const float *__restrict__ slabs, int parts, int64_t side, int64_t ld, float alpha,
                  const float *__restrict__ rest, __half *__restrict__ gram, int planes, int *err) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int64_t z = blockIdx.y, i = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x;
  const int64_t r = i / (ld / 8), c = i % (ld / 8) * 8;
  if (r >= side || !SSD_IN_BOUNDS(c + 8 <= ld, err, 536)) return;
  const float *p = slabs + z * parts * side * ld + r * ld + c;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int q = 0; q < parts; ++q, p += side * ld) {
    const float4 *s = reinterpret_cast<const float4 *>(p);
    const float4 a = s[0], b = s[1];
    v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
    v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
  }
  const float f = rest ? alpha * rest[z] * rest[z] : alpha;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] *= f;
  __half *o = gram + z * planes * side * ld + r * ld + c;
  *reinterpret_cast<uint4 *>(o) = pack8(v, planes == 2);
  if (planes == 2) *reinterpret_cast<uint4 *>(o + side * ld) = pack8(v, false);
}

// ----------------------------------------------------------------- the host

constexpr int kSplitBN = 128;  // columns to a tile of A in parts
// A goes in parts where that saves more stages than this.  Five steps, us: saving 8 of 16
// stages 1000 x 100 into bf16 takes 119 -> 127, 16 of 24 1500 x 100 131 -> 129, 24 of 32
// 2000 x 100 140 -> 130; 5034 x 30 into bf16 175 -> 113, into fp32 (237 stages) 392 -> 140.
constexpr int kSplitSaves = 12;

struct Plan {
  int planes;  // of A, B and of the products
  int64_t side, ld, gram_ld;
  int parts;           // of the norm's sums
  int split, stages;   // parts of A's k (1: A in one go), stages of k in each
  BlockSum *part;
  float *rest, *slabs;
  __half *x[2], *gram, *poly;
  size_t bytes;
};

Plan plan_of(const OrthArgs &a, ssd_dtype out, void *ws) {
  Plan p{};
  p.planes = out == SSD_F32 ? 2 : 1;
  p.side = a.rows < a.cols ? a.rows : a.cols;
  p.ld = gemm::padded(a.cols), p.gram_ld = gemm::padded(p.side);
  // some 4 blocks an SM over all matrices, each thread with something to do
  int64_t parts = (4 * sm_count() + a.count - 1) / a.count;
  const int64_t most = (a.rows * ((a.cols + 7) / 8) + kNormThreads - 1) / kNormThreads;
  p.parts = (int)(parts < most ? parts : most);
  // A's parts: as many as there are pairs for, of some eight stages at least (counting
  // those of all planes; with five or twelve no case is faster by more than 2 %)
  const int64_t tiles = a.count * ((p.side + 255) / 256) * ((p.side + kSplitBN - 1) / kSplitBN);
  const int64_t stages = ((a.rows > a.cols ? a.rows : a.cols) + gemm::kTileK - 1) / gemm::kTileK;
  const int64_t each = p.planes == 2 ? 3 : 1, most_parts = sm_count() / 2 / tiles;
  int64_t split = stages * each / 8;
  split = split < most_parts ? split : most_parts;
  if (split > 1 && (stages - (stages + split - 1) / split) * each > kSplitSaves) {
    p.stages = (int)((stages + split - 1) / split);
    p.split = (int)((stages + p.stages - 1) / p.stages);
  } else {
    p.split = 1, p.stages = 0;
  }
  Carver c(ws);
  p.part = c.take<BlockSum>(a.count * p.parts);
  p.slabs = c.take<float>(p.split > 1 ? a.count * p.split * p.side * p.gram_ld : 0);
  p.rest = c.take<float>(a.count);
  for (int i = 0; i < 2; ++i) p.x[i] = c.take<__half>(a.count * 2 * a.rows * p.ld);
  p.gram = c.take<__half>(a.count * p.planes * p.side * p.gram_ld);
  p.poly = c.take<__half>(a.count * p.planes * p.side * p.gram_ld);
  p.bytes = c.used;
  return p;
}

// A product whose epilogue's arguments `fill` writes.
template <Kind kind, typename Fill>
cudaError_t multiply(const CUtensorMap *maps, const Product &q, int bn, Fill fill, int *err,
                     cudaStream_t st) {
  typename StepEpi<kind>::Args e{};
  fill(e);
  auto with = [&](auto segment) {
    constexpr int kSegment = decltype(segment)::value;
    return bn == 256 ? gemm::launch<StepEpi<kind>, 256, kSegment>(maps, &q, 1, false, e, err, st)
                     : gemm::launch<StepEpi<kind>, 128, kSegment>(maps, &q, 1, false, e, err, st);
  };
  if constexpr (kind == kBf16 || kind == kOne)
    return q.pairs == 1 ? with(std::integral_constant<int, 0>()) : cudaErrorInvalidValue;
  else if constexpr (kind == kF32)
    return q.pairs == 3 ? with(std::integral_constant<int, gemm::kExact>()) : cudaErrorInvalidValue;
  else
    return q.pairs == 3 ? with(std::integral_constant<int, gemm::kExact>())
                        : with(std::integral_constant<int, 0>());
}

// Columns to a tile: 256, or 128 where the tiles then take less time in all.  A
// stage of a tile of 256 takes 512 clocks of products, one of 128 half that, but
// loads three quarters as much: 330 measured.
int tile_columns(const Product &q) {
  auto rounds = [&](int64_t bn) {
    const int64_t tm = (q.M + 255) / 256, tn = (q.N + bn - 1) / bn, r = 256 / bn;
    const int64_t tiles = q.batch * (q.symmetric ? tm * tn - r * (tm * (tm - 1) / 2) : tm * tn);
    return (tiles + sm_count() / 2 - 1) / (sm_count() / 2);
  };
  return rounds(128) * 330 < rounds(256) * 512 ? 128 : 256;
}

template <typename IN>
cudaError_t run(const OrthArgs &a, ssd_dtype out, void *ws, int *err, cudaStream_t st) {
  const Plan p = plan_of(a, out, ws);
  const bool tall = a.rows > a.cols;
  const int64_t longer = tall ? a.rows : a.cols, xps = a.rows * p.ld;
  // Planes that X of step k is added in (and held in: those of an fp32 result are
  // operands too).  A bf16 G is exact in one.
  auto carried = [&](int k) {
    return p.planes == 2 || (k < a.steps - 2 && (k > 0 || sizeof(IN) == 4)) ? 2 : 1;
  };
  const dim3 grid(p.parts, (unsigned)a.count);
  const auto g = view_of<const IN>(a.update);
  const bool wide = view_aligned(a.update, sizeof(IN), 16);
  squares_kernel<IN><<<grid, kNormThreads, 0, st>>>(g, a.rows, a.cols, wide, p.part, err);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = launch_after(start_kernel<IN>, grid, kNormThreads, 0, st, g, a.rows, a.cols, wide,
                         p.part, p.parts, a.eps, p.x[0], p.ld, carried(0), p.rest, err);

  if (e != cudaSuccess) return e;

  // A = X X^T or X^T X;  B = b A + c A A;  X <- a X + B X or a X + X B
  Product gram{}, poly{}, next{};
  gram.batch = poly.batch = next.batch = (int)a.count;
  gram.pairs = poly.pairs = next.pairs = p.planes == 2 ? 3 : 1;
  gram.symmetric = poly.symmetric = 1;
  gram.M = gram.N = poly.M = poly.N = poly.K = next.K = (int)p.side, gram.K = (int)longer;
  gram.a_mn = gram.b_mn = tall, gram.a_planes = gram.b_planes = 2;
  poly.a_planes = poly.b_planes = p.planes;
  next.M = (int)a.rows, next.N = (int)a.cols, next.b_mn = !tall;
  next.a_planes = tall ? 2 : p.planes, next.b_planes = tall ? p.planes : 2;
  const int bn = tile_columns(gram), next_bn = tile_columns(next);
  Product part = gram;  // A in parts: all its tiles
  part.symmetric = 0, part.part = p.stages, part.parts = p.split, part.batch *= p.split;
  const int gram_bn = p.split > 1 ? kSplitBN : bn;

  // Every array as an operand and through panes, described once: X is one of two
  // arrays in turn.
  const int64_t gps = p.side * p.gram_ld, xz = a.count * 2, gz = a.count * p.planes;
  CUtensorMap of_gram[2][2], of_poly[2], of_next[2][2];  // [X][operand]; [operand]
  CUtensorMap pane_x[2], pane_gram, pane_poly, pane_out;
  auto x_map = [&](CUtensorMap *m, int i, bool mn, int box) {
    return gemm::make_map(m, p.x[i], a.cols, a.rows, xz, p.ld, xps, mn, box);
  };
  auto side_map = [&](CUtensorMap *m, const __half *x, int box) {
    return gemm::make_map(m, x, p.side, p.side, gz, p.gram_ld, gps, false, box);
  };
  auto side_pane = [&](CUtensorMap *m, const __half *x) {
    return gemm::make_pane_map<64>(m, x, false, p.side, p.side, gz, p.gram_ld, gps);
  };
  bool ok = side_map(&of_poly[0], p.gram, gemm::kRows) && side_map(&of_poly[1], p.gram, bn / 2) &&
            side_pane(&pane_gram, p.gram) && side_pane(&pane_poly, p.poly);
  for (int i = 0; i < 2 && ok; ++i)
    ok = x_map(&of_gram[i][0], i, tall, gemm::kRows) && x_map(&of_gram[i][1], i, tall, gram_bn / 2) &&
         gemm::make_pane_map<64>(&pane_x[i], p.x[i], false, a.cols, a.rows, xz, p.ld, xps) &&
         (tall ? x_map(&of_next[i][0], i, false, gemm::kRows) &&
                     side_map(&of_next[i][1], p.poly, next_bn / 2)
               : side_map(&of_next[i][0], p.poly, gemm::kRows) &&
                     x_map(&of_next[i][1], i, true, next_bn / 2));
  SlabEpi::Args slab{};
  slab.N = (int)p.side;
  if (p.split > 1 && ok)
    ok = gemm::make_pane_map<128>(&slab.d, p.slabs, true, p.side, p.side, a.count * p.split,
                                  p.gram_ld, gps);
  bool wide_out = false;
  if (out == SSD_BF16 && ok) {
    wide_out = view_aligned(a.out, 2, 16) && a.out->token_stride >= a.cols &&
               (a.count == 1 || a.out->batch_stride > 0);
    ok = !wide_out || gemm::make_pane_map<64>(&pane_out, a.out->data, false, a.cols, a.rows,
                                              a.count, a.out->token_stride, a.out->batch_stride);
  }
  if (!ok) return cudaErrorInvalidValue;

  for (int k = 0; k < a.steps; ++k) {
    const int i = k & 1;
    const bool last = k == a.steps - 1;
    auto gram_args = [&](auto &s) {
      s.alpha = kGramScale / (kScale * kScale), s.rest = k ? nullptr : p.rest, s.power = 2;
      s.d = pane_gram, s.out = p.gram, s.d_stored = p.planes, s.share = bn / 4, s.symmetric = 1;
      s.count = (int)a.count;
      s.ld = p.gram_ld, s.ps = gps, s.zs = p.planes * gps, s.N = (int)p.side;
    };
    auto poly_args = [&](auto &s) {
      gram_args(s);
      s.alpha = a.c / kGramScale, s.beta = a.b, s.rest = nullptr;
      s.c = pane_gram, s.c_planes = s.c_stored = p.planes, s.d = pane_poly, s.out = p.poly;
    };
    auto next_args = [&](auto &s) {
      s.alpha = 1.f / kGramScale, s.beta = a.a, s.rest = k ? nullptr : p.rest, s.power = 1;
      if (last) s.alpha /= kScale, s.beta /= kScale;
      s.c = pane_x[i], s.c_planes = carried(k), s.c_stored = 2, s.d = pane_x[!i], s.d_stored = 2;
      s.N = (int)a.cols, s.share = next_bn / 4, s.count = (int)a.count;
    };
    auto bf16_args = [&](auto &s) {
      next_args(s);
      s.d_stored = 1, s.bf16 = view_of<__nv_bfloat16>(a.out), s.wide = wide_out;
      if (wide_out) s.d = pane_out;
    };
    auto f32_args = [&](auto &s) {
      next_args(s);
      s.f32 = view_of<float>(a.out), s.wide = view_aligned(a.out, 4, 16);
    };
    if (p.split > 1) {
      e = p.planes == 1
              ? gemm::launch<SlabEpi, kSplitBN, 0>(of_gram[i], &part, 1, false, slab, err, st)
              : gemm::launch<SlabEpi, kSplitBN, gemm::kExact>(of_gram[i], &part, 1, false, slab, err,
                                                              st);
      if (e != cudaSuccess) return e;
      const int64_t groups = p.side * (p.gram_ld / 8);
      e = launch_after(join_parts_kernel,
                       dim3((unsigned)((groups + kJoinThreads - 1) / kJoinThreads), (unsigned)a.count),
                       kJoinThreads, 0, st, p.slabs, p.split, p.side, p.gram_ld,
                       kGramScale / (kScale * kScale), k ? nullptr : p.rest, p.gram, p.planes, err);
    } else {
      e = p.planes == 1 ? multiply<kOne>(of_gram[i], gram, bn, gram_args, err, st)
                        : multiply<kTwo>(of_gram[i], gram, bn, gram_args, err, st);
    }
    if (e != cudaSuccess) return e;
    e = p.planes == 1 ? multiply<kOne>(of_poly, poly, bn, poly_args, err, st)
                      : multiply<kTwo>(of_poly, poly, bn, poly_args, err, st);
    if (e != cudaSuccess) return e;
    e = last                  ? (out == SSD_BF16
                                     ? multiply<kBf16>(of_next[i], next, next_bn, bf16_args, err, st)
                                     : multiply<kF32>(of_next[i], next, next_bn, f32_args, err, st))
        : carried(k + 1) == 1 ? multiply<kOne>(of_next[i], next, next_bn, next_args, err, st)
                              : multiply<kTwo>(of_next[i], next, next_bn, next_args, err, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t orthogonalize_workspace(const OrthArgs &a, ssd_dtype, ssd_dtype out) {
  return plan_of(a, out, nullptr).bytes;
}
cudaError_t launch_orthogonalize(const OrthArgs &a, ssd_dtype in, ssd_dtype out, void *ws, int *err,
                                 cudaStream_t st) {
  return in == SSD_BF16 ? run<__nv_bfloat16>(a, out, ws, err, st)
                        : run<float>(a, out, ws, err, st);
}

}  // namespace ssd
