// Newton-Schulz orthogonalisation of matrices G [rows, cols]:
//   X = G / (|G| + eps);  steps times:  A = X X^T,  B = b A + c A A,  X <- a X + B X
// (A = X^T X and X <- a X + X B where there are more rows than columns: the
// smaller Gram matrix.)
//
// Three products a step (gemm.cuh).  A and B are symmetric: their tiles below the
// diagonal are written as the transposes of those above it.  Bound by the tensor
// cores: s^2 l + s^3 + 2 s^2 l operations a step for s = min, l = max of the sides.
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

template <typename IO>
__global__ void __launch_bounds__(kNormThreads)
squares_kernel(SeqView<const IO> g, int64_t rows, int64_t cols, float *__restrict__ part,
               int *err) {
  __shared__ float sums[kNormThreads / 32];
  const int64_t z = blockIdx.y;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  for (int64_t r = blockIdx.x * (kNormThreads / 32) + warp; r < rows;
       r += gridDim.x * (kNormThreads / 32)) {
    if (!SSD_IN_BOUNDS(z < gridDim.y, err, 80)) break;
    const IO *p = g.at(z, r);
    int64_t c = lane;
    for (; c + 96 < cols; c += 128)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float v = ld_io(p + c + 32 * k);
        s[k] = fmaf(v, v, s[k]);
      }
    for (; c < cols; c += 32) {
      const float v = ld_io(p + c);
      s[0] = fmaf(v, v, s[0]);
    }
  }
  float t = (s[0] + s[1]) + (s[2] + s[3]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
  if (lane == 0) sums[warp] = t;
  __syncthreads();
  if (threadIdx.x == 0) {
    t = sums[0];
    for (int w = 1; w < kNormThreads / 32; ++w) t += sums[w];
    part[z * gridDim.x + blockIdx.x] = t;
  }
}

__device__ __forceinline__ void split(float v, __half &hi, __half &lo) {
  hi = __float2half_rn(v);
  lo = __float2half_rn(v - __half2float(hi));
}

// The first X: G times the power of two below kScale / (|G| + eps), in two
// planes; rest[z]: what is left of that factor, in [1, 2).
template <typename IO>
__global__ void __launch_bounds__(kNormThreads)
start_kernel(SeqView<const IO> g, int64_t rows, int64_t cols, const float *__restrict__ part,
             int parts, float eps, __half *__restrict__ x, int64_t ld,
             float *__restrict__ rest, int *err) {
  const int64_t z = blockIdx.y;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  float s = 0.f;  // every warp adds the parts in the same order
  for (int i = lane; i < parts; i += 32) s += part[z * parts + i];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  const float whole = kScale / (sqrtf(s) + eps);
  const uint32_t bits = __float_as_uint(whole);
  const bool normal = bits >= 0x00800000u && bits < 0x7f800000u;
  const float pow2 = normal ? __uint_as_float(bits & 0x7f800000u) : 1.f;
  if (blockIdx.x == 0 && threadIdx.x == 0) rest[z] = whole / pow2;
  __half *hi = x + z * 2 * rows * ld, *lo = hi + rows * ld;
  for (int64_t r = blockIdx.x * (kNormThreads / 32) + warp; r < rows;
       r += gridDim.x * (kNormThreads / 32)) {
    if (!SSD_IN_BOUNDS(z < gridDim.y && cols <= ld, err, 81)) break;
    const IO *p = g.at(z, r);
#pragma unroll 4
    for (int64_t c = lane; c < cols; c += 32) {
      __half h, l;
      split(ld_io(p + c) * pow2, h, l);
      hi[r * ld + c] = h;
      lo[r * ld + c] = l;
    }
  }
}

// ------------------------------------------------------------------ epilogue

// D = (alpha sum + beta C) rest^power, as fp16 planes or, the last X, as the
// result.
enum Kind { kPlanes, kBf16, kF32 };

template <Kind kind>
struct StepEpi {
  struct Args {
    float alpha, beta;
    const float *rest;  // of the first step, else NULL
    int power;
    const __half *c;  // planes of C, NULL if there is none
    int c_planes;     // read
    int64_t c_ld, c_ps, c_zs;
    __half *out;
    int out_planes;
    int64_t ld, ps, zs;
    SeqView<__nv_bfloat16> bf16;
    SeqView<float> f32;
    int N, wide;  // columns; rows of the result start on 16 bytes
  };
  const Args &a;
  int *err;
  float alpha, beta;
  int row, M, mirror;
  int64_t batch;
  __device__ __forceinline__ StepEpi(const Args &args, int *e) : a(args), err(e) {}
  __device__ __forceinline__ void begin(const Tile &o, int r, int, int rows) {
    row = r, M = rows, mirror = o.mirror, batch = o.batch;
    float f = 1.f;
    if (a.rest) {
      f = a.rest[batch];
      if (a.power == 2) f *= f;
    }
    alpha = a.alpha * f, beta = a.beta * f;
  }
  __device__ __forceinline__ void chunk(float (&v)[gemm::kChunk], int col) {
    if (row >= M || col >= a.N) return;
#pragma unroll
    for (int i = 0; i < gemm::kChunk; ++i) v[i] *= alpha;
    if (a.c) {
      const __half *c = a.c + batch * a.c_zs + (int64_t)row * a.c_ld + col;
      for (int p = 0; p < a.c_planes; ++p) {
#pragma unroll
        for (int i = 0; i < gemm::kChunk; i += 8) {
          if (col + i >= a.c_ld) break;  // rows of whole groups of 16
          const uint4 q = *reinterpret_cast<const uint4 *>(c + p * a.c_ps + i);
          const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(w + k));
            v[i + 2 * k] = fmaf(beta, f.x, v[i + 2 * k]);
            v[i + 2 * k + 1] = fmaf(beta, f.y, v[i + 2 * k + 1]);
          }
        }
      }
    }
    if constexpr (kind == kPlanes) {
      __half *base = a.out + batch * a.zs;
      for (int p = 0; p < a.out_planes; ++p) {
        uint32_t w[gemm::kChunk / 2];
#pragma unroll
        for (int i = 0; i < gemm::kChunk / 2; ++i) {
          const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t *>(&h);
          v[2 * i] -= __low2float(h), v[2 * i + 1] -= __high2float(h);
        }
        __half *o = base + p * a.ps + (int64_t)row * a.ld + col;
#pragma unroll
        for (int i = 0; i < gemm::kChunk; i += 8)
          if (col + i < a.ld && SSD_IN_BOUNDS(col + i + 8 <= a.ld, err, 82))
            *reinterpret_cast<uint4 *>(o + i) =
                make_uint4(w[i / 2], w[i / 2 + 1], w[i / 2 + 2], w[i / 2 + 3]);
        if (mirror) {  // row and column exchanged: the lanes' rows lie side by side
          uint16_t *m = reinterpret_cast<uint16_t *>(base + p * a.ps) + (int64_t)col * a.ld + row;
#pragma unroll
          for (int i = 0; i < gemm::kChunk; ++i)
            if (col + i < a.N) m[i * a.ld] = (uint16_t)(i & 1 ? w[i / 2] >> 16 : w[i / 2]);
        }
      }
    } else {
      using IO = std::conditional_t<kind == kBf16, __nv_bfloat16, float>;
      IO *o;
      if constexpr (kind == kBf16) o = a.bf16.at(batch, row) + col;
      else o = a.f32.at(batch, row) + col;
      constexpr int V = 16 / (int)sizeof(IO);
      if (a.wide && col + gemm::kChunk <= a.N) {
#pragma unroll
        for (int i = 0; i < gemm::kChunk; i += V) {
          float q[V];
#pragma unroll
          for (int k = 0; k < V; ++k) q[k] = v[i + k];
          store_vec<V>(o + i, q);
        }
      } else {
#pragma unroll
        for (int i = 0; i < gemm::kChunk; ++i)
          if (col + i < a.N) st_io(o + i, v[i]);
      }
    }
  }
  __device__ __forceinline__ void end() {}
};

// ----------------------------------------------------------------- the host

struct Plan {
  int planes;  // of A, B and of the products
  int64_t side, ld, gram_ld;
  int parts;
  float *part, *rest;
  __half *x[2], *gram, *poly;
  size_t bytes;
};

Plan plan_of(const OrthArgs &a, ssd_dtype out, void *ws) {
  Plan p{};
  p.planes = out == SSD_F32 ? 2 : 1;
  p.side = a.rows < a.cols ? a.rows : a.cols;
  p.ld = gemm::padded(a.cols), p.gram_ld = gemm::padded(p.side);
  // some 2 blocks an SM over all matrices, 16 rows at least to each
  int64_t parts = (2 * sm_count() + a.count - 1) / a.count;
  const int64_t most = (a.rows + kNormThreads / 32 - 1) / (kNormThreads / 32);
  p.parts = (int)(parts < most ? parts : most);
  Carver c(ws);
  p.part = c.take<float>(a.count * p.parts);
  p.rest = c.take<float>(a.count);
  for (int i = 0; i < 2; ++i) p.x[i] = c.take<__half>(a.count * 2 * a.rows * p.ld);
  p.gram = c.take<__half>(a.count * p.planes * p.side * p.gram_ld);
  p.poly = c.take<__half>(a.count * p.planes * p.side * p.gram_ld);
  p.bytes = c.used;
  return p;
}

template <Kind kind>
cudaError_t multiply(const CUtensorMap *maps, const Product &q, int bn,
                     const typename StepEpi<kind>::Args &e, int *err, cudaStream_t st) {
  auto with = [&](auto segment) {
    constexpr int kSegment = decltype(segment)::value;
    return bn == 256 ? gemm::launch<StepEpi<kind>, 256, kSegment>(maps, &q, 1, false, e, err, st)
                     : gemm::launch<StepEpi<kind>, 128, kSegment>(maps, &q, 1, false, e, err, st);
  };
  if constexpr (kind != kBf16)
    if (q.pairs == 3) return with(std::integral_constant<int, gemm::kExact>());
  if constexpr (kind != kF32)
    if (q.pairs == 1) return with(std::integral_constant<int, 0>());
  return cudaErrorInvalidValue;
}

// Columns to a tile: 128 while tiles of 256 leave pairs of SMs without one.
int tile_columns(const Product &q) {
  const int64_t tm = (q.M + 255) / 256, tn = (q.N + 255) / 256;
  const int64_t tiles = q.batch * (q.symmetric ? tm * (tm + 1) / 2 : tm * tn);
  return tiles < sm_count() / 2 ? 128 : 256;
}

template <typename IN>
cudaError_t run(const OrthArgs &a, ssd_dtype out, void *ws, int *err, cudaStream_t st) {
  const Plan p = plan_of(a, out, ws);
  const bool tall = a.rows > a.cols;
  const int64_t longer = tall ? a.rows : a.cols, xps = a.rows * p.ld;
  const dim3 grid(p.parts, (unsigned)a.count);
  const auto g = view_of<const IN>(a.update);
  squares_kernel<IN><<<grid, kNormThreads, 0, st>>>(g, a.rows, a.cols, p.part, err);
  start_kernel<IN><<<grid, kNormThreads, 0, st>>>(g, a.rows, a.cols, p.part, p.parts, a.eps,
                                                  p.x[0], p.ld, p.rest, err);
  cudaError_t e = cudaGetLastError();

  const int64_t gps = p.side * p.gram_ld;
  const int64_t xz = a.count * 2, gz = a.count * p.planes;
  for (int k = 0; k < a.steps && e == cudaSuccess; ++k) {
    const __half *x = p.x[k & 1];
    const bool last = k == a.steps - 1;
    Product q{};
    q.batch = (int)a.count, q.pairs = p.planes == 2 ? 3 : 1;
    CUtensorMap maps[2];
    bool ok;

    // A = X X^T or X^T X
    q.M = q.N = (int)p.side, q.K = (int)longer;
    q.a_mn = q.b_mn = tall, q.a_planes = q.b_planes = 2, q.symmetric = 1;
    int bn = tile_columns(q);
    ok = gemm::make_map(&maps[0], x, a.cols, a.rows, xz, p.ld, xps, tall, gemm::kRows) &&
         gemm::make_map(&maps[1], x, a.cols, a.rows, xz, p.ld, xps, tall, bn / 2);
    StepEpi<kPlanes>::Args s{};
    s.alpha = kGramScale / (kScale * kScale), s.rest = k ? nullptr : p.rest, s.power = 2;
    s.out = p.gram, s.out_planes = p.planes, s.ld = p.gram_ld, s.ps = gps, s.zs = p.planes * gps;
    s.N = (int)p.side;
    if (!ok) return cudaErrorInvalidValue;
    e = multiply<kPlanes>(maps, q, bn, s, err, st);
    if (e != cudaSuccess) break;

    // B = b A + c A A
    q.K = (int)p.side, q.a_mn = q.b_mn = 0, q.a_planes = q.b_planes = p.planes;
    ok = gemm::make_map(&maps[0], p.gram, p.side, p.side, gz, p.gram_ld, gps, false, gemm::kRows) &&
         gemm::make_map(&maps[1], p.gram, p.side, p.side, gz, p.gram_ld, gps, false, bn / 2);
    s.alpha = a.c / kGramScale, s.beta = a.b, s.rest = nullptr;
    s.c = p.gram, s.c_planes = p.planes, s.c_ld = p.gram_ld, s.c_ps = gps, s.c_zs = p.planes * gps;
    s.out = p.poly;
    if (!ok) return cudaErrorInvalidValue;
    e = multiply<kPlanes>(maps, q, bn, s, err, st);
    if (e != cudaSuccess) break;

    // X <- a X + B X or a X + X B
    q.M = (int)a.rows, q.N = (int)a.cols, q.symmetric = 0;
    bn = tile_columns(q);
    if (tall) {
      q.a_planes = 2, q.b_planes = p.planes;
      ok = gemm::make_map(&maps[0], x, a.cols, a.rows, xz, p.ld, xps, false, gemm::kRows) &&
           gemm::make_map(&maps[1], p.poly, p.side, p.side, gz, p.gram_ld, gps, false, bn / 2);
    } else {
      q.a_planes = p.planes, q.b_planes = 2, q.b_mn = 1;
      ok = gemm::make_map(&maps[0], p.poly, p.side, p.side, gz, p.gram_ld, gps, false,
                          gemm::kRows) &&
           gemm::make_map(&maps[1], x, a.cols, a.rows, xz, p.ld, xps, true, bn / 2);
    }
    if (!ok) return cudaErrorInvalidValue;
    auto fill = [&](auto &u) {
      u.alpha = 1.f / kGramScale, u.beta = a.a, u.rest = k ? nullptr : p.rest, u.power = 1;
      if (last) u.alpha /= kScale, u.beta /= kScale;
      u.c = x, u.c_planes = p.planes == 2 || k < a.steps - 2 ? 2 : 1;
      u.c_ld = p.ld, u.c_ps = xps, u.c_zs = 2 * xps, u.N = (int)a.cols;
    };
    if (!last) {
      StepEpi<kPlanes>::Args u{};
      fill(u);
      u.out = p.x[~k & 1], u.out_planes = p.planes == 2 || k + 1 < a.steps - 2 ? 2 : 1;
      u.ld = p.ld, u.ps = xps, u.zs = 2 * xps;
      e = multiply<kPlanes>(maps, q, bn, u, err, st);
    } else if (out == SSD_BF16) {
      StepEpi<kBf16>::Args u{};
      fill(u);
      u.bf16 = view_of<__nv_bfloat16>(a.out), u.wide = view_aligned(a.out, 2, 16);
      e = multiply<kBf16>(maps, q, bn, u, err, st);
    } else {
      StepEpi<kF32>::Args u{};
      fill(u);
      u.f32 = view_of<float>(a.out), u.wide = view_aligned(a.out, 4, 16);
      e = multiply<kF32>(maps, q, bn, u, err, st);
    }
  }
  return e;
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
