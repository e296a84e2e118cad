// The residual's addition and the root-mean-square norm in front of a block:
//   t = x + r,  y = t rstd w,  rstd = 1 / sqrt(mean(t^2) + eps)
// y in the I/O type or in e4m3 with scales, t kept in the residual stream's type.
// Its gradients from t:  n = t rstd,  g = gy w,
//   dt = rstd (g - n mean(g n)) + gt,  dw = sum over tokens of gy n
//
// Bandwidth kernels: everything is read once and written once.  A token belongs
// to a team (a warp, or a block where a warp's registers do not hold the token),
// whose threads keep V consecutive channels a vector, K vectors each, in
// registers between the sum and the output.  Measured (bf16): 8192 x 2560 into an fp32
// stream 41 us, 6.1 TB/s; in 8 bits 16384 x 5120 98 us, 6.0 TB/s; gradients of
// 8192 x 2560 41 us, 4.1 TB/s, 7 of them the sum of the blocks' shares of dw.
#include <cuda_fp8.h>

#include "model.cuh"
#include "ptx.cuh"

namespace ssd {
namespace {

constexpr int kMaxThreads = 512;   // to a block
constexpr int kTeamThreads = 384;  // to a team while two or four vectors a thread suffice
constexpr int kWarpTeams = 8;       // to a block, where a warp holds a token
constexpr int kMaxSmem = 220 * 1024;
// Threads of walking teams to an SM (from registers; from shared memory), and slots of the ring.
constexpr int kFwdPerSm = 1024, kFwdRingPerSm = 2048, kFwdRing = 2;
constexpr int kGradPerSm = 768, kGradRing = 4;
constexpr float kTop8 = 448.f;  // the largest e4m3 value
// The smallest scale: 1 / scale stays finite.
constexpr float kLeastScale = 1.17549435e-38f;

constexpr int V = 8;  // channels to a vector

// Which channels a thread has: wide, eight consecutive ones, c .. c + 7; else
// (rows off the 16-byte grid, or an odd number of channels) the same 256 of a
// warp, 32 apart, so that the warp's accesses by elements are consecutive.
template <bool kWide>
struct Channels {
  static constexpr int kStep = kWide ? 1 : 32;
  int c, D, *err;
  __device__ __forceinline__ Channels(int vector, int d, int *e)
      : c(kWide ? vector * V : vector / 32 * 32 * V + vector % 32), D(d), err(e) {}
  __device__ __forceinline__ int at(int e) const { return c + e * kStep; }
  // (every access of eight channels at once is behind this)
  __device__ __forceinline__ bool any() const {
    return c < D && SSD_IN_BOUNDS(!kWide || c + V <= D, err, 500);
  }
};
// V channels of a row as the memory holds them (elements of 16 bits by
// themselves where they come so: packing them would wait for the loads), so that
// a token can be loaded while the one before is worked on.
template <typename T, bool kWide>
struct Raw {
  static constexpr int kWords = kWide ? V * (int)sizeof(T) / 4 : V;
  uint32_t w[kWords];
  // the missing channels are zero
  __device__ __forceinline__ void load(const T *p, const Channels<kWide> &c) {
    if constexpr (kWide) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        uint4 q = make_uint4(0, 0, 0, 0);
        if (c.any())
          q = *reinterpret_cast<const uint4 *>(reinterpret_cast<const uint32_t *>(p + c.c) + i);
        w[i] = q.x, w[i + 1] = q.y, w[i + 2] = q.z, w[i + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        w[e] = 0;
        if (c.at(e) < c.D) {
          if constexpr (sizeof(T) == 4) w[e] = __float_as_uint(p[c.at(e)]);
          else w[e] = reinterpret_cast<const uint16_t *>(p)[c.at(e)];
        }
      }
    }
  }
  __device__ __forceinline__ float at(int e) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
    else if constexpr (!kWide) return __uint_as_float(w[e] << 16);
    else return __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
  }
};
template <typename T, bool kWide>
__device__ __forceinline__ void store_row(T *p, const Channels<kWide> &c, const float (&v)[V]) {
  if constexpr (kWide) {
    store_vec<V>(p + c.c, v);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (c.at(e) < c.D) st_io(p + c.at(e), v[e]);
  }
}
// The weights of a thread's channels: kept where there are few, else read (from
// L1) at every token.
template <int K, bool kWide>
struct Weights {
  static constexpr bool kKept = K * V <= 16;
  const float *p;
  Raw<float, kWide> kept[kKept ? K : 1];
  __device__ __forceinline__ Weights(const float *weight, int tid, int team, int D, int *err)
      : p(weight) {
    if constexpr (kKept)
#pragma unroll
      for (int k = 0; k < K; ++k) kept[k].load(p, Channels<kWide>(tid + k * team, D, err));
  }
  __device__ __forceinline__ Raw<float, kWide> of(int k, const Channels<kWide> &c) const {
    if constexpr (kKept) return kept[k];
    Raw<float, kWide> r;
    r.load(p, c);
    return r;
  }
};
template <bool kWide>
__device__ __forceinline__ void store_e4m3(uint8_t *p, const Channels<kWide> &c,
                                           const float (&v)[V]) {
  uint32_t w[V / 4];
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i], v[4 * i + 1]),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2], v[4 * i + 3]),
                                                 __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | hi << 16;
  }
  if constexpr (kWide) {
    *reinterpret_cast<uint2 *>(p + c.c) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (c.at(e) < c.D) p[c.at(e)] = (uint8_t)(w[e / 4] >> (8 * (e % 4)));
  }
}

// Sums (or maxima) of M values over a warp (`teams` 1) or over the block's `warps`,
// in every thread; a fixed order.  Calls in turn use the halves of `scratch`.
template <int M, bool kMax = false>
__device__ __forceinline__ void team_all(float (&v)[M], float (*scratch)[M][32], int teams,
                                         int warps, int turn) {
  auto join = [](float a, float b) { return kMax ? fmaxf(a, b) : a + b; };
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
#pragma unroll
    for (int m = 0; m < M; ++m) v[m] = join(v[m], __shfl_xor_sync(0xffffffffu, v[m], off));
  if (teams == 1) return;
  const int lane = threadIdx.x % 32;
  if (lane == 0)
#pragma unroll
    for (int m = 0; m < M; ++m) scratch[turn][m][threadIdx.x / 32] = v[m];
  __syncthreads();
#pragma unroll
  for (int m = 0; m < M; ++m) v[m] = lane < warps ? scratch[turn][m][lane] : 0.f;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
#pragma unroll
    for (int m = 0; m < M; ++m) v[m] = join(v[m], __shfl_xor_sync(0xffffffffu, v[m], off));
}

struct Quant {
  uint8_t *q;
  int64_t bs, ts;  // of q
  float *scales;
  int block, parts;  // channels to a scale (0: the token), scales to a token
  __device__ __forceinline__ uint8_t *row(int64_t b, int64_t t) const { return q + b * bs + t * ts; }
};

// The factor of values whose largest is `top`; `scale`, where given, is its inverse.
__device__ __forceinline__ float quantiser(float top, float *scale) {
  const float m = fmaxf(top, kTop8 * kLeastScale);
  if (scale) *scale = top == 0.f ? 0.f : m * (1.f / kTop8);
  return __fdividef(0.25f * kTop8, 0.25f * m);  // (it takes no divisor beyond 2^126)
}
// V values of a warp's 256 channels in e4m3, a scale to each qu.block of them.
template <bool kWide>
__device__ __forceinline__ void quantise(float (&t)[V], const Channels<kWide> &c, const Quant &qu,
                                         uint8_t *q, float *scales) {
  const auto spread = [](float m, int lanes) {
    for (int off = lanes / 2; off > 0; off >>= 1)
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    return m;
  };
  if constexpr (kWide) {  // block / V neighbouring lanes hold a block
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) m = fmaxf(m, fabsf(t[e]));
    m = spread(m, qu.block / V);
    const bool leads = c.any() && c.c % qu.block == 0 &&
                       SSD_IN_BOUNDS(c.c / qu.block < qu.parts, c.err, 501);
    const float up = quantiser(m, leads ? scales + c.c / qu.block : nullptr);
#pragma unroll
    for (int e = 0; e < V; ++e) t[e] *= up;
  } else {  // block / 32 consecutive elements of all lanes do
    const int group = qu.block / 32;
    float m[V];
#pragma unroll
    for (int e = 0; e < V; ++e) m[e] = fabsf(t[e]);
    if (group >= 2)
#pragma unroll
      for (int e = 0; e < V; e += 2) m[e] = m[e + 1] = fmaxf(m[e], m[e + 1]);
    if (group == 4)
#pragma unroll
      for (int e = 0; e < V; e += 4) m[e] = m[e + 1] = m[e + 2] = m[e + 3] = fmaxf(m[e], m[e + 2]);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (e % group == 0) {
        const bool leads = threadIdx.x % 32 == 0 && c.at(e) < c.D &&
                           SSD_IN_BOUNDS(c.at(e) / qu.block < qu.parts, c.err, 501);
        m[e] = quantiser(spread(m[e], 32), leads ? scales + c.at(e) / qu.block : nullptr);
      } else {
        m[e] = m[e - 1];
      }
      t[e] *= m[e];
    }
  }
  if (c.any()) store_e4m3(q, c, t);
}

// Rows on their way: a ring of tokens in shared memory, filled by bulk copies that
// one thread issues.  The rows have to start on 16 bytes.
template <int kSlots>
struct Ring {
  uint8_t *at;
  uint64_t *full;
  int slot, bytes, *err;  // bytes of a slot
  uint32_t parity;
  __device__ __forceinline__ Ring(uint8_t *smem, uint64_t *bars, int slot_bytes, int *e)
      : at(smem), full(bars), slot(0), bytes(slot_bytes), err(e), parity(0) {}
  __device__ __forceinline__ void open() {
    if (threadIdx.x == 0) {
      for (int i = 0; i < kSlots; ++i) ptx::mbar_init(&full[i], 1);
      ptx::fence_mbar_init();
    }
    __syncthreads();
  }
  __device__ __forceinline__ uint8_t *base(int s) const { return at + s * bytes; }
  template <typename T>
  __device__ __forceinline__ void copy(int s, int from, const T *src, int n) const {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
            "r"(ptx::smem_u32(base(s) + from)),
        "l"(src), "r"(n * (int)sizeof(T)), "r"(ptx::smem_u32(&full[s]))
        : "memory");
  }
  __device__ __forceinline__ const uint8_t *wait() {
    ptx::mbar_wait(&full[slot], parity, err, 310);
    return base(slot);
  }
  __device__ __forceinline__ void next() {
    if (++slot == kSlots) slot = 0, parity ^= 1;
  }
};

// Teams walk the tokens with a fixed stride.  kRingRows: the team is the block and
// the rows come through the ring; otherwise the next token's loads are out, to
// registers, while a token is worked on.
enum From { kRingRows, kVectors, kElements };
template <typename IO, typename ST, int K, bool kQuant, From from>
__global__ void __launch_bounds__(kMaxThreads)
add_norm_kernel(SeqView<const IO> x, SeqView<const ST> residual, const float *__restrict__ weight,
                SeqView<IO> y, SeqView<ST> total, Quant qu, int64_t L, int64_t rows, int D,
                float eps, int warps, int *err) {
  __shared__ float scratch[2][1][32], tops[2][1][32];
  __shared__ __align__(8) uint64_t bars[kFwdRing];
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr bool kRing = from == kRingRows, kWide = from != kElements;
  const int team = 32 * warps, per = !kRing && warps == 1 ? blockDim.x / 32 : 1;
  const int64_t first = (int64_t)blockIdx.x * per + (per > 1 ? threadIdx.x / 32 : 0);
  const int64_t step = (int64_t)gridDim.x * per;
  if (first >= rows) return;
  const int tid = per > 1 ? threadIdx.x % 32 : threadIdx.x;
  const Weights<K, kWide> weights(weight, tid, team, D, err);
  Raw<IO, kWide> xn[K];
  Raw<ST, kWide> rn[K];
  auto load = [&](const IO *xr, const ST *rr) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const Channels<kWide> c(tid + k * team, D, err);
      xn[k].load(xr, c);
      if (residual.p) rn[k].load(rr, c);
    }
  };
  auto fetch = [&](int64_t row) {
    if (!SSD_IN_BOUNDS(row < rows, err, 502)) return;
    const uint32_t b = (uint32_t)row / (uint32_t)L, at = (uint32_t)row - b * (uint32_t)L;
    load(x.at(b, at), residual.at(b, at));
  };
  const int xb = D * (int)sizeof(IO), rb = residual.p ? D * (int)sizeof(ST) : 0;
  Ring<kFwdRing> ring(smem, bars, xb + rb, err);
  auto send = [&](int slot, int64_t row) {  // one thread
    const uint32_t b = (uint32_t)row / (uint32_t)L, at = (uint32_t)row - b * (uint32_t)L;
    ptx::mbar_arrive_expect_tx(&bars[slot], xb + rb);
    ring.copy(slot, 0, x.at(b, at), D);
    if (rb) ring.copy(slot, xb, residual.at(b, at), D);
  };
  if constexpr (kRing) {
    ring.open();
    if (threadIdx.x == 0)
      for (int i = 0; i < kFwdRing && first + i * step < rows; ++i) send(i, first + i * step);
  } else {
    fetch(first);
  }
  int turn = 0;
  for (int64_t row = first; row < rows; row += step, turn ^= 1) {
    const uint32_t b = (uint32_t)row / (uint32_t)L, at = (uint32_t)row - b * (uint32_t)L;
    if constexpr (kRing) {
      const uint8_t *p = ring.wait();
      load(reinterpret_cast<const IO *>(p), reinterpret_cast<const ST *>(p + xb));
    }
    float t[K][V], s[1] = {0.f};
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        t[k][e] = residual.p ? xn[k].at(e) + rn[k].at(e) : xn[k].at(e);
        s[0] = fmaf(t[k][e], t[k][e], s[0]);
      }
    if (!kRing && row + step < rows) fetch(row + step);
    team_all(s, scratch, kRing ? 2 : warps, warps, turn);
    if constexpr (kRing) {  // every thread has read the slot
      if (threadIdx.x == 0 && row + kFwdRing * step < rows) send(ring.slot, row + kFwdRing * step);
      ring.next();
    }
    const float rstd = rsqrtf(s[0] / (float)D + eps);
    float top[1] = {0.f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const Channels<kWide> c(tid + k * team, D, err);
      if (c.any()) {
        if (total.p) store_row(total.at(b, at), c, t[k]);
        const Raw<float, kWide> w = weights.of(k, c);
#pragma unroll
        for (int e = 0; e < V; ++e) t[k][e] = t[k][e] * rstd * w.at(e);
        if constexpr (!kQuant) store_row(y.at(b, at), c, t[k]);
      }
      if constexpr (kQuant) {
        if (qu.block) {
          quantise(t[k], c, qu, qu.row(b, at), qu.scales + row * qu.parts);
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) top[0] = fmaxf(top[0], fabsf(t[k][e]));
        }
      }
    }
    if constexpr (kQuant) {
      if (qu.block == 0) {
        team_all<1, true>(top, tops, kRing ? 2 : warps, warps, turn);
        const float up = quantiser(top[0], tid == 0 ? qu.scales + row : nullptr);
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const Channels<kWide> c(tid + k * team, D, err);
          if (!c.any()) continue;
#pragma unroll
          for (int e = 0; e < V; ++e) t[k][e] *= up;
          store_e4m3(qu.row(b, at), c, t[k]);
        }
      }
    }
  }
}

template <typename IO, typename ST, int K, From from>
__global__ void __launch_bounds__(kMaxThreads)
add_norm_grad_kernel(SeqView<const ST> total, const float *__restrict__ weight,
                     SeqView<const IO> gy, SeqView<const ST> gtotal, SeqView<IO> dx,
                     SeqView<ST> dres, float *__restrict__ part, int64_t L, int64_t rows, int D,
                     float eps, int warps, int *err) {
  __shared__ float scratch[2][2][32];
  __shared__ __align__(8) uint64_t bars[kGradRing];
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr bool kRing = from == kRingRows, kWide = from != kElements;
  const int team = 32 * warps, per = !kRing && warps == 1 ? blockDim.x / 32 : 1;
  const int64_t first = (int64_t)blockIdx.x * per + (per > 1 ? threadIdx.x / 32 : 0);
  const int64_t step = (int64_t)gridDim.x * per;
  const int tid = per > 1 ? threadIdx.x % 32 : threadIdx.x;
  ptx::griddep_launch_dependents();  // (the sum over the blocks waits for them)
  const Weights<K, kWide> weights(weight, tid, team, D, err);
  // (two vectors of three tensors twice would not fit the registers)
  constexpr bool kNext = !kRing && K == 1;
  Raw<ST, kWide> t[K], gt[K], tn[kNext ? K : 1], gtn[kNext ? K : 1];
  Raw<IO, kWide> g[K], gn[kNext ? K : 1];
  auto load = [&](const ST *tr, const IO *gr, const ST *ur, auto &t, auto &g, auto &gt) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const Channels<kWide> c(tid + k * team, D, err);
      t[k].load(tr, c);
      g[k].load(gr, c);
      if (gtotal.p) gt[k].load(ur, c);
    }
  };
  auto fetch = [&](int64_t row, auto &t, auto &g, auto &gt) {
    if (!SSD_IN_BOUNDS(row < rows, err, 503)) return;
    const uint32_t b = (uint32_t)row / (uint32_t)L, at = (uint32_t)row - b * (uint32_t)L;
    load(total.at(b, at), gy.at(b, at), gtotal.at(b, at), t, g, gt);
  };
  const int tb = D * (int)sizeof(ST), gb = D * (int)sizeof(IO), ub = gtotal.p ? tb : 0;
  Ring<kGradRing> ring(smem, bars, tb + gb + ub, err);
  auto send = [&](int slot, int64_t row) {  // one thread
    const uint32_t b = (uint32_t)row / (uint32_t)L, at = (uint32_t)row - b * (uint32_t)L;
    ptx::mbar_arrive_expect_tx(&bars[slot], tb + gb + ub);
    ring.copy(slot, 0, total.at(b, at), D);
    ring.copy(slot, tb, gy.at(b, at), D);
    if (ub) ring.copy(slot, tb + gb, gtotal.at(b, at), D);
  };
  if constexpr (kRing) {
    ring.open();
    if (threadIdx.x == 0)
      for (int i = 0; i < kGradRing && first + i * step < rows; ++i) send(i, first + i * step);
  } else if (kNext && first < rows) {
    if constexpr (kNext) fetch(first, tn, gn, gtn);
  }
  float dw[K][V];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) dw[k][e] = 0.f;
  int turn = 0;
  for (int64_t row = first; row < rows; row += step, turn ^= 1) {
    const uint32_t b = (uint32_t)row / (uint32_t)L, at = (uint32_t)row - b * (uint32_t)L;
    if constexpr (kRing) {
      const uint8_t *p = ring.wait();
      load(reinterpret_cast<const ST *>(p), reinterpret_cast<const IO *>(p + tb),
           reinterpret_cast<const ST *>(p + tb + gb), t, g, gt);
    } else if constexpr (kNext) {
      t[0] = tn[0], g[0] = gn[0], gt[0] = gtn[0];
      if (row + step < rows) fetch(row + step, tn, gn, gtn);
    } else {
      fetch(row, t, g, gt);
    }
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const Raw<float, kWide> w = weights.of(k, Channels<kWide>(tid + k * team, D, err));
#pragma unroll
      for (int e = 0; e < V; ++e) {
        s[0] = fmaf(t[k].at(e), t[k].at(e), s[0]);
        s[1] = fmaf(g[k].at(e) * w.at(e), t[k].at(e), s[1]);
      }
    }
    team_all(s, scratch, kRing ? 2 : warps, warps, turn);
    if constexpr (kRing) {  // every thread has read the slot
      if (threadIdx.x == 0 && row + kGradRing * step < rows)
        send(ring.slot, row + kGradRing * step);
      ring.next();
    }
    const float rstd = rsqrtf(s[0] / (float)D + eps), mean = s[1] * rstd / (float)D;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const Channels<kWide> c(tid + k * team, D, err);
      if (!c.any()) continue;
      const Raw<float, kWide> w = weights.of(k, c);
      float o[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float n = t[k].at(e) * rstd;
        dw[k][e] = fmaf(g[k].at(e), n, dw[k][e]);
        o[e] = rstd * (g[k].at(e) * w.at(e) - n * mean);
        if (gtotal.p) o[e] += gt[k].at(e);
      }
      if (dx.p) store_row(dx.at(b, at), c, o);
      if (dres.p) store_row(dres.at(b, at), c, o);
    }
  }
  if (!part) return;
  if (per > 1) {  // one share a block: the warps' in their order (K is 1)
    __shared__ float shares[kWarpTeams][32 * V];
    float *mine = shares[threadIdx.x / 32] + threadIdx.x % 32;
#pragma unroll
    for (int e = 0; e < V; ++e) mine[32 * e] = dw[0][e];
    __syncthreads();
    if (threadIdx.x >= 32) return;
    for (int w = 1; w < per; ++w)
#pragma unroll
      for (int e = 0; e < V; ++e) dw[0][e] += shares[w][32 * e + threadIdx.x];
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const Channels<kWide> c(tid + k * team, D, err);
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (c.at(e) < D) part[(int64_t)blockIdx.x * D + c.at(e)] = dw[k][e];
  }
}

// How a token is shared out: vectors to a thread, warps to its team, threads to a
// block.
struct Shares {
  int K, warps, threads;
};
Shares shares_of(int64_t D) {
  const int64_t vecs = (D + V - 1) / V;
  Shares s{1, 1, 32 * kWarpTeams};
  if (vecs <= 32) return s;
  while (s.K < 4 && vecs > s.K * kTeamThreads) s.K *= 2;
  s.threads = (int)(((vecs + s.K - 1) / s.K + 31) / 32 * 32), s.warps = s.threads / 32;
  return s;
}

template <typename F>
cudaError_t with_vectors(int K, F f) {
  switch (K) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 4: return f(std::integral_constant<int, 4>());
  }
  return cudaErrorInvalidValue;
}

// Blocks that walk `rows` tokens, `per` at a time, with `bytes` of shared memory:
// as many as run at once.
int64_t blocks_of(int64_t rows, int64_t per, int threads, int per_sm, int64_t bytes) {
  int64_t one = per_sm / threads;
  if (bytes * one > kMaxSmem) one = kMaxSmem / bytes;
  const int64_t most = sm_count() * (one > 1 ? one : 1), all = (rows + per - 1) / per;
  return all < most ? all : most;
}
// The attribute is the kernel's, whatever this call needs.
template <typename F>
cudaError_t allow_smem(F *kernel) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
}
template <typename IO, typename ST>
cudaError_t forward(const AddNormArgs &a, int *err, cudaStream_t st) {
  const Shares s = shares_of(a.D);
  const int64_t rows = a.b * a.L, per = s.warps == 1 ? s.threads / 32 : 1;
  const bool quant = a.scales != nullptr;
  const bool wide = a.D % V == 0 && ptr_aligned(a.weight, 16) && view_aligned(a.x, sizeof(IO), 16) &&
                    view_aligned(a.residual, sizeof(ST), 16) &&
                    view_aligned(a.total, sizeof(ST), 16) &&
                    (quant ? view_aligned(a.y, 1, V) : view_aligned(a.y, sizeof(IO), 16));
  Quant q{};
  if (quant) {
    q.q = static_cast<uint8_t *>(a.y->data), q.bs = a.y->batch_stride, q.ts = a.y->token_stride;
    q.scales = a.scales, q.block = (int)a.block;
    q.parts = a.block ? (int)((a.D + a.block - 1) / a.block) : 1;
  }
  // One vector a thread is as fast from registers (8192 x 2560 into an fp32 stream
  // 41 us, 45 through the ring); two are not (8192 x 5120 70, 58), nor is the
  // quantised form, which works longer on a token (16384 x 5120 151, 105).
  const int64_t slots = kFwdRing * a.D * (sizeof(IO) + (a.residual ? sizeof(ST) : 0));
  const bool ring = wide && s.warps > 1 && (quant || s.K > 1) && slots <= kMaxSmem;
  const int64_t blocks = ring ? blocks_of(rows, per, s.threads, kFwdRingPerSm, slots)
                              : blocks_of(rows, per, s.threads, kFwdPerSm, 0);
  return with_vectors(s.K, [&](auto k) {
    constexpr int K = decltype(k)::value;
    auto go = [&](auto *kernel) {
      const cudaError_t e = ring ? allow_smem(kernel) : cudaSuccess;
      if (e != cudaSuccess) return e;
      kernel<<<(unsigned)blocks, s.threads, ring ? slots : 0, st>>>(
          view_of<const IO>(a.x), view_of<const ST>(a.residual), a.weight,
          quant ? SeqView<IO>{} : view_of<IO>(a.y), view_of<ST>(a.total), q, a.L, rows, (int)a.D,
          a.eps, s.warps, err);
      return cudaGetLastError();
    };
    return quant ? (ring   ? go(add_norm_kernel<IO, ST, K, true, kRingRows>)
                    : wide ? go(add_norm_kernel<IO, ST, K, true, kVectors>)
                           : go(add_norm_kernel<IO, ST, K, true, kElements>))
                 : (ring   ? go(add_norm_kernel<IO, ST, K, false, kRingRows>)
                    : wide ? go(add_norm_kernel<IO, ST, K, false, kVectors>)
                           : go(add_norm_kernel<IO, ST, K, false, kElements>));
  });
}

// The blocks that walk the gradients' tokens, whatever the rows' alignment (which
// the workspace's size does not know): those of the ring where it fits.
struct GradWalk {
  Shares s;
  int64_t per, slots, blocks;
};
template <typename IO, typename ST>
GradWalk grad_walk(const AddNormArgs &a) {
  GradWalk w{shares_of(a.D), 1, kGradRing * a.D * (int64_t)(sizeof(IO) + 2 * sizeof(ST)), 0};
  if (w.s.warps == 1) w.per = w.s.threads / 32;
  if (w.s.warps == 1 || w.slots > kMaxSmem) w.slots = 0;
  w.blocks = blocks_of(a.b * a.L, w.per, w.s.threads, w.per > 1 ? 2 * kGradPerSm : kGradPerSm,
                       w.slots);
  return w;
}

template <typename IO, typename ST>
cudaError_t backward(const AddNormArgs &a, void *ws, int *err, cudaStream_t st) {
  const bool wide = a.D % V == 0 && ptr_aligned(a.weight, 16) &&
                    view_aligned(a.total, sizeof(ST), 16) && view_aligned(a.gy, sizeof(IO), 16) &&
                    view_aligned(a.gtotal, sizeof(ST), 16) && view_aligned(a.dx, sizeof(IO), 16) &&
                    view_aligned(a.dresidual, sizeof(ST), 16);
  const GradWalk w = grad_walk<IO, ST>(a);
  const bool ring = wide && w.slots > 0;
  float *part = a.dweight ? static_cast<float *>(ws) : nullptr;
  const cudaError_t e = with_vectors(w.s.K, [&](auto k) {
    constexpr int K = decltype(k)::value;
    auto go = [&](auto *kernel) {
      const cudaError_t f = ring ? allow_smem(kernel) : cudaSuccess;
      if (f != cudaSuccess) return f;
      kernel<<<(unsigned)w.blocks, w.s.threads, ring ? w.slots : 0, st>>>(
          view_of<const ST>(a.total), a.weight, view_of<const IO>(a.gy),
          view_of<const ST>(a.gtotal), view_of<IO>(a.dx), view_of<ST>(a.dresidual), part, a.L,
          a.b * a.L, (int)a.D, a.eps, w.s.warps, err);
      return cudaGetLastError();
    };
    return ring   ? go(add_norm_grad_kernel<IO, ST, K, kRingRows>)
           : wide ? go(add_norm_grad_kernel<IO, ST, K, kVectors>)
                  : go(add_norm_grad_kernel<IO, ST, K, kElements>);
  });
  if (e != cudaSuccess || !part) return e;
  ColSum c{};
  c.nseg = 1;
  c.seg[0] = {part, a.dweight, w.blocks, a.D};
  return launch_colsum(c, err, st);
}

template <typename IO, typename ST>
size_t grad_workspace(const AddNormArgs &a) {
  const GradWalk w = grad_walk<IO, ST>(a);
  return sizeof(float) * (size_t)(w.blocks * a.D);
}

}  // namespace

size_t add_norm_backward_workspace(const AddNormArgs &a, ssd_dtype io, ssd_dtype stream) {
  if (io == SSD_F32) return grad_workspace<float, float>(a);
  return stream == SSD_F32 ? grad_workspace<__nv_bfloat16, float>(a)
                           : grad_workspace<__nv_bfloat16, __nv_bfloat16>(a);
}
cudaError_t launch_add_norm(const AddNormArgs &a, ssd_dtype io, ssd_dtype stream, int *err,
                            cudaStream_t st) {
  if (io == SSD_F32) return forward<float, float>(a, err, st);
  return stream == SSD_F32 ? forward<__nv_bfloat16, float>(a, err, st)
                           : forward<__nv_bfloat16, __nv_bfloat16>(a, err, st);
}
cudaError_t launch_add_norm_backward(const AddNormArgs &a, ssd_dtype io, ssd_dtype stream, void *ws,
                                     int *err, cudaStream_t st) {
  if (io == SSD_F32) return backward<float, float>(a, ws, err, st);
  return stream == SSD_F32 ? backward<__nv_bfloat16, float>(a, ws, err, st)
                           : backward<__nv_bfloat16, __nv_bfloat16>(a, ws, err, st);
}

}  // namespace ssd
