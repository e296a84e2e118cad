// Group norm per token with a SiLU gate, channels last.  Over each group of
// D / G channels of a token:
//   r = x silu(z) or x;  r -= mean(r) (centred);  n = r / sqrt(mean(r^2) + eps)
//   v = n weight + bias;  y = v silu(z) or v
//
// A bandwidth kernel: x and z read once, y written once.  The product x silu(z)
// is rounded by itself (no fused multiply-add with the mean), so that the r in
// r - mean(r) is the r that the mean was taken of: of a group of one channel
// the difference is exactly zero, where 1 / sqrt(eps) would enlarge a rounding.
// Of a group of equal r it is the rounding of their mean, a few ulp of r.
#include <type_traits>

#include "layer.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Sum of v over the block, in every thread; a fixed order.
__device__ __forceinline__ float block_sum(float v, float *scratch) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if (threadIdx.x % 32 == 0) scratch[threadIdx.x / 32] = v;
  __syncthreads();
  float s = scratch[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) s += scratch[w];
  __syncthreads();
  return s;
}

template <typename IO, int V>
__global__ void __launch_bounds__(kThreads)
norm_kernel(SeqView<const IO> x, const float *__restrict__ weight, const float *__restrict__ bias,
            SeqView<const IO> z, SeqView<IO> y, int64_t L, int group, float eps, int gate,
            bool center, int64_t nb, int *err) {
  __shared__ float scratch[kWarps];
  const int64_t b = blockIdx.x / L, t = blockIdx.x % L;
  const int64_t c0 = (int64_t)blockIdx.y * group;
  if (!SSD_IN_BOUNDS(b < nb && t < L, err, 40)) return;
  const IO *xr = x.at(b, t) + c0;
  const IO *zr = gate ? z.at(b, t) + c0 : nullptr;
  IO *yr = y.at(b, t) + c0;
  auto value = [&](int i, float (&r)[V]) {
    load_vec<V>(xr + i, r);
    if (gate == SSD_GATE_INPUT) {
      float g[V];
      load_vec<V>(zr + i, g);
#pragma unroll
      for (int k = 0; k < V; ++k) r[k] = __fmul_rn(r[k], silu(g[k]));
    }
  };
  float mean = 0.f, r[V];
  if (center) {
    float s = 0.f;
    for (int i = threadIdx.x * V; i < group; i += kThreads * V) {
      value(i, r);
#pragma unroll
      for (int k = 0; k < V; ++k) s += r[k];
    }
    mean = block_sum(s, scratch) / (float)group;
  }
  float s = 0.f;
  for (int i = threadIdx.x * V; i < group; i += kThreads * V) {
    value(i, r);
#pragma unroll
    for (int k = 0; k < V; ++k) s = fmaf(r[k] - mean, r[k] - mean, s);
  }
  const float rstd = rsqrtf(block_sum(s, scratch) / (float)group + eps);
  for (int i = threadIdx.x * V; i < group; i += kThreads * V) {
    value(i, r);
    float g[V];
    if (gate == SSD_GATE_OUTPUT) load_vec<V>(zr + i, g);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      float v = (r[k] - mean) * rstd * weight[c0 + i + k];
      if (bias) v += bias[c0 + i + k];
      r[k] = gate == SSD_GATE_OUTPUT ? v * silu(g[k]) : v;
    }
    store_vec<V>(yr + i, r);
  }
}

// What the gradients of one group of one token need.
struct Stat {
  float mean, rstd, qn, q;  // mean(r), 1 / root, mean(q n), mean(q)
};

// r, n and dL/dv of V channels.
template <int V, typename IO>
__device__ __forceinline__ void parts(const IO *xr, const IO *zr, const IO *gr, int64_t i,
                                      int gate, float (&x)[V], float (&z)[V], float (&gy)[V],
                                      float (&r)[V], float (&gv)[V]) {
  load_vec<V>(xr + i, x);
  load_vec<V>(gr + i, gy);
  if (gate) load_vec<V>(zr + i, z);
#pragma unroll
  for (int k = 0; k < V; ++k) {
    r[k] = gate == SSD_GATE_INPUT ? __fmul_rn(x[k], silu(z[k])) : x[k];
    gv[k] = gate == SSD_GATE_OUTPUT ? gy[k] * silu(z[k]) : gy[k];
  }
}

template <typename IO, int V>
__global__ void __launch_bounds__(kThreads)
norm_stat_kernel(SeqView<const IO> x, const float *__restrict__ weight, SeqView<const IO> z,
                 SeqView<const IO> gy, Stat *__restrict__ stat, int64_t L, int group, float eps,
                 int gate, bool center, int64_t nb, int *err) {
  __shared__ float scratch[kWarps];
  const int64_t b = blockIdx.x / L, t = blockIdx.x % L;
  const int64_t c0 = (int64_t)blockIdx.y * group;
  if (!SSD_IN_BOUNDS(b < nb && t < L, err, 41)) return;
  const IO *xr = x.at(b, t) + c0, *gr = gy.at(b, t) + c0;
  const IO *zr = gate ? z.at(b, t) + c0 : nullptr;
  float xv[V], zv[V], gyv[V], r[V], gv[V];
  Stat st{};
  if (center) {
    float s = 0.f;
    for (int i = threadIdx.x * V; i < group; i += kThreads * V) {
      parts<V>(xr, zr, gr, i, gate, xv, zv, gyv, r, gv);
#pragma unroll
      for (int k = 0; k < V; ++k) s += r[k];
    }
    st.mean = block_sum(s, scratch) / (float)group;
  }
  float s = 0.f, qr = 0.f, q = 0.f;
  for (int i = threadIdx.x * V; i < group; i += kThreads * V) {
    parts<V>(xr, zr, gr, i, gate, xv, zv, gyv, r, gv);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const float d = r[k] - st.mean, w = gv[k] * weight[c0 + i + k];
      s = fmaf(d, d, s);
      qr = fmaf(w, d, qr);
      q += w;
    }
  }
  st.rstd = rsqrtf(block_sum(s, scratch) / (float)group + eps);
  st.qn = block_sum(qr, scratch) * st.rstd / (float)group;
  st.q = center ? block_sum(q, scratch) / (float)group : 0.f;
  if (threadIdx.x == 0) stat[(int64_t)blockIdx.x * gridDim.y + blockIdx.y] = st;
}

// A thread owns V columns and walks a slice of the rows, so dweight and dbias
// need no exchange within the slice.
template <typename IO, int V>
__global__ void __launch_bounds__(kThreads)
norm_grad_kernel(SeqView<const IO> x, const float *__restrict__ weight,
                 const float *__restrict__ bias, SeqView<const IO> z, SeqView<const IO> gy,
                 const Stat *__restrict__ stat, SeqView<IO> dx, SeqView<IO> dz,
                 float *__restrict__ part_w, float *__restrict__ part_b, int64_t L, int64_t D,
                 int64_t rows, int64_t per, int group, int gate, int *err) {
  const int64_t c = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * V;
  if (c >= D) return;
  if (!SSD_IN_BOUNDS(c + V <= D, err, 42)) return;
  const int64_t r0 = blockIdx.y * per, r1 = r0 + per < rows ? r0 + per : rows;
  const int64_t G = D / group, grp = c / group;
  float w[V], bi[V], dw[V], db[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    w[k] = weight[c + k];
    bi[k] = bias ? bias[c + k] : 0.f;
    dw[k] = db[k] = 0.f;
  }
  for (int64_t row = r0; row < r1; ++row) {
    const int64_t b = row / L, t = row % L;
    const Stat st = stat[row * G + grp];
    float xv[V], zv[V], gyv[V], r[V], gv[V], ox[V], oz[V];
    parts<V>(x.at(b, t), gate ? z.at(b, t) : nullptr, gy.at(b, t), c, gate, xv, zv, gyv, r, gv);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const float n = (r[k] - st.mean) * st.rstd;
      dw[k] = fmaf(gv[k], n, dw[k]);
      db[k] += gv[k];
      const float gr = st.rstd * (gv[k] * w[k] - n * st.qn - st.q);
      ox[k] = gate == SSD_GATE_INPUT ? gr * silu(zv[k]) : gr;
      if (gate)
        oz[k] = (gate == SSD_GATE_INPUT ? gr * xv[k] : gyv[k] * fmaf(n, w[k], bi[k])) *
                dsilu(zv[k]);
    }
    store_vec<V>(dx.at(b, t) + c, ox);
    if (gate) store_vec<V>(dz.at(b, t) + c, oz);
  }
#pragma unroll
  for (int k = 0; k < V; ++k) {
    part_w[blockIdx.y * D + c + k] = dw[k];
    part_b[blockIdx.y * D + c + k] = db[k];
  }
}

// The kernels below read memory once.  A team of threads (a warp, or a whole
// block for a group of more than 32 K V channels) takes one group of one token
// at a time, K vectors of V channels to a thread, and walks the tokens with a
// fixed stride: dweight and dbias stay in registers, the weights come from L1
// at every token (held, they would cost as many registers).  Vectors of 16 bytes come kStages - 1 tokens ahead through shared
// memory, each thread copying its own, so no barrier waits for memory.
// Measured, bf16 and gated: 8192 x 5120 in 47 us (252 MB, 5.4 TB/s), the
// gradients of 8192 x 4096 in 8 groups in 68 (336 MB, 4.9 TB/s).  At odd offsets
// 8192 x 2003 takes 42 us and its gradients 74 (50 at 2000 channels).  Wider
// groups (above 8192 channels; above 4096 in fp32, or where vectors of 16 bytes
// do not fit) take the kernels above, which read memory twice: the gradients of
// 4096 x 5120 in fp32 132 us, of 4096 x 4096 66.

// V elements as the memory holds them.
template <typename IO, int V>
struct Raw {
  static constexpr int kBytes = V * (int)sizeof(IO);
  static constexpr int kWords = kBytes < 4 ? 1 : kBytes / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const IO *p) {
    if constexpr (kBytes == 16) {
      const uint4 q = *reinterpret_cast<const uint4 *>(p);
      w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
    } else if constexpr (kBytes == 8) {
      const uint2 q = *reinterpret_cast<const uint2 *>(p);
      w[0] = q.x, w[1] = q.y;
    } else if constexpr (kBytes == 4) {
      w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else {
      w[0] = *reinterpret_cast<const uint16_t *>(p);
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(IO) == 4)
      return __uint_as_float(w[i]);
    else
      return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
};

// Sums of M values over the team, in every thread; a fixed order.  `turn`
// alternates the scratch rows, so one barrier a call is enough.
template <int M>
__device__ __forceinline__ void team_sum(float (&v)[M], float (*scratch)[M][32], int warps,
                                         int &turn) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
#pragma unroll
    for (int m = 0; m < M; ++m) v[m] += __shfl_xor_sync(0xffffffffu, v[m], off);
  if (warps == 1) return;
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
    for (int m = 0; m < M; ++m) v[m] += __shfl_xor_sync(0xffffffffu, v[m], off);
  turn ^= 1;
}

// T tensors' vectors of a thread, for kStages tokens.
constexpr int kStages = 2;
template <typename IO, int V, int K, int T>
struct Ahead {
  static constexpr bool kAsync = V * sizeof(IO) == 16;
  uint4 *slots;  // this thread's first; the others blockDim apart
  int stage;
  __device__ __forceinline__ Ahead(void *smem)
      : slots(static_cast<uint4 *>(smem) + threadIdx.x), stage(0) {}
  __device__ __forceinline__ uint4 *slot(int s, int tensor, int k) const {
    return slots + ((s * T + tensor) * K + k) * (int)blockDim.x;
  }
  // Vector k of a tensor of the token `ahead` turns from the present one.
  __device__ __forceinline__ void copy(int ahead, int tensor, int k, const IO *p) {
    int s = stage + ahead;
    if (s >= kStages) s -= kStages;
    copy16(slot(s, tensor, k), p);
  }
  __device__ __forceinline__ void take(int tensor, int k, Raw<IO, V> &r) const {
    const uint4 q = *slot(stage, tensor, k);
    if constexpr (kAsync) r.w[0] = q.x, r.w[1] = q.y, r.w[2] = q.z, r.w[3] = q.w;
  }
  __device__ __forceinline__ void turn() { stage = stage + 1 == kStages ? 0 : stage + 1; }
};

// A token by sequence and position, walked by a stride without a division
// while it stays in its sequence.
struct Place {
  uint32_t b, t, L;
  __device__ __forceinline__ Place(int64_t row, int64_t len)
      : b((uint32_t)row / (uint32_t)len), t((uint32_t)row % (uint32_t)len), L((uint32_t)len) {}
  __device__ __forceinline__ void step(uint32_t n) {
    t += n;
    if (t >= L) {
      b += t / L;
      t %= L;
    }
  }
};

struct Teams {
  int threads;     // of a team: 32, or the block
  int64_t strides; // teams per group
};

constexpr int kMaxTeam = 512;
constexpr int kFwdBlocks = 2, kGradBlocks = 1;  // of that size to an SM

// V fp32 parameters; `vec`: the parameters start on a vector boundary.
__device__ __forceinline__ bool params_aligned(const float *weight, const float *bias) {
  return ((reinterpret_cast<uintptr_t>(weight) | reinterpret_cast<uintptr_t>(bias)) & 15) == 0;
}
template <int V>
__device__ __forceinline__ void load_params(const float *p, bool vec, float (&v)[V]) {
  if (V % 4 == 0 && vec) {
#pragma unroll
    for (int e = 0; e + 3 < V; e += 4) {
      const float4 f = *reinterpret_cast<const float4 *>(p + e);
      v[e] = f.x, v[e + 1] = f.y, v[e + 2] = f.z, v[e + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = p[e];
  }
}

template <typename IO, int V, int K, int gate>
__global__ void __launch_bounds__(kMaxTeam, kFwdBlocks)
norm_team_kernel(SeqView<const IO> x, const float *__restrict__ weight,
                 const float *__restrict__ bias, SeqView<const IO> z, SeqView<IO> y, int64_t L,
                 int64_t rows, int64_t G, int group, float eps, bool center, Teams tm,
                 int *err) {
  __shared__ float scratch[2][1][32];
  const int per_block = blockDim.x / tm.threads, warps = tm.threads / 32;
  const int64_t team = (int64_t)blockIdx.x * per_block + threadIdx.x / tm.threads;
  const int tid = threadIdx.x % tm.threads;
  if (team >= tm.strides * G) return;  // whole warps, or no thread of the block
  const int64_t c0 = team % G * group;
  int turn = 0;
  const float inv = 1.f / (float)group;
  const bool vec_params = params_aligned(weight, bias);
  extern __shared__ __align__(16) unsigned char smem[];
  Ahead<IO, V, K, 2> ahead(smem);
  const int64_t first = team / G;
  Place here(first, L), next(first, L);
  auto at = [&](const SeqView<const IO> &m, const Place &r, int i) {
    return m.at(r.b, r.t) + c0 + i;
  };
  auto issue = [&](int64_t row, int turns) {  // and on to the next
    if (row < rows)
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int i = (tid + k * tm.threads) * V;
        if (i >= group || !SSD_IN_BOUNDS(c0 + group <= G * group, err, 43)) continue;
        ahead.copy(turns, 0, k, at(x, next, i));
        if (gate) ahead.copy(turns, 1, k, at(z, next, i));
      }
    next.step((uint32_t)tm.strides);
    copies_issued();
  };
  if constexpr (decltype(ahead)::kAsync)
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) issue(first + k * tm.strides, k);
  for (int64_t row = first; row < rows; row += tm.strides, here.step((uint32_t)tm.strides)) {
    Raw<IO, V> xr[K], zr[K];
    if constexpr (decltype(ahead)::kAsync) {
      issue(row + (kStages - 1) * tm.strides, kStages - 1);
      copies_landed<kStages - 1>();
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = (tid + k * tm.threads) * V;
      if constexpr (decltype(ahead)::kAsync) {
        xr[k].clear(), zr[k].clear();
        if (i >= group) continue;
        ahead.take(0, k, xr[k]);
        if (gate) ahead.take(1, k, zr[k]);
      } else {  // without a branch, so that all the loads go out together
        if (!SSD_IN_BOUNDS(c0 + group <= G * group, err, 43)) return;
        xr[k].load(at(x, here, i < group ? i : 0));
        if (gate) zr[k].load(at(z, here, i < group ? i : 0));
      }
    }
    if constexpr (!decltype(ahead)::kAsync)
#pragma unroll
      for (int k = 0; k < K; ++k)
        if ((tid + k * tm.threads) * V >= group) xr[k].clear(), zr[k].clear();
    ahead.turn();
    float r[K][V], s[1] = {0.f};
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        r[k][e] = xr[k].at(e);
        if (gate == SSD_GATE_INPUT) r[k][e] = __fmul_rn(r[k][e], silu(zr[k].at(e)));
        if (center) s[0] += r[k][e];
      }
    if (center) {
      team_sum(s, scratch, warps, turn);
      const float mean = s[0] * inv;
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e)
          r[k][e] = (tid + k * tm.threads) * V < group ? r[k][e] - mean : 0.f;
    }
    s[0] = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) s[0] = fmaf(r[k][e], r[k][e], s[0]);
    team_sum(s, scratch, warps, turn);
    const float rstd = rsqrtf(s[0] * inv + eps);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = (tid + k * tm.threads) * V;
      const int64_t p = c0 + (i < group ? i : 0);
      float o[V], w[V];
      load_params<V>(weight + p, vec_params, w);
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = r[k][e] * rstd * w[e];
      if (bias) {
        load_params<V>(bias + p, vec_params, w);
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] += w[e];
      }
      if (gate == SSD_GATE_OUTPUT)
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] *= silu(zr[k].at(e));
      if (i < group) store_vec<V>(y.at(here.b, here.t) + c0 + i, o);
    }
  }
}

template <typename IO, int V, int K, int gate, bool BIAS>
__global__ void __launch_bounds__(kMaxTeam, kGradBlocks)
norm_team_grad_kernel(SeqView<const IO> x, const float *__restrict__ weight,
                      const float *__restrict__ bias, SeqView<const IO> z, SeqView<const IO> gy,
                      SeqView<IO> dx, SeqView<IO> dz, float *__restrict__ part_w,
                      float *__restrict__ part_b, int64_t L, int64_t rows, int64_t G, int group,
                      float eps, bool center, Teams tm, int *err) {
  __shared__ float scratch1[2][1][32], scratch3[2][3][32];
  const int per_block = blockDim.x / tm.threads, warps = tm.threads / 32;
  const int64_t team = (int64_t)blockIdx.x * per_block + threadIdx.x / tm.threads;
  const int tid = threadIdx.x % tm.threads;
  if (team >= tm.strides * G) return;
  const int64_t c0 = team % G * group;
  int turn1 = 0, turn3 = 0;
  const float inv = 1.f / (float)group;
  const bool vec_params = params_aligned(weight, bias);
  float dw[K][V], db[BIAS ? K : 1][V];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      dw[k][e] = 0.f;
      if (BIAS) db[k][e] = 0.f;
    }
  extern __shared__ __align__(16) unsigned char smem[];
  Ahead<IO, V, K, 3> ahead(smem);
  const int64_t first = team / G;
  Place here(first, L), next(first, L);
  auto at = [&](const SeqView<const IO> &m, const Place &r, int i) {
    return m.at(r.b, r.t) + c0 + i;
  };
  auto issue = [&](int64_t row, int turns) {  // and on to the next
    if (row < rows)
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int i = (tid + k * tm.threads) * V;
        if (i >= group || !SSD_IN_BOUNDS(c0 + group <= G * group, err, 44)) continue;
        ahead.copy(turns, 0, k, at(x, next, i));
        ahead.copy(turns, 1, k, at(gy, next, i));
        if (gate) ahead.copy(turns, 2, k, at(z, next, i));
      }
    next.step((uint32_t)tm.strides);
    copies_issued();
  };
  if constexpr (decltype(ahead)::kAsync)
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) issue(first + k * tm.strides, k);
  for (int64_t row = first; row < rows; row += tm.strides, here.step((uint32_t)tm.strides)) {
    Raw<IO, V> xc[K], zc[K], gc[K];
    if constexpr (decltype(ahead)::kAsync) {
      issue(row + (kStages - 1) * tm.strides, kStages - 1);
      copies_landed<kStages - 1>();
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = (tid + k * tm.threads) * V;
      if constexpr (decltype(ahead)::kAsync) {
        xc[k].clear(), zc[k].clear(), gc[k].clear();
        if (i >= group) continue;
        ahead.take(0, k, xc[k]);
        ahead.take(1, k, gc[k]);
        if (gate) ahead.take(2, k, zc[k]);
      } else {  // without a branch, so that all the loads go out together
        if (!SSD_IN_BOUNDS(c0 + group <= G * group, err, 44)) return;
        const int j = i < group ? i : 0;
        xc[k].load(at(x, here, j));
        gc[k].load(at(gy, here, j));
        if (gate) zc[k].load(at(z, here, j));
      }
    }
    if constexpr (!decltype(ahead)::kAsync)
#pragma unroll
      for (int k = 0; k < K; ++k)
        if ((tid + k * tm.threads) * V >= group) xc[k].clear(), zc[k].clear(), gc[k].clear();
    ahead.turn();
    float sig[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) sig[k][e] = gate ? sigmoid(zc[k].at(e)) : 0.f;
    // r and dL/dv of one channel
    auto r_of = [&](int k, int e) {
      const float v = xc[k].at(e);
      return gate == SSD_GATE_INPUT ? __fmul_rn(v, zc[k].at(e) * sig[k][e]) : v;
    };
    auto gv_of = [&](int k, int e) {
      const float v = gc[k].at(e);
      return gate == SSD_GATE_OUTPUT ? v * (zc[k].at(e) * sig[k][e]) : v;
    };
    float mean = 0.f;
    if (center) {
      float s[1] = {0.f};
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) s[0] += r_of(k, e);
      team_sum(s, scratch1, warps, turn1);
      mean = s[0] * inv;
    }
    float s[3] = {0.f, 0.f, 0.f};  // sums of d^2, q d, q with d = r - mean
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = (tid + k * tm.threads) * V;
      const bool ok = i < group;
      float w[V];
      load_params<V>(weight + c0 + (ok ? i : 0), vec_params, w);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float d = ok ? r_of(k, e) - mean : 0.f, q = ok ? gv_of(k, e) * w[e] : 0.f;
        s[0] = fmaf(d, d, s[0]);
        s[1] = fmaf(q, d, s[1]);
        if (center) s[2] += q;
      }
    }
    team_sum(s, scratch3, warps, turn3);
    const float rstd = rsqrtf(s[0] * inv + eps);
    const float qn = s[1] * rstd * inv, qm = center ? s[2] * inv : 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = (tid + k * tm.threads) * V;
      const int64_t p = c0 + (i < group ? i : 0);
      float ox[V], oz[V], w[V], bi[V];
      load_params<V>(weight + p, vec_params, w);
      if (BIAS && gate == SSD_GATE_OUTPUT) {
#pragma unroll
        for (int e = 0; e < V; ++e) bi[e] = 0.f;
        if (bias) load_params<V>(bias + p, vec_params, bi);
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float zv = zc[k].at(e), xv = xc[k].at(e), sg = sig[k][e], sz = zv * sg;
        const float gv = gv_of(k, e);
        const float n = (r_of(k, e) - mean) * rstd;
        dw[k][e] = fmaf(gv, n, dw[k][e]);
        if (BIAS) db[k][e] += gv;
        const float g = rstd * (gv * w[e] - n * qn - qm);
        const float slope = sg * fmaf(zv, 1.f - sg, 1.f);  // silu'
        ox[e] = gate == SSD_GATE_INPUT ? g * sz : g;
        if (gate == SSD_GATE_INPUT) oz[e] = slope * (g * xv);
        if (gate == SSD_GATE_OUTPUT)
          oz[e] = slope * (gc[k].at(e) * (BIAS ? fmaf(n, w[e], bi[e]) : n * w[e]));
      }
      if (i >= group) continue;
      store_vec<V>(dx.at(here.b, here.t) + c0 + i, ox);
      if (gate) store_vec<V>(dz.at(here.b, here.t) + c0 + i, oz);
    }
  }
  const int64_t D = G * group, slice = team / G;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int i = (tid + k * tm.threads) * V;
    if (i >= group) continue;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      part_w[slice * D + c0 + i + e] = dw[k][e];
      if (BIAS) part_b[slice * D + c0 + i + e] = db[k][e];
    }
  }
}

template <typename T>
struct tag {
  using type = T;
};
template <typename F>
cudaError_t dispatch(ssd_dtype io, bool vec, F f) {
  auto by_vec = [&](auto io_c) {
    return vec ? f(io_c, std::integral_constant<int, 4>{})
               : f(io_c, std::integral_constant<int, 1>{});
  };
  return io == SSD_BF16 ? by_vec(tag<__nv_bfloat16>{}) : by_vec(tag<float>{});
}

// Elements per vector that the sizes and every address allow: 16 bytes, two
// elements, or one.
int vector_of(const NormArgs &a, ssd_dtype io) {
  const size_t e = io == SSD_BF16 ? 2 : 4;
  auto fits = [&](size_t n) {
    return (a.D / a.G) % n == 0 && view_aligned(a.x, e, n * e) && view_aligned(a.z, e, n * e) &&
           view_aligned(a.y, e, n * e) && view_aligned(a.gy, e, n * e) &&
           view_aligned(a.dx, e, n * e) && view_aligned(a.dz, e, n * e);
  };
  return fits(16 / e) ? (int)(16 / e) : fits(2) ? 2 : 1;
}
// Vectors per thread: 16 channels where they come eight at a time (bf16), 8 of
// any other (fp32's registers are twice as many).
constexpr int vectors_per_thread(int V) { return V == 8 || V == 4 ? 2 : V == 2 ? 4 : 8; }

// Shared memory of a block of `block` threads for T tensors' vectors ahead.
constexpr int ahead_bytes(int V, size_t elem, int K, int T, int block) {
  return V * elem == 16 ? kStages * T * K * 16 * block : 0;
}
// Lets `kernel` have the shared memory of its largest block.  Always the same
// amount: the attribute belongs to the kernel, not to the call, so an amount
// of this call's own could fall between another thread's and its launch.
template <typename F>
cudaError_t allow_smem(F kernel, int bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

// The team for a group, or 0 threads where a block's registers do not hold it.
int team_threads(const NormArgs &a, ssd_dtype io) {
  const int V = vector_of(a, io), per = V * vectors_per_thread(V);
  const int64_t n = (a.D / a.G + per - 1) / per;
  return n > kMaxTeam ? 0 : (int)((n + 31) / 32 * 32);
}
// Teams: about `warps` warps to an SM in all.
Teams teams_of(const NormArgs &a, int threads, int warps) {
  Teams t;
  t.threads = threads;
  const int64_t want = (int64_t)sm_count() * warps * 32 / threads;
  t.strides = (want + a.G - 1) / a.G;
  if (t.strides > a.b * a.L) t.strides = a.b * a.L;
  return t;
}
constexpr int kFwdWarps = 30, kGradWarps = 16;  // what fits at once

template <typename F>
cudaError_t dispatch_team(ssd_dtype io, int V, int gate, F f) {
  using std::integral_constant;
  auto by_gate = [&](auto io_c, auto v_c) {
    if (gate == SSD_GATE_INPUT) return f(io_c, v_c, integral_constant<int, SSD_GATE_INPUT>{});
    if (gate == SSD_GATE_OUTPUT) return f(io_c, v_c, integral_constant<int, SSD_GATE_OUTPUT>{});
    return f(io_c, v_c, integral_constant<int, SSD_GATE_NONE>{});
  };
  if (io == SSD_BF16) {
    if (V == 8) return by_gate(tag<__nv_bfloat16>{}, integral_constant<int, 8>{});
    if (V == 2) return by_gate(tag<__nv_bfloat16>{}, integral_constant<int, 2>{});
    return by_gate(tag<__nv_bfloat16>{}, integral_constant<int, 1>{});
  }
  if (V == 4) return by_gate(tag<float>{}, integral_constant<int, 4>{});
  if (V == 2) return by_gate(tag<float>{}, integral_constant<int, 2>{});
  return by_gate(tag<float>{}, integral_constant<int, 1>{});
}

bool vectored(const NormArgs &a, ssd_dtype io) {
  const size_t e = io == SSD_BF16 ? 2 : 4, bytes = 4 * e;
  return (a.D / a.G) % 4 == 0 && view_aligned(a.x, e, bytes) && view_aligned(a.z, e, bytes) &&
         view_aligned(a.y, e, bytes) && view_aligned(a.gy, e, bytes) &&
         view_aligned(a.dx, e, bytes) && view_aligned(a.dz, e, bytes);
}

// Row slices of the gradient kernel and the rows of each.
int64_t slice_rows(const NormArgs &a) {
  const int64_t rows = a.b * a.L;
  const int64_t per = (rows + 255) / 256;
  return per < 4 ? 4 : per;
}
int64_t slices(const NormArgs &a) { return (a.b * a.L + slice_rows(a) - 1) / slice_rows(a); }

}  // namespace

cudaError_t launch_gated_norm(const NormArgs &a, ssd_dtype io, int *err, cudaStream_t st) {
  if (const int threads = team_threads(a, io)) {
    const Teams tm = teams_of(a, threads, kFwdWarps);
    const int block = threads == 32 ? 256 : threads;
    const int64_t blocks = (tm.strides * a.G * threads + block - 1) / block;
    return dispatch_team(io, vector_of(a, io), a.gate, [&](auto io_c, auto v_c, auto gate_c) {
      using IO = typename decltype(io_c)::type;
      constexpr int V = decltype(v_c)::value;
      constexpr int K = vectors_per_thread(V), gate = decltype(gate_c)::value;
      const auto kernel = norm_team_kernel<IO, V, K, gate>;
      const cudaError_t e = allow_smem(kernel, ahead_bytes(V, sizeof(IO), K, 2, kMaxTeam));
      if (e != cudaSuccess) return e;
      kernel<<<(unsigned)blocks, block, ahead_bytes(V, sizeof(IO), K, 2, block), st>>>(
          view_of<const IO>(a.x), a.weight, a.bias, view_of<const IO>(a.z), view_of<IO>(a.y), a.L,
          a.b * a.L, a.G, (int)(a.D / a.G), a.eps, a.center, tm, err);
      return cudaGetLastError();
    });
  }
  return dispatch(io, vectored(a, io), [&](auto io_c, auto v_c) {
    using IO = typename decltype(io_c)::type;
    const dim3 grid((unsigned)(a.b * a.L), (unsigned)a.G);
    norm_kernel<IO, decltype(v_c)::value><<<grid, kThreads, 0, st>>>(
        view_of<const IO>(a.x), a.weight, a.bias, view_of<const IO>(a.z), view_of<IO>(a.y), a.L,
        (int)(a.D / a.G), a.eps, a.gate, a.center, a.b, err);
    return cudaGetLastError();
  });
}

// The team for a group may differ between the size's query and the call (the
// addresses' alignment is not known to the query): room for either.
size_t gated_norm_backward_workspace(const NormArgs &a, ssd_dtype io) {
  const size_t two = sizeof(Stat) * (size_t)(a.b * a.L * a.G) +
                     2 * sizeof(float) * (size_t)(slices(a) * a.D);
  const int64_t most = teams_of(a, 32, kGradWarps).strides;  // the smallest team has most
  const size_t one = 2 * sizeof(float) * (size_t)(most * a.D);
  return one > two ? one : two;
}

cudaError_t launch_gated_norm_backward(const NormArgs &a, ssd_dtype io, void *ws, int *err,
                                       cudaStream_t st) {
  if (const int threads = team_threads(a, io)) {
    const Teams tm = teams_of(a, threads, kGradWarps);
    float *part_w = static_cast<float *>(ws), *part_b = part_w + tm.strides * a.D;
    const int block = threads == 32 ? 256 : threads;
    const int64_t blocks = (tm.strides * a.G * threads + block - 1) / block;
    const cudaError_t e = dispatch_team(io, vector_of(a, io), a.gate, [&](auto io_c, auto v_c, auto gate_c) {
      using IO = typename decltype(io_c)::type;
      constexpr int V = decltype(v_c)::value;
      constexpr int K = vectors_per_thread(V), gate = decltype(gate_c)::value;
      auto go = [&](auto bias_c) {
        const auto kernel = norm_team_grad_kernel<IO, V, K, gate, decltype(bias_c)::value>;
        const cudaError_t e1 = allow_smem(kernel, ahead_bytes(V, sizeof(IO), K, 3, kMaxTeam));
        if (e1 != cudaSuccess) return e1;
        kernel<<<(unsigned)blocks, block, ahead_bytes(V, sizeof(IO), K, 3, block), st>>>(
            view_of<const IO>(a.x), a.weight, a.bias, view_of<const IO>(a.z),
            view_of<const IO>(a.gy), view_of<IO>(a.dx), view_of<IO>(a.dz), part_w, part_b, a.L,
            a.b * a.L, a.G, (int)(a.D / a.G), a.eps, a.center, tm, err);
        return cudaGetLastError();
      };
      return a.bias || a.dbias ? go(std::true_type{}) : go(std::false_type{});
    });
    if (e != cudaSuccess) return e;
    ColSum s{};
    s.nseg = 2;
    s.seg[0] = {part_w, a.dweight, tm.strides, a.D};
    s.seg[1] = {part_b, a.dbias, tm.strides, a.D};
    return launch_colsum(s, err, st);
  }
  Stat *stat = static_cast<Stat *>(ws);
  float *part_w = reinterpret_cast<float *>(stat + a.b * a.L * a.G);
  float *part_b = part_w + slices(a) * a.D;
  const cudaError_t e = dispatch(io, vectored(a, io), [&](auto io_c, auto v_c) {
    using IO = typename decltype(io_c)::type;
    constexpr int V = decltype(v_c)::value;
    const int group = (int)(a.D / a.G);
    norm_stat_kernel<IO, V><<<dim3((unsigned)(a.b * a.L), (unsigned)a.G), kThreads, 0, st>>>(
        view_of<const IO>(a.x), a.weight, view_of<const IO>(a.z), view_of<const IO>(a.gy), stat,
        a.L, group, a.eps, a.gate, a.center, a.b, err);
    const cudaError_t e1 = cudaGetLastError();
    if (e1 != cudaSuccess) return e1;
    const dim3 grid((unsigned)((a.D / V + kThreads - 1) / kThreads), (unsigned)slices(a));
    norm_grad_kernel<IO, V><<<grid, kThreads, 0, st>>>(
        view_of<const IO>(a.x), a.weight, a.bias, view_of<const IO>(a.z),
        view_of<const IO>(a.gy), stat, view_of<IO>(a.dx), view_of<IO>(a.dz), part_w, part_b, a.L,
        a.D, a.b * a.L, slice_rows(a), group, a.gate, err);
    return cudaGetLastError();
  });
  if (e != cudaSuccess) return e;
  ColSum s{};
  s.nseg = 2;
  s.seg[0] = {part_w, a.dweight, slices(a), a.D};
  s.seg[1] = {part_b, a.dbias, slices(a), a.D};
  return launch_colsum(s, err, st);
}

}  // namespace ssd
