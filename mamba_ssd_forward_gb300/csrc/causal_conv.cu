// Short causal convolution along the tokens, per channel, with SiLU:
//   v_t = bias + sum_{k<W} w_k x_{t-W+1+k},   y_t = silu(v_t)
// where the W - 1 tokens before the first are the rows of a state.
//
// A bandwidth kernel: x read once, y written once; 2W + 4 operations per
// element.  A thread takes V neighbouring channels and a run of tokens, with
// the last W - 1 inputs in registers, so x is read once but for the W - 1
// tokens in front of each run (which the neighbouring run brought into L2).
// Tokens come by asynchronous copies through a ring of the thread's own in
// shared memory, which keeps eight rows in flight without their registers.
// Measured at W = 4: 2 x 4096 x 5376 in bf16 in 35 us (5.0 TB/s; 26 us at the
// copy bandwidth), the gradients of 4 x 2048 x 1792 in fp32 in 41 (the same
// bytes).  Half of the issue slots are taken, and warps wait for rows the rest.
#include <type_traits>

#include "layer.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 256;
constexpr int kRingThreads = 128, kRingBlocks = 4;
constexpr int kRing = 8, kRingBack = 4, kBackBlocks = 2, kBackBlocks1 = 3;

template <int V>
__device__ __forceinline__ void zero(float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = 0.f;
}

// The convolution's parameters of channels c .. c + V - 1.
template <int W, int V>
struct Taps {
  float w[W][V], bias[V];
  __device__ __forceinline__ void load(const float *weight, const float *b, int64_t c, int64_t D,
                                       int *err) {
    if (!SSD_IN_BOUNDS(c + V <= D, err, 30)) return;
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
      for (int k = 0; k < W; ++k) w[k][i] = weight[(c + i) * W + k];
      bias[i] = b ? b[c + i] : 0.f;
    }
  }
};

// The same for a whole warp whose lanes stand at vectors first, first + 1, ..
// (mod nv): read in the order of memory and handed out through `box`, 32 V
// quads of the warp's own, each channel's weights one quad.  Lanes reading
// their own channels directly would touch 32 lines a load: 58 us for 8192
// tokens of 5376 channels, against 37.
template <int W, int V>
__device__ __forceinline__ void warp_taps(Taps<W, V> &p, float4 *box, const float *weight,
                                          const float *b, uint32_t first, uint32_t nv, int64_t D,
                                          int *err) {
  const int lane = threadIdx.x % 32;
  const bool quads = W == 4 && (reinterpret_cast<uintptr_t>(weight) & 15) == 0;
  auto place = [](int f) { return f ^ (f / V % 8); };  // spreads a lane's quads over the banks
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int f = j * 32 + lane;
    const int64_t ch = (int64_t)((first + f / V) % nv) * V + f % V;
    if (!SSD_IN_BOUNDS(ch < D, err, 36)) continue;
    const float *w = weight + ch * W;
    float4 q;
    if (quads) {
      q = *reinterpret_cast<const float4 *>(w);
    } else {
      q.x = w[0], q.y = w[1];
      if (W > 2) q.z = w[2];
      if (W > 3) q.w = w[W - 1];
    }
    box[place(f)] = q;
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float4 q = box[place(lane * V + i)];
    p.w[0][i] = q.x, p.w[1][i] = q.y;
    if (W > 2) p.w[W > 2 ? 2 : 0][i] = q.z;
    if (W > 3) p.w[W > 3 ? 3 : 0][i] = q.w;
  }
  const int64_t c = (int64_t)((first + lane) % nv) * V;
  if (b && (reinterpret_cast<uintptr_t>(b) & 15) == 0 && V % 4 == 0) {
#pragma unroll
    for (int i = 0; i + 3 < V; i += 4) {
      const float4 q = *reinterpret_cast<const float4 *>(b + c + i);
      p.bias[i] = q.x, p.bias[i + 1] = q.y, p.bias[i + 2] = q.z, p.bias[i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) p.bias[i] = b ? b[c + i] : 0.f;
  }
}

// Row p of the inputs, p in [-(W-1), len): a row of the state below zero.
template <int W, int V, typename IO>
__device__ __forceinline__ void input_row(const SeqView<const IO> &x, const IO *state, int64_t b,
                                          int64_t p, int64_t c, int64_t D, int64_t L, int *err,
                                          float (&v)[V]) {
  zero(v);
  if (!SSD_IN_BOUNDS(p >= -(W - 1) && p < L && c + V <= D, err, 31)) return;
  if (p >= 0)
    load_vec<V>(x.at(b, p) + c, v);
  else if (state)
    load_vec<V>(state + (b * (W - 1) + (p + W - 1)) * D + c, v);
}

// Rows on any boundary, a channel to a thread, loads in batches of A rows: 48 us
// for 8192 bf16 tokens of 5376 channels at odd offsets, against 33 of the ring
// kernel on aligned ones (A was chosen at 53 us: A = 4 67, A = 16 56).
template <typename IO, int W>
__global__ void __launch_bounds__(kThreads)
conv_kernel(SeqView<const IO> x, const float *__restrict__ weight, const float *__restrict__ bias,
            const IO *__restrict__ state, const int32_t *__restrict__ lengths, SeqView<IO> y,
            IO *__restrict__ final_state, int64_t L, int64_t D, int run, bool act, int *err) {
  constexpr int A = 8, V = 1;  // rows loaded before the arithmetic of the first
  const int64_t idx = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t c = idx % D;
  const int64_t t0 = idx / D * run;
  const int64_t b = blockIdx.y;
  if (t0 >= L) return;
  const int64_t len = tokens_of(lengths, b, L);
  const int64_t t1 = t0 + run < L ? t0 + run : L;
  const int64_t te = t1 < len ? t1 : len;
  if (t0 < te) {
    Taps<W, V> p;
    p.load(weight, bias, c, D, err);
    float win[W - 1][V];
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      input_row<W, V>(x, state, b, t0 - (W - 1) + j, c, D, L, err, win[j]);
    if (!SSD_IN_BOUNDS(te <= L && c + V <= D, err, 32)) return;
    const IO *from = x.at(b, t0) + c;
    IO *to = y.at(b, t0) + c;
    for (int left = (int)(te - t0); left > 0; left -= A) {
      float in[A][V];
#pragma unroll
      for (int u = 0; u < A; ++u) {
        zero(in[u]);
        if (u < left) load_vec<V>(from, in[u]);
        from += x.ts;
      }
#pragma unroll
      for (int u = 0; u < A; ++u) {
        float out[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float v = p.bias[i];
#pragma unroll
          for (int k = 0; k < W - 1; ++k) v = fmaf(p.w[k][i], win[k][i], v);
          v = fmaf(p.w[W - 1][i], in[u][i], v);
          out[i] = act ? silu(v) : v;
#pragma unroll
          for (int k = 0; k < W - 2; ++k) win[k][i] = win[k + 1][i];
          win[W - 2][i] = in[u][i];
        }
        if (u < left) store_vec<V>(to, out);
        to += y.ts;
      }
    }
  }
  float none[V];
  zero(none);
  for (int64_t t = te > t0 ? te : t0; t < t1; ++t) store_vec<V>(y.at(b, t) + c, none);
  if (t0 == 0 && final_state) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      float v[V];
      input_row<W, V>(x, state, b, len - (W - 1) + j, c, D, L, err, v);
      store_vec<V>(final_state + (b * (W - 1) + j) * D + c, v);
    }
  }
}

template <typename IO, int W, int V>
__global__ void __launch_bounds__(kThreads)
conv_step_kernel(SeqView<const IO> x, const float *__restrict__ weight,
                 const float *__restrict__ bias, IO *__restrict__ state, SeqView<IO> y, int64_t nb,
                 int64_t D, bool act, int *err) {
  const int64_t nv = D / V;
  const int64_t idx = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t c = idx % nv * V, b = idx / nv;
  if (b >= nb) return;
  if (!SSD_IN_BOUNDS(c + V <= D, err, 33)) return;
  float win[W][V], out[V];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) load_vec<V>(state + (b * (W - 1) + j) * D + c, win[j]);
  load_vec<V>(x.at(b, 0) + c, win[W - 1]);
  Taps<W, V> p;
  p.load(weight, bias, c, D, err);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float v = p.bias[i];
#pragma unroll
    for (int k = 0; k < W; ++k) v = fmaf(p.w[k][i], win[k][i], v);
    out[i] = act ? silu(v) : v;
  }
  store_vec<V>(y.at(b, 0) + c, out);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) store_vec<V>(state + (b * (W - 1) + j) * D + c, win[j + 1]);
}

// Rows of 8 or 16 bytes a thread, copied kRing - 1 rows ahead into the thread's
// own slots of shared memory: no barrier waits for memory, and what is in
// flight does not cost registers.
template <typename IO, int V, int RING, int T>
struct Ring {
  static constexpr int kBytes = V * (int)sizeof(IO);
  unsigned char *slots;  // this thread's first
  __device__ __forceinline__ Ring(void *smem)
      : slots(static_cast<unsigned char *>(smem) + threadIdx.x * kBytes) {}
  __device__ __forceinline__ IO *slot(int row, int tensor) const {
    return reinterpret_cast<IO *>(slots + (row * T + tensor) * (int)blockDim.x * kBytes);
  }
  __device__ __forceinline__ void copy(int row, int tensor, const IO *p) const {
    if constexpr (kBytes == 16)
      copy16(slot(row, tensor), p);
    else
      copy8(slot(row, tensor), p);
  }
};

// The forward with the rows coming through a ring; RING rows unrolled, so that
// slots and the window need no index arithmetic.
template <typename IO, int W, int V, bool ACT>
__global__ void __launch_bounds__(kRingThreads, kRingBlocks)
conv_ring_kernel(SeqView<const IO> x, const float *__restrict__ weight,
                 const float *__restrict__ bias, const IO *__restrict__ state,
                 const int32_t *__restrict__ lengths, SeqView<IO> y, IO *__restrict__ final_state,
                 int64_t L, int64_t D, int run, int *err) {
  constexpr int R = kRing;
  __shared__ __align__(16) unsigned char smem[R * kRingThreads * V * sizeof(IO)];
  __shared__ float4 box[kRingThreads * V];
  const Ring<IO, V, R, 1> ring(smem);
  const uint32_t nv = (uint32_t)(D / V);
  const uint32_t idx = blockIdx.x * kRingThreads + threadIdx.x;
  const int64_t c = (int64_t)(idx % nv) * V;
  const int64_t t0 = (int64_t)(idx / nv) * run;
  const int64_t b = blockIdx.y;
  const int64_t len = tokens_of(lengths, b, L);
  const int64_t t1 = t0 + run < L ? t0 + run : L;
  const int n = (int)((t1 < len ? t1 : len) - t0);  // tokens of this run, maybe none
  const IO *px = x.at(b, t0) + c;
  IO *py = y.at(b, t0) + c;
#pragma unroll
  for (int k = 0; k < R - 1; ++k) {
    if (k < n && SSD_IN_BOUNDS(t0 + k < L && c + V <= D, err, 35)) ring.copy(k, 0, px);
    px += x.ts;
    copies_issued();
  }
  Taps<W, V> p;
  warp_taps<W, V>(p, box + threadIdx.x / 32 * 32 * V, weight, bias, idx / 32 * 32, nv, D, err);
  if (t0 >= L) return;  // only now: the warp's lanes share the weights' loads
  if (n > 0) {
    float win[W - 1][V];
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      input_row<W, V>(x, state, b, t0 - (W - 1) + j, c, D, L, err, win[j]);
    auto row = [&](int u) {
      float in[V], out[V];
      load_vec<V>(ring.slot(u, 0), in);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float v = p.bias[i];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) v = fmaf(p.w[j][i], win[j][i], v);
        v = fmaf(p.w[W - 1][i], in[i], v);
        out[i] = ACT ? silu(v) : v;
#pragma unroll
        for (int j = 0; j < W - 2; ++j) win[j][i] = win[j + 1][i];
        win[W - 2][i] = in[i];
      }
      store_vec<V>(py, out);
    };
    int k0 = 0;
    for (; k0 + 2 * R - 1 <= n; k0 += R)  // every row and every copy there
#pragma unroll
      for (int u = 0; u < R; ++u) {
        if (SSD_IN_BOUNDS(t0 + k0 + u + R - 1 < L && c + V <= D, err, 35))
          ring.copy((u + R - 1) % R, 0, px);
        px += x.ts;
        copies_issued();
        copies_landed<R - 1>();
        row(u);
        py += y.ts;
      }
    for (; k0 < n; k0 += R)
#pragma unroll
      for (int u = 0; u < R; ++u) {
        const int k = k0 + u;
        if (k + R - 1 < n && SSD_IN_BOUNDS(t0 + k + R - 1 < L && c + V <= D, err, 35))
          ring.copy((u + R - 1) % R, 0, px);
        px += x.ts;
        copies_issued();
        copies_landed<R - 1>();
        if (k < n) row(u);
        py += y.ts;
      }
  }
  float none[V];
  zero(none);
  for (int64_t t = n > 0 ? t0 + n : t0; t < t1; ++t) store_vec<V>(y.at(b, t) + c, none);
  if (t0 == 0 && final_state) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      float v[V];
      input_row<W, V>(x, state, b, len - (W - 1) + j, c, D, L, err, v);
      store_vec<V>(final_state + (b * (W - 1) + j) * D + c, v);
    }
  }
}

// Backward.  With g_t = gy_t silu'(v_t) (v recomputed from the window),
//   dx_p = sum_k w_k g_{p+W-1-k},  dw_k = sum_t g_t x_{t-W+1+k},  dbias = sum_t g_t,
// dx at p < 0 being the state's gradient.  A block is 32 channel vectors by
// kRuns runs of tokens; a thread walks its run and the W - 1 tokens after it
// (whose g its last dx need), with the last W - 1 inputs and g and the sums of
// dw and dbias in registers.  The block adds its runs' sums in order and writes
// one partial row; a column sum finishes.  x and gy read once, dx written once.
// ASYNC: rows of 8 or 16 bytes through a ring, as in the forward.
constexpr int kRuns = 8;

template <typename IO, int W, int V, bool ASYNC, bool ACT>
__global__ void __launch_bounds__(32 * kRuns, V > 1 ? kBackBlocks : kBackBlocks1)
conv_bwd_kernel(SeqView<const IO> x, const float *__restrict__ weight,
                const float *__restrict__ bias, const IO *__restrict__ state,
                SeqView<const IO> gy, const IO *__restrict__ gfinal,
                const int32_t *__restrict__ lengths, SeqView<IO> dx, IO *__restrict__ dstate,
                float *__restrict__ part_w, float *__restrict__ part_b, int64_t L, int64_t D,
                int run, int *err) {
  constexpr int R = ASYNC ? kRingBack : 8;
  static_assert(R >= W - 1, "the first turns are those before the loop's second round");
  constexpr size_t kSums = kRuns * 32 * V * (W + 1) * sizeof(float);
  constexpr size_t kSlots = ASYNC ? (size_t)R * 2 * 32 * kRuns * V * sizeof(IO) : 0;
  constexpr size_t kBox = ASYNC ? 32 * V * sizeof(float4) : 16;
  __shared__ __align__(16) unsigned char smem[kSums > kSlots ? kSums : kSlots];
  __shared__ __align__(16) unsigned char box[kBox * (ASYNC ? kRuns : 1)];
  const Ring<IO, V, R, 2> ring(smem);
  const int lane = threadIdx.x % 32, slot = threadIdx.x / 32;
  const int64_t c = ((int64_t)blockIdx.x * 32 + lane) * V;
  const int64_t b = blockIdx.z;
  const int64_t t0 = ((int64_t)blockIdx.y * kRuns + slot) * run;
  const int64_t len = tokens_of(lengths, b, L);
  float dw[W][V], db[V];
#pragma unroll
  for (int k = 0; k < W; ++k) zero(dw[k]);
  zero(db);
  Taps<W, V> p;
  if constexpr (ASYNC)  // every lane takes part, beyond the last vector with another's
    warp_taps<W, V>(p, reinterpret_cast<float4 *>(box + slot * kBox), weight, bias,
                    blockIdx.x * 32, (uint32_t)(D / V), D, err);
  if (c < D && t0 < L && SSD_IN_BOUNDS(c + V <= D, err, 34)) {
    if constexpr (!ASYNC) p.load(weight, bias, c, D, err);
    const int64_t t1 = t0 + run < L ? t0 + run : L;
    const int own = (int)(t1 - t0);
    const int all = own + W - 1;  // turns; turn k completes dx of token t0 + k - (W - 1)
    // turns that have a token
    const int n = len - t0 < all ? (len > t0 ? (int)(len - t0) : 0) : all;
    const IO *px = x.at(b, t0) + c, *pg = gy.at(b, t0) + c;
    IO *pd = dx.p ? dx.at(b, t0) + c - (W - 1) * dx.ts : nullptr;
    auto issue = [&](int k, int row, bool sure) {
      if ((sure || k < n) && SSD_IN_BOUNDS(t0 + k < L, err, 34)) {
        ring.copy(row, 0, px);
        ring.copy(row, 1, pg);
      }
      px += x.ts, pg += gy.ts;
      copies_issued();
    };
    if (ASYNC)
#pragma unroll
      for (int k = 0; k < R - 1; ++k) issue(k, k, false);
    float win[W - 1][V], gs[W - 1][V];  // the last inputs and g, oldest first
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      zero(win[j]);
      zero(gs[j]);
      if (n > 0) input_row<W, V>(x, state, b, t0 - (W - 1) + j, c, D, L, err, win[j]);
    }
    float nx[ASYNC ? 1 : R][V], ng[ASYNC ? 1 : R][V];  // without a ring: a round's rows
    // one turn; `inner`: a turn within the run whose token, dx and copies are
    // there and whose dx gets nothing of the final state's gradient
    auto turn = [&](int k, int u, auto inner_c) {
      constexpr bool inner = decltype(inner_c)::value;
      float in[V], g[V], o[V];
      zero(in);
      zero(g);
      if (ASYNC) {
        issue(k + R - 1, (u + R - 1) % R, inner);
        copies_landed<R - 1>();
        if (inner || k < n) {
          load_vec<V>(ring.slot(u, 0), in);
          load_vec<V>(ring.slot(u, 1), g);
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) in[i] = nx[u][i], g[i] = ng[u][i];
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float v = p.bias[i];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) v = fmaf(p.w[j][i], win[j][i], v);
        v = fmaf(p.w[W - 1][i], in[i], v);
        if (ACT) g[i] = inner || k < n ? g[i] * dsilu(v) : 0.f;
        o[i] = p.w[0][i] * g[i];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) o[i] = fmaf(p.w[W - 1 - j][i], gs[j][i], o[i]);
        const float gw = inner || k < own ? g[i] : 0.f;  // tokens after the run are another's
#pragma unroll
        for (int j = 0; j < W - 1; ++j) dw[j][i] = fmaf(gw, win[j][i], dw[j][i]);
        dw[W - 1][i] = fmaf(gw, in[i], dw[W - 1][i]);
        db[i] += gw;
#pragma unroll
        for (int j = 0; j < W - 2; ++j) win[j][i] = win[j + 1][i], gs[j][i] = gs[j + 1][i];
        win[W - 2][i] = in[i];
        gs[W - 2][i] = g[i];
      }
      if (inner) {
        if (pd) store_vec<V>(pd, o);
      } else if (k >= W - 1 || t0 == 0) {  // the first run owns the state's rows too
        const int64_t q = t0 + k - (W - 1);
        if (gfinal && q < len && q >= len - (W - 1)) {
          float f[V];
          load_vec<V>(gfinal + (b * (W - 1) + (q - len + W - 1)) * D + c, f);
#pragma unroll
          for (int i = 0; i < V; ++i) o[i] += f[i];
        }
        if (q >= 0) {
          if (pd) store_vec<V>(pd, o);
        } else if (dstate) {
          store_vec<V>(dstate + (b * (W - 1) + (q + W - 1)) * D + c, o);
        }
      }
      if (pd) pd += dx.ts;
    };
    const int within = n < own ? n : own;
    for (int k0 = 0; k0 < all; k0 += R) {
      if constexpr (!ASYNC)
#pragma unroll
        for (int u = 0; u < R; ++u) {
          zero(nx[u]);
          zero(ng[u]);
          if (k0 + u < n && SSD_IN_BOUNDS(t0 + k0 + u < L, err, 34)) {
            load_vec<V>(px, nx[u]);
            load_vec<V>(pg, ng[u]);
          }
          px += x.ts, pg += gy.ts;
        }
      if (k0 >= R && k0 + R <= within && k0 + 2 * R - 1 <= n) {
#pragma unroll
        for (int u = 0; u < R; ++u) turn(k0 + u, u, std::true_type{});
      } else {
#pragma unroll
        for (int u = 0; u < R; ++u)
          if (k0 + u < all) turn(k0 + u, u, std::false_type{});
      }
    }
  }
  copies_landed<0>();
  __syncthreads();  // the ring's memory becomes that of the sums
  float *sums = reinterpret_cast<float *>(smem);
  constexpr int kPer = 32 * V * (W + 1);
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int k = 0; k < W; ++k) sums[slot * kPer + (lane * V + i) * W + k] = dw[k][i];
    sums[slot * kPer + 32 * V * W + lane * V + i] = db[i];
  }
  __syncthreads();
  const int64_t row = b * gridDim.y + blockIdx.y;
  const int64_t c0 = (int64_t)blockIdx.x * 32 * V;
  for (int j = threadIdx.x; j < kPer; j += 32 * kRuns) {
    float s = sums[j];
#pragma unroll
    for (int r = 1; r < kRuns; ++r) s += sums[r * kPer + j];
    if (j < 32 * V * W) {
      const int64_t k = c0 * W + j;
      if (k < D * W) part_w[row * D * W + k] = s;
    } else {
      const int64_t k = c0 + (j - 32 * V * W);
      if (k < D) part_b[row * D + k] = s;
    }
  }
}

template <typename T>
struct tag {
  using type = T;
};

// (I/O type, width, channels per thread): `wide` channels where every row
// starts on such a boundary, else single channels.
template <int BF16, int F32, typename F>
cudaError_t dispatch(ssd_dtype io, int W, bool vec, F f) {
  auto by_vec = [&](auto io_c, auto w_c, auto wide) {
    return vec ? f(io_c, w_c, wide) : f(io_c, w_c, std::integral_constant<int, 1>{});
  };
  auto by_w = [&](auto io_c, auto wide) {
    if (W == 2) return by_vec(io_c, std::integral_constant<int, 2>{}, wide);
    if (W == 3) return by_vec(io_c, std::integral_constant<int, 3>{}, wide);
    return by_vec(io_c, std::integral_constant<int, 4>{}, wide);
  };
  return io == SSD_BF16 ? by_w(tag<__nv_bfloat16>{}, std::integral_constant<int, BF16>{})
                        : by_w(tag<float>{}, std::integral_constant<int, F32>{});
}

bool vectored(const ConvArgs &a, ssd_dtype io, int bf16) {
  const size_t e = io == SSD_BF16 ? 2 : 4, n = io == SSD_BF16 ? bf16 : 4, bytes = n * e;
  return a.D % n == 0 && view_aligned(a.x, e, bytes) && view_aligned(a.y, e, bytes) &&
         view_aligned(a.gy, e, bytes) && view_aligned(a.dx, e, bytes) &&
         ptr_aligned(a.state, bytes) && ptr_aligned(a.gfinal, bytes) &&
         ptr_aligned(a.final_state, bytes) && ptr_aligned(a.dstate, bytes);
}

// Tokens per run of the forward: the run whose rounds of resident blocks are
// shortest in all, a run's start costing about ten tokens.  2 x 4096 x 5376: 39
// us at 32 tokens (2.2 rounds), 35 at 72 (one); longer runs spread the memory's
// accesses too far (four times as many tokens: 117 us at 72, 133 at 288).
int fwd_run(const ConvArgs &a, int64_t nv, int threads, int per_sm) {
  const int64_t room = (int64_t)sm_count() * per_sm;
  int best = 4;
  int64_t least = 0;
  for (int run = 4; run <= 72; run += 4) {
    const int64_t blocks = (nv * ((a.L + run - 1) / run) + threads - 1) / threads * a.b;
    const int64_t cost = (blocks + room - 1) / room * (run + 10);
    if (run == 4 || cost < least) best = run, least = cost;
  }
  return best;
}

// The same of the backward, kRuns runs and 32 vectors of four channels (or 32
// channels that are not whole fours) to a block: long enough for the grid's
// second dimension, and the same whatever the alignment, which the workspace's
// size does not know.  A run's start, its last tokens' neighbours and a block's
// sums cost about 16 tokens.  2 x 4096 x 2688 in bf16: 46 us at 80 tokens (one
// round), 58 at 64 (1.1).
int bwd_run(const ConvArgs &a) {
  const int wide = a.D % 4 == 0 ? 128 : 32;
  const int64_t room = (int64_t)sm_count() * (wide == 128 ? kBackBlocks : kBackBlocks1);
  const int64_t tiles = (a.D + wide - 1) / wide * a.b;
  int best = 8;
  int64_t least = 0;
  for (int run = 8; run <= 128; run += 8) {
    const int64_t blocks = tiles * ((a.L + run * kRuns - 1) / (run * kRuns));
    const int64_t cost = (blocks + room - 1) / room * (run + 16);
    if (run == 8 || cost < least) best = run, least = cost;
  }
  const int64_t longest = (a.L + 65535 * kRuns - 1) / (65535 * kRuns);
  return (int)(best > longest ? best : longest);
}
int64_t bwd_rows(const ConvArgs &a) {
  const int64_t per = (int64_t)bwd_run(a) * kRuns;
  return (a.L + per - 1) / per;
}

}  // namespace

cudaError_t launch_causal_conv(const ConvArgs &a, ssd_dtype io, int *err, cudaStream_t st) {
  const bool vec = vectored(a, io, 8);
  return dispatch<8, 4>(io, a.W, vec, [&](auto io_c, auto w_c, auto v_c) {
    using IO = typename decltype(io_c)::type;
    constexpr int W = decltype(w_c)::value, V = decltype(v_c)::value;
    const int64_t nv = a.D / V;
    const int run = fwd_run(a, nv, V > 1 ? kRingThreads : kThreads, V > 1 ? kRingBlocks : 8);
    const int64_t items = nv * ((a.L + run - 1) / run);
    auto blocks = [&](int threads) {
      return dim3((unsigned)((items + threads - 1) / threads), (unsigned)a.b);
    };
    const SeqView<const IO> x = view_of<const IO>(a.x);
    const SeqView<IO> y = view_of<IO>(a.y);
    const IO *state = static_cast<const IO *>(a.state);
    IO *fin = static_cast<IO *>(a.final_state);
    if constexpr (V > 1) {
      if (items >= (int64_t)1 << 31) return cudaErrorInvalidValue;  // an output of 1 TB
      auto go = [&](auto act) {
        conv_ring_kernel<IO, W, V, decltype(act)::value>
            <<<blocks(kRingThreads), kRingThreads, 0, st>>>(x, a.weight, a.bias, state, a.lengths,
                                                            y, fin, a.L, a.D, run, err);
        return cudaGetLastError();
      };
      return a.silu ? go(std::true_type{}) : go(std::false_type{});
    } else {
      conv_kernel<IO, W><<<blocks(kThreads), kThreads, 0, st>>>(
          x, a.weight, a.bias, state, a.lengths, y, fin, a.L, a.D, run, a.silu, err);
      return cudaGetLastError();
    }
  });
}

cudaError_t launch_causal_conv_step(const ConvArgs &a, ssd_dtype io, int *err, cudaStream_t st) {
  const bool vec = vectored(a, io, 4);
  return dispatch<4, 4>(io, a.W, vec, [&](auto io_c, auto w_c, auto v_c) {
    using IO = typename decltype(io_c)::type;
    constexpr int V = decltype(v_c)::value;
    const int64_t items = a.b * (a.D / V);
    conv_step_kernel<IO, decltype(w_c)::value, V>
        <<<(unsigned)((items + kThreads - 1) / kThreads), kThreads, 0, st>>>(
            view_of<const IO>(a.x), a.weight, a.bias, static_cast<IO *>(a.final_state),
            view_of<IO>(a.y), a.b, a.D, a.silu, err);
    return cudaGetLastError();
  });
}

size_t causal_conv_backward_workspace(const ConvArgs &a, ssd_dtype) {
  return sizeof(float) * (size_t)(a.b * bwd_rows(a) * a.D * (a.W + 1));
}

cudaError_t launch_causal_conv_backward(const ConvArgs &a, ssd_dtype io, void *ws, int *err,
                                        cudaStream_t st) {
  const bool vec = vectored(a, io, 4);
  const int64_t rows = a.b * bwd_rows(a);
  float *part_w = static_cast<float *>(ws), *part_b = part_w + rows * a.D * a.W;
  const cudaError_t e = dispatch<4, 4>(io, a.W, vec, [&](auto io_c, auto w_c, auto v_c) {
    using IO = typename decltype(io_c)::type;
    constexpr int V = decltype(v_c)::value;
    const dim3 grid((unsigned)((a.D + 32 * V - 1) / (32 * V)), (unsigned)bwd_rows(a),
                    (unsigned)a.b);
    auto go = [&](auto act) {
      conv_bwd_kernel<IO, decltype(w_c)::value, V, (V > 1), decltype(act)::value>
          <<<grid, 32 * kRuns, 0, st>>>(
              view_of<const IO>(a.x), a.weight, a.bias, static_cast<const IO *>(a.state),
              view_of<const IO>(a.gy), static_cast<const IO *>(a.gfinal), a.lengths,
              view_of<IO>(a.dx), static_cast<IO *>(a.dstate), part_w, part_b, a.L, a.D,
              bwd_run(a), err);
      return cudaGetLastError();
    };
    return a.silu ? go(std::true_type{}) : go(std::false_type{});
  });
  if (e != cudaSuccess) return e;
  ColSum s{};
  s.nseg = 2;
  s.seg[0] = {part_w, a.dweight, rows, a.D * a.W};
  s.seg[1] = {part_b, a.dbias, rows, a.D};
  return launch_colsum(s, err, st);
}

}  // namespace ssd
