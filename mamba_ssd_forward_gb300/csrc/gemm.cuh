// Matrix products on the fifth-generation tensor cores with an epilogue of the
// caller's, for the operators whose work is products (vocab_loss.cu,
// orthogonalize.cu):
//   D[m][n] = sum_k A[m][k] B[n][k],  16-bit operands, fp32 sums.
//
// Operands lie K-major (k contiguous) or MN-major (m or n contiguous), as they
// come, and both ways land by TMA in 128-byte-swizzled rows, so nothing is
// transposed.  An operand may come in two planes, x = hi + lo, each 11 bits of
// an fp32 value (fp16 after a scaling by a power of two): then the products
// lo hi, hi lo, hi hi are summed one after the other, which drops lo lo alone,
// 2^-24 relative.
//
// Why this shape: a 256 x kBN tile belongs to a pair of blocks (a cluster) whose
// tensor cores work as one (cta_group::2): each block keeps 128 rows of A, half
// of the columns' rows of B and 128 rows of sums.  Per 64 k a block loads
// 32 KB for 128 x 256 x 64 multiply-adds, two thirds of what a block alone with
// a tile of 128 x 256 loads: 64 instead of 96 bytes a clock at the full rate,
// where the L2 hands out about 70 to each SM.  Persistent blocks walk the tiles; two
// accumulators in tensor memory let the epilogue of a tile run under the products
// of the next one.
//
// The tensor cores cut what each 16 k add to a sum towards zero at 24 bits, about
// 2^-25 of the sum each time, all to the same side.  Products whose result is to
// have fp32's precision are therefore taken in segments of kSegment stages, which
// the epilogue's threads add up in registers (rounded to nearest): 64 x 4
// k a segment measured 4e-6 -> 3e-7 off for sums of 3200 terms.
//
// Warps: 0 loads (TMA), 1 issues the products (the pair's first block only), the
// others run the epilogue, eight or sixteen of them: warp w reads lanes 32 (w mod 4)
// .. + 31 (a thread is a row), each four of them their share of the tile's columns.
// Every wait is bounded.
#pragma once

#include <cuda_fp16.h>

#include <atomic>

#include "layer.cuh"
#include "ptx.cuh"
#include "ssd_internal.cuh"
#include "tmap.cuh"

namespace ssd {
namespace gemm {

constexpr int kTileM = 256, kRows = 128, kTileK = 64;  // of a pair; of a block; per stage
constexpr int kChunk = 32;  // columns an epilogue thread holds at a time
constexpr int kExact = 4;   // stages to a segment where fp32's precision is asked for
constexpr int kBytesA = kRows * 128;

constexpr int kPaneBytes = 65536;  // of all epilogue warps
constexpr int kPaneBars = 2;       // of a warp

// kStaged: the epilogue's warps have panes.
template <int kBN, bool kStaged>
struct Shape {
  static constexpr int kBytesB = kBN / 2 * 128;
  static constexpr int kStage = kBytesA + kBytesB;
  static constexpr int kPanes = kStaged ? kPaneBytes : 0;
  static constexpr int kStages = (229376 - kPanes) / kStage;
  static constexpr int kSmem = kStages * kStage + kPanes + 1024;
  static constexpr uint32_t kTmemCols = 2 * kBN;
};

// One product.  M or K is read on the device where live_m, live_k say so.
struct Product {
  int M, N, K, batch;
  const int *live_m, *live_k;
  int a_mn, b_mn;          // MN-major operands
  int pairs;               // 1, or 3 with operands of two planes
  int a_planes, b_planes;  // planes that each operand's array holds
  int symmetric;           // D is: only tiles on and above the diagonal
  int part, parts;         // part > 0: every `parts` batches are one, each sums `part` stages of k
};

// What a block does of a tile: rows m .. m + 127, columns n .. n + kBN - 1.
struct Tile {
  int which, batch, m, n;
  int k0, steps;  // first stage of k, and stages, of one pair of planes
  int mirror;                     // D is symmetric and this tile lies above the diagonal
};

template <int kBN>
struct Walk {  // the tiles of up to two products, in order; in shared memory
  Product p[2];
  int M[2], K[2], tm[2], tn[2], per[2];
  int total, first;  // tiles; those of product 0

  __device__ __forceinline__ void plan(const Product &a, const Product &b, int count) {
    p[0] = a, p[1] = b;
    total = first = 0;
    for (int i = 0; i < count; ++i) {
      M[i] = p[i].live_m ? min(*p[i].live_m, p[i].M) : p[i].M;
      K[i] = p[i].live_k ? min(*p[i].live_k, p[i].K) : p[i].K;
      tm[i] = (M[i] + kTileM - 1) / kTileM;
      tn[i] = (p[i].N + kBN - 1) / kBN;
      constexpr int r = kTileM / kBN;  // column tiles to a row tile
      per[i] = p[i].symmetric ? tm[i] * tn[i] - r * (tm[i] * (tm[i] - 1) / 2) : tm[i] * tn[i];
      total += per[i] * p[i].batch;
      if (i == 0) first = total;
    }
  }

  __device__ __forceinline__ Tile at(int t, int rank) const {
    Tile o;
    const int i = t >= first;
    if (i) t -= first;
    o.which = i;
    o.batch = t / per[i];
    t -= o.batch * per[i];
    int mi, ni;
    if (p[i].symmetric) {
      constexpr int r = kTileM / kBN;
      mi = 0;
      for (int left = tn[i]; t >= left; left -= r) t -= left, ++mi;
      ni = mi * r + t;
    } else {
      // bands of eight row tiles, column by column: the blocks at work share
      // few rows of both operands in L2
      const int band = t / (8 * tn[i]), high = min(8, tm[i] - 8 * band);
      t -= band * 8 * tn[i];
      ni = t / high;
      mi = 8 * band + t % high;
    }
    o.m = mi * kTileM + rank * kRows;
    o.n = ni * kBN;
    o.k0 = p[i].part ? o.batch % p[i].parts * p[i].part : 0;
    o.steps = (K[i] + kTileK - 1) / kTileK - o.k0;
    if (p[i].part) o.steps = max(0, min(o.steps, p[i].part));
    o.mirror = p[i].symmetric && o.n >= (mi + 1) * kTileM;
    return o;
  }
};

// ------------------------------------------------- instructions of the pair

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n barrier.cluster.wait.aligned;" ::: "memory");
}
// The address of a barrier in the pair's first block.
__device__ __forceinline__ uint32_t in_first(const uint64_t *bar) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(ptx::smem_u32(bar)));
  return a;
}
__device__ __forceinline__ void arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// A load into this block's memory that signals a barrier of the pair.
__device__ __forceinline__ void load(void *dst, const CUtensorMap *map, int c0, int c1, int c2,
                                     uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(ptx::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                    uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives at the barrier at this address in both blocks when the products
// issued so far are done.
__device__ __forceinline__ void commit_both(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(ptx::smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void tmem_alloc(uint32_t *dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   ptx::smem_u32(dst)),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols)
               : "memory");
}

// A value that is the same in all lanes, said so.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// Instruction descriptor of 256 x n products with fp32 sums: fp16 (0) or bf16
// (1) operands.
__device__ __forceinline__ uint32_t idesc(int n, int bf16, int a_mn, int b_mn) {
  return (1u << 4) | ((uint32_t)bf16 << 7) | ((uint32_t)bf16 << 10) | ((uint32_t)a_mn << 15) |
         ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kTileM >> 4) << 24);
}
// Descriptor of a landed operand at address 0 (the address is added in units of
// 16 bytes; shared memory has 2^14 of them at most).  K-major: rows of 128
// bytes, 8-row groups 1024 bytes apart, 16 k are 32 bytes along the row.
// MN-major: blocks of 64 (m or n) x 64 k, 8192 bytes apart, 16 k are 16 rows.
__device__ __forceinline__ uint64_t desc(int mn) {
  return ptx::smem_desc(0, mn ? 8192 : 16, 1024, ptx::kSw128);
}

// Loads kCount rows (m or n, from r0) x 64 k (from k0) of an operand.
template <int kCount>
__device__ __forceinline__ void load_operand(uint8_t *dst, const CUtensorMap *map, int mn, int r0,
                                             int k0, int z, uint32_t bar) {
  if (!mn) {
    load(dst, map, k0, r0, z, bar);
  } else {
#pragma unroll
    for (int j = 0; j < kCount / 64; ++j) load(dst + 8192 * j, map, r0 + 64 * j, k0, z, bar);
  }
}

// One lane of a converged warp, the same each time.  (With it rather than a
// comparison of the lane the compiler keeps what the instructions below take in
// uniform registers.)
__device__ __forceinline__ bool elected() {
  uint32_t e;
  asm volatile(
      "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(e));
  return e != 0;
}
// A warp's panes in shared memory.  A thread holds a row of the tile; through a
// pane, 32 rows, values go to memory and come from it by TMA, which clips what
// lies outside the array.  (Row by row from registers every access would touch 32
// lines: measured 16000 clocks a tile against 6000 of products.)  Rows of 128 or 64
// bytes, swizzled; a warp has 8 KB of panes, or 4 KB where there are sixteen warps.
template <int kRowBytes>
struct Panes {
  static constexpr int kBytes = 32 * kRowBytes;
  uint8_t *at;
  uint64_t *bars;  // kPaneBars
  int *err;
  int lane;
  uint32_t phases;  // a bit for each barrier
  __device__ __forceinline__ Panes(uint8_t *p, uint64_t *b, int *e)
      : at(p), bars(b), err(e), lane(threadIdx.x & 31), phases(0) {}
  // byte offset of 16-byte piece `piece` of row r
  __device__ __forceinline__ static int swizzled(int r, int piece) {
    return r * kRowBytes + ((kRowBytes == 128 ? piece ^ (r & 7) : piece ^ ((r >> 1) & 3)) << 4);
  }
  // 16 bytes of this thread's row
  __device__ __forceinline__ uint4 &cell(int pane, int piece) const {
    return *reinterpret_cast<uint4 *>(at + pane * kBytes + swizzled(lane, piece));
  }
  // 4 bytes of row r
  __device__ __forceinline__ uint32_t word(int pane, int r, int w) const {
    return *reinterpret_cast<const uint32_t *>(at + pane * kBytes + swizzled(r, w >> 2) +
                                               (w & 3) * 4);
  }
  // All but the newest kLeft groups of stores have read their panes.
  template <int kLeft>
  __device__ __forceinline__ void reuse() const {
    if (elected()) ptx::bulk_wait_read<kLeft>();
    __syncwarp();
  }
  // The warp has written (or read) its panes: the elected lane may store (or load) them.
  __device__ __forceinline__ void written() const {
    ptx::fence_async_smem();
    __syncwarp();
  }
  __device__ __forceinline__ void store(int pane, const CUtensorMap *map, int col, int row,
                                        int z) const {  // the elected lane, then commit
    ptx::tma_store_3d(map, at + pane * kBytes, col, row, z);
  }
  __device__ __forceinline__ void add(int pane, const CUtensorMap *map, int col, int row,
                                      int z) const {  // fp32
    asm volatile(
        "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group"
        " [%0, {%2, %3, %4}], [%1];" ::"l"(reinterpret_cast<uint64_t>(map)),
        "r"(ptx::smem_u32(at + pane * kBytes)), "r"(col), "r"(row), "r"(z)
        : "memory");
  }
  // Loads n panes from `pane` on (z, z + 1, ..); the stores from them have to be
  // read.  fetched: they are there.
  __device__ __forceinline__ void fetch(int bar, int pane, int n, const CUtensorMap *map, int col,
                                        int row, int z) const {
    if (elected()) {
      ptx::mbar_arrive_expect_tx(&bars[bar], n * kBytes);
      for (int i = 0; i < n; ++i)
        ptx::tma_load_3d(at + (pane + i) * kBytes, map, col, row, z + i, &bars[bar]);
    }
  }
  __device__ __forceinline__ void fetched(int bar) {
    ptx::mbar_wait(&bars[bar], (phases >> bar) & 1, err, 304);
    phases ^= 1u << bar;
  }
};

// kSegment: stages to a segment, 0: all k in one.
// Epi: constructed from its Args and panes by every epilogue thread, then per tile
// begin(tile, row, column, rows), chunk(v, column, j) for each 32 columns of the
// thread's row, end().  kWarps: epilogue warps; kStaged: they use panes, of type Pane.
template <class Epi, int kBN, int kSegment>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(32 * (2 + Epi::kWarps), 1)
product_kernel(const __grid_constant__ CUtensorMap a0, const __grid_constant__ CUtensorMap b0,
               const __grid_constant__ CUtensorMap a1, const __grid_constant__ CUtensorMap b1,
               const __grid_constant__ Product p0, const __grid_constant__ Product p1,
               const int count, const int bf16, const __grid_constant__ typename Epi::Args args,
               int *err) {
  using S = Shape<kBN, Epi::kStaged>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  // full: a stage landed in both blocks (the first block's is waited on);
  // empty: its products are done; accfull: a tile's are; accfree: both blocks'
  // epilogues have read them (the first block's)
  __shared__ __align__(8) uint64_t full[S::kStages], empty[S::kStages], accfull[2], accfree[2];
  __shared__ __align__(8) uint64_t landed[Epi::kWarps][kPaneBars];  // panes of each epilogue warp
  __shared__ uint32_t tmem_slot;
  __shared__ Walk<kBN> walk;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();

  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      ptx::mbar_init(&full[i], 1);
      ptx::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&accfull[i], 1);
      ptx::mbar_init(&accfree[i], 2 * Epi::kWarps);
    }
    for (int i = 0; i < Epi::kWarps * kPaneBars; ++i) ptx::mbar_init(&landed[0][i], 1);
    ptx::fence_mbar_init();
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();  // (the numbers of rows are an earlier launch's)
    walk.plan(p0, p1, count);
  }
  if (warp == 2 && elected()) {  // (parameters: no earlier launch's)
    ptx::prefetch_tmap(&a0);
    ptx::prefetch_tmap(&b0);
    if (count > 1) {
      ptx::prefetch_tmap(&a1);
      ptx::prefetch_tmap(&b1);
    }
  }
  if (warp == 1) tmem_alloc(&tmem_slot, S::kTmemCols);
  ptx::tc_fence_before();
  __syncthreads();
  cluster_sync();
  ptx::tc_fence_after();
  ptx::griddep_wait();
  const uint32_t tmem = tmem_slot;
  const int step = gridDim.x / 2, start = blockIdx.x / 2;

  // The loops of warps 0 and 1 are latency bound (a stage is 512 clocks of
  // products): what does not change within a tile is in registers, and one lane
  // is elected where an instruction is a single thread's.
  if (warp == 0) {
    int s = 0, round = 0;
    const uint32_t bars = in_first(full);
    for (int t = start; t < walk.total; t += step) {
      const Tile o = walk.at(t, rank);
      const int which = uniform(o.which), k0 = uniform(o.k0), k1 = k0 + uniform(o.steps);
      const Product &p = which ? p1 : p0;
      const CUtensorMap *ma = which ? &a1 : &a0, *mb = which ? &b1 : &b0;
      const int a_mn = p.a_mn, b_mn = p.b_mn, pairs = p.pairs;
      const int m = uniform(o.m), n = uniform(o.n) + rank * (kBN / 2);
      const int z = uniform(p.part ? o.batch / p.parts : o.batch), za = z * p.a_planes, zb = z * p.b_planes;
      for (int pair = 0; pair < pairs; ++pair) {
        // with three: lo hi, hi lo, hi hi
        const int z0 = za + (pairs == 3 && pair == 0), z1 = zb + (pairs == 3 && pair == 1);
        for (int k = k0; k < k1; ++k) {
          if (round) ptx::mbar_wait(&empty[s], (round - 1) & 1, err, 300);
          if (elected()) {
            if (rank == 0) ptx::mbar_arrive_expect_tx(&full[s], 2 * S::kStage);
            uint8_t *at = smem + s * S::kStage;
            load_operand<kRows>(at, ma, a_mn, m, k * kTileK, z0, bars + 8 * s);
            load_operand<kBN / 2>(at + kBytesA, mb, b_mn, n, k * kTileK, z1, bars + 8 * s);
          }
          __syncwarp();
          if (++s == S::kStages) s = 0, ++round;
        }
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      int s = 0, parity = 0, n = 0;
      const uint32_t ring = ptx::smem_u32(smem) >> 4;
      for (int t = start; t < walk.total; t += step) {
        const Tile o = walk.at(t, rank);
        const Product &p = uniform(o.which) ? p1 : p0;
        const uint32_t id = idesc(kBN, bf16, p.a_mn, p.b_mn);
        const uint64_t da = desc(p.a_mn), db = desc(p.b_mn);
        const uint32_t ia = p.a_mn ? 128 : 2, ib = p.b_mn ? 128 : 2;  // to the next 16 k, by 16 bytes
        const int steps = uniform(o.steps) * p.pairs, each = kSegment ? kSegment : steps;
        int k = 0;
        do {  // a segment (an empty one where there are no k)
          const uint32_t d = tmem + (n & 1) * kBN;
          if (n >= 2) ptx::mbar_wait(&accfree[n & 1], ((n >> 1) - 1) & 1, err, 301);
          ptx::tc_fence_after();
          const int end = min(k + each, steps), begin = k;
          for (; k < end; ++k) {
            ptx::mbar_wait(&full[s], parity, err, 302);
            ptx::tc_fence_after();
            const uint32_t at = ring + s * (S::kStage / 16), bt = at + kBytesA / 16;
            if (elected()) {
#pragma unroll
              for (int kk = 0; kk < kTileK / 16; ++kk)
                mma(d, da + at + kk * ia, db + bt + kk * ib, id, k > begin || kk > 0);
              commit_both(&empty[s]);
            }
            __syncwarp();
            if (++s == S::kStages) s = 0, parity ^= 1;
          }
          if (elected()) commit_both(&accfull[n & 1]);
          __syncwarp();
          ++n;
        } while (k < steps);
      }
    }
  } else {
    constexpr int kShare = kBN / (Epi::kWarps / 4), kChunks = kShare / kChunk;
    static_assert(kChunks * kChunk == kShare, "");
    const int quad = warp & 3, c0 = (warp - 2) / 4 * kShare;
    uint8_t *panes = smem + S::kStages * S::kStage + (warp - 2) * (kPaneBytes / Epi::kWarps);
    Epi epi(args, typename Epi::Pane(panes, landed[warp - 2], err), err);
    int n = 0;
    // 32 columns of the accumulator at `at`; the last ones hand it back
    auto read = [&](uint32_t at, int j, uint32_t (&r0)[16], uint32_t (&r1)[16]) {
      ptx::tmem_ld16(at + j * kChunk, r0);
      ptx::tmem_ld16(at + j * kChunk + 16, r1);
      ptx::tmem_ld_wait();
      ptx::reg_fence(r0);
      ptx::reg_fence(r1);
      if (j == kChunks - 1) {
        ptx::tc_fence_before();
        __syncwarp();
        if (elected()) arrive_at(in_first(&accfree[n & 1]));
      }
    };
    for (int t = start; t < walk.total; t += step) {
      const Tile o = walk.at(t, rank);
      const Product &p = walk.p[o.which];
      epi.begin(o, o.m + quad * 32 + lane, o.n + c0, walk.M[o.which]);
      const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16) + c0;
      if constexpr (kSegment == 0) {
        ptx::mbar_wait(&accfull[n & 1], (n >> 1) & 1, err, 303);
        ptx::tc_fence_after();
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
          uint32_t r0[16], r1[16];
          read(lanes + (n & 1) * kBN, j, r0, r1);
          float v[kChunk];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            v[i] = o.steps ? __uint_as_float(r0[i]) : 0.f;
            v[16 + i] = o.steps ? __uint_as_float(r1[i]) : 0.f;
          }
          epi.chunk(v, o.n + c0 + j * kChunk, j);
        }
        ++n;
      } else {
        float v[kChunks][kChunk];
#pragma unroll
        for (int j = 0; j < kChunks; ++j)
#pragma unroll
          for (int i = 0; i < kChunk; ++i) v[j][i] = 0.f;
        const int steps = o.steps * p.pairs;
        int k = 0;
        do {
          ptx::mbar_wait(&accfull[n & 1], (n >> 1) & 1, err, 303);
          ptx::tc_fence_after();
#pragma unroll
          for (int j = 0; j < kChunks; ++j) {
            uint32_t r0[16], r1[16];
            read(lanes + (n & 1) * kBN, j, r0, r1);
            if (steps) {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                v[j][i] += __uint_as_float(r0[i]);
                v[j][16 + i] += __uint_as_float(r1[i]);
              }
            }
          }
          ++n;
          k += kSegment;
        } while (k < steps);
#pragma unroll
        for (int j = 0; j < kChunks; ++j) epi.chunk(v[j], o.n + c0 + j * kChunk, j);
      }
      epi.end();
    }
    if constexpr (Epi::kStaged) {
      if (elected()) ptx::bulk_wait<0>();  // the panes are read and their values written
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  cluster_sync();  // the pair's barriers and tensor memory are in use until here
  if (warp == 1) tmem_dealloc(tmem, S::kTmemCols);
}

// ----------------------------------------------------------------- the host

// Map of an operand array [z][rows][cols] of 16-bit elements, `ld` elements to a
// row and `zs` to a z; `box`: rows (m or n) that a block loads of it.
inline bool make_map(CUtensorMap *map, const void *base, int64_t cols, int64_t rows, int64_t z,
                     int64_t ld, int64_t zs, bool mn, int box) {
  const uint64_t dims[3] = {(uint64_t)cols, (uint64_t)rows, (uint64_t)z};
  const uint64_t strides[2] = {(uint64_t)ld * 2, (uint64_t)(z > 1 ? zs : ld) * 2};
  const uint32_t b[3] = {64, (uint32_t)(mn ? 64 : box), 1};
  return make_tmap_sw128(map, base, true, 3, dims, strides, b);
}

// Map of an array [z][rows][cols] for panes.
template <int kRowBytes>
bool make_pane_map(CUtensorMap *map, const void *base, bool fp32, int64_t cols, int64_t rows,
                   int64_t z, int64_t ld, int64_t zs) {
  const uint64_t e = fp32 ? 4 : 2;
  const uint64_t dims[3] = {(uint64_t)cols, (uint64_t)rows, (uint64_t)z};
  const uint64_t strides[2] = {(uint64_t)ld * e, (uint64_t)(z > 1 ? zs : ld) * e};
  const uint32_t b[3] = {(uint32_t)(kRowBytes / e), 32, 1};
  return (kRowBytes == 128 ? make_tmap_sw128 : make_tmap_sw64)(map, base, !fp32, 3, dims, strides,
                                                               b);
}

// Elements to a row of an operand array: rows start on 32 bytes.
inline int64_t padded(int64_t cols) { return (cols + 15) / 16 * 16; }

// Launches `count` products (one or two) as one grid.
template <class Epi, int kBN, int kSegment = 0>
cudaError_t launch(const CUtensorMap *maps, const Product *p, int count, bool bf16,
                   const typename Epi::Args &args, int *err, cudaStream_t st) {
  using S = Shape<kBN, Epi::kStaged>;
  auto *kernel = product_kernel<Epi, kBN, kSegment>;
  // set once a device (64 of them): every caller stores the same value
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  int64_t tiles = 0;
  for (int i = 0; i < count; ++i)
    tiles += (int64_t)p[i].batch * ((p[i].M + kTileM - 1) / kTileM) * ((p[i].N + kBN - 1) / kBN);
  const int pairs = sm_count() / 2;
  const unsigned grid = 2 * (unsigned)(tiles < pairs ? tiles : pairs);
  if (!grid) return cudaSuccess;
  const int last = count - 1;
  return launch_after(kernel, dim3(grid), 32 * (2 + Epi::kWarps), S::kSmem, st, maps[0], maps[1],
                      maps[2 * last], maps[2 * last + 1], p[0], p[last], count, (int)bf16, args,
                      err);
}

}  // namespace gemm
}  // namespace ssd
