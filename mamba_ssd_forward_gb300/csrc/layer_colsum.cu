// Column sums of partial arrays (the parameter gradients' last step): one
// block per 32 columns, 16 row slices whose partial sums are added in slice
// order.  The order depends on the sizes only, so results repeat bit for bit.
// Bandwidth-bound on arrays that are small next to what produced them.
#include "layer.cuh"

namespace ssd {
namespace {

constexpr int kCols = 32, kSlices = 16;

__global__ void __launch_bounds__(kCols *kSlices) colsum_kernel(ColSum a, int *err) {
  __shared__ float part[kSlices][kCols];
  int64_t blk = blockIdx.x;
  int s = 0;
  for (; s < a.nseg - 1; ++s) {
    const int64_t nb = (a.seg[s].n + kCols - 1) / kCols;
    if (blk < nb) break;
    blk -= nb;
  }
  const ColSum::Seg g = a.seg[s];
  const int col = threadIdx.x % kCols, slice = threadIdx.x / kCols;
  const int64_t i = blk * kCols + col;
  float acc = 0.f;
  if (i < g.n && SSD_IN_BOUNDS(g.rows >= 0, err, 60)) {
    const float *p = g.src + i;
#pragma unroll 8
    for (int64_t r = slice; r < g.rows; r += kSlices) acc += p[r * g.n];
  }
  part[slice][col] = acc;
  __syncthreads();
  if (slice == 0 && i < g.n) {
    acc = part[0][col];
#pragma unroll
    for (int k = 1; k < kSlices; ++k) acc += part[k][col];
    g.dst[i] = acc;
  }
}

}  // namespace

cudaError_t launch_colsum(const ColSum &in, int *err, cudaStream_t st) {
  ColSum a{};
  int64_t blocks = 0;
  for (int s = 0; s < in.nseg; ++s)
    if (in.seg[s].dst && in.seg[s].n > 0) {
      a.seg[a.nseg++] = in.seg[s];
      blocks += (in.seg[s].n + kCols - 1) / kCols;
    }
  if (!blocks) return cudaSuccess;
  colsum_kernel<<<(unsigned)blocks, kCols * kSlices, 0, st>>>(a, err);
  return cudaGetLastError();
}

}  // namespace ssd
