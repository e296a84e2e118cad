// Shared by the operators around the blocks of a language model (add_norm.cu,
// vocab_loss.cu, orthogonalize.cu) and their entry points (model_api.cu).
#pragma once

#include "layer.cuh"
#include "ssd_model.h"

namespace ssd {

// Bytes of a workspace, handed out in order on 256-byte boundaries.
struct Carver {
  char *base;
  size_t used = 0;
  explicit Carver(void *p) : base(static_cast<char *>(p)) {}
  template <typename T>
  T *take(int64_t n) {
    T *p = reinterpret_cast<T *>(base + used);
    used += ((size_t)n * sizeof(T) + 255) / 256 * 256;
    return p;
  }
};

struct LossArgs {
  int64_t b, L, n, d, V, ignore;  // n = b L tokens
  int reduction;
  const ssd_seq *x, *weight;      // weight: V rows, token_stride apart
  const int64_t *targets;
  float *loss, *total, *lse;      // forward: [n], the sum or mean, [n]
  const float *lse_in, *gloss;    // backward; gloss [n], or one value with a reduction
  const ssd_seq *dx;
  void *dweight;
};
size_t vocab_loss_workspace(const LossArgs &a, ssd_dtype io);
cudaError_t launch_vocab_loss(const LossArgs &a, ssd_dtype io, void *ws, int *err,
                              cudaStream_t st);
size_t vocab_loss_backward_workspace(const LossArgs &a, ssd_dtype io);
cudaError_t launch_vocab_loss_backward(const LossArgs &a, ssd_dtype io, void *ws, int *err,
                                       cudaStream_t st);

struct OrthArgs {
  int64_t count, rows, cols;
  int steps;
  float a, b, c, eps;
  const ssd_seq *update, *out;  // batch_stride between matrices, token_stride between rows
};
size_t orthogonalize_workspace(const OrthArgs &a, ssd_dtype in, ssd_dtype out);
cudaError_t launch_orthogonalize(const OrthArgs &a, ssd_dtype in, ssd_dtype out, void *ws, int *err,
                                 cudaStream_t st);

struct AddNormArgs {
  int64_t b, L, D, block;  // block: channels to a scale (quantised)
  float eps;
  const ssd_seq *x, *residual, *y, *total, *gy, *gtotal, *dx, *dresidual;
  const float *weight;
  float *scales, *dweight;
};
// y in the I/O type, or where `scales` is given in e4m3 (block 0: a scale a token)
cudaError_t launch_add_norm(const AddNormArgs &a, ssd_dtype io, ssd_dtype stream, int *err,
                            cudaStream_t st);
size_t add_norm_backward_workspace(const AddNormArgs &a, ssd_dtype io, ssd_dtype stream);
cudaError_t launch_add_norm_backward(const AddNormArgs &a, ssd_dtype io, ssd_dtype stream, void *ws,
                                     int *err, cudaStream_t st);

}  // namespace ssd
