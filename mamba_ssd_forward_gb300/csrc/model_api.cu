// C ABI of the operators around the blocks of a language model (ssd_model.h):
// argument checks and the launches, nothing else.
#include "args.cuh"
#include "model.cuh"

namespace {

using namespace ssd::args;

constexpr int64_t kMaxSide = 1 << 20;     // rows and columns of a matrix
constexpr int64_t kMaxTiles = 1ll << 30;  // tiles of a product are counted in 31 bits

int64_t tiles(int64_t n) { return (n + 127) / 128; }

ssd_status loss_args(const ssd_loss_dims *d, ssd_dtype t, const ssd_seq *weight,
                     ssd::LossArgs *a) {
  if (!d || !valid_dtype(t) || d->vocab < 1 || d->reduction < SSD_REDUCE_NONE ||
      d->reduction > SSD_REDUCE_MEAN)
    return SSD_ERR_INVALID_ARG;
  const ssd_status s = common_dims(d->batch, d->seqlen, d->channels, kMaxTokens);
  if (s != SSD_OK) return s;
  if (d->channels > 65536 || d->vocab > (1 << 24) ||
      (double)d->batch * d->seqlen > (double)(1 << 30) ||
      (double)tiles(d->batch * d->seqlen) * tiles(d->vocab) > (double)kMaxTiles)
    return SSD_ERR_UNSUPPORTED;
  if (!has(weight) || !natural(weight->data, elem(t)) || weight->token_stride < 0 ||
      (double)weight->token_stride * d->vocab > kBig / 8)
    return SSD_ERR_INVALID_ARG;
  *a = ssd::LossArgs{};
  a->b = d->batch, a->L = d->seqlen, a->n = a->b * a->L, a->d = d->channels, a->V = d->vocab;
  a->ignore = d->ignore_index, a->reduction = d->reduction, a->weight = weight;
  return SSD_OK;
}

ssd_status orth_args(const ssd_orth_dims *d, ssd_dtype in, ssd_dtype out, ssd::OrthArgs *a) {
  if (!d || !valid_dtype(in) || !valid_dtype(out) || d->count < 1 || d->rows < 1 || d->cols < 1 ||
      d->steps < 1 || d->steps > 100 || !std::isfinite(d->a) || !std::isfinite(d->b) ||
      !std::isfinite(d->c) || !(d->eps > 0.f) || !std::isfinite(d->eps))
    return SSD_ERR_INVALID_ARG;
  if (d->count > 32767 || d->rows > kMaxSide || d->cols > kMaxSide ||
      (double)d->count * tiles(d->rows) * tiles(d->cols) > (double)kMaxTiles ||
      (double)d->count * tiles(d->rows < d->cols ? d->rows : d->cols) *
              tiles(d->rows < d->cols ? d->rows : d->cols) > (double)kMaxTiles)
    return SSD_ERR_UNSUPPORTED;
  *a = ssd::OrthArgs{};
  a->count = d->count, a->rows = d->rows, a->cols = d->cols, a->steps = d->steps;
  a->a = d->a, a->b = d->b, a->c = d->c, a->eps = d->eps;
  return SSD_OK;
}

ssd_status add_norm_args(const ssd_add_norm_dims *d, ssd_dtype t, ssd_dtype stream,
                         ssd::AddNormArgs *a) {
  if (!d || !valid_dtype(t) || (stream != t && stream != SSD_F32) || !(d->eps > 0.f) ||
      !std::isfinite(d->eps))
    return SSD_ERR_INVALID_ARG;
  const ssd_status s = common_dims(d->batch, d->seqlen, d->channels, kMaxTokens);
  if (s != SSD_OK) return s;
  if (d->channels > 16384 || (double)d->batch * d->seqlen > (double)kMaxTokens)
    return SSD_ERR_UNSUPPORTED;
  *a = ssd::AddNormArgs{};
  a->b = d->batch, a->L = d->seqlen, a->D = d->channels, a->eps = d->eps;
  return SSD_OK;
}

// What both forms of the forward pass take.
bool add_norm_inputs(ssd::AddNormArgs *a, ssd_dtype t, ssd_dtype stream, const ssd_seq *x,
                     const ssd_seq *residual, const float *weight, const ssd_seq *total) {
  if (!req_view(x, t, a->b, a->L) || !opt_view(residual, stream, a->b, a->L) || !req(weight) ||
      !opt_out(total, stream, a->b, a->L, a->D))
    return false;
  a->x = x, a->residual = or_null(residual), a->weight = weight, a->total = or_null(total);
  return true;
}

}  // namespace

extern "C" {

ssd_status ssd_add_norm(const ssd_add_norm_dims *dims, ssd_dtype dtype, ssd_dtype stream_dtype,
                        const ssd_seq *x, const ssd_seq *residual, const float *weight,
                        const ssd_seq *y, const ssd_seq *total, void *stream) {
  ssd::AddNormArgs a;
  const ssd_status s = add_norm_args(dims, dtype, stream_dtype, &a);
  if (s != SSD_OK) return s;
  if (!add_norm_inputs(&a, dtype, stream_dtype, x, residual, weight, total) ||
      !req_out(y, dtype, a.b, a.L, a.D))
    return SSD_ERR_INVALID_ARG;
  a.y = y;
  int *err = ssd::device_error_word();
  if (!err) return SSD_ERR_CUDA;
  return from_cuda(ssd::launch_add_norm(a, dtype, stream_dtype, err, (cudaStream_t)stream));
}

ssd_status ssd_add_norm_quantized(const ssd_add_norm_dims *dims, ssd_dtype dtype,
                                  ssd_dtype stream_dtype, int64_t block, const ssd_seq *x,
                                  const ssd_seq *residual, const float *weight, const ssd_seq *q,
                                  float *scales, const ssd_seq *total, void *stream) {
  ssd::AddNormArgs a;
  const ssd_status s = add_norm_args(dims, dtype, stream_dtype, &a);
  if (s != SSD_OK) return s;
  if ((block != 0 && block != 32 && block != 64 && block != 128) ||
      !add_norm_inputs(&a, dtype, stream_dtype, x, residual, weight, total) || !has(q) ||
      q->batch_stride < 0 || q->token_stride < 0 ||
      (double)q->batch_stride * a.b + (double)q->token_stride * a.L > kBig / 8 ||
      !apart(q, a.b, a.L, a.D) || !req(scales))
    return SSD_ERR_INVALID_ARG;
  a.y = q, a.scales = scales, a.block = block;
  int *err = ssd::device_error_word();
  if (!err) return SSD_ERR_CUDA;
  return from_cuda(ssd::launch_add_norm(a, dtype, stream_dtype, err, (cudaStream_t)stream));
}

size_t ssd_add_norm_backward_workspace_size(const ssd_add_norm_dims *dims, ssd_dtype dtype,
                                            ssd_dtype stream_dtype) {
  ssd::AddNormArgs a;
  return add_norm_args(dims, dtype, stream_dtype, &a) == SSD_OK
             ? ssd::add_norm_backward_workspace(a, dtype, stream_dtype)
             : 0;
}

ssd_status ssd_add_norm_backward(const ssd_add_norm_dims *dims, ssd_dtype dtype,
                                 ssd_dtype stream_dtype, const ssd_seq *total,
                                 const float *weight, const ssd_seq *gy, const ssd_seq *gtotal,
                                 const ssd_seq *dx, const ssd_seq *dresidual, float *dweight,
                                 void *workspace, size_t ws_bytes, void *stream) {
  ssd::AddNormArgs a;
  const ssd_status s = add_norm_args(dims, dtype, stream_dtype, &a);
  if (s != SSD_OK) return s;
  if (!req_view(total, stream_dtype, a.b, a.L) || !req(weight) ||
      !req_view(gy, dtype, a.b, a.L) || !opt_view(gtotal, stream_dtype, a.b, a.L) ||
      !opt_out(dx, dtype, a.b, a.L, a.D) || !opt_out(dresidual, stream_dtype, a.b, a.L, a.D) ||
      !opt(dweight) ||
      (dweight && !good_ws(workspace, ws_bytes,
                           ssd::add_norm_backward_workspace(a, dtype, stream_dtype))))
    return SSD_ERR_INVALID_ARG;
  a.total = total, a.weight = weight, a.gy = gy, a.gtotal = or_null(gtotal), a.dx = or_null(dx);
  a.dresidual = or_null(dresidual), a.dweight = dweight;
  if (!a.dx && !a.dresidual && !dweight) return SSD_OK;
  int *err = ssd::device_error_word();
  if (!err) return SSD_ERR_CUDA;
  return from_cuda(
      ssd::launch_add_norm_backward(a, dtype, stream_dtype, workspace, err, (cudaStream_t)stream));
}

size_t ssd_linear_cross_entropy_workspace_size(const ssd_loss_dims *dims, ssd_dtype dtype,
                                               const ssd_seq *weight) {
  ssd::LossArgs a;
  return loss_args(dims, dtype, weight, &a) == SSD_OK ? ssd::vocab_loss_workspace(a, dtype) : 0;
}

ssd_status ssd_linear_cross_entropy(const ssd_loss_dims *dims, ssd_dtype dtype, const ssd_seq *x,
                                    const ssd_seq *weight, const int64_t *targets, float *loss,
                                    float *total, float *lse, void *workspace, size_t ws_bytes,
                                    void *stream) {
  ssd::LossArgs a;
  const ssd_status s = loss_args(dims, dtype, weight, &a);
  if (s != SSD_OK) return s;
  const bool reduced = a.reduction != SSD_REDUCE_NONE;
  if (!req_view(x, dtype, a.b, a.L) || !req(targets, 8) || !req(lse) || !opt(loss) ||
      !opt(total) || reduced != (total != nullptr) || (!reduced && !loss) ||
      !good_ws(workspace, ws_bytes, ssd::vocab_loss_workspace(a, dtype)))
    return SSD_ERR_INVALID_ARG;
  a.x = x, a.targets = targets, a.loss = loss, a.total = total, a.lse = lse;
  int *err = ssd::device_error_word();
  if (!err) return SSD_ERR_CUDA;
  return from_cuda(ssd::launch_vocab_loss(a, dtype, workspace, err, (cudaStream_t)stream));
}

size_t ssd_linear_cross_entropy_backward_workspace_size(const ssd_loss_dims *dims,
                                                        ssd_dtype dtype, const ssd_seq *weight) {
  ssd::LossArgs a;
  return loss_args(dims, dtype, weight, &a) == SSD_OK
             ? ssd::vocab_loss_backward_workspace(a, dtype)
             : 0;
}

ssd_status ssd_linear_cross_entropy_backward(const ssd_loss_dims *dims, ssd_dtype dtype,
                                             const ssd_seq *x, const ssd_seq *weight,
                                             const int64_t *targets, const float *lse,
                                             const float *gloss, const ssd_seq *dx, void *dweight,
                                             void *workspace, size_t ws_bytes, void *stream) {
  ssd::LossArgs a;
  const ssd_status s = loss_args(dims, dtype, weight, &a);
  if (s != SSD_OK) return s;
  if (!req_view(x, dtype, a.b, a.L) || !req(targets, 8) || !req(lse) || !opt(gloss) ||
      !opt_out(dx, dtype, a.b, a.L, a.d) || !opt(dweight, elem(dtype)) ||
      !good_ws(workspace, ws_bytes, ssd::vocab_loss_backward_workspace(a, dtype)))
    return SSD_ERR_INVALID_ARG;
  a.x = x, a.targets = targets, a.lse_in = lse, a.gloss = gloss, a.dx = or_null(dx);
  a.dweight = dweight;
  if (!a.dx && !a.dweight) return SSD_OK;
  int *err = ssd::device_error_word();
  if (!err) return SSD_ERR_CUDA;
  return from_cuda(
      ssd::launch_vocab_loss_backward(a, dtype, workspace, err, (cudaStream_t)stream));
}

size_t ssd_orthogonalize_workspace_size(const ssd_orth_dims *dims, ssd_dtype in_dtype,
                                        ssd_dtype out_dtype) {
  ssd::OrthArgs a;
  return orth_args(dims, in_dtype, out_dtype, &a) == SSD_OK
             ? ssd::orthogonalize_workspace(a, in_dtype, out_dtype)
             : 0;
}

ssd_status ssd_orthogonalize(const ssd_orth_dims *dims, ssd_dtype in_dtype, ssd_dtype out_dtype,
                             const ssd_seq *update, const ssd_seq *result, void *workspace,
                             size_t ws_bytes, void *stream) {
  ssd::OrthArgs a;
  const ssd_status s = orth_args(dims, in_dtype, out_dtype, &a);
  if (s != SSD_OK) return s;
  if (!req_view(update, in_dtype, a.count, a.rows) ||
      !req_out(result, out_dtype, a.count, a.rows, a.cols) ||
      !good_ws(workspace, ws_bytes, ssd::orthogonalize_workspace(a, in_dtype, out_dtype)))
    return SSD_ERR_INVALID_ARG;
  a.update = update, a.out = result;
  int *err = ssd::device_error_word();
  if (!err) return SSD_ERR_CUDA;
  return from_cuda(ssd::launch_orthogonalize(a, in_dtype, out_dtype, workspace, err,
                                             (cudaStream_t)stream));
}

}  // extern "C"
