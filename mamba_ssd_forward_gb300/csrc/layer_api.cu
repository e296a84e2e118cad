// C ABI of the operators around the scan (ssd_layer.h): argument checks and
// the launches, nothing else.
#include "args.cuh"

namespace {

using namespace ssd::args;

ssd_status conv_args(const ssd_conv_dims *d, ssd_dtype t, ssd::ConvArgs *a) {
  if (!d || !valid_dtype(t) || d->width < 1 ||
      (d->activation != SSD_ACT_NONE && d->activation != SSD_ACT_SILU))
    return SSD_ERR_INVALID_ARG;
  const ssd_status s = common_dims(d->batch, d->seqlen, d->channels);
  if (s != SSD_OK) return s;
  if (d->width < 2 || d->width > 4) return SSD_ERR_UNSUPPORTED;
  *a = ssd::ConvArgs{};
  a->b = d->batch, a->L = d->seqlen, a->D = d->channels;
  a->W = (int)d->width, a->silu = d->activation == SSD_ACT_SILU;
  return SSD_OK;
}

ssd_status scan_args(const ssd_scan_dims *d, ssd_dtype t, ssd::ScanArgs *a) {
  if (!d || !valid_dtype(t) || d->dstate < 1 || d->ngroups < 1 ||
      (d->dt_softplus != 0 && d->dt_softplus != 1))
    return SSD_ERR_INVALID_ARG;
  const ssd_status s = common_dims(d->batch, d->seqlen, d->channels);
  if (s != SSD_OK) return s;
  if (d->channels % d->ngroups) return SSD_ERR_INVALID_ARG;
  if (d->dstate > 64 || d->ngroups > 65535 ||
      (double)d->batch * d->seqlen * d->channels * d->dstate > kBig / 8)
    return SSD_ERR_UNSUPPORTED;
  *a = ssd::ScanArgs{};
  a->b = d->batch, a->L = d->seqlen, a->D = d->channels, a->N = d->dstate, a->G = d->ngroups;
  a->softplus = d->dt_softplus;
  return SSD_OK;
}

ssd_status norm_args(const ssd_norm_dims *d, ssd_dtype t, ssd::NormArgs *a) {
  if (!d || !valid_dtype(t) || d->ngroups < 1 || !(d->eps > 0.f) || !std::isfinite(d->eps) ||
      d->gate < SSD_GATE_NONE || d->gate > SSD_GATE_OUTPUT || (d->center != 0 && d->center != 1))
    return SSD_ERR_INVALID_ARG;
  const ssd_status s = common_dims(d->batch, d->seqlen, d->channels, kMaxTokens);
  if (s != SSD_OK) return s;
  if (d->channels % d->ngroups) return SSD_ERR_INVALID_ARG;
  if (d->channels / d->ngroups > 65536 || d->ngroups > 65535 ||
      (double)d->batch * d->seqlen > (double)kMaxTokens)
    return SSD_ERR_UNSUPPORTED;
  *a = ssd::NormArgs{};
  a->b = d->batch, a->L = d->seqlen, a->D = d->channels, a->G = d->ngroups;
  a->eps = d->eps, a->gate = d->gate, a->center = d->center;
  return SSD_OK;
}

// The views and parameters that every call of the scan takes.
bool scan_inputs(ssd::ScanArgs *a, ssd_dtype t, const ssd_seq *u, const ssd_seq *dt,
                 const float *A, const ssd_seq *B, const ssd_seq *C, const float *D,
                 const ssd_seq *z, const float *dt_bias) {
  const int64_t b = a->b, L = a->L;
  if (!req_view(u, t, b, L) || !req_view(dt, t, b, L) || !req_view(B, t, b, L) ||
      !req_view(C, t, b, L) || !opt_view(z, t, b, L) || !req(A) || !opt(D) || !opt(dt_bias))
    return false;
  a->u = u, a->dt = dt, a->A = A, a->B = B, a->C = C, a->Dskip = D, a->z = or_null(z);
  a->dt_bias = dt_bias;
  return true;
}

}  // namespace

extern "C" {

ssd_status ssd_causal_conv(const ssd_conv_dims *dims, ssd_dtype dtype, const ssd_seq *x,
                           const float *weight, const float *bias, const void *state,
                           const int32_t *lengths, const ssd_seq *y, void *final_state,
                           void *stream) {
  ssd::ConvArgs a;
  const ssd_status s = conv_args(dims, dtype, &a);
  if (s != SSD_OK) return s;
  if (!req_view(x, dtype, a.b, a.L) || !req_out(y, dtype, a.b, a.L, a.D) || !req(weight) ||
      !opt(bias) || !opt(state, elem(dtype)) || !opt(lengths) || !opt(final_state, elem(dtype)) ||
      x->data == y->data)  // a run reads the tokens in front of it, which are another's
    return SSD_ERR_INVALID_ARG;
  a.x = x, a.y = y, a.weight = weight, a.bias = bias, a.state = state, a.lengths = lengths;
  a.final_state = final_state;
  int *err = ssd::device_error_word();
  if (!err) return SSD_ERR_CUDA;
  return from_cuda(ssd::launch_causal_conv(a, dtype, err, (cudaStream_t)stream));
}

ssd_status ssd_causal_conv_step(const ssd_conv_dims *dims, ssd_dtype dtype, const ssd_seq *x,
                                const float *weight, const float *bias, void *state,
                                const ssd_seq *y, void *stream) {
  ssd::ConvArgs a;
  const ssd_status s = conv_args(dims, dtype, &a);
  if (s != SSD_OK) return s;
  if (a.L != 1 || !req_view(x, dtype, a.b, 0) || !req_token(y, dtype, a.b, a.D) || !req(weight) ||
      !opt(bias) || !req(state, elem(dtype)))
    return SSD_ERR_INVALID_ARG;
  a.x = x, a.y = y, a.weight = weight, a.bias = bias, a.final_state = state;
  int *err = ssd::device_error_word();
  if (!err) return SSD_ERR_CUDA;
  return from_cuda(ssd::launch_causal_conv_step(a, dtype, err, (cudaStream_t)stream));
}

size_t ssd_causal_conv_backward_workspace_size(const ssd_conv_dims *dims, ssd_dtype dtype) {
  ssd::ConvArgs a;
  return conv_args(dims, dtype, &a) == SSD_OK ? ssd::causal_conv_backward_workspace(a, dtype) : 0;
}

ssd_status ssd_causal_conv_backward(const ssd_conv_dims *dims, ssd_dtype dtype, const ssd_seq *x,
                                    const float *weight, const float *bias, const void *state,
                                    const ssd_seq *gy, const void *gfinal, const int32_t *lengths,
                                    const ssd_seq *dx, float *dweight, float *dbias, void *dstate,
                                    void *workspace, size_t ws_bytes, void *stream) {
  ssd::ConvArgs a;
  const ssd_status s = conv_args(dims, dtype, &a);
  if (s != SSD_OK) return s;
  const size_t e = elem(dtype);
  if (!req_view(x, dtype, a.b, a.L) || !req_view(gy, dtype, a.b, a.L) ||
      !opt_out(dx, dtype, a.b, a.L, a.D) || !req(weight) || !opt(bias) || !opt(state, e) ||
      !opt(gfinal, e) || !opt(lengths) || !opt(dweight) || !opt(dbias) || !opt(dstate, e) ||
      !good_ws(workspace, ws_bytes, ssd::causal_conv_backward_workspace(a, dtype)))
    return SSD_ERR_INVALID_ARG;
  a.x = x, a.gy = gy, a.dx = or_null(dx), a.weight = weight, a.bias = bias, a.state = state;
  a.gfinal = gfinal, a.lengths = lengths, a.dweight = dweight, a.dbias = dbias;
  a.dstate = dstate;
  int *err = ssd::device_error_word();
  if (!err) return SSD_ERR_CUDA;
  return from_cuda(
      ssd::launch_causal_conv_backward(a, dtype, workspace, err, (cudaStream_t)stream));
}

size_t ssd_selective_scan_workspace_size(const ssd_scan_dims *dims, ssd_dtype dtype) {
  ssd::ScanArgs a;
  return scan_args(dims, dtype, &a) == SSD_OK ? ssd::selective_scan_workspace(a, dtype) : 0;
}

ssd_status ssd_selective_scan(const ssd_scan_dims *dims, ssd_dtype dtype, const ssd_seq *u,
                              const ssd_seq *dt, const float *A, const ssd_seq *B,
                              const ssd_seq *C, const float *D, const ssd_seq *z,
                              const float *dt_bias, const float *h0, const int32_t *lengths,
                              const ssd_seq *y, float *final_state, void *workspace,
                              size_t ws_bytes, void *stream) {
  ssd::ScanArgs a;
  const ssd_status s = scan_args(dims, dtype, &a);
  if (s != SSD_OK) return s;
  if (!scan_inputs(&a, dtype, u, dt, A, B, C, D, z, dt_bias) || !opt(h0) || !opt(lengths) ||
      !req_out(y, dtype, a.b, a.L, a.D) || !opt(final_state) ||
      (h0 && final_state == h0) ||  // every segment of a sequence starts from h0
      !good_ws(workspace, ws_bytes, ssd::selective_scan_workspace(a, dtype)))
    return SSD_ERR_INVALID_ARG;
  a.h0 = h0, a.lengths = lengths, a.y = y, a.final_state = final_state;
  int *err = ssd::device_error_word();
  if (!err) return SSD_ERR_CUDA;
  return from_cuda(ssd::launch_selective_scan(a, dtype, workspace, err, (cudaStream_t)stream));
}

ssd_status ssd_selective_scan_step(const ssd_scan_dims *dims, ssd_dtype dtype, const ssd_seq *u,
                                   const ssd_seq *dt, const float *A, const ssd_seq *B,
                                   const ssd_seq *C, const float *D, const ssd_seq *z,
                                   const float *dt_bias, float *state, const ssd_seq *y,
                                   void *stream) {
  ssd::ScanArgs a;
  const ssd_status s = scan_args(dims, dtype, &a);
  if (s != SSD_OK) return s;
  if (a.L != 1 || !scan_inputs(&a, dtype, u, dt, A, B, C, D, z, dt_bias) || !req(state) ||
      !req_token(y, dtype, a.b, a.D))
    return SSD_ERR_INVALID_ARG;
  a.y = y, a.final_state = state;
  int *err = ssd::device_error_word();
  if (!err) return SSD_ERR_CUDA;
  return from_cuda(ssd::launch_selective_scan_step(a, dtype, err, (cudaStream_t)stream));
}

size_t ssd_selective_scan_backward_workspace_size(const ssd_scan_dims *dims, ssd_dtype dtype) {
  ssd::ScanArgs a;
  return scan_args(dims, dtype, &a) == SSD_OK ? ssd::selective_scan_backward_workspace(a, dtype)
                                              : 0;
}

ssd_status ssd_selective_scan_backward(
    const ssd_scan_dims *dims, ssd_dtype dtype, const ssd_seq *u, const ssd_seq *dt,
    const float *A, const ssd_seq *B, const ssd_seq *C, const float *D, const ssd_seq *z,
    const float *dt_bias, const float *h0, const ssd_seq *gy, const float *gfinal,
    const int32_t *lengths, const ssd_scan_grads *out, void *workspace, size_t ws_bytes,
    void *stream) {
  ssd::ScanArgs a;
  const ssd_status s = scan_args(dims, dtype, &a);
  if (s != SSD_OK) return s;
  if (!scan_inputs(&a, dtype, u, dt, A, B, C, D, z, dt_bias) || !opt(h0) || !opt(lengths) ||
      !req_view(gy, dtype, a.b, a.L) || !opt(gfinal) || !out ||
      !good_ws(workspace, ws_bytes, ssd::selective_scan_backward_workspace(a, dtype)))
    return SSD_ERR_INVALID_ARG;
  if (!req_out(&out->du, dtype, a.b, a.L, a.D) || !req_out(&out->ddt, dtype, a.b, a.L, a.D) ||
      !req_out(&out->dB, dtype, a.b, a.L, a.G * a.N) ||
      !req_out(&out->dC, dtype, a.b, a.L, a.G * a.N) ||
      !opt_out(&out->dz, dtype, a.b, a.L, a.D) || (has(&out->dz) && !a.z) || !opt(out->dA) ||
      !opt(out->dD) || !opt(out->ddt_bias) || !opt(out->dh0))
    return SSD_ERR_INVALID_ARG;
  a.h0 = h0, a.lengths = lengths, a.gy = gy, a.gfinal = gfinal, a.out = out;
  int *err = ssd::device_error_word();
  if (!err) return SSD_ERR_CUDA;
  return from_cuda(
      ssd::launch_selective_scan_backward(a, dtype, workspace, err, (cudaStream_t)stream));
}

ssd_status ssd_gated_norm(const ssd_norm_dims *dims, ssd_dtype dtype, const ssd_seq *x,
                          const float *weight, const float *bias, const ssd_seq *z,
                          const ssd_seq *y, void *stream) {
  ssd::NormArgs a;
  const ssd_status s = norm_args(dims, dtype, &a);
  if (s != SSD_OK) return s;
  if (!req_view(x, dtype, a.b, a.L) || !req_out(y, dtype, a.b, a.L, a.D) || !req(weight) ||
      !opt(bias) || has(z) != (a.gate != SSD_GATE_NONE) || !opt_view(z, dtype, a.b, a.L))
    return SSD_ERR_INVALID_ARG;
  a.x = x, a.y = y, a.z = or_null(z), a.weight = weight, a.bias = bias;
  int *err = ssd::device_error_word();
  if (!err) return SSD_ERR_CUDA;
  return from_cuda(ssd::launch_gated_norm(a, dtype, err, (cudaStream_t)stream));
}

size_t ssd_gated_norm_backward_workspace_size(const ssd_norm_dims *dims, ssd_dtype dtype) {
  ssd::NormArgs a;
  return norm_args(dims, dtype, &a) == SSD_OK ? ssd::gated_norm_backward_workspace(a, dtype) : 0;
}

ssd_status ssd_gated_norm_backward(const ssd_norm_dims *dims, ssd_dtype dtype, const ssd_seq *x,
                                   const float *weight, const float *bias, const ssd_seq *z,
                                   const ssd_seq *gy, const ssd_seq *dx, const ssd_seq *dz,
                                   float *dweight, float *dbias, void *workspace,
                                   size_t ws_bytes, void *stream) {
  ssd::NormArgs a;
  const ssd_status s = norm_args(dims, dtype, &a);
  if (s != SSD_OK) return s;
  const bool gated = a.gate != SSD_GATE_NONE;
  if (!req_view(x, dtype, a.b, a.L) || !req_view(gy, dtype, a.b, a.L) ||
      !req_out(dx, dtype, a.b, a.L, a.D) || !req(weight) || !opt(bias) || has(z) != gated ||
      !opt_view(z, dtype, a.b, a.L) || has(dz) != gated || !opt_out(dz, dtype, a.b, a.L, a.D) ||
      !opt(dweight) || !opt(dbias) ||
      !good_ws(workspace, ws_bytes, ssd::gated_norm_backward_workspace(a, dtype)))
    return SSD_ERR_INVALID_ARG;
  a.x = x, a.gy = gy, a.dx = dx, a.z = or_null(z), a.dz = or_null(dz), a.weight = weight;
  a.bias = bias, a.dweight = dweight, a.dbias = dbias;
  int *err = ssd::device_error_word();
  if (!err) return SSD_ERR_CUDA;
  return from_cuda(
      ssd::launch_gated_norm_backward(a, dtype, workspace, err, (cudaStream_t)stream));
}

static bool good_grads(const ssd_grad *grads, int n) {
  if (n < 0 || (n > 0 && !grads)) return false;
  double total = 0;
  for (int i = 0; i < n; ++i) {
    const ssd_grad &g = grads[i];
    if (g.n < 0 || !valid_dtype((ssd_dtype)g.dtype)) return false;
    if (g.n > 0 && (!req(g.src, elem((ssd_dtype)g.dtype)) || !req(g.dst, elem((ssd_dtype)g.dtype))))
      return false;
    total += (double)g.n;
  }
  return total < kBig / 8;
}

size_t ssd_clip_grad_norm_workspace_size(const ssd_grad *grads, int n_grads) {
  return good_grads(grads, n_grads) ? ssd::clip_grad_workspace(grads, n_grads) : 0;
}

ssd_status ssd_clip_grad_norm(const ssd_grad *grads, int n_grads, float max_norm, float eps,
                              float *norm, void *workspace, size_t ws_bytes, void *stream) {
  if (!good_grads(grads, n_grads) || !(max_norm >= 0.f) || !(eps >= 0.f) ||
      !std::isfinite(eps) || !req(norm) ||
      !good_ws(workspace, ws_bytes, ssd::clip_grad_workspace(grads, n_grads)))
    return SSD_ERR_INVALID_ARG;
  int *err = ssd::device_error_word();
  if (!err) return SSD_ERR_CUDA;
  return from_cuda(ssd::launch_clip_grad(grads, n_grads, max_norm, eps, norm, workspace, err,
                                         (cudaStream_t)stream));
}

}  // extern "C"
