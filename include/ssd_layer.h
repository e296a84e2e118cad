/*
 * ssd_layer.h -- C ABI of the operators that stand around a state space scan
 * in a layer: the short causal convolution in front of it, the selective scan
 * (a decay per channel and state, next to the per-head decay of ssd_forward),
 * the gated group norm behind it, and the global gradient norm with clipping.
 * Part of libssd_gb300.
 *
 * Conventions: those of ssd.h (device pointers, `stream`, checks before any
 * launch, status codes, nothing allocated, nothing synchronised), except
 * where said here:
 * - Activations are views (ssd_seq): element strides between sequences and
 *   between tokens, channels dense.  A slice of a wider projection is passed
 *   as it is.  A view or parameter needs the alignment of its element only;
 *   base addresses and strides that are multiples of 16 bytes run the
 *   vectorised kernels.  Strides are >= 0; an output view whose elements
 *   share an address is refused.
 * - At most 65535 sequences (the norm: 2^31 - 1 tokens in all), 2^31 - 1
 *   tokens a sequence and 2^24 channels, else SSD_ERR_UNSUPPORTED.
 * - State tensors (convolution state, h0, final states, their gradients) are
 *   dense.  Parameters and their gradients are dense fp32.
 * - `lengths` (device int32 [batch], NULL = every sequence has seqlen tokens)
 *   makes sequence i end after its first lengths[i] tokens (clamped to
 *   [0, seqlen]; 0 is a sequence without tokens).  What the inputs hold past
 *   a sequence's end is not read; outputs and gradients there are zero.
 *   Final states are those after the last real token (the initial state for
 *   a sequence without one).
 * - Arithmetic, states and sums are fp32 with either I/O type; an SSD_BF16
 *   output is rounded once.  Sums over tokens, channels or sequences are
 *   taken in a fixed order: calls of equal sizes, types, strides and
 *   alignments of the addresses on the same kind of device give the same
 *   bits.  (Aligned and unaligned views may differ in theirs.)
 * - Outputs must not overlap inputs, nor one another, unless said otherwise.
 *   (Refused where it is cheap to see: y at x's address in ssd_causal_conv,
 *   final_state at h0's in ssd_selective_scan.)
 * - A workspace (>= the matching *_workspace_size bytes, 256-byte aligned)
 *   needs no initialisation: each call writes what it reads there.  Every
 *   call reports to the library-wide error word (ssd_device_error).
 */
#ifndef SSD_GB300_LAYER_H
#define SSD_GB300_LAYER_H

#include "ssd.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A [batch, seqlen, channels] view: element (i, t, c) is at
 * data[i * batch_stride + t * token_stride + c]. */
typedef struct {
  void *data;
  int64_t batch_stride, token_stride;
} ssd_seq;

/* ------------------------------------------------------ causal convolution */

typedef enum { SSD_ACT_NONE = 0, SSD_ACT_SILU = 1 } ssd_activation;

/* batch, seqlen, channels >= 1; width W in {2, 3, 4} (else
 * SSD_ERR_UNSUPPORTED). */
typedef struct {
  int64_t batch, seqlen, channels, width;
  int32_t activation; /* ssd_activation */
} ssd_conv_dims;

/* y_t[c] = act(bias[c] + sum_{k < W} weight[c][k] x_{t - W + 1 + k}[c]),
 * where x_{-(W-1)} .. x_{-1} are the rows of `state` (NULL = zeros).
 * x, y: views, io.  weight [channels, W] f32, bias [channels] f32 (nullable).
 * state, final_state [batch, W - 1, channels] io, oldest first, nullable:
 * final_state receives the last W - 1 inputs, so a later call or
 * ssd_causal_conv_step continues from it. */
SSD_API ssd_status ssd_causal_conv(const ssd_conv_dims *dims, ssd_dtype dtype, const ssd_seq *x,
                                   const float *weight, const float *bias, const void *state,
                                   const int32_t *lengths, const ssd_seq *y, void *final_state,
                                   void *stream);

SSD_API size_t ssd_causal_conv_backward_workspace_size(const ssd_conv_dims *dims,
                                                       ssd_dtype dtype);

/* Gradients of a loss through ssd_causal_conv given gy = dL/dy (view, io) and
 * gfinal = dL/dfinal_state (io, nullable).  With v_t the pre-activation
 * (recomputed) and g_t = gy_t act'(v_t):
 *   dx_t = sum_k weight[.][k] g_{t + W - 1 - k}  (+ gfinal's row of input t)
 *   dweight[c][k] = sum_t g_t x_{t - W + 1 + k},   dbias = sum_t g_t
 * dx: view, io; dweight, dbias f32; dstate io; each nullable. */
SSD_API ssd_status ssd_causal_conv_backward(const ssd_conv_dims *dims, ssd_dtype dtype,
                                            const ssd_seq *x, const float *weight,
                                            const float *bias, const void *state,
                                            const ssd_seq *gy, const void *gfinal,
                                            const int32_t *lengths, const ssd_seq *dx,
                                            float *dweight, float *dbias, void *dstate,
                                            void *workspace, size_t ws_bytes, void *stream);

/* One token of every sequence: seqlen must be 1 (the token strides are not
 * used).  `state` is read, shifted and written in place. */
SSD_API ssd_status ssd_causal_conv_step(const ssd_conv_dims *dims, ssd_dtype dtype,
                                        const ssd_seq *x, const float *weight, const float *bias,
                                        void *state, const ssd_seq *y, void *stream);

/* ---------------------------------------------------------- selective scan */

/* batch, seqlen, channels, dstate, ngroups >= 1, channels % ngroups == 0,
 * dstate N <= 64, ngroups <= 65535 (else SSD_ERR_UNSUPPORTED). */
typedef struct {
  int64_t batch, seqlen, channels, dstate, ngroups;
  int32_t dt_softplus; /* 0: the step is dt + dt_bias; 1: softplus of it */
} ssd_scan_dims;

/* The scan with a decay per channel d and state n; g = d / (channels/ngroups):
 *   s_t = dt_t[d] + dt_bias[d], or log(1 + exp(.)) of it
 *   h_t[d][n] = exp(s_t A[d][n]) h_{t-1}[d][n] + s_t u_t[d] B_t[g][n]
 *   y_t[d] = (sum_n h_t[d][n] C_t[g][n] + D[d] u_t[d]) silu(z_t[d])
 * u, dt, z, y: views of `channels`, io (z->data NULL or z NULL: no gate).
 * B, C: views of ngroups * dstate, io.  A [channels, dstate] f32; D, dt_bias
 * [channels] f32, nullable (0).  h0, final_state [batch, channels, dstate]
 * f32, nullable. */
SSD_API size_t ssd_selective_scan_workspace_size(const ssd_scan_dims *dims, ssd_dtype dtype);

SSD_API ssd_status ssd_selective_scan(const ssd_scan_dims *dims, ssd_dtype dtype,
                                      const ssd_seq *u, const ssd_seq *dt, const float *A,
                                      const ssd_seq *B, const ssd_seq *C, const float *D,
                                      const ssd_seq *z, const float *dt_bias, const float *h0,
                                      const int32_t *lengths, const ssd_seq *y,
                                      float *final_state, void *workspace, size_t ws_bytes,
                                      void *stream);

/* The gradients of ssd_selective_scan: views in, views out.  A NULL output
 * (pointer or data) is not written; du, ddt, dB and dC are required. */
typedef struct {
  ssd_seq du, ddt, dz;  /* views of `channels`, io */
  ssd_seq dB, dC;       /* views of ngroups * dstate, io */
  float *dA;            /* [channels, dstate] */
  float *dD, *ddt_bias; /* [channels] */
  float *dh0;           /* [batch, channels, dstate] */
} ssd_scan_grads;

SSD_API size_t ssd_selective_scan_backward_workspace_size(const ssd_scan_dims *dims,
                                                          ssd_dtype dtype);

/* Given gy = dL/dy (view, io) and gfinal = dL/dfinal_state (f32, nullable),
 * with o_t = gy_t silu(z_t) and the adjoint state
 *   G_t[d][n] = o_t[d] C_t[n] + exp(s_{t+1} A) G_{t+1},  G past the end = gfinal:
 *   du_t = s_t sum_n G_t B_t + D o_t        ds_t = sum_n G_t (u_t B_t + A e_t h_{t-1})
 *   dA = sum_{i,t} s_t G_t e_t h_{t-1}      dB_t[g] = sum_{d in g} G_t s_t u_t
 *   dC_t[g] = sum_{d in g} o_t h_t          dD = sum o_t u_t
 *   ddt_t = ds_t softplus'(.)               ddt_bias = sum ddt_t (before rounding)
 *   dz_t = gy_t (sum_n h_t C_t + D u_t) silu'(z_t),   dh0 = e_1 G_1
 * with e_t = exp(s_t A).  The states are recomputed in the workspace. */
SSD_API ssd_status ssd_selective_scan_backward(
    const ssd_scan_dims *dims, ssd_dtype dtype, const ssd_seq *u, const ssd_seq *dt,
    const float *A, const ssd_seq *B, const ssd_seq *C, const float *D, const ssd_seq *z,
    const float *dt_bias, const float *h0, const ssd_seq *gy, const float *gfinal,
    const int32_t *lengths, const ssd_scan_grads *out, void *workspace, size_t ws_bytes,
    void *stream);

/* One token of every sequence: seqlen must be 1.  `state` [batch, channels,
 * dstate] f32 is read and overwritten in place. */
SSD_API ssd_status ssd_selective_scan_step(const ssd_scan_dims *dims, ssd_dtype dtype,
                                           const ssd_seq *u, const ssd_seq *dt, const float *A,
                                           const ssd_seq *B, const ssd_seq *C, const float *D,
                                           const ssd_seq *z, const float *dt_bias, float *state,
                                           const ssd_seq *y, void *stream);

/* --------------------------------------------------------- gated group norm */

/* Where silu(z) multiplies. */
typedef enum { SSD_GATE_NONE = 0, SSD_GATE_INPUT = 1, SSD_GATE_OUTPUT = 2 } ssd_gate;

/* batch, seqlen, channels, ngroups >= 1, channels % ngroups == 0, at most
 * 65536 channels in a group (else SSD_ERR_UNSUPPORTED); eps > 0. */
typedef struct {
  int64_t batch, seqlen, channels, ngroups;
  float eps;
  int32_t gate;   /* ssd_gate */
  int32_t center; /* 1: subtract the group's mean first */
} ssd_norm_dims;

/* Per token, over the channels of each group:
 *   r = x silu(z) (SSD_GATE_INPUT) or x;  r -= mean(r) with `center`
 *   v = r / sqrt(mean(r^2) + eps) * weight + bias
 *   y = v silu(z) (SSD_GATE_OUTPUT) or v
 * x, z, y: views, io; weight, bias [channels] f32, bias nullable; z is
 * required unless SSD_GATE_NONE, where it must be NULL.  y may be x's or z's
 * own buffer (the same view). */
SSD_API ssd_status ssd_gated_norm(const ssd_norm_dims *dims, ssd_dtype dtype, const ssd_seq *x,
                                  const float *weight, const float *bias, const ssd_seq *z,
                                  const ssd_seq *y, void *stream);

SSD_API size_t ssd_gated_norm_backward_workspace_size(const ssd_norm_dims *dims,
                                                      ssd_dtype dtype);

/* Gradients given gy = dL/dy.  With n the normalised r, q = dL/dv * weight
 * and r' the reciprocal root:
 *   dL/dr = r' (q - n mean(q n) [- mean(q) with `center`])
 * and from there dx, dz (required with a gate); dweight = sum dL/dv n,
 * dbias = sum dL/dv (f32, each nullable). */
SSD_API ssd_status ssd_gated_norm_backward(const ssd_norm_dims *dims, ssd_dtype dtype,
                                           const ssd_seq *x, const float *weight,
                                           const float *bias, const ssd_seq *z,
                                           const ssd_seq *gy, const ssd_seq *dx,
                                           const ssd_seq *dz, float *dweight, float *dbias,
                                           void *workspace, size_t ws_bytes, void *stream);

/* -------------------------------------------- gradient norm and clipping */

/* One tensor of `n` elements (n may be 0); dst is where the scaled values go,
 * in the same type (dst == src: in place; otherwise no overlap). */
typedef struct {
  const void *src;
  void *dst;
  int64_t n;
  int32_t dtype; /* ssd_dtype */
} ssd_grad;

SSD_API size_t ssd_clip_grad_norm_workspace_size(const ssd_grad *grads, int n_grads);

/* norm = sqrt(sum over every tensor and element of g^2), written to *norm
 * (device f32); dst = src * min(1, max_norm / (norm + eps)).  A norm that is
 * not a number makes every output not a number; an infinite one makes finite
 * elements zero (not numbers, where max_norm is infinite too).  `grads` is a
 * host array, read before the call returns; no two dst may overlap.
 * max_norm >= 0, eps >= 0 with max_norm finite or +infinity.  Squares are
 * summed in fp32: an element beyond 1.8e19 makes the norm infinite. */
SSD_API ssd_status ssd_clip_grad_norm(const ssd_grad *grads, int n_grads, float max_norm,
                                      float eps, float *norm, void *workspace, size_t ws_bytes,
                                      void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSD_GB300_LAYER_H */
