// Argument checks shared by the entry points of the operators (layer_api.cu,
// model_api.cu).
#pragma once

#include <cmath>

#include "layer.cuh"

namespace ssd {
namespace args {

constexpr int64_t kMaxTokens = 0x7fffffffLL;  // tokens index grids in 31 bits
constexpr int64_t kMaxBatch = 65535;          // sequences index a grid's second dimension
constexpr double kBig = 4.0e18;               // element counts stay within 62 bits

inline bool valid_dtype(ssd_dtype t) { return t == SSD_F32 || t == SSD_BF16; }
inline size_t elem(ssd_dtype t) { return t == SSD_BF16 ? 2 : 4; }
inline bool natural(const void *p, size_t bytes) { return ptr_aligned(p, bytes); }
inline bool req(const void *p, size_t bytes = 4) { return p && natural(p, bytes); }
inline bool opt(const void *p, size_t bytes = 4) { return natural(p, bytes); }  // NULL is aligned
inline ssd_status from_cuda(cudaError_t e) { return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA; }

inline bool has(const ssd_seq *s) { return s && s->data; }
// A view given as data: natural alignment and strides that keep its addresses
// within 62 bits.
inline bool good(const ssd_seq *s, ssd_dtype t, int64_t b, int64_t L) {
  return natural(s->data, elem(t)) && s->batch_stride >= 0 && s->token_stride >= 0 &&
         (double)s->batch_stride * b + (double)s->token_stride * L < kBig / 8;
}
inline bool req_view(const ssd_seq *s, ssd_dtype t, int64_t b, int64_t L) {
  return has(s) && good(s, t, b, L);
}
inline bool opt_view(const ssd_seq *s, ssd_dtype t, int64_t b, int64_t L) {
  return !has(s) || good(s, t, b, L);
}
// Whether no two elements of a view share an address: its b x L rows of `width`
// elements lie apart.
inline bool apart(const ssd_seq *s, int64_t b, int64_t L, int64_t width) {
  const int64_t bs = s->batch_stride, ts = s->token_stride;
  if ((b > 1 && bs < width) || (L > 1 && ts < width)) return false;
  if (b == 1 || L == 1 || bs >= (L - 1) * ts + width || ts >= (b - 1) * bs + width) return true;
  for (int64_t k = 1; k < b; ++k) {  // sequences k apart against tokens j, j + 1 apart
    const int64_t j = k * bs / ts, rest = k * bs % ts;
    if (j >= L) break;
    if (rest < width || (j + 1 < L && ts - rest < width)) return false;
  }
  return true;
}
inline bool req_out(const ssd_seq *s, ssd_dtype t, int64_t b, int64_t L, int64_t width) {
  return req_view(s, t, b, L) && apart(s, b, L, width);
}
inline bool opt_out(const ssd_seq *s, ssd_dtype t, int64_t b, int64_t L, int64_t width) {
  return !has(s) || req_out(s, t, b, L, width);
}
inline bool req_token(const ssd_seq *s, ssd_dtype t, int64_t b, int64_t width) {  // one row each
  return req_view(s, t, b, 0) && apart(s, b, 1, width);
}
inline bool good_ws(const void *ws, size_t have, size_t need) {
  return need == 0 || (ws && natural(ws, 256) && have >= need);
}
inline const ssd_seq *or_null(const ssd_seq *s) { return has(s) ? s : nullptr; }

inline ssd_status common_dims(int64_t b, int64_t L, int64_t D, int64_t most = kMaxBatch) {
  if (b < 1 || L < 1 || D < 1) return SSD_ERR_INVALID_ARG;
  if (b > most || L > kMaxTokens || D > (1 << 24)) return SSD_ERR_UNSUPPORTED;
  if ((double)b * L * D > kBig / 8) return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

}  // namespace args
}  // namespace ssd
