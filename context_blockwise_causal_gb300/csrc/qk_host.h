// Host side of the rotations that entry points share: checks of the plan and
// of strided rows, and the kernels' fields.
#pragma once
#include <cstdint>

#include "../../include/cpattn.h"
#include "api_common.h"
#include "qk_rows.cuh"
#include "rope_turns.h"

namespace cpattn {

// Checks the rotary plan for b x n tokens and fills the kernel's fields.
inline int fill_rotary(const cpattn_rotary* r, int b, int n, int d, int inverse, QkArgs* a) {
  if (!r) return CPATTN_ERR_NULL_PTR;
  if (b < 1 || n < 1 || (d != 64 && d != 128)) return CPATTN_ERR_INVALID_ARG;
  if (r->layout != CPATTN_ROPE_HALF && r->layout != CPATTN_ROPE_INTERLEAVED) return CPATTN_ERR_INVALID_ARG;
  if (r->rot_dim < 16 || r->rot_dim > d || r->rot_dim % 16 != 0) return CPATTN_ERR_INVALID_ARG;
  if (!(r->magnitude > 0.f && r->magnitude <= 3.0e38f)) return CPATTN_ERR_INVALID_ARG;
  if (!r->inv_freq) return CPATTN_ERR_NULL_PTR;
  for (int i = 0; i < r->rot_dim / 2; ++i)
    if (!(r->inv_freq[i] >= 0.0 && r->inv_freq[i] <= 1.0e6)) return CPATTN_ERR_INVALID_ARG;
  if (r->positions) {
    // explicit positions take the place of every other source
    if (r->rank >= 0 || r->cu_seqlens || r->positions_batch < 0) return CPATTN_ERR_INVALID_ARG;
    if (!aligned4(r->positions)) return CPATTN_ERR_MISALIGNED;
  } else if (r->rank < 0) {
    if (n != r->s) return CPATTN_ERR_INVALID_ARG;
  } else {
    if (r->cp < 1 || r->s < 1 || r->rank >= r->cp || r->s % (2 * int64_t(r->cp)) != 0 || n != r->s / r->cp)
      return CPATTN_ERR_INVALID_ARG;
  }
  if (r->cu_seqlens && (b != 1 || r->nseq < 1)) return CPATTN_ERR_INVALID_ARG;
  if (r->cu_seqlens && !aligned4(r->cu_seqlens)) return CPATTN_ERR_MISALIGNED;
  a->b = b;
  a->n = n;
  a->s = r->s;
  a->cp = r->cp;
  a->rank = r->rank < 0 ? -1 : r->rank;
  a->cu_seqlens = r->cu_seqlens;
  a->nseq = r->cu_seqlens ? r->nseq : 0;
  a->positions = r->positions;
  a->pos_batch = r->positions_batch;
  a->rot = r->rot_dim;
  a->inverse = inverse ? 1 : 0;
  a->magnitude = r->magnitude;
  for (int i = 0; i < kQkMaxPairs; ++i) a->turns[i] = i < r->rot_dim / 2 ? turn_fraction(r->inv_freq[i]) : 0;
  return CPATTN_OK;
}

// Features of a token, queries' and keys' heads together, stay below this: the
// kernels count heads, and features from a token's first head, in 32 bits.
constexpr int64_t kQkMaxFeatures = int64_t(1) << 31;

// Strides of one tensor's rows [b, n, h, d]: 16-byte pieces, tokens apart by
// at least their heads; for an output, batch elements apart by their tokens.
inline int check_rows(const void* p, int64_t batch, int64_t token, int b, int n, int h, int d, bool output) {
  if (!p) return CPATTN_ERR_NULL_PTR;
  if (h < 1 || batch < 0 || token < 0 || batch % 8 != 0 || token % 8 != 0) return CPATTN_ERR_INVALID_ARG;
  const int64_t row = int64_t(h) * d;
  if (row >= kQkMaxFeatures) return CPATTN_ERR_INVALID_ARG;
  if (n > 1 && token < row) return CPATTN_ERR_INVALID_ARG;
  const int64_t span = int64_t(n - 1) * token + row;  // elements of one batch element
  if (output && b > 1 && batch < span) {
    // batch elements may also lie inside each other's token stride, e.g. [n, b, h, d]
    if (!(batch >= row && (n == 1 || token >= int64_t(b - 1) * batch + row))) return CPATTN_ERR_INVALID_ARG;
  }
  if (!aligned16(p)) return CPATTN_ERR_MISALIGNED;
  return CPATTN_OK;
}

inline void set_tensor(QkTensor* t, const cpattn_rows* x, const cpattn_rows* dy, const cpattn_rows* y, const void* w, int h) {
  t->x = static_cast<const __nv_bfloat16*>(x->data);
  t->x_batch = x->batch_stride;
  t->x_token = x->token_stride;
  t->dy = dy ? static_cast<const __nv_bfloat16*>(dy->data) : nullptr;
  t->dy_batch = dy ? dy->batch_stride : 0;
  t->dy_token = dy ? dy->token_stride : 0;
  t->y = static_cast<__nv_bfloat16*>(y->data);
  t->y_batch = y->batch_stride;
  t->y_token = y->token_stride;
  t->w = w;
  t->h = h;
}

inline int check_rows(const cpattn_rows* r, int b, int n, int h, int d, bool output) {
  if (!r) return CPATTN_ERR_NULL_PTR;
  return check_rows(r->data, r->batch_stride, r->token_stride, b, n, h, d, output);
}

}  // namespace cpattn
