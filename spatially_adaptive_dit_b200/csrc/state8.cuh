// state8.cuh -- the 8-bit state: argument checks shared by the kernels that
// write it (state8.cu) and that attend over it (attn_state8.cu).
#pragma once

#include "internal.h"

namespace sd {

// Codes [B, H, N, d] of one 8-bit type, d contiguous, other strides multiples
// of 16 elements, 16-byte aligned.
inline safedit_status check_codes(const safedit_tensor* t) {
  if (!t) return SAFEDIT_ERR_INVALID_ARG;
  if (t->dtype != SAFEDIT_I8 && t->dtype != SAFEDIT_E4M3) return SAFEDIT_ERR_DTYPE;
  safedit_tensor plain = *t;
  plain.dtype = SAFEDIT_U8;
  const safedit_status st = check_tensor(&plain, 4);
  if (st != SAFEDIT_OK) return st;
  if (t->strides[3] != 1 || !aligned16(t->data)) return SAFEDIT_ERR_ALIGNMENT;
  for (int k = 0; k < 3; ++k)
    if (t->strides[k] % 16 != 0 || t->strides[k] < 0) return SAFEDIT_ERR_ALIGNMENT;
  return SAFEDIT_OK;
}

inline bool state8_block_ok(int32_t block) { return block == 16 || block == 32 || block == 64 || block == 128; }

// Scales [B, H, ceil(N / block)] f32 of `codes`, blocks contiguous.
inline safedit_status check_scales(const safedit_tensor* t, const safedit_tensor* codes, int32_t block) {
  const safedit_status st = check_tensor(t, 3);
  if (st != SAFEDIT_OK) return st;
  if (t->dtype != SAFEDIT_F32) return SAFEDIT_ERR_DTYPE;
  if (t->dims[0] != codes->dims[0] || t->dims[1] != codes->dims[1] ||
      t->dims[2] != (codes->dims[2] + block - 1) / block)
    return SAFEDIT_ERR_SHAPE;
  if (t->strides[2] != 1 || t->strides[0] < 0 || t->strides[1] < 0) return SAFEDIT_ERR_ALIGNMENT;
  return SAFEDIT_OK;
}

}  // namespace sd
