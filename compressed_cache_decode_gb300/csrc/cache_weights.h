// cache_weights.h — the summation over the heads shared by the calls that
// accumulate attention weights per cache row.
#pragma once

#include <cstdint>

#include "lrkv.h"

namespace lrkv {

// weights_out[b][j] = decay * weights[b][j] * (j < L_b - 1) + sum over the
// heads of 2^(scores[b][h][j] - lse[b][h] log2 e), rows [0, L_b); scores
// [B][H][max_len] in the log2 domain.  decay 0 reads no earlier weight.
lrkv_status weights_sum_launch(int B, int H, int max_len, const int32_t* seq_lens, const float* scores,
                               const float* lse, float decay, const float* weights, float* weights_out,
                               void* stream);

// Host checks of a weight accumulation's own arguments.
inline lrkv_status weights_check(float decay, const float* weights, const float* weights_out) {
  if (!(decay >= 0.f) || decay > 3.0e38f || !weights_out) return LRKV_ERR_INVALID_ARG;
  return decay > 0.f && !weights ? LRKV_ERR_INVALID_ARG : LRKV_OK;
}

}  // namespace lrkv
