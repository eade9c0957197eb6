// cache8.h — the factored cache in 8 bits: what its calls share.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "lrkv.h"

namespace lrkv {

constexpr int kBlock8 = LRKV_BLOCK8;

// Host checks of the shapes and the cache's pointers, shared by the calls.
inline lrkv_status cache8_check_dims(const lrkv_dims* d) {
  if (!d) return LRKV_ERR_INVALID_ARG;
  if (d->batch < 1 || d->heads < 1 || d->head_dim < 1 || d->rank < 0 || d->max_len < 1) return LRKV_ERR_INVALID_ARG;
  if (d->dtype != LRKV_F32 && d->dtype != LRKV_BF16) return LRKV_ERR_INVALID_ARG;
  if (!(d->scale == d->scale)) return LRKV_ERR_INVALID_ARG;  // NaN scale
  if (d->head_dim % 16 != 0 || d->head_dim > 256 || d->rank % 2 != 0 || d->rank > 64 || d->heads > 256 ||
      (static_cast<long long>(d->heads) * d->rank) % 16 != 0 || d->batch > 4096)
    return LRKV_ERR_UNSUPPORTED;
  if (static_cast<long long>(d->batch) * d->max_len > (1LL << 31) - 1) return LRKV_ERR_UNSUPPORTED;
  return LRKV_OK;
}

inline bool cache8_a16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline lrkv_status cache8_check(const lrkv_dims* d, const lrkv_cache8* c) {
  if (!c || !c->k_s || !c->v_s || !c->k_s_scale || !c->v_s_scale) return LRKV_ERR_INVALID_ARG;
  if (!cache8_a16(c->k_s) || !cache8_a16(c->v_s) || !cache8_a16(c->k_s_scale) || !cache8_a16(c->v_s_scale))
    return LRKV_ERR_INVALID_ARG;
  if (d->rank == 0) return LRKV_OK;
  if (!c->z_k || !c->z_v || !c->z_k_scale || !c->z_v_scale) return LRKV_ERR_INVALID_ARG;
  if (!cache8_a16(c->z_k) || !cache8_a16(c->z_v) || !cache8_a16(c->z_k_scale) || !cache8_a16(c->z_v_scale))
    return LRKV_ERR_INVALID_ARG;
  return LRKV_OK;
}

// The paging of a call (block_table NULL: contiguous, page_size and num_pages not read).
inline lrkv_status cache8_check_paging(const lrkv_dims* d, int page_size, int num_pages, const int32_t* block_table) {
  if (!block_table) return LRKV_OK;
  if (page_size < kBlock8 || (page_size & (page_size - 1)) != 0 || num_pages < 1) return LRKV_ERR_INVALID_ARG;
  if (d->max_len % page_size != 0) return LRKV_ERR_INVALID_ARG;
  if (static_cast<long long>(num_pages) * page_size > (1LL << 31) - 1) return LRKV_ERR_UNSUPPORTED;
  return LRKV_OK;
}

// Two fp32 values as e4m3 (low byte: lo), rounded to nearest even, magnitudes
// past 448 to 448, NaN to NaN.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// The two values of a pair of e4m3 bytes.
__device__ __forceinline__ float2 from_e4m3x2(uint32_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(v)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

}  // namespace lrkv
