// The paged 8-bit KV cache as the kernels see it, and its host checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/pkv.h"
#include "api_common.h"

namespace pkv {

constexpr float kE4m3Max = 448.0f;

// Two fp32 values to two e4m3 codes (lo in the low byte): nearest even,
// limited to +-448, NaN kept.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two e4m3 codes (16 bits) to two fp16 values; exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
  return r;
}

// Refuses a cache the kernels cannot address; PKV_OK otherwise.
inline int cache_error(const pkv_kv_cache* c) {
  if (c == nullptr) return fail(PKV_EINVAL, "cache is NULL");
  if (c->k == nullptr || c->v == nullptr || c->k_scale == nullptr || c->v_scale == nullptr)
    return fail(PKV_EINVAL, "cache has a NULL pointer");
  if (c->page_size < 1 || c->num_pages < 1 || c->num_pages > INT32_MAX / c->page_size)
    return fail(PKV_EINVAL, "cache of %lld pages of %d tokens: need 1 <= tokens < 2^31",
                (long long)c->num_pages, c->page_size);
  if (c->kv_heads < 1 || c->kv_heads > 65535)
    return fail(PKV_EINVAL, "kv_heads=%d outside [1, 65535]", c->kv_heads);
  if (c->head_dim < 16 || c->head_dim > PKV_MAX_HEAD_DIM || c->head_dim % 16 != 0)
    return fail(PKV_EINVAL, "head_dim=%d is not a multiple of 16 in [16, %d]", c->head_dim,
                PKV_MAX_HEAD_DIM);
  const int64_t strides[3] = {c->page_stride, c->token_stride, c->head_stride};
  const int64_t counts[3] = {c->num_pages, c->page_size, c->kv_heads};
  // Kernels reach a code by 32 bits of 16-byte steps: 64 GiB in all.
  const int64_t spans[3] = {int64_t{1} << 35, int64_t{1} << 34, int64_t{1} << 34};
  for (int i = 0; i < 3; ++i) {
    if (strides[i] < 0 || strides[i] % 16 != 0 || strides[i] > spans[i] / counts[i])
      return fail(PKV_EINVAL, "cache stride %lld is not a multiple of 16 within the limits",
                  (long long)strides[i]);
  }
  if (!aligned16(c->k) || !aligned16(c->v))
    return fail(PKV_EINVAL, "cache is not 16-byte aligned");
  return PKV_OK;
}

// Refuses a [tokens, heads, head_dim] tensor of 2-byte elements whose rows
// are not all 16-byte aligned.
inline int rows_error(const char* name, const void* p, int64_t token_stride, int64_t head_stride) {
  if (p == nullptr) return fail(PKV_EINVAL, "%s is NULL", name);
  if (!aligned16(p) || token_stride % 8 != 0 || head_stride % 8 != 0 || token_stride < 0 ||
      head_stride < 0)
    return fail(PKV_EINVAL, "%s has rows that are not 16-byte aligned", name);
  return PKV_OK;
}

template <typename T> struct Pair;  // two packed 16-bit values <-> two fp32
template <> struct Pair<__nv_bfloat16> {
  static __device__ __forceinline__ float2 unpack(uint32_t x) {
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};
template <> struct Pair<__half> {
  static __device__ __forceinline__ float2 unpack(uint32_t x) {
    return __half22float2(*reinterpret_cast<const __half2*>(&x));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 r = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};

}  // namespace pkv
