// Sixteen elements of a row on their way into an MX tensor: loads, amax, codes.
// Shared by the quantiser and by kernels that quantise what they compute.
#pragma once

#include "mx.h"

namespace lq {

constexpr int kUnit = 16;  // columns per thread

// max over the lane pair (2 i, 2 i + 1)
__device__ __forceinline__ uint32_t pair_max(uint32_t v) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false);
  return v > o ? v : o;
}

// a bf16 pair's bits (by value: a vector element must not be bit-cast in place)
__device__ __forceinline__ bf16x2 pair(uint32_t w) { return __builtin_bit_cast(bf16x2, w); }

// 16 elements of a unit as loaded: bf16 pairs or floats
template <bool BF16>
struct Unit;
template <>
struct Unit<true> {
  u32x4 v[2];
  __device__ __forceinline__ void load(const void* X, int64_t e) {
    const u32x4_a2* p = reinterpret_cast<const u32x4_a2*>((const uint16_t*)X + e);
    v[0] = p[0];
    v[1] = p[1];
  }
  __device__ __forceinline__ void load_some(const void* X, int64_t e, int n) {
    uint32_t h[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) h[i] = i < n ? ((const uint16_t*)X)[e + i] : 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i >> 2][i & 3] = h[2 * i] | (h[2 * i + 1] << 16);
  }
  // bits of max |x| as a float32
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w = v[i >> 2][i & 3];
      const uint32_t lo = (w << 16) & 0x7FFF0000u, hi = w & 0x7FFF0000u;
      m = m > lo ? m : lo;
      m = m > hi ? m : hi;
    }
    return m;
  }
  __device__ __forceinline__ u32x4 fp8(float s) const {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s16x2 c = {0, 0};
      const uint32_t a = v[i >> 1][2 * (i & 1)], b = v[i >> 1][2 * (i & 1) + 1];
      c = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(c, pair(a), s, false);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(c, pair(b), s, true);
      o[i] = __builtin_bit_cast(uint32_t, c);
    }
    return o;
  }
  __device__ __forceinline__ u32x2 fp4(float s) const {
    u32x2 o;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t c = 0;
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, pair(v[i][0]), s, 0);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, pair(v[i][1]), s, 1);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, pair(v[i][2]), s, 2);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, pair(v[i][3]), s, 3);
      o[i] = c;
    }
    return o;
  }
};
template <>
struct Unit<false> {
  f32x4 v[4];
  __device__ __forceinline__ void load(const void* X, int64_t e) {
    const f32x4_a4* p = reinterpret_cast<const f32x4_a4*>((const float*)X + e);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = p[i];
  }
  __device__ __forceinline__ void load_some(const void* X, int64_t e, int n) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i >> 2][i & 3] = i < n ? ((const float*)X)[e + i] : 0.0f;
  }
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t a = __float_as_uint(v[i >> 2][i & 3]) & 0x7FFFFFFFu;
      m = m > a ? m : a;
    }
    return m;
  }
  __device__ __forceinline__ u32x4 fp8(float s) const {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s16x2 c = {0, 0};
      c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, v[i][0], v[i][1], s, false);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, v[i][2], v[i][3], s, true);
      o[i] = __builtin_bit_cast(uint32_t, c);
    }
    return o;
  }
  __device__ __forceinline__ u32x2 fp4(float s) const {
    u32x2 o;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t c = 0;
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2 * i][0], v[2 * i][1], s, 0);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2 * i][2], v[2 * i][3], s, 1);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2 * i + 1][0], v[2 * i + 1][1], s, 2);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2 * i + 1][2], v[2 * i + 1][3], s, 3);
      o[i] = c;
    }
    return o;
  }
};

}  // namespace lq
