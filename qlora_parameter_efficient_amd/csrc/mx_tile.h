// Helpers of the MX product kernels that stage operand tiles in LDS with
// gfx950's direct-to-LDS loads: the loads and their wait, LDS operand reads,
// the tiles' swizzles, and the operands of the rank-r expand.
#pragma once

#include "mx.h"

namespace lq {

__device__ __forceinline__ uint32_t mx_lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

// 1 if a < b, else 0, for uniform a and b less than 2^31 apart, in a scalar
// register: a comparison the compiler sees may end up in a vector register,
// which the scalar operands of the asm below do not take.
__device__ __forceinline__ int mx_less(int a, int b) {
  int o;
  asm("s_sub_i32 %0, %1, %2\n\ts_lshr_b32 %0, %0, 31" : "=&s"(o) : "s"(a), "s"(b) : "scc");
  return o;
}

// 16 bytes per lane from global memory (base + off) to LDS at lds + 16 lane.
// Issued from asm so that the compiler does not make later LDS reads of the
// other stage wait for it; the kernel waits itself (mx_wait_loads) before the
// barrier that publishes a stage.  No register results; the address operands
// are read when it issues.  go (uniform) = 0 skips the load, with a branch that
// the compiler does not see (a visible one would split the kernels' loop body).
__device__ __forceinline__ void mx_dma16(const char* base, uint32_t off, uint32_t lds, int go) {
  asm volatile(
      "s_cmp_eq_u32 %3, 0\n\t"
      "s_mov_b32 m0, %2\n\t"
      "s_cbranch_scc1 1f\n\t"
      "global_load_lds_dwordx4 %0, %1\n"
      "1:"
      :
      : "v"(off), "s"(base), "s"(lds), "s"(go)
      : "memory", "scc", "m0");
}

// The same, 4 bytes per lane to LDS at lds + 4 lane.
__device__ __forceinline__ void mx_dma4(const void* base, uint32_t off, uint32_t lds, int go) {
  asm volatile(
      "s_cmp_eq_u32 %3, 0\n\t"
      "s_mov_b32 m0, %2\n\t"
      "s_cbranch_scc1 1f\n\t"
      "global_load_lds_dword %0, %1\n"
      "1:"
      :
      : "v"(off), "s"(base), "s"(lds), "s"(go)
      : "memory", "scc", "m0");
}

// Wait for this wave's loads: all but the newest N if ``some`` (uniform) is
// nonzero, else all of them.
template <int N>
__device__ __forceinline__ void mx_wait_loads(int some) {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile(
      "s_cmp_eq_u32 %0, 0\n\t"
      "s_cbranch_scc1 1f\n\t"
      "s_waitcnt vmcnt(%1)\n\t"
      "s_branch 2f\n"
      "1:\n\t"
      "s_waitcnt vmcnt(0)\n"
      "2:"
      :
      : "s"(some), "n"(N)
      : "memory", "scc");
}
__device__ __forceinline__ void mx_wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

__device__ __forceinline__ u32x4 mx_read16(uint32_t addr) {
  typedef __attribute__((address_space(3))) const u32x4* lds_ptr;
  return *(lds_ptr)(uintptr_t)addr;
}

// Chunk swizzle of tiles with 128-byte rows: 16-byte chunk c of row x sits at
// c ^ mx_swz128(x), so that one chunk column of 16 consecutive rows covers 16
// distinct groups of four banks (64 banks).  64-byte rows: c ^ mx_swz64(x).
__device__ __forceinline__ int mx_swz128(int x) { return (x & 7) ^ ((x >> 3) & 1); }
__device__ __forceinline__ int mx_swz64(int x) { return (x >> 2) & 3; }

// s v[0..7] as an operand of the expand, in two bf16 parts, h = bf16(s v) and
// l = bf16(s v - h), together off by 2^-16 of the value (one part alone, 2^-8, is
// as much as the rounding of the output, and more where ranks cancel); v is a
// float32 row of length r at rank j0, ranks past r are zero
struct MxVParts {
  u32x4 h, l;
};
__device__ __forceinline__ MxVParts mx_v_operand(const float* row, int j0, int r, float s) {
  float e[8];
  if (j0 + 8 <= r && (reinterpret_cast<uintptr_t>(row + j0) & 15) == 0) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(row + j0);
    const f32x4 b = *reinterpret_cast<const f32x4*>(row + j0 + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      e[i] = a[i];
      e[4 + i] = b[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = j0 + i < r ? row[j0 + i] : 0.0f;
  }
  MxVParts o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = s * e[2 * i], b = s * e[2 * i + 1];
    o.h[i] = pack_bf16x2(a, b);
    const float ha = lo_bf16(o.h[i]), hb = hi_bf16(o.h[i]);
    // (the rest of an infinity or NaN is 0)
    o.l[i] = pack_bf16x2(fabsf(ha) < __builtin_inff() ? a - ha : 0.0f,
                         fabsf(hb) < __builtin_inff() ? b - hb : 0.0f);
  }
  return o;
}

__device__ __forceinline__ u32x4 mx_pack8(const uint16_t (&v)[8]) {
  return u32x4{(uint32_t)v[0] | ((uint32_t)v[1] << 16), (uint32_t)v[2] | ((uint32_t)v[3] << 16),
               (uint32_t)v[4] | ((uint32_t)v[5] << 16), (uint32_t)v[6] | ((uint32_t)v[7] << 16)};
}

// ranks j0 .. j0 + 7 of a bf16 row of length r, zeros past r
__device__ __forceinline__ u32x4 mx_e_row(const uint16_t* row, int j0, int r) {
  if (j0 + 8 <= r && (reinterpret_cast<uintptr_t>(row + j0) & 15) == 0)
    return *reinterpret_cast<const u32x4*>(row + j0);
  uint16_t v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = j0 + i < r ? row[j0 + i] : (uint16_t)0;
  return mx_pack8(v);
}

// A[j0 + i][k], i < 8 (A r x ld bf16), zeros past r
__device__ __forceinline__ u32x4 mx_e_col(const uint16_t* A, int64_t ld, int64_t k, int j0, int r) {
  uint16_t v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = j0 + i < r ? A[(int64_t)(j0 + i) * ld + k] : (uint16_t)0;
  return mx_pack8(v);
}

}  // namespace lq
