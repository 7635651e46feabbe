// MX quantiser and dequantiser: one power-of-two scale per 32 columns of a
// row, elements E4M3 or E2M1.
//
//   e = min { e in [-127, 127] : amax <= largest 2^e },  code = RNE(x 2^-e)
//
// The scale byte comes from amax's bits: with amax = 1.f 2^(E - 127),
// largest = 1.75 2^8 (E4M3) or 1.5 2^2 (E2M1), b = E - 8 (or 2), plus one
// where the fraction exceeds that of the largest element, never below 0.
//
// Both kernels are bound by HBM.  A thread owns half a block (16 columns), so
// a lane pair shares a block and one DPP move completes its amax; codes leave
// as one 16-byte (FP8) or 8-byte (FP4) store per thread.  A tensor whose rows
// hold whole blocks is one flat run of blocks; other widths locate each unit's
// row and read the row's last block element by element.
#include "dispatch.h"
#include "mx.h"

namespace lq {
namespace {

constexpr int kThreads = 256;
constexpr int kUnit = 16;  // columns per thread

typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef f32x4 f32x4_a4 __attribute__((aligned(4)));

// max over the lane pair (2 i, 2 i + 1)
__device__ __forceinline__ uint32_t pair_max(uint32_t v) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false);
  return v > o ? v : o;
}

// scale byte of a block from the bits of its amax (sign cleared)
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  constexpr int top = FMT == LQ_MX_FP8 ? 8 : 2;
  constexpr uint32_t frac = FMT == LQ_MX_FP8 ? 0x600000u : 0x400000u;
  const int E = (int)(amax >> 23);
  if (E == 255) return 255u;
  const int b = E - top + ((amax & 0x7FFFFFu) > frac ? 1 : 0);
  return (uint32_t)(b > 0 ? b : 0);
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

// units = rows kp / 16; FLAT: cols % 32 == 0, so unit u starts at element 16 u
template <bool BF16, int FMT, bool FLAT>
__global__ __launch_bounds__(kThreads) void mx_quantize_kernel(const void* __restrict__ X,
                                                               int64_t units, int64_t cols,
                                                               int64_t per_row,
                                                               uint8_t* __restrict__ codes,
                                                               uint8_t* __restrict__ scales) {
  const int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (u >= units) return;  // units is even: lane pairs leave together
  Unit<BF16> x;
  if (FLAT) {
    x.load(X, kUnit * u);
  } else {
    const int64_t row = u / per_row;
    const int64_t c = (u - row * per_row) * kUnit;
    const int64_t left = cols - c;
    if (left >= kUnit)
      x.load(X, row * cols + c);
    else
      x.load_some(X, row * cols + (left > 0 ? c : 0), left > 0 ? (int)left : 0);
  }
  const uint32_t b = scale_byte<FMT>(pair_max(x.amax()));
  const float s = mx_scale(b);
  if (FMT == LQ_MX_FP8) {
    u32x4 o = x.fp8(s);
    *reinterpret_cast<u32x4*>(codes + kUnit * u) = sel4(b != 255u, o);
  } else {
    u32x2 o = x.fp4(s);
    if (b == 255u) o = u32x2{0u, 0u};
    *reinterpret_cast<u32x2*>(codes + (kUnit / 2) * u) = o;
  }
  if (!(u & 1)) scales[u >> 1] = (uint8_t)b;
}

typedef float f32x2v __attribute__((ext_vector_type(2)));

template <bool BF16, int FMT, bool FLAT>
__global__ __launch_bounds__(kThreads) void mx_dequantize_kernel(
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t units,
    int64_t cols, int64_t per_row, void* __restrict__ out) {
  const int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (u >= units) return;
  uint32_t w[4];
  if (FMT == LQ_MX_FP8) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(codes + kUnit * u);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = v[i];
  } else {
    const u32x2 v = *reinterpret_cast<const u32x2*>(codes + (kUnit / 2) * u);
    w[0] = v[0];
    w[1] = v[1];
  }
  const float s = mx_scale(scales[u >> 1]);
  int64_t e = kUnit * u, left = kUnit;
  if (!FLAT) {
    const int64_t row = u / per_row;
    const int64_t c = (u - row * per_row) * kUnit;
    e = row * cols + c;
    left = cols - c;
  }
  if (BF16) {
    u32x4 o[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      o[i] = FMT == LQ_MX_FP8 ? mx8_bf16(w[2 * i], w[2 * i + 1], s) : mx4_bf16(w[i], s);
    uint16_t* dst = (uint16_t*)out + e;
    if (FLAT || left >= kUnit) {
      reinterpret_cast<u32x4_a2*>(dst)[0] = o[0];
      reinterpret_cast<u32x4_a2*>(dst)[1] = o[1];
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < left) dst[i] = (uint16_t)(o[i >> 3][(i >> 1) & 3] >> (16 * (i & 1)));
    }
  } else {
    f32x4 o[4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f32x2v v;
      if (FMT == LQ_MX_FP8) {
        v = (i & 1) ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[i >> 1], s, true)
                    : __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[i >> 1], s, false);
      } else {
        const int j = i & 3;
        v = j == 0   ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i >> 2], s, 0)
            : j == 1 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i >> 2], s, 1)
            : j == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i >> 2], s, 2)
                     : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i >> 2], s, 3);
      }
      o[i >> 1][2 * (i & 1)] = v[0];
      o[i >> 1][2 * (i & 1) + 1] = v[1];
    }
    float* dst = (float*)out + e;
    if (FLAT || left >= kUnit) {
#pragma unroll
      for (int i = 0; i < 4; ++i) reinterpret_cast<f32x4_a4*>(dst)[i] = o[i];
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < left) dst[i] = o[i >> 2][i & 3];
    }
  }
}

template <bool BF16, int FMT>
void launch_q(const void* X, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scales,
              hipStream_t st) {
  const int64_t per_row = cdiv(cols, kMxB) * 2, units = rows * per_row;
  const dim3 grid((unsigned)cdiv(units, kThreads)), block(kThreads);
  if (cols % kMxB == 0)
    hipLaunchKernelGGL((mx_quantize_kernel<BF16, FMT, true>), grid, block, 0, st, X, units, cols,
                       per_row, codes, scales);
  else
    hipLaunchKernelGGL((mx_quantize_kernel<BF16, FMT, false>), grid, block, 0, st, X, units, cols,
                       per_row, codes, scales);
}

template <bool BF16, int FMT>
void launch_d(const lq_mx_tensor& q, void* out, hipStream_t st) {
  const int64_t per_row = cdiv(q.cols, kMxB) * 2, units = q.rows * per_row;
  const dim3 grid((unsigned)cdiv(units, kThreads)), block(kThreads);
  if (q.cols % kMxB == 0)
    hipLaunchKernelGGL((mx_dequantize_kernel<BF16, FMT, true>), grid, block, 0, st, q.codes,
                       q.scales, units, q.cols, per_row, out);
  else
    hipLaunchKernelGGL((mx_dequantize_kernel<BF16, FMT, false>), grid, block, 0, st, q.codes,
                       q.scales, units, q.cols, per_row, out);
}

}  // namespace

namespace dispatch {

int mx_quantize(const void* X, lq_dtype xdt, int64_t rows, int64_t cols, int32_t fmt,
                uint8_t* codes, uint8_t* scales, hipStream_t st) {
  if (xdt == LQ_BF16)
    fmt == LQ_MX_FP8 ? launch_q<true, LQ_MX_FP8>(X, rows, cols, codes, scales, st)
                     : launch_q<true, LQ_MX_FP4>(X, rows, cols, codes, scales, st);
  else
    fmt == LQ_MX_FP8 ? launch_q<false, LQ_MX_FP8>(X, rows, cols, codes, scales, st)
                     : launch_q<false, LQ_MX_FP4>(X, rows, cols, codes, scales, st);
  return hip_fail(hipGetLastError(), "mx_quantize launch");
}

int mx_dequantize(const lq_mx_tensor& q, void* out, lq_dtype odt, hipStream_t st) {
  if (odt == LQ_BF16)
    q.format == LQ_MX_FP8 ? launch_d<true, LQ_MX_FP8>(q, out, st)
                          : launch_d<true, LQ_MX_FP4>(q, out, st);
  else
    q.format == LQ_MX_FP8 ? launch_d<false, LQ_MX_FP8>(q, out, st)
                          : launch_d<false, LQ_MX_FP4>(q, out, st);
  return hip_fail(hipGetLastError(), "mx_dequantize launch");
}

}  // namespace dispatch
}  // namespace lq
