// Internal definitions of the microscaled (MX) kernels: the element formats'
// conversions on gfx950 and the launchers called by the ABI layer.
//
// gfx950 converts between packed E2M1 / E4M3 codes and float32 / bf16 with a
// block scale in one instruction (v_cvt_scalef32_*): the scale operand is a
// float32 whose exponent field is the block's scale byte, so a scale byte b is
// passed as the bits b << 23, which the instructions read as 2^(b - 127) also
// for b = 0 (2^-127) and as NaN for b = 255.  The roundings (ties to even,
// subnormal results) are those of the format's definition.
#pragma once

#include "../../include/lq_mx.h"
#include "device_util.h"

namespace lq {

constexpr int64_t kMxB = LQ_MX_BLOCK;

__host__ __device__ inline int64_t mx_pitch(int32_t fmt, int64_t cols) {
  return cdiv(cols, kMxB) * (kMxB * fmt / 8);
}
__host__ __device__ inline int64_t mx_spitch(int64_t cols) { return cdiv(cols, kMxB); }

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// 16-byte accesses to rows that are aligned to their elements only
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef f32x4 f32x4_a4 __attribute__((aligned(4)));

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

__device__ __forceinline__ float mx_scale(uint32_t b) { return __uint_as_float(b << 23); }

// Eight E2M1 codes (element e in bits 4e .. 4e + 3) times 2^(b - 127) as bf16
// in element order: exact (bf16 subnormals rounded to nearest even)
__device__ __forceinline__ u32x4 mx4_bf16(uint32_t w, float s) {
  return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3))};
}

// Eight E4M3 codes (two words) times 2^(b - 127) as bf16
__device__ __forceinline__ u32x4 mx8_bf16(uint32_t w0, uint32_t w1, float s) {
  return u32x4{
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, false)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, true)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, false)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, true))};
}

// One block of 32 codes held by a lane (FP8: 32 bytes, FP4: 16 bytes)
template <int FMT>
struct MxBlock {
  u32x4 w[FMT == LQ_MX_FP8 ? 2 : 1];
  uint32_t b;  // scale byte
  __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* scales) {
#pragma unroll
    for (int i = 0; i < (FMT == LQ_MX_FP8 ? 2 : 1); ++i)
      w[i] = *reinterpret_cast<const u32x4*>(codes + 16 * i);
    b = *scales;
  }
  // elements 8 d .. 8 d + 7 as bf16
  __device__ __forceinline__ u32x4 part(int d) const {
    const float s = mx_scale(b);
    if (FMT == LQ_MX_FP8) return mx8_bf16(w[d >> 1][2 * (d & 1)], w[d >> 1][2 * (d & 1) + 1], s);
    return mx4_bf16(w[0][d], s);
  }
};

namespace dispatch {

int mx_quantize(const void* X, lq_dtype xdt, int64_t rows, int64_t cols, int32_t fmt,
                uint8_t* codes, uint8_t* scales, hipStream_t st);
int mx_dequantize(const lq_mx_tensor& q, void* out, lq_dtype odt, hipStream_t st);

// T = X A^T (M x r float32) from an MX tensor.
int mx_shrink(const lq_mx_tensor& X, const void* A, int64_t r, float* T, hipStream_t st);
// U = dY B (M x r float32) from bf16 dY and B (N x r); Bt: N r bf16 of scratch.
int mx_u(const void* dY, int64_t M, int64_t N, const void* B, int64_t r, void* Bt, float* U,
         hipStream_t st);

// Y = X W^T + s T B^T, X and W MX tensors (W MXFP4); T M x r float32 or r = 0.
// part: mx_gemm_ws_bytes bytes.
size_t mx_gemm_ws_bytes(int64_t M, int64_t N, int64_t K);
int mx_gemm(const lq_mx_tensor& X, const lq_mx_tensor& W, const float* T, const void* B,
            int64_t r, float s, void* Y, void* part, hipStream_t st);

// out (bf16, n values, n % 8 == 0) = the splits' float32 partial sums, each of
// n values, added in order
int mx_sum_splits(const float* part, void* out, int64_t n, int splits, hipStream_t st);

// dX = dY W + s U A (bf16, M x K; W MXFP4, U = dY B M x r float32); part:
// mx_dx_ws_bytes bytes.
size_t mx_dx_ws_bytes(int64_t M, int64_t N, int64_t K);
int mx_dx(const void* dY, int64_t M, const lq_mx_tensor& W, const float* U, const void* A,
          int64_t r, float s, void* dX, void* part, hipStream_t st);

// The same with a dense bf16 W (N, K <= 65536).  mx_dx_fills: not tiles of 64
// rows in one round (too many to split, too few to fill the chip).
bool mx_dx_fills(int64_t M, int64_t N, int64_t K);
int mx_dx_dense(const void* dY, int64_t M, const lq_weight& W, const float* U, const void* A,
                int64_t r, float s, void* dX, void* part, hipStream_t st);

// Few rows (M <= LQ_MX_ROWS_BF16), X bf16: Y = X W^T + s (X A^T) B^T, W
// streamed once per 16 rows.  Tp: mx_stream_ws_bytes bytes of partial sums.
size_t mx_stream_ws_bytes(int64_t M, int64_t K, int64_t r);
int mx_stream_fwd(const void* X, int64_t M, const lq_mx_tensor& W, const void* A, const void* B,
                  int64_t r, float s, void* Y, float* T_out, float* Tp, hipStream_t st);

// dA = s U^T X, dB = s dY^T T (float32; X an MX tensor; U, T M x r float32),
// in a fixed order; part: mx_grad_bytes bytes.
size_t mx_grad_bytes(int64_t M, int64_t N, int64_t K, int64_t r);
int mx_grads(const lq_mx_tensor& X, const float* U, const void* dY, const float* T, int64_t N,
             int64_t r, float s, int accumulate, float* dA, float* dB, void* part,
             hipStream_t st);

// dX of a dense or NF4 layer by whichever path the shape, the weight and the
// workspace (big_ws, or NULL) select (lora_grad.hip).  U: M x r float32
// scratch, which receives U = dY B on the paths that form it there; U_out: the
// same buffer (U is then written on every path) or NULL.
int bf16_dx_any(const void* dY, int64_t M, const lq_weight& W, const void* A, const void* B,
                int64_t r, float s, void* dX, float* U, float* U_out, void* big_ws,
                hipStream_t st);

}  // namespace dispatch

// Workspace of the backward from an MX checkpoint: [U][T][B transposed]
// [gradient partials], then the dX path's own part.  Without dA and dB no T and
// no partials.
struct MxBwdWs {
  size_t u, t, bt, part, rest;  // byte offsets; rest: the end
};
inline MxBwdWs mx_bwd_ws(int64_t M, int64_t N, int64_t K, int64_t r, bool grads) {
  auto up = [](size_t b) { return (b + 255) & ~(size_t)255; };
  MxBwdWs w;
  w.u = 0;
  w.t = up((size_t)(M * r) * 4);
  w.bt = w.t + (grads ? up((size_t)(M * r) * 4) : 0);
  w.part = w.bt + up((size_t)(N * r) * 2);
  w.rest = w.part + (grads ? up(dispatch::mx_grad_bytes(M, N, K, r)) : 0);
  return w;
}

// Argument checks of an MX tensor operand (sets the error): its format among
// ``formats`` (bit mask of LQ_MX_*), its shape, its buffers.
int mx_check_tensor(const lq_mx_tensor* q, const char* name, int32_t formats, int64_t rows,
                    int64_t cols);
// ... of the pointers the product kernels read or write with 16-byte accesses
int mx_check_aligned(const void* p, const char* name);

}  // namespace lq
