// MX quantiser and dequantiser: one power-of-two scale per 32 columns of a
// row, elements E4M3 or E2M1.
//
//   e = min { e in [-127, 127] : amax <= largest 2^e },  code = RNE(x 2^-e)
//
// The scale byte comes from amax's bits: with amax = 1.f 2^(E - 127),
// largest = 1.75 2^8 (E4M3) or 1.5 2^2 (E2M1), b = E - 8 (or 2), plus one
// where the fraction exceeds that of the largest element, never below 0.
//
// Both kernels are bound by HBM.  Quantiser: a thread owns half a block (16
// columns), so a lane pair shares a block and one DPP move completes its amax;
// codes leave as one 16-byte (FP8) or 8-byte (FP4) store per thread (with one
// 16-byte load a thread, consecutive as below, it takes the same 51 us, and
// float32 8.1 against 7.6).
// Dequantiser: a thread owns two 16-byte pieces of the output, consecutive
// lanes consecutive pieces (with 16 float32 of a row per thread, four stores 64
// bytes apart, 2049 x 4095 to float32 took 15 us).  A tensor whose rows hold
// whole blocks is one flat run; other widths locate each piece's row and
// handle the row's end element by element.  Measured: 8192 x 11008 bf16 to E4M3 51
// us (5.3 TB/s of reads and writes) and back 40 (6.9; tensors this size half
// stay in the last-level cache); 2049 x 4095 float32 to E2M1 7.6 us and back 8.3;
// 16 x 4096 2.2 us each, a launch.
#include "dispatch.h"
#include "mx_unit.h"

namespace lq {
namespace {

constexpr int kThreads = 256;

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

// Output elements of a piece (16 bytes), pieces of a thread
template <bool BF16>
struct Piece {
  static constexpr int E = BF16 ? 8 : 4;
  static constexpr int N = 2;
};

// the E codes of a piece: FP8 8 or 4 bytes, FP4 4 or 2
template <int BYTES>
__device__ __forceinline__ u32x2 load_codes(const uint8_t* p) {
  if (BYTES == 8) return *reinterpret_cast<const u32x2*>(p);
  return u32x2{BYTES == 4 ? *reinterpret_cast<const uint32_t*>(p)
                          : (uint32_t)*reinterpret_cast<const uint16_t*>(p), 0u};
}

// pieces = rows kp / E; FLAT: cols % 32 == 0, so piece u starts at element E u
template <bool BF16, int FMT, bool FLAT>
__global__ __launch_bounds__(kThreads) void mx_dequantize_kernel(
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t pieces,
    int64_t cols, int64_t per_row, void* __restrict__ out) {
  constexpr int E = Piece<BF16>::E, PN = Piece<BF16>::N, CB = E * FMT / 8;
  const int64_t u0 = (blockIdx.x + (int64_t)blockIdx.y * gridDim.x) * (kThreads * PN) + threadIdx.x;
  u32x2 w[PN];
  uint32_t b[PN];
#pragma unroll
  for (int i = 0; i < PN; ++i) {
    int64_t u = u0 + kThreads * i;
    u = u < pieces ? u : pieces - 1;
    w[i] = load_codes<CB>(codes + CB * u);
    b[i] = scales[u / (32 / E)];
  }
#pragma unroll
  for (int i = 0; i < PN; ++i) {
    const int64_t u = u0 + kThreads * i;
    if (u >= pieces) break;
    const float s = mx_scale(b[i]);
    int64_t e = E * u, left = E;
    if (!FLAT) {
      // (the division in 32 bits where the tensor allows: a few instructions)
      const int64_t row = (pieces >> 32) == 0 ? (int64_t)((uint32_t)u / (uint32_t)per_row) : u / per_row;
      const int64_t c = (u - row * per_row) * E;
      e = row * cols + c;
      left = cols - c;
    }
    if (BF16) {
      const u32x4 o = FMT == LQ_MX_FP8 ? mx8_bf16(w[i][0], w[i][1], s) : mx4_bf16(w[i][0], s);
      uint16_t* dst = (uint16_t*)out + e;
      if (FLAT || left >= E) {
        *reinterpret_cast<u32x4_a2*>(dst) = o;
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < left) dst[k] = (uint16_t)(o[k >> 1] >> (16 * (k & 1)));
      }
    } else {
      f32x2v lo, hi;
      if (FMT == LQ_MX_FP8) {
        lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[i][0], s, false);
        hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[i][0], s, true);
      } else {
        lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i][0], s, 0);
        hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i][0], s, 1);
      }
      const f32x4 o = f32x4{lo[0], lo[1], hi[0], hi[1]};
      float* dst = (float*)out + e;
      if (FLAT || left >= E) {
        *reinterpret_cast<f32x4_a4*>(dst) = o;
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (k < left) dst[k] = o[k];
      }
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
  using P = Piece<BF16>;
  const int64_t per_row = cdiv(q.cols, kMxB) * (kMxB / P::E), pieces = q.rows * per_row;
  // 2^35 elements to float32 take 2^32 threads, one more than a launch's first
  // dimension may hold
  const int64_t blocks = cdiv(pieces, kThreads * P::N), wide = (int64_t)1 << 22;
  const dim3 grid((unsigned)(blocks < wide ? blocks : wide), (unsigned)cdiv(blocks, wide));
  const dim3 block(kThreads);
  if (q.cols % kMxB == 0)
    hipLaunchKernelGGL((mx_dequantize_kernel<BF16, FMT, true>), grid, block, 0, st, q.codes,
                       q.scales, pieces, q.cols, per_row, out);
  else
    hipLaunchKernelGGL((mx_dequantize_kernel<BF16, FMT, false>), grid, block, 0, st, q.codes,
                       q.scales, pieces, q.cols, per_row, out);
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
