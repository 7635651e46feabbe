// Forward of few rows (M <= 64, bf16 activations) on an MXFP4 base.
//
//   Y = X W^T + s T B^T,  T = X A^T
//
// Few rows are bound by streaming W (4.25 bits per weight).  A workgroup owns
// 16 output rows n; lane (q, l16) of wave w takes row n0 + l16 and the blocks
// 4 t + q, t = w, w + waves, ...: 16 code bytes and one scale byte, turned into
// 32 bf16 weights by 16 conversion instructions and multiplied by four
// v_mfma_f32_16x16x32_bf16 (X padded to 16 rows; the 32 reduction elements of
// a lane are relabelled so that they are contiguous on both operands).
#include "dispatch.h"
#include "mx.h"

namespace lq {
namespace {

constexpr int kWaves = 16;   // stream kernel
constexpr int kTP = 16;      // partial sums of T (workgroups of the T kernel per 16 rows)

// ------------------------------------------------ T of few bf16 rows
// Workgroup (b, chunk): columns [b K / kTP ..) of the chunk's 16 rows, its
// four waves each a part; partial sums to Tp[chunk][b][16][r].
template <int JT>
__global__ __launch_bounds__(256) void mx_tpart_kernel(const uint16_t* __restrict__ X, int64_t M,
                                                       int64_t K, const uint16_t* __restrict__ A,
                                                       int r, float* __restrict__ Tp) {
  __shared__ f32x4 part[4][JT][64];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int l16 = lane & 15, q = lane >> 4;
  const int64_t m0 = 16 * (int64_t)blockIdx.y;
  int64_t m = m0 + l16;
  m = m < M ? m : M - 1;
  const int64_t G = K / 32;  // 32-wide groups, dealt round robin to the 4 kTP waves
  f32x4 acc[JT];
#pragma unroll
  for (int j = 0; j < JT; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int64_t g = (int64_t)blockIdx.x * 4 + wave; g < G; g += 4 * kTP) {
    const int64_t k = 32 * g + 8 * q;
    const u32x4 xf = *reinterpret_cast<const u32x4*>(X + m * K + k);
    u32x4 af[JT];
#pragma unroll
    for (int j = 0; j < JT; ++j) {
      const int row = 16 * j + l16 < r ? 16 * j + l16 : r - 1;
      af[j] = *reinterpret_cast<const u32x4*>(A + (int64_t)row * K + k);
    }
#pragma unroll
    for (int j = 0; j < JT; ++j) acc[j] = mfma16(xf, af[j], acc[j]);
  }
#pragma unroll
  for (int j = 0; j < JT; ++j) part[wave][j][lane] = acc[j];
  __syncthreads();
  if (wave) return;
  float* o = Tp + ((int64_t)blockIdx.y * kTP + blockIdx.x) * 16 * r;
#pragma unroll
  for (int j = 0; j < JT; ++j) {
    const f32x4 a = part[0][j][lane], b = part[1][j][lane], c = part[2][j][lane],
                d = part[3][j][lane];
    const int col = 16 * j + l16;
    if (col < r) {
#pragma unroll
      for (int i = 0; i < 4; ++i) o[(4 * q + i) * r + col] = (a[i] + b[i]) + (c[i] + d[i]);
    }
  }
}

// ------------------------------------------------------- the weight stream
struct StreamParams {
  const uint16_t* X;  // M x K
  int64_t M, N, K;
  const uint8_t* codes;   // N x K / 2
  const uint8_t* scales;  // N x K / 32
  const float* Tp;        // [chunk][kTP][16][r]
  const uint16_t* B;      // N x r
  float* T_out;           // M x r or NULL (written by the chunk's workgroup 0)
  int32_t r;
  float s;
  uint16_t* Y;
};

// XS: bf16 elements of X staged in LDS (rows of K, 16-byte chunk c of row m at
// c ^ (m & 15) when K % 128 == 0); 0: X read from global memory.
template <int XS>
__global__ __launch_bounds__(64 * kWaves) void mx_stream_kernel(StreamParams p) {
  constexpr int NT = 64 * kWaves;
  constexpr int CH = 2;
  __shared__ __attribute__((aligned(16))) uint16_t xs[XS > 0 ? XS : 8];
  __shared__ f32x4 part[kWaves][64];
  __shared__ float tT[16 * 64];
  __shared__ float tB[16 * 64];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int l16 = lane & 15, q = lane >> 4;
  const int64_t m0 = 16 * (int64_t)blockIdx.y;
  const int M = (int)(p.M - m0 < 16 ? p.M - m0 : 16);
  const int64_t N = p.N, K = p.K;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int r = p.r;
  const uint16_t* X = p.X + m0 * K;

  const int64_t n = n0 + l16;  // N % 16 == 0
  const bool mrow = l16 < M;
  const int64_t xm = mrow ? l16 : 0;
  const int64_t G = K / 32;
  const int64_t steps = (G + 3) / 4;
  f32x4 acc[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  MxBlock<LQ_MX_FP4> w[CH];
  bool ok[CH];
  int64_t kb[CH];
  auto load = [&](int64_t base) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int64_t g = 4 * (base + kWaves * i) + q;
      ok[i] = g < G;
      kb[i] = ok[i] ? g : 0;
      w[i].load(p.codes + n * (K / 2) + 16 * kb[i], p.scales + n * (K / 32) + kb[i]);
    }
  };
  load(wave);
  if (XS > 0) {
    const int64_t nxc = M * K / 8, rowc = K / 8;
    for (int64_t c = tid; c < nxc; c += NT) {
      const int64_t m = c / rowc, ch = c - m * rowc;
      *reinterpret_cast<u32x4*>(xs + m * K + 8 * (ch ^ (m & 15))) =
          *reinterpret_cast<const u32x4*>(X + 8 * c);
    }
  }
  // inputs of the expand
  for (int e = tid; e < M * r; e += NT) {
    const float* t = p.Tp + (int64_t)blockIdx.y * kTP * 16 * r + e;
    float v = 0.0f;
#pragma unroll
    for (int b = 0; b < kTP; ++b) v += t[b * 16 * r];
    const int m = e / r, j = e - m * r;
    tT[m * 64 + j] = v;
    if (p.T_out && blockIdx.x == 0) p.T_out[m0 * r + e] = v;
  }
  for (int e = tid; e < 16 * r; e += NT) {
    const int nn = e / r, j = e - nn * r;
    tB[nn * 64 + j] = bf16_to_f32(p.B[n0 * r + e]);
  }
  __syncthreads();
  for (int64_t base = wave; base < steps; base += kWaves * CH) {
    if (base != wave) load(base);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      u32x4 xf[4];
#pragma unroll
      for (int d = 0; d < 4; ++d)
        xf[d] = XS > 0 ? *reinterpret_cast<const u32x4*>(xs + xm * K + 8 * ((4 * kb[i] + d) ^ (xm & 15)))
                       : *reinterpret_cast<const u32x4*>(X + xm * K + 32 * kb[i] + 8 * d);
#pragma unroll
      for (int d = 0; d < 4; ++d)
        acc[i] = mfma16(sel4(ok[i], w[i].part(d)), sel4(ok[i] && mrow, xf[d]), acc[i]);
    }
  }
#pragma unroll
  for (int v = 0; v < 4; ++v) acc[0][v] += acc[1][v];
  part[wave][lane] = acc[0];
  __syncthreads();
  if (wave != 0) return;
  f32x4 sum = part[0][lane];
#pragma unroll
  for (int wv = 1; wv < kWaves; ++wv) {
    const f32x4 o = part[wv][lane];
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] += o[i];
  }
  if (!mrow) return;
  float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int j = 0; j < r; ++j) {
    const float t = tT[l16 * 64 + j];
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = fmaf(t, tB[(4 * q + i) * 64 + j], d[i]);
  }
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = r ? sum[i] + p.s * d[i] : sum[i];
  *reinterpret_cast<u32x2*>(p.Y + (m0 + l16) * N + n0 + 4 * q) =
      u32x2{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
}

}  // namespace

namespace dispatch {

size_t mx_stream_ws_bytes(int64_t M, int64_t K, int64_t r) {
  (void)K;
  return (size_t)(cdiv(M, 16) * kTP * 16 * r) * 4;
}

int mx_stream_fwd(const void* X, int64_t M, const lq_mx_tensor& W, const void* A, const void* B,
                  int64_t r, float s, void* Y, float* T_out, float* Tp, hipStream_t st) {
  const int64_t K = W.cols;
  const unsigned chunks = (unsigned)cdiv(M, 16);
  if (r) {
    const dim3 grid(kTP, chunks), block(256);
    const uint16_t *x = (const uint16_t*)X, *a = (const uint16_t*)A;
    if (r <= 16)
      hipLaunchKernelGGL(mx_tpart_kernel<1>, grid, block, 0, st, x, M, K, a, (int)r, Tp);
    else if (r <= 32)
      hipLaunchKernelGGL(mx_tpart_kernel<2>, grid, block, 0, st, x, M, K, a, (int)r, Tp);
    else
      hipLaunchKernelGGL(mx_tpart_kernel<4>, grid, block, 0, st, x, M, K, a, (int)r, Tp);
    const int e = hip_fail(hipGetLastError(), "mx_tpart launch");
    if (e) return e;
  }
  StreamParams p;
  p.X = (const uint16_t*)X;
  p.M = M;
  p.N = W.rows;
  p.K = K;
  p.codes = W.codes;
  p.scales = W.scales;
  p.Tp = Tp;
  p.B = (const uint16_t*)B;
  p.T_out = T_out;
  p.r = (int32_t)r;
  p.s = s;
  p.Y = (uint16_t*)Y;
  const dim3 grid((unsigned)(W.rows / 16), chunks), block(64 * kWaves);
  const int64_t xe = (M < 16 ? M : 16) * K;
  if (K % 128 == 0 && xe <= 16384)
    hipLaunchKernelGGL(mx_stream_kernel<16384>, grid, block, 0, st, p);
  else if (K % 128 == 0 && xe <= 65536)
    hipLaunchKernelGGL(mx_stream_kernel<65536>, grid, block, 0, st, p);
  else
    hipLaunchKernelGGL(mx_stream_kernel<0>, grid, block, 0, st, p);
  return hip_fail(hipGetLastError(), "mx_stream launch");
}

}  // namespace dispatch
}  // namespace lq
