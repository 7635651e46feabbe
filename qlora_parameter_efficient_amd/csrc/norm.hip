// Root-mean-square norm of a residual stream, forward and backward
// (lq_rmsnorm_fwd, lq_rmsnorm_bwd).
//
//   H = X + R (rounded),  c = 1 / sqrt(mean(H^2) + eps),  y = H w c
//   dX = c (g - H c^2 mean(g H)) + dH,  g = dY w;   dW = sum_i dY H c
//
// Both are bound by HBM: every element is read once and written once, and a row
// stays in registers between its sums and its stores (past 16384 columns what does
// not fit is read again).  A thread owns 16 columns of a row at a time, so that a lane
// pair, or eight lanes, hold one block of an MX output and a few DPP moves complete
// the block's amax; y is quantised from its float32 value, never stored in between.
// Measured: 2048 x 4096 bf16 with residual, y and MXFP8 out 15.8 us (4.7 TB/s),
// backward of 8192 x 4096 with dW 50 + 5 us (5.3 TB/s in the first), 777 x 4095
// float32 to y and MXFP4 8.4 us, one row of 4096 2.6 us.
#include <type_traits>

#include "block.h"
#include "mx_unit.h"

namespace lq {
namespace {

typedef u32x2 u32x2_a2 __attribute__((aligned(2)));

// Which columns a thread's unit u is.  LONG (bf16 rows, and rows that are read
// twice): 16 in a run.  Else (float32 rows up to 16384): four runs of 4, consecutive
// as the threads are, since runs of 64 bytes make each of their four loads touch
// every line that the wave has (us, long runs / short: float32 forward 2048 x 4096
// 32 / 21, 4096 x 11008 161 / 132, 777 x 4095 16.2 / 10.4, backward 2048 x 4096 29 /
// 24, but 1000 x 30000 forward 140 / 167 and backward 146 / 173; bf16 in runs of 4:
// forward 2048 x 4096 with MX output 15.8 / 18.7, backward 8192 x 4096 50 / 78).
template <bool LONG, int TPR>
struct Cols {
  static constexpr int kRun = LONG ? 16 : 4, kRuns = 16 / kRun;
  // first column of run k
  static __device__ __forceinline__ int at(int t, int u, int k = 0) {
    return kRun * (t + TPR * (kRuns * u + k));
  }
};

// n (some: 1 to 15) of 16 consecutive values at e as floats, zeros past them
template <bool BF16>
__device__ __forceinline__ void load_run(const void* p, int64_t e, int n, float* x, std::integral_constant<int, 16>) {
  Unit<BF16> u;
  if (n >= 16)
    u.load(p, e);
  else
    u.load_some(p, e, n);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if constexpr (BF16) {
      const uint32_t w = u.v[i >> 3][(i >> 1) & 3];
      x[i] = i & 1 ? hi_bf16(w) : lo_bf16(w);
    } else {
      x[i] = u.v[i >> 2][i & 3];
    }
  }
}
// ... of four
template <bool BF16>
__device__ __forceinline__ void load_run(const void* p, int64_t e, int n, float* x, std::integral_constant<int, 4>) {
  if (n >= 4) {
    if constexpr (BF16) {
      const u32x2 w = *reinterpret_cast<const u32x2_a2*>((const uint16_t*)p + e);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = i & 1 ? hi_bf16(w[i >> 1]) : lo_bf16(w[i >> 1]);
    } else {
      const f32x4 v = *reinterpret_cast<const f32x4_a4*>((const float*)p + e);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = v[i];
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = 0.0f;
    if (i < n)
      x[i] = BF16 ? bf16_to_f32(((const uint16_t*)p)[e + i]) : ((const float*)p)[e + i];
  }
}

// a thread's unit u of the row of K values of type EB ? bf16 : float32 at e
template <bool EB, bool LONG, int TPR>
__device__ __forceinline__ void load_unit(const void* p, int64_t e, int K, int t, int u, float (&x)[16]) {
  using C = Cols<LONG, TPR>;
#pragma unroll
  for (int k = 0; k < C::kRuns; ++k) {
    const int c = C::at(t, u, k);
    load_run<EB>(p, e + c, K - c, x + C::kRun * k, std::integral_constant<int, C::kRun>{});
  }
}

template <bool EB, bool LONG, int TPR>
__device__ __forceinline__ void store_unit(void* p, int64_t row, int K, int t, int u, const float (&x)[16]) {
  using C = Cols<LONG, TPR>;
  if constexpr (EB) {
    static_assert(LONG, "bf16 rows are stored in long runs");
    const int c = C::at(t, u), n = K - c;
    uint16_t* d = (uint16_t*)p + row + c;
    u32x4 v[2];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i >> 2][i & 3] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    if (n >= 16) {
      reinterpret_cast<u32x4_a2*>(d)[0] = v[0];
      reinterpret_cast<u32x4_a2*>(d)[1] = v[1];
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < n) d[i] = (uint16_t)(v[i >> 3][(i >> 1) & 3] >> (16 * (i & 1)));
    }
  } else {
#pragma unroll
    for (int k = 0; k < C::kRuns; ++k) {
      const int c = C::at(t, u, k), n = K - c;
      float* d = (float*)p + row + c;
      const float* v = x + C::kRun * k;
      if (n >= C::kRun) {
#pragma unroll
        for (int i = 0; i < C::kRun / 4; ++i)
          reinterpret_cast<f32x4_a4*>(d)[i] = f32x4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
      } else {
#pragma unroll
        for (int i = 0; i < C::kRun; ++i)
          if (i < n) d[i] = v[i];
      }
    }
  }
}

template <bool LONG, int TPR>
__device__ __forceinline__ void load_gain(const void* W, bool wbf16, int K, int t, int u, float (&w)[16]) {
  if (wbf16)
    load_unit<true, LONG, TPR>(W, 0, K, t, u, w);
  else
    load_unit<false, LONG, TPR>(W, 0, K, t, u, w);
}

// max over eight lanes 8 i .. 8 i + 7
__device__ __forceinline__ uint32_t max8(uint32_t v) {
#define LQ_MAX(ctrl)                                                                       \
  {                                                                                        \
    const uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, ctrl, 0xF, 0xF, false);  \
    v = v > o ? v : o;                                                                     \
  }
  LQ_MAX(0xB1)   // lane ^ 1
  LQ_MAX(0x4E)   // lane ^ 2
  LQ_MAX(0x141)  // mirrored within eight
#undef LQ_MAX
  return v;
}

// codes and scales of a unit; row: its first block's place in elements, kp: the
// row's columns with padding (a lane pair or eight lanes hold one block)
template <int FMT, bool LONG, int TPR>
__device__ __forceinline__ void quantise(const float (&y)[16], int64_t row, int K, int kp, int t, int u,
                                         uint8_t* codes, uint8_t* scales) {
  using C = Cols<LONG, TPR>;
  if constexpr (LONG) {
    // one past the row's end is padding (a short row's second unit: zeros)
    const int col = C::at(t, u), n = K - col;
    if (col >= kp) return;
    Unit<false> q;
#pragma unroll
    for (int i = 0; i < 16; ++i) q.v[i >> 2][i & 3] = i < n ? y[i] : 0.0f;
    const uint32_t b = scale_byte<FMT>(pair_max(q.amax()));
    const float sc = mx_scale(b);
    const int64_t un = (row + col) >> 4;
    if constexpr (FMT == LQ_MX_FP8) {
      *reinterpret_cast<u32x4*>(codes + 16 * un) = sel4(b != 255u, q.fp8(sc));
    } else {
      u32x2 o = q.fp4(sc);
      if (b == 255u) o = u32x2{0u, 0u};
      *reinterpret_cast<u32x2*>(codes + 8 * un) = o;
    }
    if (!(un & 1)) scales[un >> 1] = (uint8_t)b;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int col = C::at(t, u, k), n = K - col;
      if (col >= kp) return;
      float v[4];
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = i < n ? y[4 * k + i] : 0.0f;
        const uint32_t a = __float_as_uint(v[i]) & 0x7FFFFFFFu;
        m = m > a ? m : a;
      }
      const uint32_t b = scale_byte<FMT>(max8(m));
      const float sc = mx_scale(b);
      const int64_t at = row + col;
      if constexpr (FMT == LQ_MX_FP8) {
        s16x2 c = {0, 0};
        c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, v[0], v[1], sc, false);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, v[2], v[3], sc, true);
        *reinterpret_cast<uint32_t*>(codes + at) = b != 255u ? __builtin_bit_cast(uint32_t, c) : 0u;
      } else {
        uint32_t c = 0;
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], sc, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], sc, 1);
        *reinterpret_cast<uint16_t*>(codes + (at >> 1)) = b != 255u ? (uint16_t)c : (uint16_t)0;
      }
      if (!(at & 31)) scales[at >> 5] = (uint8_t)b;
    }
  }
}

// Sum over the TPR threads of a row; scratch: one float per wave of the
// workgroup and value.  Every thread gets the same bits.
template <int TPR, int NV>
__device__ __forceinline__ void row_sum(float (&v)[NV], float* scratch) {
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int o = 32; o; o >>= 1) v[k] += __shfl_xor(v[k], o);
  if (TPR == 64) return;
  constexpr int W = TPR / 64;
  const int wave = threadIdx.x >> 6;
  __syncthreads();  // the scratch of the row before is read
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int k = 0; k < NV; ++k) scratch[k * W + wave] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) s += scratch[k * W + i];
    v[k] = s;
  }
}

struct NormParams {
  const void* X;   // forward: X; backward: H
  const void* R;   // forward: R or NULL; backward: dH or NULL
  const void* dY;  // backward
  const void* W;
  void* H;  // forward: H_out or NULL; backward: dX or NULL
  void* Y;
  uint8_t* codes;
  uint8_t* scales;
  const float* rstd_in;
  float* rstd;  // forward: rstd_out or NULL
  float* part;  // backward: partial sums of dW, gridDim.x x K, or NULL
  int64_t M;
  int32_t K, wbf16;
  float eps;
};

// TPR threads per row (64: four rows per workgroup), U units of 16 columns each:
// columns 16 (t + TPR u).  KEEP: the gain stays in registers too.
template <bool BF16, int FMT, int TPR, int U, bool KEEP>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void rmsnorm_fwd_kernel(NormParams p) {
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
  constexpr bool LONG = BF16 || !KEEP;
  using C = Cols<LONG, TPR>;
  __shared__ float scratch[16];
  const int t = threadIdx.x % TPR, K = p.K;
  const int kp = (int)(mx_spitch(K) * kMxB);
  const float inv_k = 1.0f / (float)K;
  for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; row < p.M;
       row += (int64_t)gridDim.x * RPB) {
    float h[U][16], w[KEEP ? U : 1][16], s[1] = {0.0f};
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (C::at(t, u) >= K) {
#pragma unroll
        for (int i = 0; i < 16; ++i) h[u][i] = 0.0f;
        continue;
      }
      load_unit<BF16, LONG, TPR>(p.X, row * K, K, t, u, h[u]);
      if (KEEP) load_gain<LONG, TPR>(p.W, p.wbf16, K, t, u, w[KEEP ? u : 0]);
      if (p.R) {
        float r[16];
        load_unit<BF16, LONG, TPR>(p.R, row * K, K, t, u, r);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          h[u][i] += r[i];
          if (BF16) h[u][i] = bf16_to_f32(f32_to_bf16(h[u][i]));
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) s[0] += h[u][i] * h[u][i];
    }
    row_sum<TPR, 1>(s, scratch);
    const float c = 1.0f / sqrtf(s[0] * inv_k + p.eps);
    if (p.rstd && t == 0) p.rstd[row] = c;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = C::at(t, u) < K;
      if (in && p.H) store_unit<BF16, LONG, TPR>(p.H, row * K, K, t, u, h[u]);
      float y[16];
      if (!KEEP && in) load_gain<LONG, TPR>(p.W, p.wbf16, K, t, u, w[0]);
#pragma unroll
      for (int i = 0; i < 16; ++i) y[i] = h[u][i] * c * w[KEEP ? u : 0][i];
      if (in && p.Y) store_unit<BF16, LONG, TPR>(p.Y, row * K, K, t, u, y);
      if constexpr (FMT != 0) quantise<FMT, LONG, TPR>(y, row * kp, K, kp, t, u, p.codes, p.scales);
    }
  }
}

// Rows blockIdx, blockIdx + gridDim, ...: each thread adds its columns' shares
// of dW over the workgroup's rows in registers; the workgroups' sums are added
// by dw_reduce_kernel.  KEEP: H, dY and the gain stay in registers from the sums
// on.
template <bool BF16, int TPR, int U, bool KEEP>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void rmsnorm_bwd_kernel(NormParams p) {
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1, UK = KEEP ? U : 1;
  constexpr bool LONG = BF16 || !KEEP;
  using C = Cols<LONG, TPR>;
  __shared__ float scratch[32];
  const int t = threadIdx.x % TPR, K = p.K;
  const float inv_k = 1.0f / (float)K;
  float w[UK][16], dw[U][16];
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int i = 0; i < 16; ++i) dw[u][i] = 0.0f;
    if (KEEP) {
#pragma unroll
      for (int i = 0; i < 16; ++i) w[KEEP ? u : 0][i] = 0.0f;
      if (C::at(t, u) < K) load_gain<LONG, TPR>(p.W, p.wbf16, K, t, u, w[KEEP ? u : 0]);
    }
  }
  for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; row < p.M;
       row += (int64_t)gridDim.x * RPB) {
    float h[UK][16], d[UK][16], s[2] = {0.0f, 0.0f};
    auto load = [&](int k, int u) {
      load_unit<BF16, LONG, TPR>(p.X, row * K, K, t, u, h[k]);
      load_unit<BF16, LONG, TPR>(p.dY, row * K, K, t, u, d[k]);
      if (!KEEP) load_gain<LONG, TPR>(p.W, p.wbf16, K, t, u, w[k]);
    };
    // (bf16 rows in turn where they do not fit: the loads of four units at once spill,
    // 1000 x 30000 100 us against 86)
#pragma unroll(BF16 && !KEEP ? 1 : U)
    for (int u = 0; u < U; ++u) {
      const int k = KEEP ? u : 0;
      if (C::at(t, u) >= K) {
        if (KEEP)
#pragma unroll
          for (int i = 0; i < 16; ++i) h[k][i] = d[k][i] = 0.0f;
        continue;
      }
      load(k, u);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[0] += d[k][i] * w[k][i] * h[k][i];
        s[1] += h[k][i] * h[k][i];
      }
    }
    row_sum<TPR, 2>(s, scratch);
    const float c = p.rstd_in ? p.rstd_in[row] : 1.0f / sqrtf(s[1] * inv_k + p.eps);
    const float m = s[0] * inv_k * c * c;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = KEEP ? u : 0;
      if (C::at(t, u) >= K) continue;
      if (!KEEP) load(k, u);
      if (p.part)
#pragma unroll
        for (int i = 0; i < 16; ++i) dw[u][i] += d[k][i] * (h[k][i] * c);
      if (p.H) {
        float g[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) g[i] = c * (d[k][i] * w[k][i] - h[k][i] * m);
        if (p.R) {
          float r[16];
          load_unit<BF16, LONG, TPR>(p.R, row * K, K, t, u, r);
#pragma unroll
          for (int i = 0; i < 16; ++i) g[i] += r[i];
        }
        store_unit<BF16, LONG, TPR>(p.H, row * K, K, t, u, g);
      }
    }
  }
  if (!p.part) return;
  // one row of partial sums per row group of the workgroup
  float* out = p.part + ((int64_t)blockIdx.x * RPB + threadIdx.x / TPR) * K;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (C::at(t, u) < K) store_unit<false, LONG, TPR>(out, 0, K, t, u, dw[u]);
  }
}

// dW[c] (+)= sum of P partial rows: 32 columns per workgroup, 32 groups of rows
// that are added in order, eight loads at a time, and then across the groups
__global__ __launch_bounds__(1024) void dw_reduce_kernel(const float* part, int P, int K, float* dW,
                                                         int accumulate) {
  __shared__ float sum[32][33];
  const int l = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + l;
  float s = 0.0f;
  if (c < K) {
    int i = grp;
    for (; i + 7 * 32 < P; i += 8 * 32) {
      float x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = part[(int64_t)(i + 32 * k) * K + c];
#pragma unroll
      for (int k = 0; k < 8; ++k) s += x[k];
    }
    for (; i < P; i += 32) s += part[(int64_t)i * K + c];
  }
  sum[grp][l] = s;
  __syncthreads();
  if (grp || c >= K) return;
#pragma unroll
  for (int i = 1; i < 32; ++i) s += sum[i][l];
  dW[c] = accumulate ? dW[c] + s : s;
}

// threads per row and units per thread by the row's length
int norm_shape(int64_t K) { return K <= 1024 ? 0 : K <= 4096 ? 1 : K <= 8192 ? 2 : K <= 16384 ? 3 : 4; }
int rows_per_block(int64_t K) { return norm_shape(K) == 0 ? 4 : 1; }

// workgroups: one per row (or four) up to what a launch's first dimension holds
unsigned fwd_grid(int64_t M, int64_t K) {
  const int64_t b = cdiv(M, rows_per_block(K));
  return (unsigned)(b < (1 << 20) ? b : 1 << 20);
}

// Backward: about what the chip holds at once, so that dW's partial sums, one row of
// them for each row at work, stay few (us, 1024 workgroups / so many: 8192 x 1024 27 /
// 21, 8192 x 4096 56.4 / 54.8, 8192 x 8192 111 / 105, 1024 x 8192 30 / 21; with half
// as many 22, 72, 116 for the first three); a number that leaves a second row to a few
// is evened out (777 x 4095 float32 18.8 / 16.7), of many rows not (8192 x 4096 54.8 /
// 56.9)
int64_t bwd_most(int64_t K) {
  const int shape = norm_shape(K);
  return shape == 1 ? 768 : shape >= 3 ? 256 : 512;
}
unsigned bwd_grid(int64_t M, int64_t K) {
  const int64_t b = cdiv(M, rows_per_block(K)), most = bwd_most(K);
  return (unsigned)(b < 2 * most ? cdiv(b, cdiv(b, most)) : most);
}

template <bool BF16, int FMT>
void launch_fwd(const NormParams& p, hipStream_t st) {
  const dim3 g(fwd_grid(p.M, p.K));
  switch (norm_shape(p.K)) {
    case 0: hipLaunchKernelGGL((rmsnorm_fwd_kernel<BF16, FMT, 64, 1, true>), g, dim3(256), 0, st, p); break;
    case 1: hipLaunchKernelGGL((rmsnorm_fwd_kernel<BF16, FMT, 256, 1, true>), g, dim3(256), 0, st, p); break;
    case 2: hipLaunchKernelGGL((rmsnorm_fwd_kernel<BF16, FMT, 512, 1, true>), g, dim3(512), 0, st, p); break;
    case 3: hipLaunchKernelGGL((rmsnorm_fwd_kernel<BF16, FMT, 1024, 1, true>), g, dim3(1024), 0, st, p); break;
    default: hipLaunchKernelGGL((rmsnorm_fwd_kernel<BF16, FMT, 1024, 4, false>), g, dim3(1024), 0, st, p);
  }
}

template <bool BF16>
void launch_bwd(const NormParams& p, hipStream_t st) {
  const dim3 g(bwd_grid(p.M, p.K));
  switch (norm_shape(p.K)) {
    case 0: hipLaunchKernelGGL((rmsnorm_bwd_kernel<BF16, 64, 1, true>), g, dim3(256), 0, st, p); break;
    case 1: hipLaunchKernelGGL((rmsnorm_bwd_kernel<BF16, 256, 1, true>), g, dim3(256), 0, st, p); break;
    case 2: hipLaunchKernelGGL((rmsnorm_bwd_kernel<BF16, 512, 1, true>), g, dim3(512), 0, st, p); break;
    case 3: hipLaunchKernelGGL((rmsnorm_bwd_kernel<BF16, 1024, 1, true>), g, dim3(1024), 0, st, p); break;
    default: hipLaunchKernelGGL((rmsnorm_bwd_kernel<BF16, 1024, 4, false>), g, dim3(1024), 0, st, p);
  }
}

}  // namespace

namespace dispatch {

// (for M rows or fewer: an evened-out grid may be smaller than that of fewer rows)
size_t rmsnorm_part_bytes(int64_t M, int64_t K) {
  const int64_t b = cdiv(M, rows_per_block(K)), most = bwd_most(K);
  return (size_t)(b < most ? b : most) * rows_per_block(K) * (size_t)K * 4;
}

int rmsnorm_fwd(const void* X, const void* R, int64_t M, int64_t K, lq_dtype dt, const void* W,
                lq_dtype wdt, float eps, void* H, void* Y, int32_t fmt, uint8_t* codes,
                uint8_t* scales, float* rstd, hipStream_t st) {
  NormParams p{};
  p.X = X;
  p.R = R;
  p.W = W;
  p.H = H;
  p.Y = Y;
  p.codes = codes;
  p.scales = scales;
  p.rstd = rstd;
  p.M = M;
  p.K = (int32_t)K;
  p.wbf16 = wdt == LQ_BF16;
  p.eps = eps;
  const bool b = dt == LQ_BF16;
  if (!codes)
    b ? launch_fwd<true, 0>(p, st) : launch_fwd<false, 0>(p, st);
  else if (fmt == LQ_MX_FP8)
    b ? launch_fwd<true, LQ_MX_FP8>(p, st) : launch_fwd<false, LQ_MX_FP8>(p, st);
  else
    b ? launch_fwd<true, LQ_MX_FP4>(p, st) : launch_fwd<false, LQ_MX_FP4>(p, st);
  return hip_fail(hipGetLastError(), "rmsnorm_fwd launch");
}

int rmsnorm_bwd(const void* dY, const void* H, int64_t M, int64_t K, lq_dtype dt, const void* W,
                lq_dtype wdt, float eps, const float* rstd, const void* dH, void* dX, float* dW,
                int accumulate, float* part, hipStream_t st) {
  NormParams p{};
  p.X = H;
  p.R = dH;
  p.dY = dY;
  p.W = W;
  p.H = dX;
  p.rstd_in = rstd;
  p.part = dW ? part : nullptr;
  p.M = M;
  p.K = (int32_t)K;
  p.wbf16 = wdt == LQ_BF16;
  p.eps = eps;
  dt == LQ_BF16 ? launch_bwd<true>(p, st) : launch_bwd<false>(p, st);
  if (dW)
    hipLaunchKernelGGL(dw_reduce_kernel, dim3((unsigned)cdiv(K, 32)), dim3(1024), 0, st, part,
                       (int)(bwd_grid(M, K) * rows_per_block(K)), (int)K, dW, accumulate);
  return hip_fail(hipGetLastError(), "rmsnorm_bwd launch");
}

}  // namespace dispatch
}  // namespace lq
