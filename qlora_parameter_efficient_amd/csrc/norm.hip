// Root-mean-square norm of a residual stream, forward and backward
// (lq_rmsnorm_fwd, lq_rmsnorm_bwd).
//
//   H = X + R (rounded),  c = 1 / sqrt(mean(H^2) + eps),  y = H w c
//   dX = c (g - H c^2 mean(g H)) + dH,  g = dY w;   dW = sum_i dY H c
//
// Both are bound by HBM: every element is read once and written once, and a row
// stays in registers between its sums and its stores (past 16384 columns what does
// not fit is read again).  A thread owns units of 16 consecutive columns, so that a
// lane pair holds one block of an MX output and one DPP move completes the block's
// amax, as in the quantiser; y is quantised from its float32 value, never stored
// in between.  Measured: 2048 x 4096 bf16 with residual, y and MXFP8 out 15.5 us (4.8
// TB/s), backward of 8192 x 4096 with dW 50 + 5 us (5.3 TB/s in the first), 777 x
// 4095 float32 to y and MXFP4 11 us, one row of 4096 2.6 us.  (Pieces of 16 bytes, consecutive as the threads are, took 61 us
// against 54 in the backward of 8192 x 4096 and as long in the forward.)
#include "block.h"
#include "mx_unit.h"

namespace lq {
namespace {

// a thread's 16 values of type BF16 ? bf16 : float32 as floats; n < 16: the
// row's last unit, the rest is 0
template <bool BF16>
__device__ __forceinline__ void load_unit(const void* p, int64_t e, int n, float (&x)[16]) {
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

template <bool BF16>
__device__ __forceinline__ void store_unit(void* p, int64_t e, int n, const float (&x)[16]) {
  if constexpr (BF16) {
    uint16_t* d = (uint16_t*)p + e;
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
    float* d = (float*)p + e;
    if (n >= 16) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        reinterpret_cast<f32x4_a4*>(d)[i] =
            f32x4{x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]};
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < n) d[i] = x[i];
    }
  }
}

__device__ __forceinline__ void load_gain(const void* W, bool bf16, int c, int n, float (&w)[16]) {
  if (bf16)
    load_unit<true>(W, c, n, w);
  else
    load_unit<false>(W, c, n, w);
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
  __shared__ float scratch[16];
  const int t = threadIdx.x % TPR, K = p.K;
  const int64_t kp = mx_spitch(K) * kMxB;
  const float inv_k = 1.0f / (float)K;
  for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; row < p.M;
       row += (int64_t)gridDim.x * RPB) {
    float h[U][16], w[KEEP ? U : 1][16], s[1] = {0.0f};
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = 16 * (t + TPR * u), n = K - c;
      if (n <= 0) {
#pragma unroll
        for (int i = 0; i < 16; ++i) h[u][i] = 0.0f;
        continue;
      }
      const int64_t e = row * K + c;
      load_unit<BF16>(p.X, e, n, h[u]);
      if (KEEP) load_gain(p.W, p.wbf16, c, n, w[KEEP ? u : 0]);
      if (p.R) {
        float r[16];
        load_unit<BF16>(p.R, e, n, r);
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
      const int col = 16 * (t + TPR * u), n = K - col;
      const int64_t e = row * K + col;
      if (n > 0 && p.H) store_unit<BF16>(p.H, e, n, h[u]);
      float y[16];
      if (!KEEP && n > 0) load_gain(p.W, p.wbf16, col, n, w[0]);
#pragma unroll
      for (int i = 0; i < 16; ++i) y[i] = h[u][i] * c * w[KEEP ? u : 0][i];
      if (n > 0 && p.Y) store_unit<BF16>(p.Y, e, n, y);
      if constexpr (FMT != 0) {
        // both units of a block are in one lane pair; one past the row's end is
        // padding (a short row's second unit: zeros)
        if (col < kp) {
          Unit<false> q;
#pragma unroll
          for (int i = 0; i < 16; ++i) q.v[i >> 2][i & 3] = i < n ? y[i] : 0.0f;
          const uint32_t b = scale_byte<FMT>(pair_max(q.amax()));
          const float sc = mx_scale(b);
          const int64_t un = (row * kp + col) >> 4;
          if constexpr (FMT == LQ_MX_FP8) {
            *reinterpret_cast<u32x4*>(p.codes + 16 * un) = sel4(b != 255u, q.fp8(sc));
          } else {
            u32x2 o = q.fp4(sc);
            if (b == 255u) o = u32x2{0u, 0u};
            *reinterpret_cast<u32x2*>(p.codes + 8 * un) = o;
          }
          if (!(un & 1)) p.scales[un >> 1] = (uint8_t)b;
        }
      }
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
  __shared__ float scratch[32];
  const int t = threadIdx.x % TPR, K = p.K;
  const float inv_k = 1.0f / (float)K;
  float w[UK][16], dw[U][16];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = 16 * (t + TPR * u), n = K - c;
#pragma unroll
    for (int i = 0; i < 16; ++i) dw[u][i] = 0.0f;
    if (KEEP) {
#pragma unroll
      for (int i = 0; i < 16; ++i) w[KEEP ? u : 0][i] = 0.0f;
      if (n > 0) load_gain(p.W, p.wbf16, c, n, w[KEEP ? u : 0]);
    }
  }
  for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; row < p.M;
       row += (int64_t)gridDim.x * RPB) {
    float h[UK][16], d[UK][16], s[2] = {0.0f, 0.0f};
    auto load = [&](int k, int c, int n) {
      load_unit<BF16>(p.X, row * K + c, n, h[k]);
      load_unit<BF16>(p.dY, row * K + c, n, d[k]);
      if (!KEEP) load_gain(p.W, p.wbf16, c, n, w[k]);
    };
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = 16 * (t + TPR * u), n = K - c, k = KEEP ? u : 0;
      if (n <= 0) {
        if (KEEP)
#pragma unroll
          for (int i = 0; i < 16; ++i) h[k][i] = d[k][i] = 0.0f;
        continue;
      }
      load(k, c, n);
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
      const int col = 16 * (t + TPR * u), n = K - col, k = KEEP ? u : 0;
      if (n <= 0) continue;
      const int64_t e = row * K + col;
      if (!KEEP) load(k, col, n);
      if (p.part)
#pragma unroll
        for (int i = 0; i < 16; ++i) dw[u][i] += d[k][i] * (h[k][i] * c);
      if (p.H) {
        float g[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) g[i] = c * (d[k][i] * w[k][i] - h[k][i] * m);
        if (p.R) {
          float r[16];
          load_unit<BF16>(p.R, e, n, r);
#pragma unroll
          for (int i = 0; i < 16; ++i) g[i] += r[i];
        }
        store_unit<BF16>(p.H, e, n, g);
      }
    }
  }
  if (!p.part) return;
  // one row of partial sums per row group of the workgroup
  float* out = p.part + ((int64_t)blockIdx.x * RPB + threadIdx.x / TPR) * K;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = 16 * (t + TPR * u), n = K - c;
    if (n > 0) store_unit<false>(out, c, n, dw[u]);
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

// backward: few enough that dW's partial sums stay small
unsigned bwd_grid(int64_t M, int64_t K) {
  const int64_t b = cdiv(M, rows_per_block(K)), most = norm_shape(K) >= 3 ? 256 : 1024;
  return (unsigned)(b < most ? b : most);
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

size_t rmsnorm_part_bytes(int64_t M, int64_t K) {
  return (size_t)bwd_grid(M, K) * rows_per_block(K) * (size_t)K * 4;
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
