// Rank-r shrinks of the MX layer, in float32: T = X A^T of an MX tensor X
// (M x K) and U = dY B of a bf16 dY (M x N).
//
// Both are out[m][j] = sum_k Z[m][k] G[j][k] with G r x K row-major.  For U, G
// is B's transpose: where r % 4 == 0 the rows of B (K x r) are staged as they
// lie and read by the transposing ds_read_b64_tr_b16; otherwise a small kernel
// writes the transpose to the workspace first (another launch, 4.7 us).
//
// Bound by the load path (Z from HBM once, r K bf16 of G from L2 per
// workgroup); the products are a few percent of the matrix units' time.  Two
// kernels:
//
// mx_shrink_tile_kernel (U, and T where K % 128 == 0 and the scales lie on
// words: they are read as 4-byte words).  A workgroup of eight waves owns 16 H rows and walks
// the reduction in steps of 256 columns.  The step's Z rows (and scales) and G
// rows go straight from global memory into LDS in whole lines, NST - 1 steps
// ahead; wave w multiplies columns 32 w .. of the step, one
// v_mfma_f32_16x16x32_bf16 per 16 x 16 block of the output (a lane's 8 columns
// of an MX row are converted as they are read).  16-byte chunks are swizzled by
// row so that the 16 rows of a read fall on distinct banks.  M = 2048,
// K = 4096, r = 16: T of an 8-bit X 7.0 us (1.2 TB/s, launch and the pipeline's
// filling included), U 6.0 us (2.8 TB/s); M = 8192, r = 64: U of N = 4096 23.7 us
// (2.8 TB/s), T of a 4-bit X of K = 4096 16.0 (512 KB of A per workgroup from L2).  With few rows a workgroup's steps
// bound it, 0.28 us each (M = 1001, K = 11008: 13.0 us).
//
// mx_shrink_kernel (the rest).  A workgroup owns 16 H rows and deals the
// 128-column steps of the reduction to its waves; lane (q, l16) of a wave takes
// one block of 32 columns of row l16 of each 16-row group with its scale and
// the same columns of row l16 of each 16-rank group of G, the 32 columns of a
// lane relabelled so that they are contiguous.  The next step's loads are
// issued before this step's products.  Each load touches 32 lines, which costs
// twice the tile kernel's time (T at M = 2048, K = 4096, r = 16: 12.5 us).
//
// In both the waves' sums are added in order through LDS.
#include <type_traits>

#include "dispatch.h"
#include "mx_tile.h"

namespace lq {
namespace {

template <int FZ, int JT, int H, int NW>
__global__ __launch_bounds__(64 * NW) void mx_shrink_kernel(const uint8_t* __restrict__ Z,
                                                            const uint8_t* __restrict__ Zs,
                                                            int64_t M, int64_t K,
                                                            const uint16_t* __restrict__ G, int r,
                                                            float* __restrict__ out) {
  __shared__ f32x4 part[NW][H * JT][64];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int l16 = lane & 15, q = lane >> 4;
  const int64_t m0 = 16 * H * (int64_t)blockIdx.x;
  const int blocks = (int)(K / 32), steps = (blocks + 3) / 4;
  const int64_t pitch = K * FZ / 8;
  const uint8_t *zr[H], *sr[H];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    int64_t m = m0 + 16 * h + l16;
    m = m < M ? m : M - 1;
    zr[h] = Z + m * pitch;
    sr[h] = Zs + m * blocks;
  }
  const uint16_t* gr[JT];
#pragma unroll
  for (int j = 0; j < JT; ++j) {
    const int row = 16 * j + l16 < r ? 16 * j + l16 : r - 1;
    gr[j] = G + (int64_t)row * K;
  }
  struct In {
    MxBlock<FZ> z[H];
    u32x4 g[JT][4];
  };
  // a lane whose block is past the row reads block 0 and is masked below
  auto load = [&](int t, In& in) {
    int b = 4 * t + q;
    b = b < blocks ? b : 0;
#pragma unroll
    for (int h = 0; h < H; ++h) in.z[h].load(zr[h] + (int64_t)b * (4 * FZ), sr[h] + b);
#pragma unroll
    for (int j = 0; j < JT; ++j)
#pragma unroll
      for (int d = 0; d < 4; ++d)
        in.g[j][d] = *reinterpret_cast<const u32x4*>(gr[j] + 32 * b + 8 * d);
  };
  f32x4 acc[H][JT];
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int j = 0; j < JT; ++j) acc[h][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  auto products = [&](int t, const In& in) {
    const bool ok = 4 * t + q < blocks;
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const u32x4 zf = sel4(ok, in.z[h].part(d));
#pragma unroll
        for (int j = 0; j < JT; ++j) acc[h][j] = mfma16(zf, sel4(ok, in.g[j][d]), acc[h][j]);
      }
  };
  if (wave < steps) {  // uniform
    In in[2];
    load(wave, in[0]);
    for (int t = wave;; t += 2 * NW) {
      const int t1 = t + NW, t2 = t + 2 * NW;
      load(t1 < steps ? t1 : t, in[1]);
      __builtin_amdgcn_sched_barrier(0);
      products(t, in[0]);
      if (t1 >= steps) break;
      load(t2 < steps ? t2 : t1, in[0]);
      __builtin_amdgcn_sched_barrier(0);
      products(t1, in[1]);
      if (t2 >= steps) break;
    }
  }
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int j = 0; j < JT; ++j) part[wave][h * JT + j][lane] = acc[h][j];
  __syncthreads();
  for (int c = wave; c < H * JT; c += NW) {
    f32x4 s = part[0][c][lane];
#pragma unroll
    for (int w = 1; w < NW; ++w) {
      const f32x4 o = part[w][c][lane];
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] += o[i];
    }
    const int h = c / JT, j = 16 * (c - h * JT) + l16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t m = m0 + 16 * h + 4 * q + i;
      if (m < M && j < r) out[m * r + j] = s[i];
    }
  }
}

// ------------------------------- K % 64 == 0 of bf16 rows, K % 128 == 0 of MX
template <int FZ, int JT, int H>
struct TileShape {
  static constexpr int NW = 8;
  static constexpr int ZRow = 256 * FZ / 8, ZBytes = 16 * H * ZRow;
  static constexpr int GBytes = 16 * JT * 512;
  static constexpr int SBytes = FZ == 16 ? 0 : 256;       // 8 scale bytes a row, 32 rows
  static constexpr int Stage = ZBytes + GBytes + SBytes;
  static constexpr int NST = 4 * Stage <= 80 * 1024 ? 4 : 3;
  static constexpr int Red = NW * H * JT * 64 * 16;       // the waves' sums
  static constexpr int Used = NST * Stage + 1024;         // and a place for spare loads
  static constexpr int Smem = Used > Red ? Used : Red;
  static constexpr int ZI = ZBytes / 1024, ZU = (ZI + NW - 1) / NW;  // loads per step, per wave
  static constexpr int Loads = ZU + JT + (FZ == 16 ? 0 : 1);
};

__device__ __forceinline__ u32x2 shrink_tr(const char* p) {
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) s16x4* lds_ptr;
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p)));
}

// GT: G is given as K x r (r % 4 == 0).  TAIL: K % 256 != 0, the last step ends
// inside its columns (apart, because the checks cost 0.1 us per 256 columns).
template <int FZ, int JT, int H, bool GT, bool TAIL>
__global__ __launch_bounds__(512) void mx_shrink_tile_kernel(const uint8_t* __restrict__ Z,
                                                             const uint8_t* __restrict__ Zs,
                                                             int64_t M, int64_t K,
                                                             const uint16_t* __restrict__ G, int r,
                                                             float* __restrict__ out) {
  using S = TileShape<FZ, JT, H>;
  constexpr int NST = S::NST, ZC = S::ZRow / 16;  // chunks per Z row
  __shared__ __attribute__((aligned(1024))) char smem[S::Smem];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, q = lane >> 4;
  const int64_t m0 = 16 * H * (int64_t)blockIdx.x;
  const int64_t zpitch = K * FZ / 8;
  const int blocks = (int)(K / 32), steps = (blocks + 7) / 8;
  const uint32_t sbase = mx_lds_addr(smem);
  auto zswz = [](int row) { return ZC == 8 ? mx_swz128(row) : row & 15; };

  // load offsets relative to the step; Z load i covers 1024 / ZRow rows, G load
  // i rows 2 i and 2 i + 1, and wave 0 loads the scales.  Every wave makes the
  // same number of loads (its waits count them); a spare one reads one address
  // with all its lanes, into a place of its own.  cols: the step's columns; a
  // lane whose chunk lies past them reads the first chunk again.
  uint32_t goff[JT], zoff[S::ZU], soff = 0;
  int zi[S::ZU];
  auto offsets = [&](uint32_t cols) {
#pragma unroll
    for (int u = 0; u < S::ZU; ++u) {
      zi[u] = wave * S::ZU + u;
      const int row = zi[u] * (1024 / S::ZRow) + lane / ZC;
      int64_t m = m0 + row;
      m = m < M ? m : M - 1;
      const uint32_t at = 16u * ((lane % ZC) ^ zswz(row));
      zoff[u] = zi[u] < S::ZI ? (uint32_t)(m * zpitch) + (at < cols * FZ / 8 ? at : 0u) : 0u;
    }
#pragma unroll
    for (int u = 0; u < JT; ++u) {
      if (GT) {  // the step's 2 r cols bytes in order
        const uint32_t at = (wave * JT + u) * 1024 + lane * 16;
        goff[u] = at < 2 * r * cols ? at : 0u;
      } else {
        const int row = 2 * (wave * JT + u) + (lane >> 5);
        const int j = row < r ? row : r - 1;
        const uint32_t at = 16u * ((lane & 31) ^ (row & 15));
        goff[u] = (uint32_t)((int64_t)j * K * 2) + (at < 2 * cols ? at : 0u);
      }
    }
    if (FZ != 16) {
      int64_t m = m0 + (lane >> 1) % (16 * H);
      m = m < M ? m : M - 1;
      soff = wave == 0 ? (uint32_t)(m * blocks + (cols > 128 ? 4 * (lane & 1) : 0)) : 0u;
    }
  };
  offsets(256);
  const uint32_t spare = sbase + NST * S::Stage;
  auto issue = [&](int t, int b, int go) {
    if (TAIL && go && 8 * t + 8 > blocks) offsets(32 * (blocks - 8 * t));  // the last step's
    const uint32_t st = sbase + b * S::Stage;
#pragma unroll
    for (int u = 0; u < S::ZU; ++u)
      mx_dma16(reinterpret_cast<const char*>(Z) + (int64_t)t * S::ZRow, zoff[u],
               zi[u] < S::ZI ? st + zi[u] * 1024 : spare, go);
#pragma unroll
    for (int u = 0; u < JT; ++u)
      mx_dma16(reinterpret_cast<const char*>(G) + (int64_t)t * 512 * (GT ? r : 1), goff[u],
               st + S::ZBytes + (wave * JT + u) * 1024, go);
    if (FZ != 16)
      mx_dma4(Zs + (int64_t)t * 8, soff, wave == 0 ? st + S::ZBytes + S::GBytes : spare, go);
  };

  f32x4 acc[H][JT];
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int j = 0; j < JT; ++j) acc[h][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int t = 0; t < NST - 1; ++t) {
    const int go = mx_less(t, steps);
    issue(go ? t : 0, t, go);
  }
  int b = 0;
  for (int t = 0; t < steps; ++t) {
    // step t has landed (those after it may be on their way), and every wave
    // has read step t - 1, whose stage the next loads take
    mx_wait_loads<(NST - 2) * S::Loads>(mx_less(t + NST - 1, steps + 1));
    __syncthreads();
    {
      const int go = mx_less(t + NST - 1, steps);
      issue(go ? t + NST - 1 : t, b == 0 ? NST - 1 : b - 1, go);
    }
    const char* st = smem + b * S::Stage;
    b = b + 1 == NST ? 0 : b + 1;
    if (TAIL && 8 * t + wave >= blocks) break;  // past the last step's columns
    u32x4 zf[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int row = 16 * h + l16;
      const char* zr = st + row * S::ZRow;
      if (FZ == 16) {
        zf[h] = *reinterpret_cast<const u32x4*>(zr + 16 * ((4 * wave + q) ^ zswz(row)));
      } else {
        const float sc =
            mx_scale(*reinterpret_cast<const uint8_t*>(st + S::ZBytes + S::GBytes + 8 * row + wave));
        if (FZ == LQ_MX_FP8) {
          const u32x2 w = *reinterpret_cast<const u32x2*>(
              zr + 16 * ((2 * wave + (q >> 1)) ^ zswz(row)) + 8 * (q & 1));
          zf[h] = mx8_bf16(w[0], w[1], sc);
        } else {
          zf[h] = mx4_bf16(*reinterpret_cast<const uint32_t*>(zr + 16 * (wave ^ zswz(row)) + 4 * q),
                           sc);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < JT; ++j) {
      u32x4 gf;
      if (GT) {  // lane c of a 16-lane group: row c / 4, columns 4 (c % 4) ..; gets column c
        const char* a = st + S::ZBytes +
                        2 * ((32 * wave + 8 * q + (l16 >> 2)) * r + 16 * j + 4 * (l16 & 3));
        const u32x2 lo = shrink_tr(a), hi = shrink_tr(a + 8 * r);
        gf = u32x4{lo[0], lo[1], hi[0], hi[1]};
      } else {
        gf = *reinterpret_cast<const u32x4*>(st + S::ZBytes + (16 * j + l16) * 512 +
                                             16 * ((4 * wave + q) ^ l16));
      }
#pragma unroll
      for (int h = 0; h < H; ++h) acc[h][j] = mfma16(zf[h], gf, acc[h][j]);
    }
  }
  __syncthreads();  // the sums overwrite the stages
  f32x4(*part)[H * JT][64] = reinterpret_cast<f32x4(*)[H * JT][64]>(smem);
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int j = 0; j < JT; ++j) part[wave][h * JT + j][lane] = acc[h][j];
  __syncthreads();
  for (int c = wave; c < H * JT; c += S::NW) {
    f32x4 s = part[0][c][lane];
#pragma unroll
    for (int w = 1; w < S::NW; ++w) {
      const f32x4 o = part[w][c][lane];
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] += o[i];
    }
    const int h = c / JT, j = 16 * (c - h * JT) + l16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t m = m0 + 16 * h + 4 * q + i;
      if (m < M && j < r) out[m * r + j] = s[i];
    }
  }
}

// Bt[j][n] = B[n][j]: 64 rows of B per workgroup through LDS
__global__ __launch_bounds__(256) void mx_transpose_kernel(const uint16_t* __restrict__ B,
                                                           int64_t N, int r,
                                                           uint16_t* __restrict__ Bt) {
  __shared__ uint16_t t[64 * 65];
  const int64_t n0 = 64 * (int64_t)blockIdx.x;  // N % 64 == 0
  for (int e = threadIdx.x; e < 64 * r; e += 256) {
    const int n = e / r, j = e - n * r;
    t[j * 65 + n] = B[n0 * r + e];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 64 * r; e += 256) Bt[(int64_t)(e >> 6) * N + n0 + (e & 63)] = t[(e >> 6) * 65 + (e & 63)];
}

// Rows per workgroup: 16 while that fills the chip, 32 beyond (G is read half
// as often).  gt: G is K x r, see mx_shrink_tile_kernel.
template <int FZ, int JT>
void launch_rows(const void* Z, const uint8_t* Zs, int64_t M, int64_t K, const uint16_t* G, int r,
                 bool gt, float* out, hipStream_t st) {
  const uint8_t* z = (const uint8_t*)Z;
  const bool wide = M > 4096;
  const dim3 grid((unsigned)cdiv(M, wide ? 32 : 16));
  constexpr bool U = FZ == 16;
  if (U || (K % 128 == 0 && (uintptr_t)Zs % 4 == 0)) {  // scales are read as 4-byte words
    auto tile = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, grid, dim3(512), 0, st, z, Zs, M, K, G, r, out);
    };
    auto rows = [&](auto g, auto tail) {
      constexpr bool GT = decltype(g)::value, TAIL = decltype(tail)::value;
      wide ? tile(mx_shrink_tile_kernel<FZ, JT, 2, GT, TAIL>)
           : tile(mx_shrink_tile_kernel<FZ, JT, 1, GT, TAIL>);
    };
    const std::false_type no{};
    const std::true_type yes{};
    const std::integral_constant<bool, U> u{};
    if (U && gt)
      K % 256 ? rows(u, yes) : rows(u, no);
    else
      K % 256 ? rows(no, yes) : rows(no, no);
  } else if constexpr (!U) {
    constexpr int NW = JT == 1 ? 16 : 8;
    auto rows = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, grid, dim3(64 * NW), 0, st, z, Zs, M, K, G, r, out);
    };
    wide ? rows(mx_shrink_kernel<FZ, JT, 2, NW>) : rows(mx_shrink_kernel<FZ, JT, 1, NW>);
  }
}

template <int FZ>
int launch_z(const void* Z, const uint8_t* Zs, int64_t M, int64_t K, const uint16_t* G, int64_t r,
             bool gt, float* out, hipStream_t st) {
  if (r <= 16)
    launch_rows<FZ, 1>(Z, Zs, M, K, G, (int)r, gt, out, st);
  else if (r <= 32)
    launch_rows<FZ, 2>(Z, Zs, M, K, G, (int)r, gt, out, st);
  else
    launch_rows<FZ, 4>(Z, Zs, M, K, G, (int)r, gt, out, st);
  return hip_fail(hipGetLastError(), "mx_shrink launch");
}

}  // namespace

namespace dispatch {

int mx_shrink(const lq_mx_tensor& X, const void* A, int64_t r, float* T, hipStream_t st) {
  return X.format == LQ_MX_FP8
             ? launch_z<LQ_MX_FP8>(X.codes, X.scales, X.rows, X.cols, (const uint16_t*)A, r, false,
                                   T, st)
             : launch_z<LQ_MX_FP4>(X.codes, X.scales, X.rows, X.cols, (const uint16_t*)A, r, false,
                                   T, st);
}

int mx_u(const void* dY, int64_t M, int64_t N, const void* B, int64_t r, void* Bt, float* U,
         hipStream_t st) {
  const void* G = B;
  const bool gt = r % 4 == 0;
  if (r > 1 && !gt) {  // one rank: B is its own transpose
    hipLaunchKernelGGL(mx_transpose_kernel, dim3((unsigned)(N / 64)), dim3(256), 0, st,
                       (const uint16_t*)B, N, (int)r, (uint16_t*)Bt);
    const int e = hip_fail(hipGetLastError(), "mx_transpose launch");
    if (e) return e;
    G = Bt;
  }
  return launch_z<16>(dY, nullptr, M, N, (const uint16_t*)G, r, gt, U, st);
}

}  // namespace dispatch
}  // namespace lq
