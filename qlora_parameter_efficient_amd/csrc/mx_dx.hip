// Input gradient of the MXFP4 layer:
//
//   dX = dY W + (s U) A       dY bf16 (M x N), W MXFP4 or bf16 (N x K), U = dY B
//                             (M x r float32), A bf16 (r x K)
//
// The reduction runs over N while a scale covers 32 columns k of one row n, so
// the scaled matrix instructions do not apply (a scale would change within
// each product group).  W's elements are exact in bf16; the kernel converts
// its 4-bit codes to bf16 inside the loop and multiplies by
// v_mfma_f32_32x32x16_bf16.  Against a bf16 copy of W0 in memory this reads a
// quarter of the weight bytes through the load path, which (not the matrix
// units) limits a loop that loads both operands as bf16.
//
// Tiles.  Four waves own a 256 (k) x 64 JM (m) output tile, wave (wi, wj) its
// 128 x 32 JM block, computed transposed (k = MFMA rows: a lane holds four
// consecutive outputs of one row).  Steps of 64 reduction rows n, four 16-wide
// substeps.  LDS holds
//   * two dY tiles (64 JM rows of 128 bytes, chunks swizzled by row), straight
//     from global memory;
//   * two bf16 W tiles, 64 rows n of 512 bytes, chunk c of row n at
//     c ^ 2 (n & 3) ^ 8 (c >> 1 & 1).  Thread (n, q) converts blocks q and
//     q + 4 of row n, a 16-byte chunk at a time between the products; its codes
//     and scale bytes come straight into registers, a step ahead.  Operands
//     (one column k, eight consecutive n) come back by the transposing
//     ds_read_b64_tr_b16.
// One barrier per step, before the last substep's products (see mxg_kernel):
// after it the tiles just read are free, so the last substep converts the W
// tile two steps ahead, and the next step's first substep issues the loads
// behind that.  Per step and compute unit LDS moves about 96 (JM = 2) or
// 128 KB of operand reads and 48 or 64 KB of writes, against 1,024 or 2,048 cycles
// of products.  Measured: 2048 x 4096 x 4096 76 to 79 us (0.9 PFLOP/s), 8192 x 4096
// x 11008 722 us (1.02), 1001 x 4096 x 11008 112 us (0.81).  Timed apart, dX and U
// at the first two shapes: 83 and 726 us, without the W tile's writes 78 and 690,
// without the loads 70 and 614, without both 69 and 602.  So the products with
// their operand reads are four fifths of it; the matrix units are busy 43 and 53%
// of the compute units' cycles, at 2.3 and 2.1 GHz (the instruction alone, on random
// values in registers, runs at 1.8 PFLOP/s).  Eight waves on the tile, with half
// again the operand reads, take the same time.
//
// A dense bf16 W (the backward from an MX checkpoint of a dense layer) takes
// the same loop with its W tiles loaded straight into LDS.
//
// Split: few tiles leave float32 partial sums of ranges of n, the first with
// the expand, added in order by mx_sum_splits_kernel.
#include <type_traits>

#include "dispatch.h"
#include "mx_tile.h"

namespace lq {
namespace {

constexpr int kThreads = 256;
constexpr int kTI = 256;  // output columns k per tile
constexpr int kStep = 64; // reduction rows n per step

struct MxdxParams {
  const uint16_t* dY;     // M x N
  const uint8_t* W;       // N x K / 2 codes, or bf16 N x K
  const uint8_t* Ws;      // N x K / 32 (codes)
  const float* U;         // M x r
  const uint16_t* A;      // r x K
  uint16_t* dX;           // M x K
  float* part;            // splits x M x K
  int64_t M, N, K;
  int32_t r;
  float s;
  int32_t ti, tj, splits, ksteps;
};

template <int JM>
struct MxdxShape {
  static constexpr int TJ = 64 * JM;
  static constexpr int WTile = kStep * kTI * 2;  // bf16 W tile of a step
  static constexpr int YTile = TJ * kStep * 2;   // dY tile of a step
  static constexpr int YBase = 2 * WTile;
  static constexpr int Out = TJ * kTI * 2;
  static constexpr int Smem = YBase + 2 * YTile > Out ? YBase + 2 * YTile : Out;
  static constexpr int YU = YTile / 4096;        // dY loads per wave and step
  static constexpr int WU = WTile / 4096;        // W loads per wave and step (bf16 W)
};

typedef short s16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ u32x2 read_tr(uint32_t addr) {
  typedef __attribute__((address_space(3))) s16x4* lds_ptr;
  return __builtin_bit_cast(u32x2,
                            __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(uintptr_t)addr));
}

// physical chunk of logical 16-byte chunk c in row n of a W tile
__device__ __forceinline__ int wphys(int c, int n) {
  return c ^ (2 * (n & 3)) ^ (8 * ((c >> 1) & 1));
}

// FP4: W are MXFP4 codes; else bf16 values, whose tiles come straight from global
// memory like dY's, at the places where the codes are converted.
template <bool FP4, int JM, bool SPLIT>
__global__ __launch_bounds__(kThreads) void mxdx_kernel(MxdxParams p) {
  using S = MxdxShape<JM>;
  __shared__ __attribute__((aligned(1024))) char smem[S::Smem];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wi = wave & 1, wj = wave >> 1;
  const int h = lane >> 5, l32 = lane & 31;

  const int t0 = xcd_tile(blockIdx.x, p.ti * p.tj);
  constexpr int GJ = 4;
  const int grp = t0 / (GJ * p.ti);
  const int in = t0 - grp * GJ * p.ti;
  const int gj = (p.tj - grp * GJ) < GJ ? (p.tj - grp * GJ) : GJ;
  const int tile_j = grp * GJ + in % gj;
  const int tile_i = in / gj;
  const int64_t i0 = (int64_t)tile_i * kTI, j0 = (int64_t)tile_j * S::TJ;
  const int64_t M = p.M, N = p.N, K = p.K;
  const int KT = (int)(N / kStep);  // N % 64 == 0
  const int ka = blockIdx.y * p.ksteps;
  const int kb = ka + p.ksteps < KT ? ka + p.ksteps : KT;
  const uint32_t sbase = mx_lds_addr(smem);
  const int blocks = (int)((K - i0) / 32 < 8 ? (K - i0) / 32 : 8);  // blocks of the tile in W's rows

  // ---- per-thread dY load offsets
  uint32_t yoff[S::YU];
#pragma unroll
  for (int u = 0; u < S::YU; ++u) {
    const int row = 8 * (wave * S::YU + u) + (lane >> 3);
    int64_t m = j0 + row;
    m = m < M ? m : M - 1;
    yoff[u] = (uint32_t)((m * N + 8 * ((lane & 7) ^ mx_swz128(row))) * 2);
  }
  const char* yb0 = reinterpret_cast<const char*>(p.dY);
  auto issue_y = [&](int kt, int slot, int go, int u) {
    mx_dma16(yb0 + (int64_t)kt * (kStep * 2), yoff[u],
             sbase + S::YBase + slot * S::YTile + (wave * S::YU + u) * 1024, go);
  };

  // ---- W: thread (n, q), blocks q and q + 4 of the tile (a block past K reads
  // the tile's first; its columns are not stored)
  const int cn = tid >> 2, cq = tid & 3;
  const uint8_t *wp[2], *sp[2];
#pragma unroll
  for (int i = 0; FP4 && i < 2; ++i) {
    const int blk = cq + 4 * i < blocks ? cq + 4 * i : 0;
    wp[i] = p.W + cn * (K / 2) + i0 / 2 + 16 * blk;
    sp[i] = p.Ws + cn * (K / 32) + i0 / 32 + blk;
  }
  u32x4 cw[2];
  uint32_t cs[2];
  auto load_codes = [&](int kt) {
    const int64_t row0 = (int64_t)kt * kStep;
#pragma unroll
    for (int i = 0; FP4 && i < 2; ++i) {
      cw[i] = *reinterpret_cast<const u32x4*>(wp[i] + row0 * (K / 2));
      cs[i] = sp[i][row0 * (K / 32)];
    }
  };
  uint32_t wst[8];  // LDS offsets of the thread's chunks: block i, part d at 4 i + d
#pragma unroll
  for (int c = 0; c < 8; ++c)
    wst[c] = (uint32_t)(cn * 512 + wphys(4 * (cq + 4 * (c >> 2)) + (c & 3), cn) * 16);
  // bf16 W: load u of the wave brings rows n and n + 1, lane i their chunk that
  // sits at i % 32 (one past K: the row's first)
  uint32_t wo[S::WU];
#pragma unroll
  for (int u = 0; !FP4 && u < S::WU; ++u) {
    const int n = 2 * (wave * S::WU + u) + (lane >> 5), at = lane & 31;
    const int c1 = ((at >> 1) ^ n) & 1;  // bit 1 of the chunk at this place
    const int c = at ^ (2 * (n & 3)) ^ (8 * c1);
    wo[u] = (uint32_t)(n * K * 2 + 16 * (c < 4 * blocks ? c : 0));
  }
  const char* wb0 = reinterpret_cast<const char*>(p.W) + i0 * 2;
  // piece c of 8 of the W tile of step kt into tile b
  auto convert = [&](int kt, int b, int go, int c) {
    if constexpr (FP4)
      *reinterpret_cast<u32x4*>(smem + b * S::WTile + wst[c]) =
          mx4_bf16(cw[c >> 2][c & 3], mx_scale(cs[c >> 2]));
    else
      mx_dma16(wb0 + (int64_t)kt * kStep * K * 2, wo[c],
               sbase + b * S::WTile + (wave * S::WU + c) * 1024, go);
  };
  static_assert(S::WU == 8, "pieces of a W tile");

  // ---- per-lane LDS read offsets
  const int sw = mx_swz128(l32);
  const uint32_t prow = (uint32_t)((32 * JM * wj + l32) * 128);
  uint32_t pcx[4], qtr[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) pcx[s] = (uint32_t)(((2 * s + h) ^ sw) << 4);
  // transposing reads: lane c of a 16-lane group addresses row c / 4, columns
  // 4 (c % 4) .., and receives column c of the four rows
  const int gc = l32 & 15, half = l32 >> 4, nlo = gc >> 2;
  const uint32_t qrow = (uint32_t)((8 * h + nlo) * 512);
#pragma unroll
  for (int ns = 0; ns < 4; ++ns) {
    const int col = 128 * wi + 32 * ns + 16 * half + 4 * (gc & 3);
    qtr[ns] = (uint32_t)(wphys(col >> 3, nlo) * 16 + (col & 7) * 2);
  }
  u32x4 wf[2][4], xf[2][JM];
  auto frags = [&](int b, int s, int c) {
    const uint32_t pt = sbase + S::YBase + b * S::YTile;
#pragma unroll
    for (int ms = 0; ms < JM; ++ms) xf[c][ms] = mx_read16(pt + prow + ms * 32 * 128 + pcx[s]);
#pragma unroll
    for (int ns = 0; ns < 4; ++ns) {
      const uint32_t a = sbase + b * S::WTile + qrow + (uint32_t)(16 * s * 512) + qtr[ns];
      const u32x2 lo = read_tr(a), hi = read_tr(a + 4 * 512);
      wf[c][ns] = u32x4{lo[0], lo[1], hi[0], hi[1]};
    }
  };

  f32x16 acc[4][JM];
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < JM; ++b)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[a][b][v] = 0.0f;

  // the step d steps on, or this one again where there is none (its loads are
  // then skipped or unused)
  auto next = [&](int kt, int d) { return mx_less(kt + d, kb) ? kt + d : kt; };
  // prologue: dY tiles of steps ka and ka + 1, both W tiles, the codes of
  // step ka + 2
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    load_codes(next(ka, q));
#pragma unroll
    for (int u = 0; u < S::YU; ++u) issue_y(next(ka, q), q, q == 0 ? 1 : mx_less(ka + 1, kb), u);
#pragma unroll
    for (int c = 0; c < 8; ++c) convert(next(ka, q), q, q == 0 ? 1 : mx_less(ka + 1, kb), c);
  }
  load_codes(next(ka, 2));
  mx_wait_loads();
  __syncthreads();
  frags(0, 0, 0);

  // step kt on tiles b; at its start the codes of step kt + 2 and the dY of
  // step kt + 1 are loaded or on their way.  The body has no branch.
  int kt = ka, b = 0;
  do {
    const int go1 = (mx_less(ka, kt) & mx_less(kt + 1, kb));  // dY of step kt + 1 (the first is there)
    const int k1 = next(kt, 1);
    const int go2 = FP4 ? 0 : mx_less(kt + 2, kb), k2 = go2 ? kt + 2 : kt;
    auto sub = [&](auto k) {
      constexpr int s = decltype(k)::value, c = s & 1;
      frags(b, s + 1, c ^ 1);
      __builtin_amdgcn_sched_barrier(0);  // the next reads before these products
#pragma unroll
      for (int ns = 0; ns < 4; ++ns) {
#pragma unroll
        for (int ms = 0; ms < JM; ++ms) acc[ns][ms] = mfma32(wf[c][ns], xf[c][ms], acc[ns][ms]);
        if (s == 0) {  // the loads into the tile that the last barrier freed
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int u = 0; u < S::YU; ++u)
            if (u * 4 / S::YU == ns) issue_y(k1, b ^ 1, go1, u);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    sub(std::integral_constant<int, 0>{});
    sub(std::integral_constant<int, 1>{});
    sub(std::integral_constant<int, 2>{});
    // this step's operands are in registers, the next step's tiles are there
    mx_wait_loads();
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);
    frags(b ^ 1, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int ns = 0; ns < 4; ++ns) {
#pragma unroll
      for (int ms = 0; ms < JM; ++ms) {
        acc[ns][ms] = mfma32(wf[1][ns], xf[1][ms], acc[ns][ms]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (c * JM / 2 == ns * JM + ms) convert(k2, b, go2, c);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    load_codes(next(kt, 3));
    b ^= 1;
  } while (++kt < kb);
  __syncthreads();  // the output tile overwrites the stages

  // ---- expand: acc += A-operand x (s U)-operand over rank chunks of 16, s U in
  // two bf16 parts
  const int r = SPLIT && blockIdx.y ? 0 : p.r;
  for (int c = 0; c < r; c += 16) {
    const int jr = c + 8 * h;
    u32x4 ef[4];
    MxVParts vf[JM];
#pragma unroll
    for (int ns = 0; ns < 4; ++ns) {
      int64_t k = i0 + 128 * wi + 32 * ns + l32;
      k = k < K ? k : K - 1;
      ef[ns] = mx_e_col(p.A, K, k, jr, r);
    }
#pragma unroll
    for (int ms = 0; ms < JM; ++ms) {
      int64_t m = j0 + 32 * JM * wj + 32 * ms + l32;
      m = m < M ? m : M - 1;
      vf[ms] = mx_v_operand(p.U + m * r, jr, r, p.s);
    }
#pragma unroll
    for (int ns = 0; ns < 4; ++ns)
#pragma unroll
      for (int ms = 0; ms < JM; ++ms) {
        acc[ns][ms] = mfma32(ef[ns], vf[ms].l, acc[ns][ms]);
        acc[ns][ms] = mfma32(ef[ns], vf[ms].h, acc[ns][ms]);
      }
  }

  if constexpr (SPLIT) {
    float* part = p.part + (int64_t)blockIdx.y * M * K;
#pragma unroll
    for (int ms = 0; ms < JM; ++ms) {
      const int64_t m = j0 + 32 * JM * wj + 32 * ms + l32;
#pragma unroll
      for (int ns = 0; ns < 4; ++ns)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int64_t k = i0 + 128 * wi + 32 * ns + 8 * q + 4 * h;
          if (m < M && k < K)
            *reinterpret_cast<f32x4*>(part + m * K + k) =
                f32x4{acc[ns][ms][4 * q], acc[ns][ms][4 * q + 1], acc[ns][ms][4 * q + 2],
                      acc[ns][ms][4 * q + 3]};
        }
    }
    return;
  }

  // ---- store: bf16 tile in LDS (row j, 512 bytes; chunk c at c ^ (j & 15)),
  // then 16-byte stores of whole output rows
#pragma unroll
  for (int ms = 0; ms < JM; ++ms) {
    const int j = 32 * JM * wj + 32 * ms + l32;
#pragma unroll
    for (int ns = 0; ns < 4; ++ns)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = 128 * wi + 32 * ns + 8 * q + 4 * h;
        *reinterpret_cast<u32x2*>(smem + j * 512 + ((i >> 3) ^ (j & 15)) * 16 + (i & 7) * 2) =
            u32x2{pack_bf16x2(acc[ns][ms][4 * q], acc[ns][ms][4 * q + 1]),
                  pack_bf16x2(acc[ns][ms][4 * q + 2], acc[ns][ms][4 * q + 3])};
      }
  }
  __syncthreads();
  const int cl = tid & 31;
  const int64_t k = i0 + 8 * cl;
#pragma unroll 4
  for (int it = 0; it < 8 * JM; ++it) {
    const int j = 8 * it + (tid >> 5);
    const int64_t m = j0 + j;
    const u32x4 v = mx_read16(sbase + (uint32_t)(j * 512 + ((cl ^ (j & 15)) << 4)));
    if (m < M && k < K) *reinterpret_cast<u32x4*>(p.dX + m * K + k) = v;
  }
}

// out = bf16(sum over splits): eight outputs per thread, the splits added in
// order
__global__ __launch_bounds__(256) void mx_sum_splits_kernel(const float* part, uint16_t* out,
                                                            int64_t n, int splits) {
  const int64_t i = 8 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
  if (i >= n) return;
  f32x4 a = *reinterpret_cast<const f32x4*>(part + i);
  f32x4 b = *reinterpret_cast<const f32x4*>(part + i + 4);
#pragma unroll 4
  for (int t = 1; t < splits; ++t) {
    const float* q = part + t * n + i;
    const f32x4 c = *reinterpret_cast<const f32x4*>(q), d = *reinterpret_cast<const f32x4*>(q + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a[e] += c[e];
      b[e] += d[e];
    }
  }
  *reinterpret_cast<u32x4*>(out + i) = u32x4{pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]),
                                             pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3])};
}

struct Plan {
  int jm, ti, tj, splits;
};

// The tile with the least rounds x time of a round, the wider at a tie: at
// N = 4096 a round of 256 tiles takes 105 us at 256 x 256, 65 to 75 at
// 256 x 128 and 45 to 60 at 256 x 64 (dX and U, 1001 x 4096 x 11008: 114, 138 and
// 131 us; 2048 x 4096 x 4096: 110, 79 and 89).  Two workgroups of 256 x 64 fit a
// compute unit; where a third of those places would be filled, the reduction is
// split (600 x 4096 x 4096, 160 tiles: 63 us whole, 48 in three; 512: 62 and
// 43 in four; 100: 61 and 28 in eight).
Plan plan(int64_t M, int64_t N, int64_t K) {
  static const int shapes[3][2] = {{4, 20}, {2, 14}, {1, 11}};
  Plan q{};
  q.ti = (int)cdiv(K, kTI);
  int64_t best = 0;
  for (const auto& c : shapes) {
    const int64_t tj = cdiv(M, 64 * c[0]), cost = c[1] * cdiv(q.ti * tj, 256);
    if (best && cost >= best) continue;
    best = cost;
    q.jm = c[0];
    q.tj = (int)tj;
  }
  const int64_t tiles = (int64_t)q.ti * q.tj;
  int64_t sp = q.jm == 1 && tiles <= 170 ? 512 / tiles : 1;
  const int64_t most = N / 256;  // at least four steps a split
  if (sp > most) sp = most;
  if (sp > 8) sp = 8;
  if (sp < 1) sp = 1;
  const int64_t steps = N / kStep, per = cdiv(steps, sp);
  q.splits = (int)cdiv(steps, per);
  return q;
}

template <bool FP4, int JM, bool SPLIT>
void launch(const MxdxParams& p, hipStream_t st) {
  hipLaunchKernelGGL((mxdx_kernel<FP4, JM, SPLIT>), dim3((unsigned)(p.ti * p.tj), (unsigned)p.splits),
                     dim3(kThreads), 0, st, p);
}

template <bool FP4>
int run_dx(MxdxParams& p, hipStream_t st) {
  const Plan q = plan(p.M, p.N, p.K);
  p.ti = q.ti;
  p.tj = q.tj;
  p.splits = q.splits;
  p.ksteps = (int32_t)cdiv(p.N / kStep, q.splits);
  if (q.splits > 1)
    launch<FP4, 1, true>(p, st);
  else if (q.jm == 4)
    launch<FP4, 4, false>(p, st);
  else if (q.jm == 2)
    launch<FP4, 2, false>(p, st);
  else
    launch<FP4, 1, false>(p, st);
  const int e = hip_fail(hipGetLastError(), "mx_dx launch");
  if (e || q.splits == 1) return e;
  return dispatch::mx_sum_splits(p.part, p.dX, p.M * p.K, q.splits, st);
}

}  // namespace

namespace dispatch {

int mx_sum_splits(const float* part, void* out, int64_t n, int splits, hipStream_t st) {
  hipLaunchKernelGGL(mx_sum_splits_kernel, dim3((unsigned)cdiv(n, 2048)), dim3(256), 0, st, part,
                     (uint16_t*)out, n, splits);
  return hip_fail(hipGetLastError(), "mx_sum_splits launch");
}

size_t mx_dx_ws_bytes(int64_t M, int64_t N, int64_t K) {
  const Plan q = plan(M, N, K);
  return q.splits > 1 ? (size_t)q.splits * M * K * 4 : 0;
}

int mx_dx(const void* dY, int64_t M, const lq_mx_tensor& W, const float* U, const void* A,
          int64_t r, float s, void* dX, void* part, hipStream_t st) {
  MxdxParams p = {(const uint16_t*)dY, W.codes, W.scales, U, (const uint16_t*)A, (uint16_t*)dX,
                  (float*)part, M, W.rows, W.cols, (int32_t)r, s, 0, 0, 0, 0};
  return run_dx<true>(p, st);
}

bool mx_dx_fills(int64_t M, int64_t N, int64_t K) {
  const Plan q = plan(M, N, K);
  return q.jm > 1 || q.splits > 1;
}

int mx_dx_dense(const void* dY, int64_t M, const lq_weight& W, const float* U, const void* A,
                int64_t r, float s, void* dX, void* part, hipStream_t st) {
  MxdxParams p = {(const uint16_t*)dY, (const uint8_t*)W.dense, nullptr, U, (const uint16_t*)A,
                  (uint16_t*)dX, (float*)part, M, W.N, W.K, (int32_t)r, s, 0, 0, 0, 0};
  return run_dx<false>(p, st);
}

}  // namespace dispatch
}  // namespace lq
