// Forward product of the MXFP4 layer on the scaled matrix instructions:
//
//   Y = X W^T + (s T) B^T      X MXFP8 or MXFP4 (M x K), W MXFP4 (N x K),
//                              T = X A^T (M x r float32)
//
// v_mfma_scale_f32_32x32x64_f8f6f4 multiplies the codes and applies both
// operands' block scales, so nothing is dequantised; 4-bit codes on both sides
// run at twice the rate of an 8-bit side.
//
// Operand layout of the instruction (lane l: row l % 32, half h = l / 32; the
// 64 reduction elements are two scale blocks 0 and 1):
//   4-bit codes: 16 bytes per lane, block h
//   8-bit codes: 32 bytes per lane, 16-byte half h of block 0, then of block 1
//   scale: one byte of the lane's scale register (picked by opsel), block h
// Any relabelling of the reduction that is the same on both operands leaves
// the product unchanged; the kernel uses it to make a lane's scale bytes
// adjacent: in a step of KB blocks per row, instruction kk's block h is block
// h KB / 2 + kk of the step, so a lane's scale bytes for all instructions of
// the step are one LDS word or half word.
//
// Tiles.  WI x 2 waves own a (32 IM WI) x (64 JM) output tile, i (weight rows n)
// by j (activation rows m), wave (wi, wj) a (32 IM) x (32 JM) block of 32 x 32
// accumulators: eight waves at 256 x 256 and 256 x 128 (with four, 8192 x 11008 x
// 4096 of 4-bit codes took 4% longer), four at 128 x 128, of which two fit a
// compute unit.  The output is computed transposed (n = MFMA rows), so a lane
// holds four consecutive outputs of one row.  Codes and scales of a step go
// straight from global memory into LDS (global_load_lds_dwordx4 and _dword),
// 16-byte chunks of the codes swizzled by row through the lanes' global
// addresses so that operand reads are conflict-free.  A scale load costs the
// load path a line per row however few bytes it takes, half of a step's lines
// at 4 or 8 bytes, so where K % 512 == 0 a load brings 16 bytes of each row, the
// scales of two (FP4) or four steps (with the eight waves 5% off that shape).
// Steps of 256 columns with an FP4 X, so that every row piece is a whole 128-byte
// line (with 128 columns the lines are fetched twice: 4096^3 takes 17% longer
// although twice the stages fit), and of 128 columns with an FP8 X.  Two to four LDS stages (what
// fits), one barrier per step, placed before the step's last substep of
// products (see the loop).
//
// Split K (few tiles): workgroups of one tile take ranges of the steps and
// leave float32 partial sums (the first with the expand), added in order by
// mx_sum_splits.
//
// Measured: 2048 x 4096 x 4096 MXFP8 38 us (1.8 PFLOP/s), 8192 x 11008 x 4096
// MXFP4 282 us (2.6 PFLOP/s), 1001 x 4096 x 11008 MXFP8 60 us (1.5).
// No one unit is full.  Over these kernels the matrix units are busy 49, 42 and
// 35% of the compute units' cycles, at a shader clock of 2.4 GHz (2.1 in the
// second).  At M = N = 4096 and K = 1024, 4096, 16384 a call takes 18, 41 and 136 us
// with an FP4 X and 24, 59 and 214 with an FP8 one: a further step costs 4.4 and
// 2.7 PFLOP/s, and 7 to 10 us of a call lie outside the steady loop (a tile's
// first loads, its expand and its stores leave the matrix units idle, as there
// is one workgroup per compute unit).  The same instructions alone, on random
// codes in registers, run at 7.0 to 7.4 PFLOP/s with a 4-bit X, 3.9 to 4.3 with an
// 8-bit one.
//
// Epilogue: the expand adds (s T) B^T on the finished accumulators with bf16
// MFMAs (s T in two bf16 parts, off by 2^-16, so that the adapter's term is no
// coarser here than in the forward of few bf16 rows), then the tile goes through
// LDS and leaves as 16-byte stores covering whole output lines.
#include <type_traits>

#include "dispatch.h"
#include "mx_tile.h"

namespace lq {
namespace {

struct MxgParams {
  const uint8_t* X;   // M x K codes
  const uint8_t* Xs;  // M x K / 32
  const uint8_t* W;   // N x K codes (FP4)
  const uint8_t* Ws;
  const float* T;     // M x r
  const uint16_t* B;  // N x r
  uint16_t* Y;        // M x N
  float* part;        // splits x M x N (splits > 1)
  int64_t M, N, K;
  int32_t r;
  float s;
  int32_t ti, tj, splits, ksteps;
};

// IM, JM: 32 x 32 blocks of a wave; WI x 2 waves.  Scales of a step: WIDE (rows
// of scales 16-byte aligned, K % 512 == 0) 16 bytes a row for the GS steps that
// they cover, into two buffers of their own; else 4 or 8 bytes a row with the
// step's stage.
template <int FX, int IM, int JM, int WI, bool WIDE>
struct MxgShape {
  static constexpr int NW = 2 * WI, NT = 64 * NW;          // waves, threads
  static constexpr int BK = FX == LQ_MX_FP4 ? 256 : 128;   // columns per step
  static constexpr int KB = BK / 32;                       // blocks per row and step
  static constexpr int GS = 16 / KB;                       // steps of a 16-byte scale load
  static constexpr int TI = 32 * IM * WI, TJ = 64 * JM;
  static constexpr int WRow = BK / 2, XRow = 128;          // bytes per row and step
  static constexpr int WBytes = TI * WRow, XBytes = TJ * XRow;
  static constexpr int Stage = WBytes + XBytes + (WIDE ? 0 : (TI + TJ) * KB);
  static constexpr int GBytes = (TI + TJ) * 16;            // a scale buffer (WIDE)
  // stages: as many as one workgroup per compute unit allows (256-row tiles:
  // their accumulators leave room for one), two workgroups for 128 x 128
  static constexpr int Room = (TI == 256 ? 160 : 80) * 1024 - (WIDE ? 2 * GBytes : 0);
  static constexpr int NST = Room / Stage < 4 ? Room / Stage : 4;
  static constexpr int SBase = NST * Stage;
  static constexpr int Used = SBase + (WIDE ? 2 * GBytes : 0);
  static constexpr int Out = TJ * TI * 2;                  // bf16 output tile
  static constexpr int Smem = Used > Out ? Used : Out;
  static constexpr int WU = WBytes / (1024 * NW), XU = XBytes / (1024 * NW);  // code loads per wave
  static constexpr int SRows = WIDE ? 64 : 256 / KB;       // rows of a scale load
  static constexpr int SG = (TI + TJ) / SRows;             // scale loads (WIDE: of GS steps) ...
  static constexpr int SU = (SG + NW - 1) / NW;            // ... and per wave
  static constexpr int Loads = WU + XU + SU;
  static constexpr int Counted = WIDE ? WU + XU : Loads;   // those of every step
  static constexpr int SR = (TI + TJ + NT - 1) / NT;       // scale rows per thread (TAIL)
  // a group's buffer is free when the loads of the next but one go out
  static_assert(!WIDE || NST <= GS + 1, "scale buffers");
};

__device__ __forceinline__ i32x8 widen(const u32x4& v) {
  typedef int i32x4 __attribute__((ext_vector_type(4)));
  return __builtin_shufflevector(__builtin_bit_cast(i32x4, v), __builtin_bit_cast(i32x4, v), 0, 1,
                                 2, 3, -1, -1, -1, -1);
}

__device__ __forceinline__ i32x8 join(const u32x4& a, const u32x4& b) {
  typedef int i32x4 __attribute__((ext_vector_type(4)));
  return __builtin_shufflevector(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), 0, 1,
                                 2, 3, 4, 5, 6, 7);
}

// TAIL: K is not a multiple of the step; the last step's missing blocks (an
// even number) are read from the row's first blocks of the step and zeroed on
// the weight side, with scale 1 (byte 127) on both, and the scales, whose rows
// may then start at any even address, go through registers.  It also takes whole
// steps whose scales start off a word (rows cut from a larger tensor).
// SPLIT: several workgroups per tile, float32 partial sums out.
template <int FX, int IM, int JM, int WI, bool TAIL, bool WIDE, bool SPLIT>
__global__ __launch_bounds__(128 * WI) void mxg_kernel(MxgParams p) {
  using S = MxgShape<FX, IM, JM, WI, WIDE>;
  static_assert(!(TAIL && WIDE), "a tail's scales go through registers");
  constexpr int kThreads = S::NT;
  constexpr int KB = S::KB, MK = KB / 2;  // blocks and instructions (64 wide) per step
  __shared__ __attribute__((aligned(1024))) char smem[S::Smem];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wi = wave % WI, wj = wave / WI;
  const int h = lane >> 5, l32 = lane & 31;

  // tile: each XCD a contiguous range, in groups of four activation tiles
  const int t = xcd_tile(blockIdx.x, p.ti * p.tj);
  constexpr int GJ = 4;
  const int grp = t / (GJ * p.ti);
  const int in = t - grp * GJ * p.ti;
  const int gj = (p.tj - grp * GJ) < GJ ? (p.tj - grp * GJ) : GJ;
  const int tile_j = grp * GJ + in % gj;
  const int tile_i = in / gj;
  const int64_t i0 = (int64_t)tile_i * S::TI, j0 = (int64_t)tile_j * S::TJ;
  const int64_t M = p.M, N = p.N, K = p.K;
  const int64_t wpitch = K / 2, xpitch = K * FX / 8, spitch = K / 32;
  const int KT = (int)cdiv(K, S::BK);
  const int last_nb = (int)(K / 32) - (KT - 1) * KB;  // blocks of the last step
  const int ka = blockIdx.y * p.ksteps;
  const int kb = ka + p.ksteps < KT ? ka + p.ksteps : KT;
  const uint32_t sbase = mx_lds_addr(smem);

  // ---- per-thread load offsets, relative to the step's base pointers
  constexpr int WU = S::WU, XU = S::XU, SU = S::SU;
  uint32_t woff[WU], xoff[XU];
  int wch[WU], xch[XU];
#pragma unroll
  for (int u = 0; u < WU; ++u) {
    const int row = S::WRow == 128 ? 8 * (wave * WU + u) + (lane >> 3)
                                   : 16 * (wave * WU + u) + (lane >> 2);
    wch[u] = S::WRow == 128 ? (lane & 7) ^ mx_swz128(row) : (lane & 3) ^ mx_swz64(row);
    int64_t n = i0 + row;
    n = n < N ? n : N - 1;
    woff[u] = (uint32_t)(n * wpitch + 16 * wch[u]);
  }
#pragma unroll
  for (int u = 0; u < XU; ++u) {
    const int row = 8 * (wave * XU + u) + (lane >> 3);
    xch[u] = (lane & 7) ^ mx_swz128(row);
    int64_t m = j0 + row;
    m = m < M ? m : M - 1;
    xoff[u] = (uint32_t)(m * xpitch + 16 * xch[u]);
  }
  // scale rows of this wave's SU loads: group g of SRows rows (weight rows
  // first), a word (WIDE: 16 bytes) per lane; a group past the last is loaded
  // again, to the same place (WIDE: not loaded)
  uint32_t soff[SU];
  bool sw_[SU];
  int sgrp[SU];
#pragma unroll
  for (int u = 0; u < SU; ++u) {
    int g = wave * SU + u;
    g = g < S::SG ? g : S::SG - 1;
    sgrp[u] = g;
    const int R = g * S::SRows + (WIDE ? lane : lane / (KB / 4));
    sw_[u] = g * S::SRows < S::TI;
    const int64_t row = sw_[u] ? i0 + R : j0 + R - S::TI;
    const int64_t last = (sw_[u] ? N : M) - 1;
    soff[u] = (uint32_t)((row < last ? row : last) * spitch + (WIDE ? 0 : 4 * (lane % (KB / 4))));
  }
  const char* wb0 = reinterpret_cast<const char*>(p.W);
  const char* xb0 = reinterpret_cast<const char*>(p.X);
  // load u of this wave's Loads of step kt into stage b
  auto issue_one = [&](int kt, int b, int go, int u) {
    const uint32_t st = sbase + b * S::Stage;
    const bool cut = TAIL && kt == KT - 1;
    if (u < WU) {
      const uint32_t o = cut && wch[u] >= last_nb ? woff[u] - 16 * wch[u] : woff[u];
      mx_dma16(wb0 + (int64_t)kt * S::WRow, o, st + (wave * WU + u) * 1024, go);
    } else if (u < WU + XU) {
      const int v = u - WU;
      const bool past = xch[v] >= (FX == LQ_MX_FP4 ? last_nb : 2 * last_nb);
      const uint32_t o = cut && past ? xoff[v] - 16 * xch[v] : xoff[v];
      mx_dma16(xb0 + (int64_t)kt * S::XRow, o, st + S::WBytes + (wave * XU + v) * 1024, go);
    } else if (WIDE) {  // the group's first step in this workgroup brings its scales
      const int v = u - WU - XU;
      const int first = mx_less(kt & (S::GS - 1), 1) | mx_less(kt, ka + 1);
      mx_dma16(reinterpret_cast<const char*>(sw_[v] ? p.Ws : p.Xs) + (int64_t)(kt / S::GS) * 16,
               soff[v], sbase + S::SBase + (kt / S::GS & 1) * S::GBytes + sgrp[v] * 1024,
               go & first & mx_less(wave * SU + v, S::SG));
    } else if (!TAIL) {
      const int v = u - WU - XU;
      mx_dma4((sw_[v] ? p.Ws : p.Xs) + (int64_t)kt * KB, soff[v],
              st + S::WBytes + S::XBytes + sgrp[v] * 256, go);
    }
  };
  auto issue = [&](int kt, int b, int go) {
#pragma unroll
    for (int u = 0; u < S::Loads; ++u) issue_one(kt, b, go, u);
  };
  // the loads dealt over the products of two substeps: part i of 2 IM JM
  auto issue_part = [&](int kt, int b, int go, int i) {
    constexpr int parts = 2 * IM * JM;
#pragma unroll
    for (int u = 0; u < S::Loads; ++u)
      if (u * parts / S::Loads == i) issue_one(kt, b, go, u);
  };

  // ---- TAIL: thread t carries the scale bytes of rows t, t + 256 of (weight,
  // activation); a thread past the last row stores that row's bytes again
  const uint8_t* srow[S::SR];
  uint32_t sv[S::SR][KB / 4];
  if constexpr (TAIL) {
#pragma unroll
    for (int i = 0; i < S::SR; ++i) {
      int R = tid + kThreads * i;
      R = R < S::TI + S::TJ ? R : S::TI + S::TJ - 1;
      const int64_t row = R < S::TI ? i0 + R : j0 + R - S::TI;
      const int64_t last = (R < S::TI ? N : M) - 1;
      srow[i] = (R < S::TI ? p.Ws : p.Xs) + (row < last ? row : last) * spitch;
    }
  }
  auto load_scales = [&](int kt) {
    if constexpr (TAIL) {
      const int nb = kt == KT - 1 ? last_nb : KB;
#pragma unroll
      for (int i = 0; i < S::SR; ++i) {
        const uint16_t* a = reinterpret_cast<const uint16_t*>(srow[i] + (int64_t)kt * KB);
        uint32_t v[KB / 2];
#pragma unroll
        for (int e = 0; e < KB / 2; ++e) {
          const bool in = 2 * e < nb;
          const uint32_t w = a[in ? e : 0];
          v[e] = in ? w : 0x7F7Fu;
        }
#pragma unroll
        for (int e = 0; e < KB / 4; ++e) sv[i][e] = v[2 * e] | (v[2 * e + 1] << 16);
      }
    }
  };
  auto store_scales = [&](int b) {
    if constexpr (TAIL) {
#pragma unroll
      for (int i = 0; i < S::SR; ++i) {
        int R = tid + kThreads * i;
        R = R < S::TI + S::TJ ? R : S::TI + S::TJ - 1;
#pragma unroll
        for (int e = 0; e < KB / 4; ++e)
          *reinterpret_cast<uint32_t*>(smem + b * S::Stage + S::WBytes + S::XBytes + R * KB +
                                       4 * e) = sv[i][e];
      }
    }
  };

  // ---- per-lane LDS read offsets
  const int wrow0 = 32 * IM * wi + l32, xrow0 = 32 * JM * wj + l32;
  // row offsets by multiples of 32 leave both swizzles unchanged
  const int xsw = mx_swz128(l32), wsw = S::WRow == 128 ? mx_swz128(l32) : mx_swz64(l32);
  auto read_w = [&](uint32_t st, int ns, int kk) {
    const int c = h * (KB / 2) + kk;
    return mx_read16(st + (uint32_t)((wrow0 + 32 * ns) * S::WRow + ((c ^ wsw) << 4)));
  };
  auto read_x = [&](uint32_t st, int ms, int kk) {
    const uint32_t row = st + S::WBytes + (uint32_t)((xrow0 + 32 * ms) * S::XRow);
    if (FX == LQ_MX_FP4) {
      const int c = h * (KB / 2) + kk;
      return widen(mx_read16(row + (uint32_t)((c ^ xsw) << 4)));
    }
    // half h of block kk (the instruction's block 0) and of block KB / 2 + kk
    const int c0 = 2 * kk + h, c1 = KB + 2 * kk + h;
    return join(mx_read16(row + (uint32_t)((c0 ^ xsw) << 4)),
                mx_read16(row + (uint32_t)((c1 ^ xsw) << 4)));
  };
  auto read_scale = [&](int kt, int b, int row) -> int {
    const char* a = smem + (WIDE ? S::SBase + (kt / S::GS & 1) * S::GBytes + row * 16 +
                                       (kt & (S::GS - 1)) * KB
                                 : b * S::Stage + S::WBytes + S::XBytes + row * KB) +
                    h * (KB / 2);
    if (KB == 8) return *reinterpret_cast<const int*>(a);
    return (int)*reinterpret_cast<const uint16_t*>(a);
  };

  f32x16 acc[IM][JM];
#pragma unroll
  for (int a = 0; a < IM; ++a)
#pragma unroll
    for (int b = 0; b < JM; ++b)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[a][b][v] = 0.0f;

  // The loop, pipelined across the barrier: a substep's LDS reads go out before
  // the previous substep's products, and the last substep's products run after
  // the barrier, covering the first reads of the next step and the first half
  // of the loads NST steps ahead (into the stage the barrier has just freed);
  // the second half goes out among the next step's first products (all of them
  // in one substep: 4% longer at 8192 x 11008 x 4096 MXFP4).  The body has
  // no branch: one between the products and the barrier would let the compiler
  // sink products past it, so loads past the last step are skipped inside
  // mx_dma16.
  u32x4 wf[2][IM];
  i32x8 xf[2][JM];
  int ws[2][IM], xs[2][JM];
  auto frags = [&](uint32_t st, int kt, int kk, int c) {
#pragma unroll
    for (int ns = 0; ns < IM; ++ns) {
      wf[c][ns] = read_w(st, ns, kk);
      if (TAIL) wf[c][ns] = sel4(kt < KT - 1 || h * (KB / 2) + kk < last_nb, wf[c][ns]);
    }
#pragma unroll
    for (int ms = 0; ms < JM; ++ms) xf[c][ms] = read_x(st, ms, kk);
  };
  auto read_scales = [&](int kt, int b, int q) {
#pragma unroll
    for (int ns = 0; ns < IM; ++ns) ws[q][ns] = read_scale(kt, b, wrow0 + 32 * ns);
#pragma unroll
    for (int ms = 0; ms < JM; ++ms) xs[q][ms] = read_scale(kt, b, S::TI + xrow0 + 32 * ms);
  };
  constexpr int NST = S::NST;
  // loads of the first NST steps; every split has at least one step
#pragma unroll
  for (int q = 0; q < NST; ++q) {
    const int go = mx_less(ka + q, kb);
    issue(go ? ka + q : ka, q, go);
  }
  load_scales(ka);
  store_scales(0);
  if constexpr (TAIL)
    mx_wait_loads();
  else
    mx_wait_loads<(NST - 1) * S::Counted>(mx_less(ka + NST, kb + 1));
  __syncthreads();
  int kt = ka, b = 0;
  load_scales(mx_less(ka + 1, kb) ? ka + 1 : ka);
  read_scales(ka, 0, 0);
  frags(sbase, ka, 0, 0);
  int kp = ka, bp = 0, gp = 0;  // step, stage and go of the loads under way
  do {
    const uint32_t st = sbase + b * S::Stage;
    const int bn = b + 1 == NST ? 0 : b + 1;
    auto products = [&](auto k, int ns, int ms) {
      constexpr int kk = decltype(k)::value, c = kk & 1;
      acc[ns][ms] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
          widen(wf[c][ns]), xf[c][ms], acc[ns][ms], 4, FX == LQ_MX_FP4 ? 4 : 0, kk, ws[0][ns], kk,
          xs[0][ms]);
    };
    auto sub = [&](auto k) {
      constexpr int kk = decltype(k)::value;
      frags(st, kt, kk + 1, (kk + 1) & 1);
      __builtin_amdgcn_sched_barrier(0);  // the next reads before these products
#pragma unroll
      for (int ns = 0; ns < IM; ++ns)
#pragma unroll
        for (int ms = 0; ms < JM; ++ms) {
          products(k, ns, ms);
          if (kk == 0) {  // the second half of the loads that the last step began
            __builtin_amdgcn_sched_barrier(0);
            issue_part(kp, bp, gp, IM * JM + ns * JM + ms);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      __builtin_amdgcn_sched_barrier(0);
    };
    sub(std::integral_constant<int, 0>{});
    if constexpr (MK > 2) {
      sub(std::integral_constant<int, 1>{});
      sub(std::integral_constant<int, 2>{});
    }
    // this step's operands are in registers; wait for the next step's loads
    // (those of later steps stay in flight)
    store_scales(bn);
    if constexpr (TAIL)
      mx_wait_loads();
    else
      mx_wait_loads<(NST - 2) * S::Counted>(mx_less(kt + NST, kb + 1));
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);
    const int k1 = mx_less(kt + 1, kb) ? kt + 1 : kt;
    const int go = mx_less(kt + NST, kb);
    const int kn = go ? kt + NST : kt;
    read_scales(k1, bn, 1);
    frags(sbase + bn * S::Stage, k1, 0, 0);
    load_scales(mx_less(kt + 2, kb) ? kt + 2 : k1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int ns = 0; ns < IM; ++ns) {
#pragma unroll
      for (int ms = 0; ms < JM; ++ms) {
        products(std::integral_constant<int, MK - 1>{}, ns, ms);
        __builtin_amdgcn_sched_barrier(0);
        issue_part(kn, b, go, ns * JM + ms);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int ns = 0; ns < IM; ++ns) ws[0][ns] = ws[1][ns];
#pragma unroll
    for (int ms = 0; ms < JM; ++ms) xs[0][ms] = xs[1][ms];
    kp = kn, bp = b, gp = go;
    b = bn;
  } while (++kt < kb);
  __syncthreads();  // the output tile overwrites the stages

  // ---- expand: acc += B-operand x (s T)-operand over rank chunks of 16
  const int r = SPLIT && blockIdx.y ? 0 : p.r;
  for (int c = 0; c < r; c += 16) {
    const int jr = c + 8 * h;
    u32x4 ef[IM];
    MxVParts vf[JM];
#pragma unroll
    for (int ns = 0; ns < IM; ++ns) {
      int64_t n = i0 + wrow0 + 32 * ns;
      n = n < N ? n : N - 1;
      ef[ns] = mx_e_row(p.B + n * r, jr, r);
    }
#pragma unroll
    for (int ms = 0; ms < JM; ++ms) {
      int64_t m = j0 + xrow0 + 32 * ms;
      m = m < M ? m : M - 1;
      vf[ms] = mx_v_operand(p.T + m * r, jr, r, p.s);
    }
#pragma unroll
    for (int ns = 0; ns < IM; ++ns)
#pragma unroll
      for (int ms = 0; ms < JM; ++ms) {
        acc[ns][ms] = mfma32(ef[ns], vf[ms].l, acc[ns][ms]);
        acc[ns][ms] = mfma32(ef[ns], vf[ms].h, acc[ns][ms]);
      }
  }

  if constexpr (SPLIT) {  // float32 partial sums; lane: rows n = .. + 8 q + 4 h + 0..3, column m
    float* part = p.part + (int64_t)blockIdx.y * M * N;
#pragma unroll
    for (int ms = 0; ms < JM; ++ms) {
      const int64_t m = j0 + xrow0 + 32 * ms;
#pragma unroll
      for (int ns = 0; ns < IM; ++ns)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int64_t n = i0 + 32 * IM * wi + 32 * ns + 8 * q + 4 * h;
          if (m < M && n < N)
            *reinterpret_cast<f32x4*>(part + m * N + n) =
                f32x4{acc[ns][ms][4 * q], acc[ns][ms][4 * q + 1], acc[ns][ms][4 * q + 2],
                      acc[ns][ms][4 * q + 3]};
        }
    }
    return;
  }

  // ---- store: bf16 tile in LDS (row j of 2 TI bytes, chunk c at c ^ (j & 15)),
  // then 16-byte stores of whole output rows
  constexpr int ORow = 2 * S::TI, OC = ORow / 16;  // bytes, chunks per output row
#pragma unroll
  for (int ms = 0; ms < JM; ++ms) {
    const int j = xrow0 + 32 * ms;
#pragma unroll
    for (int ns = 0; ns < IM; ++ns)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = 32 * IM * wi + 32 * ns + 8 * q + 4 * h;
        const int chunk = (i >> 3) ^ (j & 15);
        *reinterpret_cast<u32x2*>(smem + j * ORow + chunk * 16 + (i & 7) * 2) =
            u32x2{pack_bf16x2(acc[ns][ms][4 * q], acc[ns][ms][4 * q + 1]),
                  pack_bf16x2(acc[ns][ms][4 * q + 2], acc[ns][ms][4 * q + 3])};
      }
  }
  __syncthreads();
  const int cl = tid % OC;
  const int64_t n = i0 + 8 * cl;
#pragma unroll 4
  for (int it = 0; it < S::TJ * OC / kThreads; ++it) {
    const int j = it * (kThreads / OC) + tid / OC;
    const int64_t m = j0 + j;
    const u32x4 v = mx_read16(sbase + (uint32_t)(j * ORow + ((cl ^ (j & 15)) << 4)));
    if (m < M && n < N) *reinterpret_cast<u32x4*>(p.Y + m * N + n) = v;
  }
}

// Tile and split choice: the tile with the least rounds x time of a round, the
// larger at a tie.  At K = 4096 a round of 256 tiles takes about 3, 2 and 1 parts
// of 18 us at 256 x 256, 256 x 128 and 128 x 128 with an 8-bit X and of 12 with a
// 4-bit one (2048 x 4096 x 4096, calls of the three tiles: 51, 35 and 35 us 8-bit,
// 31, 24 and 25 4-bit; 4096 x 4096 x 4096: 59, 67 and 69 us, 39, 46 and 47).  Split
// K fills the chip but costs a second launch and the partial sums: it takes 4096
// columns to pay (8-bit X, 100 x 4096 x 11008: 44 us whole, 18 in eight; 512 x 4096 x
// 11008: 48 and 37 in two; 100 x 4096 x 4096: 19 and 14 in four; 512 x 4096 x 4096:
// 20 and 21 in two; 200 x 2048 x 2048: 11.0 and 11.4 in two).
struct Plan {
  int rows_i, rows_j, ti, tj, splits;
};

Plan plan(int64_t M, int64_t N, int64_t K) {
  static const int shapes[3][3] = {{256, 256, 3}, {256, 128, 2}, {128, 128, 1}};
  Plan q{};
  int64_t best = 0;
  for (const auto& c : shapes) {
    const int64_t ti = cdiv(N, c[0]), tj = cdiv(M, c[1]);
    const int64_t cost = c[2] * cdiv(ti * tj, 256);
    if (best && cost >= best) continue;
    best = cost;
    q = Plan{c[0], c[1], (int)ti, (int)tj, 1};
  }
  const int64_t tiles = (int64_t)q.ti * q.tj;  // at most 128 only at 128 x 128
  int64_t sp = tiles <= 128 ? 256 / tiles : 1;
  const int64_t most = K < 4096 ? 1 : K / (tiles <= 32 ? 1024 : 4096);
  if (sp > most) sp = most;
  if (sp > 8) sp = 8;
  q.splits = sp < 1 ? 1 : (int)sp;
  return q;
}

template <int FX, int IM, int JM, int WI, bool SPLIT>
void launch(const MxgParams& p, hipStream_t st) {
  const dim3 grid((unsigned)(p.ti * p.tj), (unsigned)p.splits), block(128 * WI);
  const uintptr_t at = (uintptr_t)p.Xs | (uintptr_t)p.Ws;  // the scale loads' alignment
  if (p.K % MxgShape<FX, IM, JM, WI, false>::BK || at % 4)
    hipLaunchKernelGGL((mxg_kernel<FX, IM, JM, WI, true, false, SPLIT>), grid, block, 0, st, p);
  else if (p.K % 512 || at % 16)
    hipLaunchKernelGGL((mxg_kernel<FX, IM, JM, WI, false, false, SPLIT>), grid, block, 0, st, p);
  else
    hipLaunchKernelGGL((mxg_kernel<FX, IM, JM, WI, false, true, SPLIT>), grid, block, 0, st, p);
}

// p.splits and p.ksteps are set so that every split has a step
template <int FX>
void launch_shape(MxgParams& p, const Plan& q, hipStream_t st) {
  const int64_t steps = cdiv(p.K, FX == LQ_MX_FP4 ? 256 : 128);
  p.ksteps = (int32_t)cdiv(steps, q.splits);
  p.splits = (int32_t)cdiv(steps, p.ksteps);
  if (q.rows_j == 256)
    launch<FX, 2, 4, 4, false>(p, st);
  else if (q.rows_i == 256)
    launch<FX, 2, 2, 4, false>(p, st);
  else if (q.splits == 1)
    launch<FX, 2, 2, 2, false>(p, st);
  else
    launch<FX, 2, 2, 2, true>(p, st);
}

}  // namespace

namespace dispatch {

size_t mx_gemm_ws_bytes(int64_t M, int64_t N, int64_t K) {
  const Plan q = plan(M, N, K);
  return q.splits > 1 ? (size_t)q.splits * M * N * 4 : 0;
}

int mx_gemm(const lq_mx_tensor& X, const lq_mx_tensor& W, const float* T, const void* B,
            int64_t r, float s, void* Y, void* part, hipStream_t st) {
  MxgParams p;
  p.X = X.codes;
  p.Xs = X.scales;
  p.W = W.codes;
  p.Ws = W.scales;
  p.T = T;
  p.B = (const uint16_t*)B;
  p.Y = (uint16_t*)Y;
  p.part = (float*)part;
  p.M = X.rows;
  p.N = W.rows;
  p.K = X.cols;
  p.r = (int32_t)r;
  p.s = s;
  const Plan q = plan(p.M, p.N, p.K);
  p.ti = q.ti;
  p.tj = q.tj;
  p.splits = q.splits;
  if (X.format == LQ_MX_FP8)
    launch_shape<LQ_MX_FP8>(p, q, st);
  else
    launch_shape<LQ_MX_FP4>(p, q, st);
  int e = hip_fail(hipGetLastError(), "mx_gemm launch");
  if (e || q.splits == 1) return e;
  return mx_sum_splits(p.part, p.Y, p.M * p.N, p.splits, st);
}

}  // namespace dispatch
}  // namespace lq
