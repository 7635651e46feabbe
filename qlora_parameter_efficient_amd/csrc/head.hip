// Loss of a frozen large-vocabulary head and the gradient of its input
// (lq_head_loss).
//
//   z = c H W^T,  lse_i = log sum_v exp z_iv,  loss_i = sum_j p_ij (lse_i - z_i,t_ij)
//   g_i D = w_i c (P_i softmax(z_i) - sum_j p_ij e(t_ij)),  P_i = sum_j p_ij
//   dH_i = g_i (D W)_i,  g_i such that D's largest entry is 1
//
// Two products of 2 M V K operations bound it; the softmax between them costs
// memory traffic only.  A piece of rows at a time: its logits as float32 (a bf16
// logit of 16 would be off by 0.03, three percent of its probability) and then D as
// bf16 (half a step, 2^-8, of each entry but the largest) lie in the workspace.  Kept
// logits are cheaper than formed ones: 12 bytes of traffic per logit against 2 K
// operations.
//
// Products.  Four waves own a 256 (weight side: v or k) x 64 JM (rows m) tile,
// wave (wi, wj) its 128 x 32 JM block, in 32 x 32 x 16 products, the weight side
// being the MFMA rows, so that a lane holds four consecutive outputs of a row.
// Steps of 64 of the reduction, both operands straight from global memory into
// one of two LDS stages (chunk swizzles as below), four 16-wide substeps whose
// operands are read one substep ahead, across the barrier too: it stands before
// the last substep's products, when every wave holds its last operands and the
// next stage has landed, and behind it go the next step's first reads and the
// loads of the step after that.
//   row tiles (H and D; W in z): rows of 128 bytes, chunk c of row x at
//     c ^ (x & 7) ^ (x >> 3 & 1)
//   W in dH: 64 reduction rows v of 512 bytes, chunk c of row v at
//     c ^ 2 (v & 3) ^ 8 (c >> 1 & 1), operands by the transposing LDS read
// The order inside a step is what the rate hangs on: operand reads one behind each
// product (in a burst they fill the LDS queue: dH of 4096 x 32000 x 4096 887 us
// against 881), no branch in the steady loop (824), and the loads of the step after
// next behind the products of two substeps, half behind the barrier and half in the
// next step (766; all behind the barrier, or over three substeps, 4 to 6% more).
//
// Measured at 4096 x 32000 x 4096: logits 871 us (1.23 PFLOP/s; of a tile's 102 us 2 to
// 3 go to its first loads, 6 to the stores of its logits, the rest to 64 steps of
// 1.45 us), softmax 195 (4.0 TB/s), dH 779 (1.38 PFLOP/s).  Over both products the
// matrix units are busy 72% of the cycles and waves wait 16% of theirs.  130 rows:
// logits 69 to 81 us (W once, 3.2 to 3.8 TB/s), dH 66 + 9.
#include <type_traits>

#include "block.h"
#include "mx_tile.h"

namespace lq {
namespace {

constexpr int kTI = 256;                    // weight side of a tile
constexpr int kStep = 64;                   // reduction per step
constexpr int kWTile = kTI * kStep * 2;     // weight tile of a step
constexpr int kThreads = 256;

struct ProdParams {
  const uint16_t* P;  // rows x KR (H or D)
  const uint16_t* Q;  // z: W, NI x KR.  dH: W, KV x NI (KV <= KR rows)
  float* Z;           // z: splits x rows x ldz; dH, split: splits x rows x NI
  uint16_t* Y;        // dH, not split: rows x NI
  const float* g;     // ... each row times g
  int32_t M, NI, KR, KV, ldz;
  float scale;
  int32_t ti, tj, splits, ksteps;
  int32_t i_first;    // first output column
};

typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u32x2 read_turned(uint32_t addr) {
  typedef __attribute__((address_space(3))) s16x4* lds_ptr;
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(uintptr_t)addr));
}

// physical chunk of logical chunk c in reduction row v of the turned weight
// tile, and back
__device__ __forceinline__ int tphys(int c, int v) { return c ^ (2 * (v & 3)) ^ (8 * ((c >> 1) & 1)); }
__device__ __forceinline__ int tlogical(int p, int v) {
  return p ^ (2 * (v & 3)) ^ (8 * (((p >> 1) & 1) ^ (v & 1)));
}

// 16 bytes per lane from base + off to LDS at lds + 16 lane; the kernel waits
// for them itself
__device__ __forceinline__ void dma16(const char* base, uint32_t off, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %2\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %0, %1"
      :
      : "v"(off), "s"(base), "s"(lds)
      : "memory", "m0");
}

// TR: the product dH = D W (W read turned); else z = c H W^T.  JM: 32-row
// blocks per wave.
template <bool TR, int JM>
__global__ __launch_bounds__(kThreads) void head_product_kernel(ProdParams p) {
  constexpr int TJ = 64 * JM, kPTile = TJ * kStep * 2, kStage = kWTile + kPTile;
  __shared__ __attribute__((aligned(1024))) char smem[2 * kStage];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wi = wave & 1, wj = wave >> 1;
  const int h = lane >> 5, l32 = lane & 31;

  // Workgroup b runs on XCD b % 8: each XCD has a contiguous range of the
  // (split, tile) list, in groups of four row tiles that share weight rows
  const int ntiles = p.ti * p.tj;
  const int w = xcd_tile(blockIdx.x, ntiles * p.splits);
  const int split = w / ntiles, t = w - split * ntiles;
  constexpr int GJ = 4;
  const int grp = t / (GJ * p.ti), in = t - grp * GJ * p.ti;
  const int gj = p.tj - grp * GJ < GJ ? p.tj - grp * GJ : GJ;
  const int i0 = p.i_first + (in / gj) * kTI, j0 = (grp * GJ + in % gj) * TJ;
  const int NI = p.NI, KR = p.KR, M = p.M;
  const int steps = KR / kStep;
  const int ka = split * p.ksteps;
  const int kb = ka + p.ksteps < steps ? ka + p.ksteps : steps;

  const uint32_t sbase = mx_lds_addr(smem);
  uint32_t poff[2 * JM], qoff[8];
#pragma unroll
  for (int u = 0; u < 2 * JM; ++u) {
    const int row = 16 * JM * wave + 8 * u + (lane >> 3);
    const int m = j0 + row < M ? j0 + row : M - 1;
    poff[u] = ((uint32_t)m * KR + 8 * ((lane & 7) ^ mx_swz128(row))) * 2;
  }
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    if (!TR) {
      const int row = 64 * wave + 8 * u + (lane >> 3);
      const int n = i0 + row < NI ? i0 + row : NI - 1;
      qoff[u] = ((uint32_t)n * KR + 8 * ((lane & 7) ^ mx_swz128(row))) * 2;
    } else {
      const int v = 16 * wave + 2 * u + (lane >> 5);
      const int c = i0 + 8 * tlogical(lane & 31, v);
      qoff[u] = ((uint32_t)v * NI + (c < NI ? c : NI - 8)) * 2;
    }
  }
  const char* pbase = reinterpret_cast<const char*>(p.P);
  const char* qbase = reinterpret_cast<const char*>(p.Q);
  const int64_t qstep = TR ? (int64_t)kStep * NI * 2 : kStep * 2;  // bytes from step to step
  // load u (0 .. 2 JM + 7) of a step into stage b; qb, pb: the step's operands;
  // past: rows of the step beyond W's last (which they read instead)
  auto issue = [&](const char* qb, const char* pb, int past, int b, int u) {
    const uint32_t st = sbase + b * kStage;
    if (u >= 8) {
      dma16(pb, poff[u - 8], st + kWTile + (16 * JM * wave + 8 * (u - 8)) * 128);
    } else if (!TR) {
      dma16(qb, qoff[u], st + (64 * wave + 8 * u) * 128);
    } else {
      uint32_t off = qoff[u];
      if (past > 0) {
        const int over = 16 * wave + 2 * u + (lane >> 5) + past - (kStep - 1);
        off -= over > 0 ? (uint32_t)over * NI * 2 : 0u;
      }
      dma16(qb, off, st + (16 * wave + 2 * u) * 512);
    }
  };
  // loads u0 .. u1 - 1 of step kt
  auto issue_some = [&](int kt, int b, int u0, int u1) {
#pragma unroll
    for (int u = u0; u < u1; ++u)
      issue(qbase + kt * qstep, pbase + (int64_t)kt * kStep * 2,
            TR ? kt * kStep + kStep - p.KV : 0, b, u);
  };

  const int sw = mx_swz128(l32);
  const uint32_t prow = (uint32_t)((32 * JM * wj + l32) * 128);
  const uint32_t qrow = (uint32_t)((128 * wi + l32) * 128);
  uint32_t cx[4], qtr[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) cx[s] = (uint32_t)(((2 * s + h) ^ sw) << 4);
  if (TR) {
    const int gc = l32 & 15, half = l32 >> 4, vlo = gc >> 2;
#pragma unroll
    for (int ns = 0; ns < 4; ++ns) {
      const int col = 128 * wi + 32 * ns + 16 * half + 4 * (gc & 3);
      qtr[ns] = (uint32_t)((8 * h + vlo) * 512 + tphys(col >> 3, vlo) * 16 + (col & 7) * 2);
    }
  }
  // operand read i of substep s (JM + 4: the activation side's, the weight side's)
  constexpr int kReads = JM + 4;
  auto load_frag = [&](uint32_t st, int s, int i, u32x4 (&wf)[4], u32x4 (&xf)[JM]) {
    if (i < JM) {
      xf[i] = mx_read16(st + kWTile + prow + i * 32 * 128 + cx[s]);
    } else if (!TR) {
      wf[i - JM] = mx_read16(st + qrow + (i - JM) * 32 * 128 + cx[s]);
    } else {
      const uint32_t a = st + (uint32_t)(16 * s * 512) + qtr[i - JM];
      const u32x2 lo = read_turned(a), hi = read_turned(a + 4 * 512);
      wf[i - JM] = u32x4{lo[0], lo[1], hi[0], hi[1]};
    }
  };

  f32x16 acc[4][JM];
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < JM; ++b)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[a][b][v] = 0.0f;
  u32x4 wf[2][4], xf[2][JM];
  constexpr int kLoads = 8 + 2 * JM, kHalf = kLoads / 2;
  // products among which a substep's reads go
  constexpr int kSpread = JM == 1 ? 3 : 2 * JM + JM / 2;

  // One step on stage B.  STEADY: step kt + 2 exists and is whole, and no branch
  // parts the products; else it is loaded at once, if it exists.
  auto step = [&](int kt, auto stage, auto steady) {
    constexpr int B = decltype(stage)::value;
    constexpr bool STEADY = decltype(steady)::value;
    const char* qb = qbase + (kt + 2) * qstep;
    const char* pb = pbase + (int64_t)(kt + 2) * kStep * 2;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int c = s & 1;
      const uint32_t st = sbase + (s < 3 ? B : B ^ 1) * kStage;
      if (s == 3) {
        // every wave holds its last operands of this stage; the next has landed
        mx_wait_loads();
        __syncthreads();
        if (!STEADY && kt + 2 < kb) issue_some(kt + 2, B, 0, kHalf);
      }
      if (!STEADY && s == 0 && kt + 1 < kb) issue_some(kt + 1, B ^ 1, kHalf, kLoads);
      __builtin_amdgcn_sched_barrier(0);
      // one read behind each product, from the first on: a burst of reads fills
      // the LDS queue and holds back the products behind it
#pragma unroll
      for (int k = 0; k < 4 * JM; ++k) {
        acc[k / JM][k % JM] = mfma32(wf[c][k / JM], xf[c][k % JM], acc[k / JM][k % JM]);
#pragma unroll
        for (int i = k * kReads / kSpread; i < (k + 1) * kReads / kSpread && i < kReads; ++i)
          load_frag(st, (s + 1) & 3, i, wf[c ^ 1], xf[c ^ 1]);
        if (STEADY && s == 3) {
#pragma unroll
          for (int u = k * kHalf / (4 * JM); u < (k + 1) * kHalf / (4 * JM); ++u)
            issue(qb, pb, 0, B, u);
        }
        if (STEADY && s == 0) {
#pragma unroll
          for (int u = k * kHalf / (4 * JM); u < (k + 1) * kHalf / (4 * JM); ++u)
            issue(qb - qstep, pb - kStep * 2, 0, B ^ 1, kHalf + u);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using Yes = std::integral_constant<bool, true>;
  using No = std::integral_constant<bool, false>;
  {
    issue_some(ka, 0, 0, kLoads);
    mx_wait_loads();
    __syncthreads();
    if (ka + 1 < kb) issue_some(ka + 1, 1, 0, kHalf);
#pragma unroll
    for (int i = 0; i < kReads; ++i) load_frag(sbase, 0, i, wf[0], xf[0]);
    // the last step of W's rows may be short
    const int whole = TR && kb * kStep > p.KV ? kb - 1 : kb;
    int kt = ka;
    for (; kt + 3 < whole; kt += 2) {
      step(kt, I0{}, Yes{});
      step(kt + 1, I1{}, Yes{});
    }
#pragma unroll 1
    for (; kt + 1 < kb; kt += 2) {
      step(kt, I0{}, No{});
      step(kt + 1, I1{}, No{});
    }
    if (kt < kb) step(kt, I0{}, No{});
  }

  if (!TR || p.splits > 1) {
    // float32, by whole lines: each wave turns 32 rows of its block at a time in
    // LDS of its own (rows of 512 bytes, chunk c at c ^ (row & 15)).  From the
    // accumulators, 32 bytes of a row at once, 4096 x 32000 x 4096 takes 1807 us
    // against 1792
    __syncthreads();
    const int ld = TR ? NI : p.ldz;
    const uint32_t mine = sbase + wave * 32 * 512;
    float* out = p.Z + (int64_t)split * M * ld;
    typedef __attribute__((address_space(3))) f32x4* lds_f4;
#pragma unroll
    for (int ms = 0; ms < JM; ++ms) {
#pragma unroll
      for (int ns = 0; ns < 4; ++ns)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x16& x = acc[ns][ms];
          const int chunk = 8 * ns + 2 * q + h;
          *(lds_f4)(uintptr_t)(mine + l32 * 512 + ((chunk ^ (l32 & 15)) << 4)) =
              TR ? f32x4{x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]}
                 : f32x4{p.scale * x[4 * q], p.scale * x[4 * q + 1], p.scale * x[4 * q + 2],
                         p.scale * x[4 * q + 3]};
        }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      const int i = i0 + 128 * wi + 4 * l32;
#pragma unroll
      for (int it = 0; it < 16; ++it) {
        const int row = 2 * it + h, m = j0 + 32 * JM * wj + 32 * ms + row;
        const f32x4 v = *(lds_f4)(uintptr_t)(mine + row * 512 + ((l32 ^ (row & 15)) << 4));
        if (m < M && i < ld)  // ld and i are multiples of 4
          *reinterpret_cast<f32x4*>(out + (int64_t)m * ld + i) = v;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
    return;
  }
  // bf16: the tile through LDS (row j of 512 bytes, chunk c at c ^ (j & 15)), whole
  // output lines from there
  float gain[JM];
#pragma unroll
  for (int ms = 0; ms < JM; ++ms) {
    const int m = j0 + 32 * JM * wj + 32 * ms + l32;
    gain[ms] = p.g[m < M ? m : M - 1];
  }
  __syncthreads();
#pragma unroll
  for (int ms = 0; ms < JM; ++ms) {
    const int j = 32 * JM * wj + 32 * ms + l32;
    const float gm = gain[ms];
#pragma unroll
    for (int ns = 0; ns < 4; ++ns)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = 128 * wi + 32 * ns + 8 * q + 4 * h;
        const f32x16& x = acc[ns][ms];
        typedef __attribute__((address_space(3))) u32x2* lds_ptr;
        *(lds_ptr)(uintptr_t)(sbase + (uint32_t)(j * 512 + (((i >> 3) ^ (j & 15)) * 16) + (i & 7) * 2)) =
            u32x2{pack_bf16x2(gm * x[4 * q], gm * x[4 * q + 1]),
                  pack_bf16x2(gm * x[4 * q + 2], gm * x[4 * q + 3])};
      }
  }
  __syncthreads();
  const int cl = tid & 31;
#pragma unroll 4
  for (int it = 0; it < 8 * JM; ++it) {
    const int j = 8 * it + (tid >> 5);
    const u32x4 v = mx_read16(sbase + (uint32_t)(j * 512 + ((cl ^ (j & 15)) << 4)));
    if (j0 + j < M && i0 + 8 * cl < NI)
      *reinterpret_cast<u32x4*>(p.Y + (int64_t)(j0 + j) * NI + i0 + 8 * cl) = v;
  }
}

// ---------------------------------------------------------------- softmax
// One workgroup per row: its maximum, its sum of exponentials, the loss, and D.
// The row stays in registers from its one read to D's store; what does not fit
// (past 65536 columns) is read three times.

struct RowParams {
  const float* Z;     // splits x rows x ldz
  const int32_t* t;   // rows x kt
  const float* pt;    // rows x kt or NULL
  const float* w;     // rows or NULL
  float* loss;
  float* lse;
  uint16_t* D;        // rows x ldd or NULL
  float* g;           // rows: the gradient of the logits is g D
  int32_t V, ldz, ldd, kt;
  int32_t splits;     // Z: so many partial sums, part elements apart
  int64_t part;
  float scale;
};

constexpr int kMaxTargets = 128;

// The sum, or the largest, over the N (16 or 64) lanes that share lane / N, in every one:
// 16 lanes by moves within the row (lane ^ 1, ^ 2, mirrored within eight and sixteen)
template <bool MAX, int N>
__device__ __forceinline__ float lanes(float v) {
  auto join = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
#define LQ_JOIN(ctrl) \
  v = join(v, __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(v), ctrl, 0xF, 0xF, false)))
  LQ_JOIN(0xB1);
  LQ_JOIN(0x4E);
  LQ_JOIN(0x141);
  LQ_JOIN(0x140);
#undef LQ_JOIN
#pragma unroll
  for (int o = 16; o < N; o *= 2) v = join(v, __shfl_xor(v, o));
  return v;
}
template <int N = 64>
__device__ __forceinline__ float lanes_sum(float v) {
  return lanes<false, N>(v);
}
template <int N = 64>
__device__ __forceinline__ float lanes_max(float v) {
  return lanes<true, N>(v);
}

// T threads; Q: groups of four values per thread that stay in registers.  Wave 0 has the
// targets, two a lane at most (lane and lane + 64): in every wave, what there is to do
// for 16 of them costs as much as the row.  Scalar registers: with more than 80 (it
// would take 97) a compute unit holds one workgroup instead of two (rows of 1000: 30 us
// against 20 for 2048 of them).
template <int T, int Q>
__global__ __launch_bounds__(T) __attribute__((amdgpu_num_sgpr(80))) void head_row_kernel(RowParams p) {
  constexpr int W = T / 64;
  __shared__ float waves[3][W];  // of each wave: its maximum, its sum, its largest that stays
  __shared__ float top_target, factor, has_target;
  __shared__ int n_ones;
  __shared__ int tgt[kMaxTargets];
  __shared__ float wgt[kMaxTargets];
  // several targets.  Bit 4 i + k: value x[i][k] of a thread is a target's; and whether
  // one is among those that it reads again
  __shared__ unsigned long long own[T];
  __shared__ uint8_t beyond[T];
  const int tid = threadIdx.x, V = p.V, kt = p.kt;
  const int64_t row = blockIdx.x;
  const float* z = p.Z + row * p.ldz;
  const float ninf = -__builtin_inff();
  int tj[2] = {-1, -1};
  float wj[2] = {0.0f, 0.0f}, zj[2] = {0.0f, 0.0f};
  const float w_row = tid == 0 && p.w ? p.w[row] : 1.0f;
  if (tid == 0) n_ones = 0;
  if (kt > 1) {
    own[tid] = 0;
    beyond[tid] = 0;
  }
  if (tid < 64)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int j = tid + 64 * u;
      if (j >= kt) continue;
      const int t = p.t[row * kt + j];
      if (t >= 0 && t < V) {
        tj[u] = t;
        wj[u] = p.pt ? p.pt[row * kt + j] : 1.0f;
      }
      tgt[j] = tj[u];
      wgt[j] = wj[u];
    }
  const int groups = (V + 3) / 4;
  f32x4 x[Q];
  auto load = [&](int g) {
    f32x4 v = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(z + 4 * g));
    for (int i = 1; i < p.splits; ++i) {
      const f32x4 y = *reinterpret_cast<const f32x4*>(z + i * p.part + 4 * g);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] += y[k];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = 4 * g + k < V ? v[k] : ninf;
    return v;
  };
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int g = tid + T * i;
    x[i] = f32x4{ninf, ninf, ninf, ninf};
    if (g < groups) x[i] = load(g);
  }
  // a target's logit, its weight at the first of several with one index, the others'
  // weights
  bool first[2] = {tj[0] >= 0, tj[1] >= 0};
  float same_w[2] = {wj[0], wj[1]}, other_w[2] = {0.0f, 0.0f};
  if (tid < 64) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (tj[u] >= 0)
        for (int k = 0; k < p.splits; ++k) zj[u] += z[k * p.part + tj[u]];
    if (kt > 1) {
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (64 * u >= kt) break;
        same_w[u] = 0.0f;
        for (int j = 0; j < kt; ++j) {
          const bool same = tgt[j] == tj[u];
          const float w = wgt[j];
          same_w[u] += same ? w : 0.0f;
          other_w[u] += same ? 0.0f : w;
          first[u] &= !same || j >= tid + 64 * u;
        }
      }
    }
  }
  float own_top = ninf;
#pragma unroll
  for (int i = 0; i < Q; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) own_top = fmaxf(own_top, x[i][k]);
  for (int g = tid + T * Q; g < groups; g += T) {
    const f32x4 v = load(g);
#pragma unroll
    for (int k = 0; k < 4; ++k) own_top = fmaxf(own_top, v[k]);
  }
  float top = lanes_max(own_top);
  if ((tid & 63) == 0) waves[0][tid >> 6] = top;
  if (tid < 64) {
    float best = fmaxf(tj[0] >= 0 ? zj[0] : ninf, tj[1] >= 0 ? zj[1] : ninf);
    if (kt > 1) best = lanes_max(best);
    if (tid == 0) top_target = best;
  }
  __syncthreads();
  if (kt > 1 && tid < 64)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (!first[u]) continue;
      const int g = tj[u] >> 2;
      if (g < T * Q)
        atomicOr(&own[g % T], 1ull << (4 * (g / T) + (tj[u] & 3)));
      else
        beyond[g % T] = 1;
    }
#pragma unroll
  for (int i = 0; i < W; ++i) top = fmaxf(top, waves[0][i]);
  // What the exponentials are taken from: an infinite maximum would make inf - inf of
  // itself (from 0 a sum with +inf in it is +inf, of all -inf it is 0, and a NaN stays)
  const bool finite = fabsf(top) < __builtin_inff();
  const float base = finite ? top : 0.0f;
  const bool top_in = finite && top_target == top;  // a target is the largest logit
  // The sum of the exponentials without the first 1 of each thread that has the largest
  // logit (n_ones of them, mostly one): where a target is that logit, 1 - p is the rest
  // over all, not what 1 / sum - 1 leaves of it.
  float sum = 0.0f, big = 0.0f;
#pragma unroll
  for (int i = 0; i < Q; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[i][k] = __expf(x[i][k] - base);
      sum += x[i][k];
    }
  bool one = finite && own_top == top;  // still to leave out
  if (one) {
    atomicAdd(&n_ones, 1);
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < Q; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bool skip = one && x[i][k] == 1.0f;
        sum += skip ? 0.0f : x[i][k];
        one &= !skip;
      }
  }
  for (int g = tid + T * Q; g < groups; g += T) {
    const f32x4 v = load(g);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float e = __expf(v[k] - base);
      const bool skip = one && e == 1.0f;
      sum += skip ? 0.0f : e;
      one &= !skip;
    }
  }
  // The largest exponential that stays in D: 1, or beside such a target the largest of
  // no target's (with one target its entry, all of the others' together, is larger)
  const bool look = kt > 1 && top_in && p.D;
  if (look) {
    __syncthreads();
    const unsigned long long mine = own[tid];
#pragma unroll
    for (int i = 0; i < Q; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        big = fmaxf(big, mine >> (4 * i + k) & 1 ? 0.0f : x[i][k]);
    for (int g = tid + T * Q; g < groups; g += T) {
      const f32x4 v = load(g);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float e = __expf(v[k] - base);
        if (beyond[tid])
          for (int j = 0; j < kt; ++j) e = tgt[j] == 4 * g + k ? 0.0f : e;
        big = fmaxf(big, e);
      }
    }
    big = lanes_max(big);
  }
  sum = lanes_sum(sum);
  if ((tid & 63) == 0) {
    waves[1][tid >> 6] = sum;
    waves[2][tid >> 6] = big;
  }
  __syncthreads();
  float out[3] = {0.0f, 0.0f, 0.0f};  // loss, lse, g
  float dj[2] = {0.0f, 0.0f};         // the targets' entries of D
  if (tid < 64) {
    const float less = lanes_sum<W>(waves[1][tid % W]) + (finite ? (float)(n_ones - 1) : 0.0f);
    sum = finite ? 1.0f + less : less;
    // (lse - z of a target from the differences to the largest logit, which are small
    // where the loss is: lse itself is rounded beside that logit)
    const float log_sum = finite ? log1pf(less) : logf(sum);
    const bool any = (__ballot(tj[0] >= 0) | __ballot(tj[1] >= 0)) != 0;
    float total = wj[0] + wj[1], loss = 0.0f, most = 0.0f;
    if (kt > 1) total = lanes_sum(total);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (tj[u] < 0) continue;
      loss += wj[u] * (log_sum + (base - zj[u]));
      // (total p - weight; of the largest logit with p = 1 - less / sum)
      dj[u] = finite && zj[u] == top ? other_w[u] - total * (less / sum)
                                     : total * (__expf(zj[u] - base) / sum) - same_w[u];
      most = fmaxf(most, fabsf(dj[u]));
    }
    if (kt > 1) {
      loss = lanes_sum(loss);
      most = lanes_max(most);
    }
    // D is the gradient over its largest entry, which is then exact in bf16.  That
    // entry is most of dH, and the same error of it in every row (w and 1 - p are often
    // the same in all) would be dH's error: up to 2^-8, where the others' errors, half
    // of that and of either sign, are mostly lost in dH's own rounding.
    const float stays = look ? lanes_max<W>(waves[2][tid % W]) : top_in ? 0.0f : 1.0f;
    // (at least so much that 1 / most and factor are finite: D's zeros must stay that)
    const float share = fabsf(total / sum);
    most = fmaxf(fmaxf(most, stays * share), 1e-37f * fmaxf(share, 1.0f));
    most = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(most)));
    const float inv = 1.0f / most;
    out[0] = loss;
    out[1] = base + log_sum;
    out[2] = any ? w_row * p.scale * most : 0.0f;
    if (tid == 0) {
      // (a NaN in a row without a target must not reach D)
      has_target = any ? 1.0f : 0.0f;
      factor = total / sum * inv;
    }
    dj[0] *= inv;
    dj[1] *= inv;
  }
  auto store_row = [&] {
    if (tid) return;
    if (p.loss) p.loss[row] = out[0];
    if (p.lse) p.lse[row] = out[1];
    if (p.D) p.g[row] = out[2];
  };
  if (!p.D) return store_row();
  __syncthreads();
  store_row();
  const float f = factor;
  const bool any = has_target != 0.0f;
  uint16_t* d = p.D + row * p.ldd;
  auto store = [&](int g, f32x4 e) {
#pragma unroll
    for (int k = 0; k < 4; ++k) e[k] = any ? e[k] * f : 0.0f;
    *reinterpret_cast<u32x2*>(d + 4 * g) = u32x2{pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3])};
  };
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int g = tid + T * i;
    if (g < p.ldd / 4) store(g, x[i]);
  }
  for (int g = tid + T * Q; g < p.ldd / 4; g += T) {
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (g < groups) {
      v = load(g);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = __expf(v[k] - base);
    }
    store(g, v);
  }
  __syncthreads();  // the targets' entries over what is stored for them
#pragma unroll
  for (int u = 0; u < 2; ++u)
    if (first[u]) d[tj[u]] = f32_to_bf16(dj[u]);
}

// out (bf16) = the splits' sums in order, row i of K times g[i]; K % 8 == 0, n < 2^31
__global__ __launch_bounds__(256) void head_sum_kernel(const float* part, uint16_t* out, const float* g,
                                                       int64_t n, int K, int splits) {
  const int64_t e = 8 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
  if (e >= n) return;
  f32x4 a = {0.0f, 0.0f, 0.0f, 0.0f}, b = a;
  for (int k = 0; k < splits; ++k) {
    const f32x4* q = reinterpret_cast<const f32x4*>(part + k * n + e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] += q[0][i];
      b[i] += q[1][i];
    }
  }
  const float gm = g[(uint32_t)e / (uint32_t)K];
  *reinterpret_cast<u32x4*>(out + e) =
      u32x4{pack_bf16x2(gm * a[0], gm * a[1]), pack_bf16x2(gm * a[2], gm * a[3]),
            pack_bf16x2(gm * b[0], gm * b[1]), pack_bf16x2(gm * b[2], gm * b[3])};
}

// ---------------------------------------------------------------- host

size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

constexpr int kCUs = 256;

struct Shape {
  int jm;  // 32-row blocks per wave: tiles of 64 jm rows
  int64_t ti, tj, splits, ksteps;
};

// Time of a product's launch in units of a 64-wide step of the 256 x 256 tile
// (1.45 us), from sweeps at K = 4096, V = 32000 over 1 to 2048 rows: a round of
// tiles costs 9 such steps outside its loop, a step of the smaller tiles the
// shares below (64-row tiles fit a compute unit twice, and then take 0.87), and
// partial sums their way to memory and back.
double launch_cost(int jm, int64_t rows, int64_t n, int64_t steps, int64_t splits, bool always_part) {
  const int64_t wgs = cdiv(n, kTI) * cdiv(rows, 64 * jm) * splits;
  const bool pairs = jm == 1 && wgs > kCUs;
  const double step = pairs ? 0.87 : jm == 1 ? 0.54 : jm == 2 ? 0.69 : jm == 3 ? 0.84 : 1.0;
  const double parts = always_part && splits == 1 ? 0.0 : (double)(always_part ? splits : splits - 1);
  return (double)cdiv(wgs, pairs ? 2 * kCUs : kCUs) * (9.0 + (double)cdiv(steps, splits) * step) +
         1.2e-6 * parts * (double)rows * (double)n;
}

// Splits of eight steps at least
int64_t split_limit(int64_t steps, int most_splits) {
  const int64_t s = cdiv(steps, 8);
  return s < most_splits ? s : most_splits;
}

// The cheapest tile and number of splits.  ``sums``: the splits are added by a
// launch of their own (dH), not by the softmax (z)
Shape best_shape(int64_t rows, int64_t n, int64_t steps, int most_splits, bool sums) {
  Shape best{};
  double least = 0.0;
  for (int jm = 1; jm <= 4; ++jm) {
    const int64_t tiles = cdiv(n, kTI) * cdiv(rows, 64 * jm);
    for (int fill = 1; fill <= 2; ++fill) {
      int64_t splits = fill * kCUs / tiles;
      const int64_t most = split_limit(steps, most_splits);
      splits = splits < most ? splits : most;
      splits = splits < 1 ? 1 : splits;
      const int64_t ks = cdiv(steps, splits);
      splits = cdiv(steps, ks);
      const double cost = launch_cost(jm, rows, n, steps, splits, sums);
      if (best.jm == 0 || cost < least) {
        least = cost;
        best = Shape{jm, cdiv(n, kTI), cdiv(rows, 64 * jm), splits, ks};
      }
    }
  }
  return best;
}

// Rows of all splits together, of so many rows or fewer, where there are splits: two
// rounds of tiles of up to 256 rows at most
int64_t most_split_rows(int64_t rows, int64_t n, int64_t steps, int most_splits) {
  const int64_t a = split_limit(steps, most_splits) * rows, b = 2 * kCUs / cdiv(n, kTI) * 256;
  return split_limit(steps, most_splits) < 2 ? 0 : a < b ? a : b;
}

constexpr int kZSplits = 4, kDhSplits = 32;
Shape z_shape(int64_t rows, int64_t V, int64_t K) {
  return best_shape(rows, V, K / kStep, kZSplits, false);
}
Shape dh_shape(int64_t rows, int64_t V, int64_t K) {
  return best_shape(rows, K, cdiv(V, kStep), kDhSplits, true);
}

// Columns of z that its first launch takes: all, or whole rounds of tiles, where
// a second launch with smaller tiles is done sooner than a last round of few
int64_t z_first_columns(const Shape& s, int64_t rows, int64_t V, int64_t K) {
  const int64_t tiles = s.ti * s.tj, rounds = tiles / kCUs;
  if (s.splits > 1 || s.jm < 3 || rounds < 1 || tiles % kCUs == 0) return V;
  const int64_t first = rounds * kCUs / s.tj * kTI;
  if (first <= 0 || first >= V) return V;
  const Shape t = best_shape(rows, V - first, K / kStep, 1, false);
  const double two = launch_cost(s.jm, rows, first, K / kStep, 1, false) + 2.0 +
                     launch_cost(t.jm, rows, V - first, K / kStep, 1, false);
  return two < launch_cost(s.jm, rows, V, K / kStep, 1, false) ? first : V;
}

int64_t ld_of(int64_t V) { return cdiv(V, 64) * 64; }

// Rows of a piece: at most 2^28 logits with their padding (1 GiB of float32), whole
// 256-row tiles; at most 2^21, since a launch's first dimension holds fewer than 2^32
// threads and the softmax has 1024 a row
int64_t piece_rows(int64_t M, int64_t V) {
  constexpr int64_t kMost = (int64_t)1 << 21;
  int64_t most = ((int64_t)1 << 28) / ld_of(V) / 256 * 256;
  most = most < 256 ? 256 : most > kMost ? kMost : most;
  return M < most ? M : most;
}

// The workspace of M rows is enough for fewer, those of the last piece among them:
// fewer rows may have more splits.
struct Layout {
  size_t z, d, g, part, end;
};
Layout layout(int64_t M, int64_t V, int64_t K, bool need_dh) {
  const int64_t rows = piece_rows(M, V), split = most_split_rows(rows, V, K / kStep, kZSplits);
  Layout l;
  l.z = 0;
  l.d = up256((size_t)(split > rows ? split : rows) * ld_of(V) * 4);
  l.g = l.d + (need_dh ? up256((size_t)rows * ld_of(V) * 2) : 0);
  l.part = l.g + (need_dh ? up256((size_t)rows * 4) : 0);
  l.end = l.part;
  if (need_dh)
    l.end += up256((size_t)most_split_rows(rows, K, cdiv(V, kStep), kDhSplits) * K * 4);
  return l;
}

template <bool TR>
int launch_product(const ProdParams& p, int jm, hipStream_t st) {
  const dim3 g((unsigned)(p.ti * p.tj * p.splits)), b(kThreads);
  const auto kernel = jm == 1   ? head_product_kernel<TR, 1>
                      : jm == 2 ? head_product_kernel<TR, 2>
                      : jm == 3 ? head_product_kernel<TR, 3>
                                : head_product_kernel<TR, 4>;
  hipLaunchKernelGGL(kernel, g, b, 0, st, p);
  return hip_fail(hipGetLastError(), TR ? "head dH launch" : "head logits launch");
}

// The fewest values per thread that hold the row, since those past its end cost as much
// (us of the whole call with 4, 8 or 13 groups / with 16: 4096 x 16000 x 64 173 / 250,
// 4096 x 32000 x 64 373 / 401, 4000 x 53000 x 64 602 / 613, 2048 x 33000 x 256 264 / 269)
void launch_rows(const RowParams& r, int64_t rows, hipStream_t st) {
  const int64_t ld = r.ldz;
  const auto kernel = ld <= 4096 * 4    ? head_row_kernel<1024, 4>
                      : ld <= 4096 * 8  ? head_row_kernel<1024, 8>
                      : ld <= 4096 * 13 ? head_row_kernel<1024, 13>
                                        : head_row_kernel<1024, 16>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)rows), dim3(1024), 0, st, r);
}

// z of columns [first, end), first a multiple of the tile
int launch_columns(ProdParams p, const Shape& s, int64_t first, int64_t end, hipStream_t st) {
  p.i_first = (int32_t)first;
  p.ti = (int32_t)cdiv(end - first, kTI);
  p.tj = (int32_t)s.tj;
  p.splits = (int32_t)s.splits;
  p.ksteps = (int32_t)s.ksteps;
  return launch_product<false>(p, s.jm, st);
}

}  // namespace

namespace dispatch {

size_t head_loss_ws(int64_t M, int64_t V, int64_t K, int32_t kt, bool need_dh) {
  (void)kt;
  return layout(M, V, K, need_dh).end;
}

int head_loss(const void* H, int64_t M, int64_t V, int64_t K, const void* W, const int32_t* t,
              const float* pt, int32_t kt, const float* w, float scale, float* loss, float* lse,
              void* dH, void* ws, hipStream_t st) {
  const Layout l = layout(M, V, K, dH != nullptr);
  const int64_t piece = piece_rows(M, V), ld = ld_of(V);
  char* base = (char*)ws;
  for (int64_t m0 = 0; m0 < M; m0 += piece) {
    const int64_t rows = M - m0 < piece ? M - m0 : piece;
    ProdParams p{};
    const Shape z = z_shape(rows, V, K);
    p.P = (const uint16_t*)H + m0 * K;
    p.Q = (const uint16_t*)W;
    p.Z = (float*)(base + l.z);
    p.M = (int32_t)rows;
    p.NI = (int32_t)V;
    p.KR = (int32_t)K;
    p.KV = (int32_t)K;
    p.ldz = (int32_t)ld;
    p.scale = scale;
    const int64_t first = z_first_columns(z, rows, V, K);
    int rc = launch_columns(p, z, 0, first, st);
    if (!rc && first < V)
      rc = launch_columns(p, best_shape(rows, V - first, K / kStep, 1, false), first, V, st);
    if (rc) return rc;
    RowParams r;
    r.Z = p.Z;
    r.t = t + m0 * kt;
    r.pt = pt ? pt + m0 * kt : nullptr;
    r.w = w ? w + m0 : nullptr;
    r.loss = loss ? loss + m0 : nullptr;
    r.lse = lse ? lse + m0 : nullptr;
    r.D = dH ? (uint16_t*)(base + l.d) : nullptr;
    r.g = (float*)(base + l.g);
    r.V = (int32_t)V;
    r.ldz = r.ldd = (int32_t)ld;
    r.kt = kt;
    r.splits = (int32_t)z.splits;
    r.part = rows * ld;
    r.scale = scale;
    launch_rows(r, rows, st);
    if ((rc = hip_fail(hipGetLastError(), "head softmax launch"))) return rc;
    if (!dH) continue;
    const Shape s = dh_shape(rows, V, K);
    ProdParams q{};
    q.P = (const uint16_t*)(base + l.d);
    q.Q = (const uint16_t*)W;
    q.Z = (float*)(base + l.part);
    q.Y = (uint16_t*)dH + m0 * K;
    q.g = r.g;
    q.M = (int32_t)rows;
    q.NI = (int32_t)K;
    q.KR = (int32_t)ld;
    q.KV = (int32_t)V;
    q.ti = (int32_t)s.ti;
    q.tj = (int32_t)s.tj;
    q.splits = (int32_t)s.splits;
    q.ksteps = (int32_t)s.ksteps;
    if ((rc = launch_product<true>(q, s.jm, st))) return rc;
    if (s.splits > 1) {
      const int64_t n = rows * K;
      hipLaunchKernelGGL(head_sum_kernel, dim3((unsigned)cdiv(n, 2048)), dim3(256), 0, st,
                         (const float*)q.Z, q.Y, r.g, n, (int)K, (int)s.splits);
      if ((rc = hip_fail(hipGetLastError(), "head sums launch"))) return rc;
    }
  }
  return LQ_OK;
}

}  // namespace dispatch
}  // namespace lq
