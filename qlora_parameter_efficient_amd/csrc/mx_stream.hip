// Forward of few rows (M <= 64, bf16 activations) on an MXFP4 base.
//
//   Y = X W^T + s T B^T,  T = X A^T
//
// Few rows are bound by streaming W (4.25 bits per weight).  A workgroup of 16
// waves takes a contiguous range of 16-row blocks of W, so that X is staged in
// LDS once per workgroup (at M = 13, N = 11008 one block each re-stages 106 KB
// of X for every 34 KB of W).  Lane (q, l16) of wave w takes row n0 + l16 and the
// K blocks 4 t + q, t = w, w + 16, ...: 16 code bytes and one scale byte, turned
// into 32 bf16 weights by 16 conversion instructions and multiplied by four
// v_mfma_f32_16x16x32_bf16 (X padded to 16 rows; the 32 reduction elements of
// a lane are relabelled so that they are contiguous on both operands).  The
// next loads go out before the current products.  The waves' sums of a block
// meet in LDS; one wave, another for each block, adds them, applies the
// expand and stores, while the others stream on.  The expand is at most four
// more matrix instructions, T in two bf16 parts (h = bf16(t), l = bf16(t - h):
// off by 2^-17 of t, far below the output's rounding); as a loop of float32
// products over r = 64 ranks it took 3 us per block.
//
// T comes from a small kernel first, as partial sums over ranges of K; but for
// a few tokens (M <= 4, r <= 16, r K <= 65536) every workgroup forms all of T
// itself, wave j the products of rank j with A's row read in whole lines.  That
// spares a launch, which is what a host that issues single calls waits for, and
// costs the device time that grows with M and with r K.  N = K = 4096, r = 16,
// this / two launches: calls from the host M = 1 8.7 / 10.9 us, 2 9.7 / 10.8, 4
// 12.1 / 10.9; in a replayed graph 8.7 to 9.2 / 8.1, 10.1 / 8.2 and 12.5 / 8.3.  So
// it pays for one or two tokens off a graph.  Past r K = 65536, K = 11008, M = 1:
// calls 15.3 / 13.0, in a graph 16.1 / 13.6.
//
// Measured: M = 1, N = K = 4096, r = 16 9.5 us (8.9 MB of W: 0.94 TB/s; without an
// adapter 5.0), M = 13, N = 11008, K = 4096, r = 64 14.4 us (24 MB: 1.7 TB/s) and
// 4.1 for T.  Past 16 rows W is read again for every 16: N = K = 4096, r = 16, M = 17,
// 32, 48 and 64 take 16, 17, 24 and 30 us.
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
  const uint16_t* A;      // r x K (TI)
  const float* Tp;        // [chunk][kTP][16][r] (not TI)
  const uint16_t* B;      // N x r
  float* T_out;           // M x r or NULL (written by the chunk's workgroup 0)
  int32_t r;
  float s;
  uint16_t* Y;
};

constexpr int kTPitch = 72;  // bf16 elements per row of T's parts and of B in LDS

// XS: bf16 elements of X staged in LDS (rows of K, 16-byte chunk c of row m at
// c ^ (m & 15): needs K % 128 == 0); 0: X read from global memory.
// TI: T formed here (inline_t below).
template <int XS, bool TI>
__global__ __launch_bounds__(64 * kWaves) void mx_stream_kernel(StreamParams p) {
  constexpr int NT = 64 * kWaves;
  constexpr int CH = 2;  // K blocks per lane and round
  __shared__ __attribute__((aligned(16))) uint16_t xs[XS > 0 ? XS : 8];
  constexpr int NB = XS > 16384 ? 1 : 2;  // buffers of the blocks' sums (what fits)
  __shared__ f32x4 part[NB][kWaves][64];
  // T's two parts and the block's rows of B, ranks r .. 63 zero
  __shared__ __attribute__((aligned(16))) uint16_t tT[2][16 * kTPitch];
  __shared__ __attribute__((aligned(16))) uint16_t tB[NB][16 * kTPitch];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int l16 = lane & 15, q = lane >> 4;
  const int64_t m0 = 16 * (int64_t)blockIdx.y;
  const int M = (int)(p.M - m0 < 16 ? p.M - m0 : 16);
  const int64_t N = p.N, K = p.K;
  const int r = p.r;
  const uint16_t* X = p.X + m0 * K;
  const int nblocks = (int)(N / 16);
  const int b0 = (int)((int64_t)blockIdx.x * nblocks / gridDim.x);
  const int b1 = (int)((int64_t)(blockIdx.x + 1) * nblocks / gridDim.x);

  const bool mrow = l16 < M;
  const int xm = mrow ? l16 : 0;
  const int G = (int)(K / 32);
  const int rounds = (G + 4 * kWaves * CH - 1) / (4 * kWaves * CH);
  struct In {
    MxBlock<LQ_MX_FP4> w[CH];
  };
  // K block of chain i in a round, clamped; a lane past K is masked
  auto kblock = [&](int round, int i) { return 4 * (wave + kWaves * (CH * round + i)) + q; };
  auto load = [&](int blk, int round, In& in) {
    const int64_t n = 16 * (int64_t)blk + l16;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      int g = kblock(round, i);
      g = g < G ? g : 0;
      in.w[i].load(p.codes + n * (K / 2) + 16 * g, p.scales + n * (K / 32) + g);
    }
  };
  In in[2];

  // rank ``wave`` of A for T: elements 512 i + 8 lane .. of its row
  constexpr int TA = 8;
  u32x4 af[TI ? TA : 1];
  const uint16_t* arow = TI ? p.A + (int64_t)(wave < r ? wave : 0) * K : nullptr;
  auto load_a = [&](int k0) {
#pragma unroll
    for (int i = 0; i < TA; ++i) {
      const int k = k0 + 512 * i + 8 * lane;
      af[TI ? i : 0] = *reinterpret_cast<const u32x4*>(arow + (k < (int)K ? k : 0));
    }
  };
  if constexpr (TI) load_a(0);
  if (XS > 0) {
    // all of a thread's chunks are loaded before any is stored; the first
    // weights go out behind them (loads return in order), so that T is formed
    // while they arrive
    constexpr int XC = XS / 8 / NT > 0 ? XS / 8 / NT : 1;
    const int nxc = (int)(M * K / 8), rowc = (int)(K / 8);
    u32x4 v[XC];
#pragma unroll
    for (int i = 0; i < XC; ++i) {
      const int c = tid + NT * i;
      v[i] = *reinterpret_cast<const u32x4*>(X + 8 * (int64_t)(c < nxc ? c : nxc - 1));
    }
    __builtin_amdgcn_sched_barrier(0);
    load(b0, 0, in[0]);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < XC; ++i) {
      const int c = tid + NT * i;
      const int m = c / rowc, ch = c - m * rowc;
      if (c < nxc) *reinterpret_cast<u32x4*>(xs + m * (int)K + 8 * (ch ^ (m & 15))) = v[i];
    }
  } else {
    load(b0, 0, in[0]);
  }
  auto xchunk = [&](int ch) {  // 8 values of row xm at 8 ch
    return XS > 0 ? *reinterpret_cast<const u32x4*>(xs + xm * (int)K + 8 * (ch ^ (xm & 15)))
                  : *reinterpret_cast<const u32x4*>(X + xm * K + 8 * (int64_t)ch);
  };
  // thread (em, ej): element (em, ej) of T, and of each block's rows of B
  static_assert(NT == 16 * 64, "one element of T and of B per thread");
  const int em = tid >> 6, ej = tid & 63;
  auto load_b = [&](int blk) {
    return ej < r ? p.B[(16 * (int64_t)blk + em) * r + ej] : (uint16_t)0;
  };
  uint16_t bnext = 0;
  if (r) {
    float v = 0.0f;
    if constexpr (TI) {
      __syncthreads();  // X is in LDS
      float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int k0 = 0;; k0 += 512 * TA) {
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          if (m >= M) break;  // uniform
#pragma unroll
          for (int i = 0; i < TA; ++i) {
            const int k = k0 + 512 * i + 8 * lane;
            const bool ok = k < (int)K;
            const u32x4 x = *reinterpret_cast<const u32x4*>(
                xs + m * (int)K + 8 * (((ok ? k : 0) >> 3) ^ (m & 15)));
            float d = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              d = fmaf(hi_bf16(x[e]), hi_bf16(af[i][e]), fmaf(lo_bf16(x[e]), lo_bf16(af[i][e]), d));
            t[m] += ok ? d : 0.0f;
          }
        }
        if (k0 + 512 * TA >= (int)K) break;
        load_a(k0 + 512 * TA);
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        if (m >= M) break;
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) t[m] += __shfl_xor(t[m], o, 64);
        if (ej == m && em < r) v = t[m];  // wave em's sums: lane m keeps row m
      }
      // element (m, rank) from lane m of wave ``rank``; zeros elsewhere
      if (ej < M && em < r) {
        const float vh = (float)(__bf16)v;
        tT[0][ej * kTPitch + em] = f32_to_bf16(v);
        tT[1][ej * kTPitch + em] =
            fabsf(vh) < __builtin_inff() ? f32_to_bf16(v - vh) : (uint16_t)0;
        if (p.T_out && blockIdx.x == 0) p.T_out[(m0 + ej) * r + em] = v;
      }
      if (em >= M || ej >= r) {
        tT[0][em * kTPitch + ej] = 0;
        tT[1][em * kTPitch + ej] = 0;
      }
    } else {
      if (em < M && ej < r) {
        const float* t = p.Tp + (int64_t)blockIdx.y * kTP * 16 * r + em * r + ej;
#pragma unroll
        for (int b = 0; b < kTP; ++b) v += t[b * 16 * r];
        if (p.T_out && blockIdx.x == 0) p.T_out[(m0 + em) * r + ej] = v;
      }
      const float vh = (float)(__bf16)v;
      tT[0][em * kTPitch + ej] = f32_to_bf16(v);
      tT[1][em * kTPitch + ej] =
          fabsf(vh) < __builtin_inff() ? f32_to_bf16(v - vh) : (uint16_t)0;
    }
    bnext = load_b(b0);
  }
  __syncthreads();

  f32x4 acc[CH];
  auto products = [&](int round, const In& v) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int g = kblock(round, i);
      const bool ok = g < G;
#pragma unroll
      for (int d = 0; d < 4; ++d)
        acc[i] = mfma16(sel4(ok, v.w[i].part(d)), sel4(ok && mrow, xchunk(4 * (ok ? g : 0) + d)),
                        acc[i]);
    }
  };
  int cur = 0;
  for (int blk = b0; blk < b1; ++blk) {
    const int buf = (blk - b0) & (NB - 1);
    const int64_t n0 = 16 * (int64_t)blk;
    const uint16_t braw = bnext;
    if (r && blk + 1 < b1) bnext = load_b(blk + 1);
#pragma unroll
    for (int i = 0; i < CH; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int round = 0; round < rounds; ++round) {
      const bool last = round + 1 == rounds;
      const int nb = last ? blk + 1 : blk;
      if (cur == 0) {  // uniform
        if (nb < b1) load(nb, last ? 0 : round + 1, in[1]);
        products(round, in[0]);
      } else {
        if (nb < b1) load(nb, last ? 0 : round + 1, in[0]);
        products(round, in[1]);
      }
      cur ^= 1;
    }
    if (NB == 1) __syncthreads();  // the previous block has been finished
    if (r) tB[buf][em * kTPitch + ej] = braw;
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[0][v] += acc[1][v];
    part[buf][wave][lane] = acc[0];
    __syncthreads();
    // one wave finishes the block; with two buffers, this one is next written
    // after the next block's barrier, which that wave reaches only then
    if (wave == ((blk - b0) & (kWaves - 1))) {
      f32x4 sum = part[buf][0][lane];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) {
        const f32x4 o = part[buf][w][lane];
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] += o[i];
      }
      f32x4 d = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      for (int c = 0; c < r; c += 32) {  // rows n as the A operand, rows m as B
        const int at = l16 * kTPitch + c + 8 * q;
        const u32x4 bf = *reinterpret_cast<const u32x4*>(&tB[buf][at]);
        d = mfma16(bf, *reinterpret_cast<const u32x4*>(&tT[1][at]), d);
        d = mfma16(bf, *reinterpret_cast<const u32x4*>(&tT[0][at]), d);
      }
      float y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = r ? sum[i] + p.s * d[i] : sum[i];
      if (mrow)
        *reinterpret_cast<u32x2*>(p.Y + (m0 + l16) * N + n0 + 4 * q) =
            u32x2{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
    }
  }
}

template <int XS, bool TI>
void launch_stream(const StreamParams& p, unsigned chunks, hipStream_t st) {
  // workgroups: as many as run at once (two per compute unit with a small X),
  // each with the same number of blocks but for one
  const int64_t nb = p.N / 16, most = XS > 16384 ? 256 : 512;
  hipLaunchKernelGGL((mx_stream_kernel<XS, TI>), dim3((unsigned)cdiv(nb, cdiv(nb, most)), chunks),
                     dim3(64 * kWaves), 0, st, p);
}

// T formed by the stream kernel itself (its X must be in LDS)
bool inline_t(int64_t M, int64_t K, int64_t r) {
  return r >= 1 && r <= 16 && M <= 4 && r * K <= 65536 && K % 128 == 0 && M * K <= 16384;
}

}  // namespace

namespace dispatch {

size_t mx_stream_ws_bytes(int64_t M, int64_t K, int64_t r) {
  return inline_t(M, K, r) ? 0 : (size_t)(cdiv(M, 16) * kTP * 16 * r) * 4;
}

int mx_stream_fwd(const void* X, int64_t M, const lq_mx_tensor& W, const void* A, const void* B,
                  int64_t r, float s, void* Y, float* T_out, float* Tp, hipStream_t st) {
  const int64_t K = W.cols;
  const unsigned chunks = (unsigned)cdiv(M, 16);
  const bool ti = inline_t(M, K, r);
  if (r && !ti) {
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
  p.A = (const uint16_t*)A;
  p.Tp = Tp;
  p.B = (const uint16_t*)B;
  p.T_out = T_out;
  p.r = (int32_t)r;
  p.s = s;
  p.Y = (uint16_t*)Y;
  const int64_t xe = (M < 16 ? M : 16) * K;
  if (ti)
    launch_stream<16384, true>(p, chunks, st);
  else if (K % 128 == 0 && xe <= 16384)
    launch_stream<16384, false>(p, chunks, st);
  else if (K % 128 == 0 && xe <= 65536)
    launch_stream<65536, false>(p, chunks, st);
  else
    launch_stream<0, false>(p, chunks, st);
  return hip_fail(hipGetLastError(), "mx_stream launch");
}

}  // namespace dispatch
}  // namespace lq
