// Adapter gradients from an MX tensor of the layer's input:
//
//   dA = s U^T X  (r x K)      dB = s dY^T T  (N x r)
//
// X MXFP8 or MXFP4 (M x K), dY bf16 (M x N), U = dY B and T = X A^T float32
// (M x r).  Both have the form out[j][c] = s sum_m V[m][j] Z[m][c] and run in
// one launch: the grid holds dA's tiles, then dB's.
//
// Precision: the outputs are float32, so V must not be rounded to bf16 before
// the matrix instruction.  It is split into three bf16 parts, v = h + m + l
// with h = bf16(v), m = bf16(v - h), l = bf16(v - h - m): 24 bits, each
// difference exact.  Z is exact in bf16 (E4M3 and E2M1 elements times a power
// of two, but for values below 2^-126), so every product is exact and only
// the float32 sums round.  (The parts of an infinite or NaN v are v, 0, 0.)
//
// A workgroup takes TC columns of Z (256, or 128 where r <= 32) and a range of
// rows in steps of 64.  A step's rows (MX blocks, one or two per thread, or
// bf16 values) and its rows of V are loaded into registers two to four steps ahead,
// converted (V into its parts) and stored in LDS in storage order during the
// previous step's products, and read back as MFMA operands with the row as the
// reduction index by the transposing ds_read_b64_tr_b16; two LDS buffers, one
// barrier per step.  Small r is HBM-bound on Z (1.03 bytes per element of X in
// MXFP8, 2 of dY); at r = 64 the three parts make 6 products per 32 x 32 block
// and their LDS traffic is the limit, which is why the tile is 256 columns wide
// there (the V part of a step is read once per 64 columns of a wave, not per
// 32).  Ranges of rows leave partial sums that mx_grad_reduce_kernel adds in a
// fixed order: no atomics.
//
// Measured (gradients + reduction): M = 2048, N = K = 4096, r = 16 10.7 + 4.8 us
// (25 MB: 2.4 TB/s; short ranges, the fill of the loads ahead bounds it); M =
// 8192, N = 4096, K = 11008, r = 64 71 + 7.6 us (0.67 PFLOP/s over the three parts).
#include "dispatch.h"
#include "mx.h"

namespace lq {
namespace {

constexpr int kThreads = 256;

struct MxGradJob {
  const void* Z;          // MX codes, or bf16 values
  const uint8_t* Zs;      // MX scales
  const float* V;         // M x r
  float* P;               // splits x r x C partial sums
  int64_t C;
  int64_t rows_per_split; // multiple of 64
  int32_t c_tiles, splits;
};

struct MxGradParams {
  MxGradJob job[2];
  int64_t M;
  int32_t r;
  int32_t blocks0;  // workgroups of job 0
};

// LDS row of one m: Z[m][c0 .. c0 + TC - 1], then the h, m and l parts of
// V[m][0 .. RP - 1]; 16-byte chunk q at q ^ (m & 3).  Pitches are 64 or 192
// bytes off a multiple of 256, so four consecutive rows of a transposing read
// fall on distinct banks.
template <int TC, int RP>
struct MxGradShape {
  static constexpr int Pitch = TC + 3 * RP + (RP == 64 ? 32 : 0);  // bf16 elements
  static constexpr int Buf = 64 * Pitch;
};
static_assert((MxGradShape<128, 32>::Pitch * 2) % 256 == 192, "bank spread");
static_assert((MxGradShape<256, 64>::Pitch * 2) % 256 == 192, "bank spread");

typedef short s16x4g __attribute__((ext_vector_type(4)));

__device__ __forceinline__ u32x2 lds_tr(const uint16_t* p) {
  typedef __attribute__((address_space(3))) s16x4g* lds_ptr;
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p)));
}

// the three bf16 parts of v
__device__ __forceinline__ void split3(float v, float& h, float& m, float& l) {
  h = (float)(__bf16)v;
  const float d = v - h;
  const bool fin = fabsf(h) < __builtin_inff();  // also false for NaN
  m = fin ? (float)(__bf16)d : 0.0f;
  l = fin ? (float)(__bf16)(d - m) : 0.0f;
}

// one step's share of Z per thread, NS = TC / 128.  MX: blocks q + 4 i of row
// tid / 4 (q = tid % 4); bf16: chunk tid % 16 + 16 i' of rows tid / 16 + 16 i.
template <int FZ, int NS>
struct Stage {
  MxBlock<FZ> b[NS];
};
template <int NS>
struct Stage<16, NS> {
  u32x4 z[4 * NS];
};

template <int FZ, int TC, int RP, bool V4>
__device__ __forceinline__ void grad_body(const MxGradParams& p, const MxGradJob& jb, int bid,
                                          bool by_col, uint16_t* tiles) {
  constexpr int NS = TC / 128;
  constexpr int JT = RP / 32;
  constexpr int PT = MxGradShape<TC, RP>::Pitch;
  constexpr int NV = RP / 16;  // float4 chunks of V per thread and step
  constexpr int NZ = 4 * NS;   // 16-byte chunks of Z per thread and step
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int h = lane >> 5, l32 = lane & 31;
  const int tl = xcd_tile(bid, jb.c_tiles * jb.splits);
  const int tc = tl % jb.c_tiles, split = tl / jb.c_tiles;
  const int64_t C = jb.C, M = p.M;
  const int64_t c0 = (int64_t)tc * TC;
  const int64_t mbeg = (int64_t)split * jb.rows_per_split;
  int64_t mend = mbeg + jb.rows_per_split;
  mend = mend < M ? mend : M;
  const int steps = mend > mbeg ? (int)cdiv(mend - mbeg, 64) : 0;
  const int r = p.r;

  f32x16 acc[NS][JT];
#pragma unroll
  for (int n = 0; n < NS; ++n)
#pragma unroll
    for (int jt = 0; jt < JT; ++jt)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[n][jt][v] = 0.0f;

  const int zc = tid & 15, zr = tid >> 4;  // bf16 staging
  const int vr = tid >> 2, vq = tid & 3;   // MX staging and V staging
  // columns past C read the tile's first ones and are zeroed when stored
  const char* Zb[NS];
  const uint8_t* Sb[NS];
  bool zok[NS];
#pragma unroll
  for (int n = 0; n < NS; ++n) {
    int64_t col = FZ == 16 ? c0 + 8 * zc + 128 * n : c0 + 32 * (vq + 4 * n);
    zok[n] = col < C;
    col = zok[n] ? col : c0;
    Zb[n] = (const char*)jb.Z + col * FZ / 8;
    Sb[n] = FZ == 16 ? nullptr : jb.Zs + col / 32;
  }
  const int64_t zpitch = C * FZ / 8, spitch = C / 32;

  struct In {
    Stage<FZ, NS> z;
    f32x4 v[NV];
  };
  auto load = [&](int step, In& st) {
    const int64_t m0r = mbeg + 64 * (int64_t)(step < steps ? step : steps - 1);
    if constexpr (FZ == 16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        int64_t m = m0r + zr + 16 * i;
        m = m < mend ? m : mend - 1;
#pragma unroll
        for (int n = 0; n < NS; ++n)
          st.z.z[4 * n + i] = *reinterpret_cast<const u32x4*>(Zb[n] + m * zpitch);
      }
    }
    int64_t m = m0r + vr;
    m = m < mend ? m : mend - 1;
    if constexpr (FZ != 16) {
#pragma unroll
      for (int n = 0; n < NS; ++n)
        st.z.b[n].load((const uint8_t*)Zb[n] + m * zpitch, Sb[n] + m * spitch);
    }
    const float* row = jb.V + m * r;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j0 = 4 * (vq + 4 * i);
      if (V4) {
        st.v[i] = *reinterpret_cast<const f32x4*>(row + (j0 < r ? j0 : 0));
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) st.v[i][e] = row[j0 + e < r ? j0 + e : 0];
      }
    }
  };
  // piece i of a step's stores: NZ chunks of Z, then NV chunks of V in parts
  auto store = [&](int step, const In& st, uint16_t* t, int i) {
    const int64_t m0r = mbeg + 64 * (int64_t)step;
    const bool vok = m0r + vr < mend;
    if (i < NZ) {
      if constexpr (FZ == 16) {
        const int m = zr + 16 * (i & 3), n = i >> 2;
        const bool ok = zok[n] && m0r + m < mend;
        *reinterpret_cast<u32x4*>(t + m * PT + 8 * ((zc + 16 * n) ^ (m & 3))) = sel4(ok, st.z.z[i]);
      } else {
        const int n = i >> 2, d = i & 3;
        *reinterpret_cast<u32x4*>(t + vr * PT + 8 * ((4 * (vq + 4 * n) + d) ^ (vr & 3))) =
            sel4(vok && zok[n], st.z.b[n].part(d));
      }
    } else {
      const int vc = vq + 4 * (i - NZ), j0 = 4 * vc;
      float a[3][4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        split3(vok && j0 + e < r ? st.v[i - NZ][e] : 0.0f, a[0][e], a[1][e], a[2][e]);
#pragma unroll
      for (int q = 0; q < 3; ++q)
        *reinterpret_cast<u32x2*>(t + vr * PT +
                                  8 * ((TC / 8 + q * (RP / 8) + (vc >> 1)) ^ (vr & 3)) +
                                  4 * (vc & 1)) =
            u32x2{pack_bf16x2(a[q][0], a[q][1]), pack_bf16x2(a[q][2], a[q][3])};
    }
  };
  constexpr int NP = NZ + NV;
  // transposing reads: lane group g = lane / 16 of lane c = lane % 16
  const int c = lane & 15, g = lane >> 4;
  const int rbase = (32 * h + (c >> 2)) * PT + 8 * ((2 * (g & 1) + ((c >> 1) & 1)) ^ (c >> 2)) +
                    4 * (c & 1);
  auto frag = [&](const uint16_t* t, int col32, int s) {
    const uint16_t* q = t + rbase + 8 * s * PT + 32 * col32;
    const u32x2 lo = lds_tr(q), hi = lds_tr(q + 4 * PT);
    return u32x4{lo[0], lo[1], hi[0], hi[1]};
  };
  // products of a step, the next step's stores among them
  auto body = [&](int step, const In& nxt, int b) {
    const uint16_t* t = tiles + b * 64 * PT;
    uint16_t* tn = tiles + (b ^ 1) * 64 * PT;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      u32x4 zf[NS];
#pragma unroll
      for (int n = 0; n < NS; ++n) zf[n] = frag(t, NS * wave + n, s);
#pragma unroll
      for (int jt = 0; jt < JT; ++jt)
#pragma unroll
        for (int part = 2; part >= 0; --part) {  // smallest first
          const u32x4 vf = frag(t, TC / 32 + part * JT + jt, s);
#pragma unroll
          for (int n = 0; n < NS; ++n) acc[n][jt] = mfma32(zf[n], vf, acc[n][jt]);
        }
#pragma unroll
      for (int i = NP * s / 4; i < NP * (s + 1) / 4; ++i) store(step + 1, nxt, tn, i);
      __builtin_amdgcn_sched_barrier(0);
    }
    __syncthreads();
  };

  if (steps > 0) {  // uniform
    constexpr int D = RP == 32 ? 4 : 2;  // steps loaded ahead (what the registers hold)
    In in[D];
#pragma unroll
    for (int q = 0; q < D; ++q) load(q, in[q]);
#pragma unroll
    for (int i = 0; i < NP; ++i) store(0, in[0], tiles, i);
    __syncthreads();
    for (int s0 = 0; s0 < steps; s0 += D) {
#pragma unroll
      for (int q = 0; q < D; ++q) {
        if (s0 + q >= steps) break;
        // past the last step: nothing at small r, where a range is a few steps
        // (11 us against 12 at M = 2048, r = 16); the last step again at r >
        // 32, where the branch costs the schedule more (79 us against 71 at M =
        // 8192, K = 11008, N = 4096, r = 64)
        if (RP == 64 || s0 + q + D < steps) load(s0 + q + D, in[q]);
        body(s0 + q, in[(q + 1) % D], q & 1);
      }
    }
  }
  // acc lane l: columns c0 + 32 (NS wave + n) + 8 q + 4 h + i, rank 32 jt + l32;
  // partial sums as [rank][column], or [column][rank] (by_col: dB's layout)
  float* P = jb.P + (int64_t)split * r * C;
#pragma unroll
  for (int n = 0; n < NS; ++n)
#pragma unroll
    for (int jt = 0; jt < JT; ++jt) {
      const int j = 32 * jt + l32;
      if (j >= r) continue;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t cc = c0 + 32 * (NS * wave + n) + 8 * q + 4 * h;
        if (cc >= C) continue;  // C is a multiple of 64
        if (by_col) {
#pragma unroll
          for (int i = 0; i < 4; ++i) P[(cc + i) * r + j] = acc[n][jt][4 * q + i];
        } else {
          *reinterpret_cast<f32x4*>(P + (int64_t)j * C + cc) =
              f32x4{acc[n][jt][4 * q], acc[n][jt][4 * q + 1], acc[n][jt][4 * q + 2],
                    acc[n][jt][4 * q + 3]};
        }
      }
    }
}

template <int FX, int TC, int RP, bool V4>
__global__ __launch_bounds__(kThreads) void mx_grad_kernel(MxGradParams p) {
  __shared__ __attribute__((aligned(16))) uint16_t tiles[2 * MxGradShape<TC, RP>::Buf];
  if ((int)blockIdx.x < p.blocks0)
    grad_body<FX, TC, RP, V4>(p, p.job[0], blockIdx.x, false, tiles);
  else
    grad_body<16, TC, RP, V4>(p, p.job[1], blockIdx.x - p.blocks0, true, tiles);
}

struct MxReduceParams {
  const float* P[2];
  float* out[2];
  int64_t C[2];
  int32_t splits[2];
  int32_t r;
  float s;
  int32_t accumulate;
};

// out = s sum_split P[split] (+ out), dA's elements then dB's, four per thread
// (both counts are multiples of 64); the splits in two interleaved chains
__global__ __launch_bounds__(256) void mx_grad_reduce_kernel(MxReduceParams p) {
  const int64_t idx = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
  const int64_t t0 = (int64_t)p.r * p.C[0];
  const int jb = idx < t0 ? 0 : 1;
  const int64_t total = (int64_t)p.r * p.C[jb];
  const int64_t i = jb ? idx - t0 : idx;
  if (i >= total) return;
  const float* P = p.P[jb] + i;
  const int ns = p.splits[jb];
  f32x4 a[2] = {f32x4{0.0f, 0.0f, 0.0f, 0.0f}, f32x4{0.0f, 0.0f, 0.0f, 0.0f}};
  int t = 0;
  for (; t + 4 <= ns; t += 4) {
    f32x4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = *reinterpret_cast<const f32x4*>(P + (int64_t)(t + u) * total);
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) a[u & 1][e] += v[u][e];
  }
  for (; t < ns; ++t) {
    const f32x4 v = *reinterpret_cast<const f32x4*>(P + (int64_t)t * total);
#pragma unroll
    for (int e = 0; e < 4; ++e) a[t & 1][e] += v[e];
  }
  float* o = p.out[jb] + i;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float v = p.s * (a[0][e] + a[1][e]);
    if (p.accumulate) v += o[e];
    o[e] = v;
  }
}

int tile_cols(int64_t r) { return r <= 32 ? 128 : 256; }

// Ranges of rows: at most 512 (r <= 32: two workgroups fit a compute unit) or
// 256 workgroups per output, so that no partly filled round follows, and at
// least 256 rows each.
int pick_splits(int64_t M, int64_t C, int64_t r) {
  int64_t want = (r <= 32 ? 512 : 256) / cdiv(C, tile_cols(r));
  const int64_t most = cdiv(M, 256);
  if (want > most) want = most;
  return want < 1 ? 1 : (int)want;
}

void set_job(MxGradJob& j, const void* Z, const uint8_t* Zs, const float* V, int64_t M, int64_t C,
             int64_t r, float* P) {
  j.Z = Z;
  j.Zs = Zs;
  j.V = V;
  j.P = P;
  j.C = C;
  j.c_tiles = (int32_t)cdiv(C, tile_cols(r));
  j.splits = pick_splits(M, C, r);
  j.rows_per_split = cdiv(cdiv(M, j.splits), 64) * 64;
}

template <int FX>
void launch_grads(const MxGradParams& p, unsigned blocks, hipStream_t st) {
  const dim3 grid(blocks), block(kThreads);
  const bool v4 = p.r % 4 == 0;
  if (p.r <= 32) {
    if (v4)
      hipLaunchKernelGGL((mx_grad_kernel<FX, 128, 32, true>), grid, block, 0, st, p);
    else
      hipLaunchKernelGGL((mx_grad_kernel<FX, 128, 32, false>), grid, block, 0, st, p);
  } else {
    if (v4)
      hipLaunchKernelGGL((mx_grad_kernel<FX, 256, 64, true>), grid, block, 0, st, p);
    else
      hipLaunchKernelGGL((mx_grad_kernel<FX, 256, 64, false>), grid, block, 0, st, p);
  }
}

}  // namespace

namespace dispatch {

size_t mx_grad_bytes(int64_t M, int64_t N, int64_t K, int64_t r) {
  return (size_t)(pick_splits(M, K, r) * r * K + pick_splits(M, N, r) * r * N) * 4;
}

int mx_grads(const lq_mx_tensor& X, const float* U, const void* dY, const float* T, int64_t N,
             int64_t r, float s, int accumulate, float* dA, float* dB, void* part,
             hipStream_t st) {
  const int64_t M = X.rows, K = X.cols;
  MxGradParams p;
  float* PA = (float*)part;
  float* PB = PA + (int64_t)pick_splits(M, K, r) * r * K;
  set_job(p.job[0], X.codes, X.scales, U, M, K, r, PA);
  set_job(p.job[1], dY, nullptr, T, M, N, r, PB);
  p.M = M;
  p.r = (int32_t)r;
  p.blocks0 = p.job[0].c_tiles * p.job[0].splits;
  const unsigned blocks = (unsigned)(p.blocks0 + p.job[1].c_tiles * p.job[1].splits);
  if (X.format == LQ_MX_FP8)
    launch_grads<LQ_MX_FP8>(p, blocks, st);
  else
    launch_grads<LQ_MX_FP4>(p, blocks, st);
  const int e = hip_fail(hipGetLastError(), "mx_grad launch");
  if (e) return e;
  MxReduceParams q;
  q.P[0] = PA;
  q.P[1] = PB;
  q.out[0] = dA;
  q.out[1] = dB;
  q.C[0] = K;
  q.C[1] = N;
  q.splits[0] = p.job[0].splits;
  q.splits[1] = p.job[1].splits;
  q.r = (int32_t)r;
  q.s = s;
  q.accumulate = accumulate;
  hipLaunchKernelGGL(mx_grad_reduce_kernel, dim3((unsigned)cdiv(r * (K + N), 1024)), dim3(256), 0,
                     st, q);
  return hip_fail(hipGetLastError(), "mx_grad_reduce launch");
}

}  // namespace dispatch
}  // namespace lq
