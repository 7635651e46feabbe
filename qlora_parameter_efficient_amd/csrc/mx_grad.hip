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
// HBM-bound on Z (1.03 bytes per element of X in MXFP8, 2 of dY).  A workgroup
// takes 128 columns of Z and a range of rows in steps of 64: the rows' codes
// (one block of 32 per thread) or bf16 values are loaded several steps ahead,
// converted to bf16 and stored in LDS in storage order with the step's V
// parts beside them, and read back as MFMA operands with the row as the
// reduction index by the transposing ds_read_b64_tr_b16.  Ranges of rows leave
// partial sums that mx_grad_reduce_kernel adds in a fixed order: no atomics.
#include "dispatch.h"
#include "mx.h"

namespace lq {
namespace {

constexpr int kThreads = 256;
constexpr int kTileC = 128;

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

// LDS row of one m: Z[m][c0 .. c0 + 127], then the h, m and l parts of
// V[m][0 .. RP - 1]; 16-byte chunk q at q ^ (m & 3).  Pitches are 64 or 192
// bytes off a multiple of 256, so four consecutive rows of a transposing read
// fall on distinct banks.
template <int RP>
struct MxGradPitch {
  static constexpr int P = RP == 32 ? 224 : 352;  // bf16 elements
};

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

// one step's share of Z per thread.  MX: thread (row = tid / 4, block =
// tid % 4) one block of 32; bf16: chunk tid & 15 of rows tid / 16 + 16 i.
template <int FZ>
struct Stage;
template <>
struct Stage<16> {
  u32x4 z[4];
};
template <>
struct Stage<LQ_MX_FP8> {
  MxBlock<LQ_MX_FP8> b;
};
template <>
struct Stage<LQ_MX_FP4> {
  MxBlock<LQ_MX_FP4> b;
};

template <int FZ, int RP, bool V4>
__device__ __forceinline__ void grad_body(const MxGradParams& p, const MxGradJob& jb, int bid,
                                          uint16_t* tiles) {
  constexpr int JT = RP / 32;
  constexpr int PT = MxGradPitch<RP>::P;
  constexpr int NV = RP / 16;  // float4 chunks of V per thread and step
  constexpr int kAhead = 4;    // steps whose loads are in flight together
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int h = lane >> 5, l32 = lane & 31;
  const int tl = xcd_tile(bid, jb.c_tiles * jb.splits);
  const int tc = tl % jb.c_tiles, split = tl / jb.c_tiles;
  const int64_t C = jb.C, M = p.M;
  const int64_t c0 = (int64_t)tc * kTileC;
  const int64_t mbeg = (int64_t)split * jb.rows_per_split;
  int64_t mend = mbeg + jb.rows_per_split;
  mend = mend < M ? mend : M;
  const int steps = mend > mbeg ? (int)cdiv(mend - mbeg, 64) : 0;
  const int r = p.r;

  f32x16 acc[JT];
#pragma unroll
  for (int jt = 0; jt < JT; ++jt)
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[jt][v] = 0.0f;

  const int zc = tid & 15, zr = tid >> 4;   // bf16 staging
  const int vr = tid >> 2, vq = tid & 3;    // MX staging and V staging
  int64_t zcol = FZ == 16 ? c0 + 8 * zc : c0 + 32 * vq;
  const bool zok = zcol < C;
  zcol = zok ? zcol : C - (FZ == 16 ? 8 : 32);
  const int64_t zpitch = C * FZ / 8, spitch = C / 32;
  const char* Zb = (const char*)jb.Z + zcol * FZ / 8;
  const uint8_t* Sb = jb.Zs + zcol / 32;

  struct In {
    Stage<FZ> z;
    f32x4 v[NV];
  };
  auto load = [&](int64_t m0r, In& st) {
    if constexpr (FZ == 16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        int64_t m = m0r + zr + 16 * i;
        m = m < mend ? m : mend - 1;
        st.z.z[i] = *reinterpret_cast<const u32x4*>(Zb + m * zpitch);
      }
    }
    int64_t m = m0r + vr;
    m = m < mend ? m : mend - 1;
    if constexpr (FZ != 16) st.z.b.load((const uint8_t*)Zb + m * zpitch, Sb + m * spitch);
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
  auto store = [&](int64_t m0r, const In& st, uint16_t* t) {
    const bool vok = m0r + vr < mend;
    if constexpr (FZ == 16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int m = zr + 16 * i;
        const bool ok = zok && m0r + m < mend;
        *reinterpret_cast<u32x4*>(t + m * PT + 8 * (zc ^ (m & 3))) = sel4(ok, st.z.z[i]);
      }
    } else {
#pragma unroll
      for (int d = 0; d < 4; ++d)
        *reinterpret_cast<u32x4*>(t + vr * PT + 8 * ((4 * vq + d) ^ (vr & 3))) =
            sel4(vok && zok, st.z.b.part(d));
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vc = vq + 4 * i, j0 = 4 * vc;
      float a[3][4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        split3(vok && j0 + e < r ? st.v[i][e] : 0.0f, a[0][e], a[1][e], a[2][e]);
#pragma unroll
      for (int q = 0; q < 3; ++q)
        *reinterpret_cast<u32x2*>(t + vr * PT + 8 * ((16 + q * (RP / 8) + (vc >> 1)) ^ (vr & 3)) +
                                  4 * (vc & 1)) =
            u32x2{pack_bf16x2(a[q][0], a[q][1]), pack_bf16x2(a[q][2], a[q][3])};
    }
  };
  // transposing reads: lane group g = lane / 16 of lane c = lane % 16
  const int c = lane & 15, g = lane >> 4;
  const int rbase = (32 * h + (c >> 2)) * PT + 8 * ((2 * (g & 1) + ((c >> 1) & 1)) ^ (c >> 2)) +
                    4 * (c & 1);
  auto frag = [&](const uint16_t* t, int col32, int s) {
    const uint16_t* q = t + rbase + 8 * s * PT + 32 * col32;
    const u32x2 lo = lds_tr(q), hi = lds_tr(q + 4 * PT);
    return u32x4{lo[0], lo[1], hi[0], hi[1]};
  };

  for (int s0 = 0; s0 < steps; s0 += kAhead) {
    In st[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const int sq = s0 + q < steps ? s0 + q : steps - 1;
      load(mbeg + (int64_t)sq * 64, st[q]);
    }
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      if (s0 + q < steps) {  // uniform
        uint16_t* t = tiles + (q & 1) * 64 * PT;
        store(mbeg + (int64_t)(s0 + q) * 64, st[q], t);
        __syncthreads();
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const u32x4 zf = frag(t, wave, s);
#pragma unroll
          for (int jt = 0; jt < JT; ++jt)
#pragma unroll
            for (int part = 2; part >= 0; --part)  // smallest first
              acc[jt] = mfma32(zf, frag(t, 4 + part * JT + jt, s), acc[jt]);
        }
      }
    }
    __syncthreads();
  }
  // acc[jt] lane l: columns c0 + 32 wave + 8 q + 4 h + i, rank j = 32 jt + l32
  float* P = jb.P + (int64_t)split * r * C;
#pragma unroll
  for (int jt = 0; jt < JT; ++jt) {
    const int j = 32 * jt + l32;
    if (j >= r) continue;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t cc = c0 + 32 * wave + 8 * q + 4 * h;
      if (cc < C)  // C is a multiple of 64
        *reinterpret_cast<f32x4*>(P + (int64_t)j * C + cc) =
            f32x4{acc[jt][4 * q], acc[jt][4 * q + 1], acc[jt][4 * q + 2], acc[jt][4 * q + 3]};
    }
  }
}

template <int FX, int RP, bool V4>
__global__ __launch_bounds__(kThreads) void mx_grad_kernel(MxGradParams p) {
  __shared__ __attribute__((aligned(16))) uint16_t tiles[2 * 64 * MxGradPitch<RP>::P];
  if ((int)blockIdx.x < p.blocks0)
    grad_body<FX, RP, V4>(p, p.job[0], blockIdx.x, tiles);
  else
    grad_body<16, RP, V4>(p, p.job[1], blockIdx.x - p.blocks0, tiles);
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

// out = s sum_split P[split] (+ out): dA (out[j][c]) then dB (out[c][j]), the
// splits in four interleaved chains (split t in chain t % 4), then pairwise
__global__ __launch_bounds__(256) void mx_grad_reduce_kernel(MxReduceParams p) {
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t t0 = (int64_t)p.r * p.C[0];
  const int jb = idx < t0 ? 0 : 1;
  const int64_t total = (int64_t)p.r * p.C[jb];
  const int64_t i = jb ? idx - t0 : idx;
  if (i >= total) return;
  int64_t src = i;
  if (jb) {
    const int64_t c = i / p.r;
    src = (i - c * p.r) * p.C[1] + c;
  }
  const float* P = p.P[jb] + src;
  const int ns = p.splits[jb];
  float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  int t = 0;
  for (; t + 4 <= ns; t += 4) {
    float v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = P[(int64_t)(t + u) * total];
#pragma unroll
    for (int u = 0; u < 4; ++u) a[u] += v[u];
  }
#pragma unroll
  for (int u = 0; u < 3; ++u)
    if (t + u < ns) a[u] += P[(int64_t)(t + u) * total];
  float v = p.s * ((a[0] + a[1]) + (a[2] + a[3]));
  if (p.accumulate) v += p.out[jb][i];
  p.out[jb][i] = v;
}

// ranges of rows: about 512 workgroups per output, at least 256 rows each
int pick_splits(int64_t M, int64_t C) {
  int64_t want = cdiv(512, cdiv(C, kTileC));
  const int64_t most = cdiv(M, 256);
  if (want > most) want = most;
  return want < 1 ? 1 : (int)want;
}

void set_job(MxGradJob& j, const void* Z, const uint8_t* Zs, const float* V, int64_t M, int64_t C,
             float* P) {
  j.Z = Z;
  j.Zs = Zs;
  j.V = V;
  j.P = P;
  j.C = C;
  j.c_tiles = (int32_t)cdiv(C, kTileC);
  j.splits = pick_splits(M, C);
  j.rows_per_split = cdiv(cdiv(M, j.splits), 64) * 64;
}

template <int FX>
void launch_grads(const MxGradParams& p, unsigned blocks, hipStream_t st) {
  const dim3 grid(blocks), block(kThreads);
  const bool v4 = p.r % 4 == 0;
  if (p.r <= 32) {
    if (v4)
      hipLaunchKernelGGL((mx_grad_kernel<FX, 32, true>), grid, block, 0, st, p);
    else
      hipLaunchKernelGGL((mx_grad_kernel<FX, 32, false>), grid, block, 0, st, p);
  } else {
    if (v4)
      hipLaunchKernelGGL((mx_grad_kernel<FX, 64, true>), grid, block, 0, st, p);
    else
      hipLaunchKernelGGL((mx_grad_kernel<FX, 64, false>), grid, block, 0, st, p);
  }
}

}  // namespace

namespace dispatch {

size_t mx_grad_bytes(int64_t M, int64_t N, int64_t K, int64_t r) {
  return (size_t)(pick_splits(M, K) * r * K + pick_splits(M, N) * r * N) * 4;
}

int mx_grads(const lq_mx_tensor& X, const float* U, const void* dY, const float* T, int64_t N,
             int64_t r, float s, int accumulate, float* dA, float* dB, void* part,
             hipStream_t st) {
  const int64_t M = X.rows, K = X.cols;
  MxGradParams p;
  float* PA = (float*)part;
  float* PB = PA + (int64_t)pick_splits(M, K) * r * K;
  set_job(p.job[0], X.codes, X.scales, U, M, K, PA);
  set_job(p.job[1], dY, nullptr, T, M, N, PB);
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
  hipLaunchKernelGGL(mx_grad_reduce_kernel, dim3((unsigned)cdiv(r * (K + N), 256)), dim3(256), 0,
                     st, q);
  return hip_fail(hipGetLastError(), "mx_grad_reduce launch");
}

}  // namespace dispatch
}  // namespace lq
