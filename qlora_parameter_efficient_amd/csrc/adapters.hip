// Low-rank adapters of many requests beside a shared projection
// (lq_adapters_fwd, lq_adapters_bwd).
//
//   Y[i] += s_a (X[i] A_a^T) B_a^T,  a = rows[i]
//   dX[i] += s_a U[i] A_a,  U[i] = dY[i] B_a
//   dA_a = s_a sum_i U[i]^T X[i],  dB_a = s_a sum_i dY[i]^T T[i]
//
// Rows are taken in tiles that share one adapter.  Up to 64 rows every workgroup
// finds its tile, of up to 16 rows, by itself: workgroup i looks at the row ids
// (one per lane, one ballot) and goes on only if row i is the first with its
// adapter, or the 17th, 33rd or 49th.  More rows are sorted by one workgroup
// first (plan_kernel), into tiles of up to 64.
//
// Shrink (T = X A^T, U = dY B): workgroups split the reduction, their partial sums
// are added in order by the expand.
// Expand (Y += s T B^T, dX += s U A): rows of B in an order (column 4 i + b of a
// 64-column block is column i of MFMA block b) that gives a lane four consecutive
// outputs of a row and 16 lanes a whole 128-byte line.
//
// Bound by memory: X, Y in and out, the factors once, and for one row by the
// latency of a chain of dependent loads (rows, place, rank, operands).  Measured
// (kernels, us): 1 x 4096 x 4096 rank 16 one launch 7.5; 48 x 11008 x 4096, nearly
// every row its own adapter of rank up to 32, shrink 6 + expand 9.5; 8192 x 4096 x
// 4096, 16 places of rank up to 64, plan 7 + shrink 18 + expand 40 (65 in all, 3.1
// TB/s of the 201 MB of X and Y; without the partial sums of T and without B the
// expand would take 31: both come from L2 for every 256 columns).  Backward of 4096 x
// 4096 x 11008, 8 places of rank up to 32: plan and turned factors 9.5, U 12, dX 45
// (4.0 TB/s), gradients 37 + 8.
#include "block.h"
#include "dispatch.h"
#include "mx_tile.h"

namespace lq {
namespace {

constexpr int kTM = 64;       // rows per tile
constexpr int kDirect = 64;   // up to so many rows workgroups find their tiles by themselves,
constexpr int kFew = 16;      // ... of so many rows at most
constexpr int kCnt = 36880;   // LDS words of the plan's workgroup: larger pools, ...
constexpr int kCntOne = 19 * 1024;  // ... and up to 1023 places (two workgroups fit a CU)

struct RowArgs {
  const int32_t* rows;
  const int32_t* ranks;
  const float* scales;
  // the plan (NULL: M <= kDirect): rows sorted by place (place ``slots``: rows
  // without an adapter), (place, first position, rows, rank) of each tile and of
  // each segment of the gradients, the first segment of each place, and its first
  // partial sum (places of several segments have one a segment)
  const int32_t* perm;
  const int4* tiles;
  const int4* segs;
  const int32_t* seg0;
  const int32_t* part0;
  const int32_t* count;  // tiles, segments
  int32_t M, slots, r;
};

__device__ __forceinline__ int place_of(int32_t a, int slots) {
  return a >= 0 && a < slots ? a : slots;
}

__device__ __forceinline__ int rank_of(const int32_t* ranks, int slots, int r, int slot) {
  if (slot >= slots) return 0;
  if (!ranks) return r;
  const int k = ranks[slot];
  return k < 0 ? 0 : k > r ? r : k;
}

struct Tile {
  int slot, n, rank;  // n = 0: none
};

// Tile and part (of ``parts``) of workgroup b: workgroups of one tile stay on one
// XCD, b % 8 (its rows and T's partial sums stay in that L2), and its parts run
// together.  Tiles go round the XCDs: consecutive ones on one XCD would share its
// factors, but the short tiles at the end leave the last XCD idle (8192 rows, 16
// places: 87 us against 78).
__device__ __forceinline__ int tile_of(const RowArgs& a, int b, int parts, int& part) {
  const int q = a.tiles ? b >> 3 : b;
  part = q % parts;
  return a.tiles ? q / parts * 8 + (b & 7) : q / parts;
}

// This workgroup's tile, and its rows' indices in rows_s (ready after the
// caller's next barrier).
__device__ __forceinline__ Tile find_tile(const RowArgs& a, int tile, int32_t* rows_s) {
  const int lane = threadIdx.x & 63;
  Tile t;
  if (!a.tiles) {
    const int id = lane < a.M ? place_of(a.rows[lane], a.slots) : -1;
    t.slot = __builtin_amdgcn_readlane(id, tile);
    t.rank = __builtin_amdgcn_readfirstlane(rank_of(a.ranks, a.slots, a.r, t.slot));
    const uint64_t same = __ballot(id == t.slot);
    const int before = __builtin_popcountll(same & ((1ull << tile) - 1));
    const int left = __builtin_popcountll(same) - before;
    t.n = before % kFew ? 0 : left < kFew ? left : kFew;
    const int at = __builtin_popcountll(same & ((1ull << lane) - 1)) - before;
    if (threadIdx.x < 64 && id == t.slot && at >= 0 && at < kFew) rows_s[at] = lane;
    return t;
  }
  const int4 d = a.tiles[tile];  // (past the last tile: not used)
  // (the same for every lane, and known to be)
  t.slot = __builtin_amdgcn_readfirstlane(d.x);
  t.n = __builtin_amdgcn_readfirstlane(tile < a.count[0] ? d.z : 0);
  t.rank = __builtin_amdgcn_readfirstlane(d.w);
  if ((int)threadIdx.x < t.n) rows_s[threadIdx.x] = a.perm[d.y + threadIdx.x];
  return t;
}

// ---------------------------------------------------------------- plan
// Stable counting sort of the rows by place, in one workgroup of 16 waves: each
// wave counts its own range of rows into counters of its own (rows of a wave
// that share a place are found with one ballot per bit of the place) and notes
// each row's position among them, the counters become the waves' first positions
// within the place, and the rows are placed; the row that begins a tile or a
// segment lists it (from the counting threads, one place after another, the lists
// took 2 to 3 us).  Rows are loaded eight at a time, since a load is the longest
// part of a step.  Of 6.2 us for 8192 rows in 16 places (without the launch, 7.3
// with it), 2.4 go until the rows are there, 1 to counting, 1 to the sums and 1.9 to
// the stores.
struct PlanArgs {
  const int32_t* rows;
  const int32_t* ranks;
  int32_t* perm;
  int4* tiles;
  int4* segs;
  int32_t* seg0;
  int32_t* part0;
  int32_t* count;
  int32_t M, slots, r, waves, bits, seg_rows;
};

// the lanes of m whose value equals this lane's
__device__ __forceinline__ uint64_t lanes_like(int v, int bits, uint64_t m) {
  uint32_t lo = (uint32_t)m, hi = (uint32_t)(m >> 32);
  for (int b = 0; b < bits; ++b) {
    const uint32_t bit = __builtin_amdgcn_sbfe(v, b, 1);  // 0 or all ones
    const uint64_t set = __ballot(bit != 0);
    lo &= ~((uint32_t)set ^ bit);
    hi &= ~((uint32_t)(set >> 32) ^ bit);
  }
  return (uint64_t)hi << 32 | lo;
}

// inclusive sums over rows of 16 lanes, and over the wave's lanes
#define LQ_SCAN(ctrl, rows) x += __builtin_amdgcn_update_dpp(0, x, ctrl, rows, 0xF, false)
__device__ __forceinline__ int row_scan(int x) {
  LQ_SCAN(0x111, 0xF);  // row_shr 1, 2, 4, 8
  LQ_SCAN(0x112, 0xF);
  LQ_SCAN(0x114, 0xF);
  LQ_SCAN(0x118, 0xF);
  return x;
}
__device__ __forceinline__ int wave_scan(int x) {
  x = row_scan(x);
  LQ_SCAN(0x142, 0xA);  // row_bcast 15, 31
  LQ_SCAN(0x143, 0xC);
  return x;
}
#undef LQ_SCAN

// exclusive sums over the workgroup's 16 waves of four values per thread; the totals
__device__ __forceinline__ void scan(int (&v)[4], int (&total)[4], int4* sh) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int x[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = wave_scan(v[k]);
  if (lane == 63) sh[wave] = make_int4(x[0], x[1], x[2], x[3]);
  __syncthreads();
  // the waves' sums, one per lane of a row of 16
  const int4 q = sh[lane & 15];
  const int w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int all = row_scan(w[k]);
    v[k] = x[k] - v[k] + (wave ? __builtin_amdgcn_readlane(all, wave - 1) : 0);
    total[k] = __builtin_amdgcn_readlane(all, 15);
  }
}

// --------------------------------------------- factors turned (backward)
// Bt[slot][j][n] = B[slot][n][j] and At[slot][k][j] = A[slot][j][k] (rows of ld
// elements) for the places that have rows: 64 columns n or k per 256 threads.
struct TurnArgs {
  const uint16_t* A;
  const uint16_t* B;
  uint16_t* At;
  uint16_t* Bt;
  int32_t N, K, r, ld;
  int32_t chunks;  // of 64 columns, of one place
  uint32_t inv;    // 2^16 / (ld / 8), rounded up: e * inv >> 16 is e / (ld / 8), e < 512
};

// Whether a row has this place (the workgroup's threads together)
__device__ __forceinline__ bool any_row(const int32_t* rows, int M, int slot) {
  for (int64_t b = 0; b < M; b += 8 * (int64_t)blockDim.x) {
    bool here = false;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int64_t i = b + k * (int64_t)blockDim.x + threadIdx.x;
      here |= i < M && rows[i] == slot;
    }
    if (__syncthreads_or(here)) return true;
  }
  return false;
}

// Chunk ``chunk`` of a place by 256 threads (tid) with 64 x 66 elements of LDS;
// every thread of the workgroup takes part in the barrier
__device__ __forceinline__ void turn_chunk(const TurnArgs& p, int slot, int chunk, int tid,
                                           uint16_t* s) {
  const int r = p.r, nb = p.N / 64;
  const bool is_b = chunk < nb, in = chunk < p.chunks;
  const int c0 = (is_b ? chunk : chunk - nb) * 64;
  // in: 64 columns of r ranks (B) or r ranks of 64 columns (A), eight elements a
  // thread where rows allow; in LDS as [rank][column]
  if (in && is_b) {
    const uint16_t* B = p.B + ((int64_t)slot * p.N + c0) * r;
    if (r % 8 == 0) {
      for (int e = tid; e < 8 * r; e += 256) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(B + 8 * e);
        const int c = e * p.inv >> 16, j = 8 * (e - c * (r / 8));
#pragma unroll
        for (int k = 0; k < 8; ++k) s[(j + k) * 66 + c] = (uint16_t)(v[k >> 1] >> (16 * (k & 1)));
      }
    } else {
      for (int e = tid; e < 64 * r; e += 256) s[(e % r) * 66 + e / r] = B[e];
    }
  } else if (in) {
    for (int e = tid; e < 8 * r; e += 256) {
      const int j = e >> 3, c = 8 * (e & 7);
      const u32x4 v = *reinterpret_cast<const u32x4*>(p.A + ((int64_t)slot * r + j) * p.K + c0 + c);
#pragma unroll
      for (int k = 0; k < 8; ++k) s[j * 66 + c + k] = (uint16_t)(v[k >> 1] >> (16 * (k & 1)));
    }
  }
  __syncthreads();
  if (in && is_b) {
    for (int e = tid; e < 8 * r; e += 256) {
      const int j = e >> 3, c = 8 * (e & 7);
      u32x4 v;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        v[k] = s[j * 66 + c + 2 * k] | ((uint32_t)s[j * 66 + c + 2 * k + 1] << 16);
      *reinterpret_cast<u32x4*>(p.Bt + ((int64_t)slot * r + j) * p.N + c0 + c) = v;
    }
  } else if (in) {
    for (int e = tid; e < 8 * p.ld; e += 256) {  // rows of ld = r rounded up to eight
      const int c = e * p.inv >> 16, j = 8 * (e - c * (p.ld / 8));
      u32x4 v;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t lo = j + 2 * k < r ? s[(j + 2 * k) * 66 + c] : 0u;
        const uint32_t hi = j + 2 * k + 1 < r ? s[(j + 2 * k + 1) * 66 + c] : 0u;
        v[k] = lo | (hi << 16);
      }
      *reinterpret_cast<u32x4*>(p.At + ((int64_t)slot * p.K + c0) * p.ld + 8 * e) = v;
    }
  }
}

constexpr int kPerThread = (LQ_ADAPTERS_MAX_SLOTS + 1024) / 1024;  // most places of a thread

// Workgroup 0: the plan.  The others (backward): four chunks each of a place's
// factors, which wait for nothing of it, but look for the place among all rows, so
// the launch takes as long as the pool is large: dX of 64 rows beside 4096 x 4096
// rank 16, six places in use, 15 us with 8 places, 23 with 64, 167 with 1024, 639 with
// 4096.  PT: places per thread; one in pools of
// up to 1023 places, where all 16 waves have counters too.
template <int PT>
__global__ __launch_bounds__(1024) void plan_kernel(PlanArgs p, TurnArgs q) {
  __shared__ __attribute__((aligned(16))) int32_t cnt[PT == 1 ? kCntOne : kCnt];
  __shared__ int4 sh[16];
  if (blockIdx.x > 0) {
    const int per_place = (q.chunks + 3) / 4, b = blockIdx.x - 1;
    const int slot = b / per_place, g = threadIdx.x >> 8;
    if (any_row(p.rows, p.M, slot))
      turn_chunk(q, slot, 4 * (b % per_place) + g, threadIdx.x & 255,
                 reinterpret_cast<uint16_t*>(cnt) + g * 64 * 66);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int S1 = p.slots + 1, W = PT == 1 ? 16 : p.waves;
  // of each place: its first position, its first tile and rank, its first segment
  int32_t *first_s = cnt + W * S1, *tile_s = first_s + S1, *seg_s = tile_s + S1;
  const int per = (int)cdiv(cdiv(p.M, 64), W) * 64;
  const int64_t lo = (int64_t)wave * per;
  const int64_t end = lo + per;
  const int64_t hi = wave < W ? (end < p.M ? end : p.M) : 0;
  const uint64_t below = (1ull << lane) - 1;
  const int c = (int)cdiv(S1, 1024);  // thread t has places c t .. c t + c - 1
  int id[8], pos[8], rank[PT];
  auto load = [&](int64_t b) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int64_t i = b + 64 * k + lane;
      id[k] = i < hi ? p.rows[i] : 0;
    }
  };
  load(lo);
#pragma unroll
  for (int k = 0; k < PT; ++k)
    rank[k] = k < c && tid * c + k < p.slots ? rank_of(p.ranks, p.slots, p.r, tid * c + k) : 0;
  for (int i = tid; i < W * S1; i += 1024) cnt[i] = 0;
  __syncthreads();
  // Counts the wave's rows by place; pos: a row's position among those that the
  // counter has seen.
  auto count = [&](int64_t b) {
    int old[8], first[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      old[k] = first[k] = 0;
      pos[k] = lane;
      id[k] = place_of(id[k], p.slots);
      if (b + 64 * k >= hi) continue;
      const bool in = b + 64 * k + lane < hi;
      uint64_t m = __ballot(in);
      // (a request's rows mostly fill the wave)
      if (__ballot(in && id[k] != __builtin_amdgcn_readfirstlane(id[k])))
        m = lanes_like(id[k], p.bits, m);
      first[k] = in ? (int)__builtin_ctzll(m) : lane;
      pos[k] = __builtin_popcountll(m & below);
      if (in && lane == first[k])
        old[k] = atomicAdd(&cnt[wave * S1 + id[k]], __builtin_popcountll(m));
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) pos[k] += __shfl(old[k], first[k]);
  };
  for (int64_t b = lo; b < hi; b += 512) {
    if (b > lo) load(b);
    count(b);
  }
  __syncthreads();
  // counts become positions
  int v[4] = {0, 0, 0, 0}, total[4], n[PT];
#pragma unroll
  for (int k = 0; k < PT; ++k) {
    const int s = tid * c + k;
    n[k] = 0;
    if (k >= c || s >= S1) continue;
    int x[16];
#pragma unroll
    for (int w = 0; w < 16; ++w) x[w] = w < W ? cnt[w * S1 + s] : 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
      if (w < W) cnt[w * S1 + s] = n[k];
      n[k] += x[w];
    }
    v[0] += n[k];
    v[1] += (n[k] + kTM - 1) / kTM;
    const int segs = s < p.slots ? (n[k] + p.seg_rows - 1) / p.seg_rows : 0;
    v[2] += segs;
    v[3] += segs > 1 ? segs : 0;
  }
  scan(v, total, sh);
#pragma unroll
  for (int k = 0; k < PT; ++k) {
    const int s = tid * c + k;
    if (k >= c || s >= S1) continue;
    first_s[s] = v[0];
    tile_s[s] = v[1] << 7 | rank[k];  // (fewer than 2^20 tiles, ranks up to 64)
    seg_s[s] = v[2];
    p.seg0[s] = v[2];
    if (s < p.slots) p.part0[s] = v[3];
    v[0] += n[k];
    v[1] += (n[k] + kTM - 1) / kTM;
    const int segs = s < p.slots ? (n[k] + p.seg_rows - 1) / p.seg_rows : 0;
    v[2] += segs;
    v[3] += segs > 1 ? segs : 0;
  }
  if (tid == 0) {
    p.count[0] = total[1];
    p.count[1] = total[2];
  }
  __syncthreads();
  // row i of place s, the d-th of its place; the first of a tile or segment lists it
  auto put = [&](int64_t i, int s, int d) {
    const int first = first_s[s];
    p.perm[first + d] = (int32_t)i;
    if (d % 32) return;
    const int left = (s < p.slots ? first_s[s + 1] : p.M) - first - d;
    const int tile = tile_s[s], rank = tile & 127;
    if (d % kTM == 0)
      p.tiles[(tile >> 7) + d / kTM] = make_int4(s, first + d, left < kTM ? left : kTM, rank);
    if (!p.segs || s >= p.slots) return;
    const int q = d / p.seg_rows;  // (a multiple of 32)
    if (q * p.seg_rows == d)
      p.segs[seg_s[s] + q] = make_int4(s, first + d, left < p.seg_rows ? left : p.seg_rows, rank);
  };
  if (per <= 512) {  // places and positions are still in registers
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int64_t i = lo + 64 * k + lane;
      if (i < hi) put(i, id[k], cnt[wave * S1 + id[k]] + pos[k]);
    }
    return;
  }
  // else the rows are counted again, from the wave's first positions on
  for (int64_t b = lo; b < hi; b += 512) {
    load(b);
    count(b);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int64_t i = b + 64 * k + lane;
      if (i < hi) put(i, id[k], pos[k]);
    }
  }
}

// -------------------------------------------------------------- shrink

struct ShrinkParams {
  RowArgs a;
  const uint16_t* X;  // M x C
  const uint16_t* A;  // slots x r x C
  float* Tp;          // splits x M x rp
  int32_t C, rp, splits, steps;   // 64-column steps of the reduction, of one split
};

// p, the same in every lane, in scalar registers
__device__ __forceinline__ const char* uniform(const void* p) {
  const uint64_t a = (uint64_t)(uintptr_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
  return (const char*)(uintptr_t)(((uint64_t)hi << 32) | lo);
}

// 16 bytes per lane from base + off to LDS at lds + 16 lane; the kernels wait for
// these loads themselves
__device__ __forceinline__ void dma16(const void* base, uint32_t off, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %2\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %0, %1"
      :
      : "v"(off), "s"(base), "s"(lds)
      : "memory", "m0");
}

// At most 16 rows: operands straight into registers, the four waves taking turns
// at the steps of the split.
template <int JB>
__device__ __forceinline__ void shrink_few(const ShrinkParams& p, const int32_t* rows_s, int n,
                                           const uint16_t* A, int rank, int s0, int s1, float* out,
                                           f32x4* red) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4, i16 = lane & 15;
  const uint16_t* xr = p.X + (int64_t)rows_s[i16 < n ? i16 : n - 1] * p.C + 8 * g;
  const uint16_t* ar[JB];
  f32x4 acc[JB];
#pragma unroll
  for (int j = 0; j < JB; ++j) {
    const int k = 16 * j + i16;
    ar[j] = A + (int64_t)(k < rank ? k : rank - 1) * p.C + 8 * g;
    acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  constexpr int D = JB == 1 ? 8 : JB == 2 ? 6 : 4;  // halves of steps in flight
  u32x4 x[D], a[D][JB];
  const int nw = (s1 - s0 - wave + 3) / 4;
  auto load = [&](int i, int b) {
    const int c = 64 * (s0 + wave + 4 * (i >> 1)) + 32 * (i & 1);
    x[b] = *reinterpret_cast<const u32x4*>(xr + c);
#pragma unroll
    for (int j = 0; j < JB; ++j) a[b][j] = *reinterpret_cast<const u32x4*>(ar[j] + c);
  };
#pragma unroll
  for (int b = 0; b < D; ++b)
    if (b < 2 * nw) load(b, b);
  for (int i = 0; i < 2 * nw; i += D)
#pragma unroll
    for (int b = 0; b < D; ++b) {
      if (i + b >= 2 * nw) break;
#pragma unroll
      for (int j = 0; j < JB; ++j) acc[j] = mfma16(x[b], a[b][j], acc[j]);
      if (i + b + D < 2 * nw) load(i + b + D, b);
    }
#pragma unroll
  for (int j = 0; j < JB; ++j) red[(wave * JB + j) * 64 + lane] = acc[j];
  __syncthreads();
  // wave w finishes block w
  if (wave >= JB) return;
  f32x4 t = red[wave * 64 + lane];
#pragma unroll
  for (int w = 1; w < 4; ++w)
#pragma unroll
    for (int e = 0; e < 4; ++e) t[e] += red[(w * JB + wave) * 64 + lane][e];
  const int j = 16 * wave + i16;
#pragma unroll
  for (int v = 0; v < 4; ++v)
    if (4 * g + v < n && j < rank) out[(int64_t)rows_s[4 * g + v] * p.rp + j] = t[v];
}

// 17 to 64 rows: steps of X (64 rows of 128 bytes) and of A go straight into one of
// three LDS stages, chunk c of row x at c ^ mx_swz128(x), by whole lines (read in
// the operands' layout, where neighbouring lanes have different rows, a load
// takes the address unit 64 cycles instead of 16); wave w owns rows 16 w .. 16 w +
// 15, so nothing is left to add.
constexpr int kStages = 3;

template <int JB>
__device__ __forceinline__ void shrink_many(const ShrinkParams& p, const int32_t* rows_s, int n,
                                            const uint16_t* A, int rank, int s0, int s1, float* out,
                                            char* lds) {
  constexpr int kX = kTM * 128, kStage = kX + 16 * JB * 128;
  constexpr int DA = (JB + 1) / 2, DL = 2 + DA;  // loads of a wave and stage: A's, all
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, i16 = lane & 15;
  const uint32_t base = mx_lds_addr(lds);
  // load u covers rows 8 u .. 8 u + 7; a wave's are wave, wave + 4, ... (past the
  // end the last again)
  uint32_t xo[2], ao[DA];
  int au[DA];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int row = 8 * (wave + 4 * k) + (lane >> 3);
    xo[k] = ((uint32_t)rows_s[row < n ? row : n - 1] * p.C + 8 * ((lane & 7) ^ mx_swz128(row))) * 2;
  }
#pragma unroll
  for (int k = 0; k < DA; ++k) {
    au[k] = wave + 4 * k < 2 * JB ? wave + 4 * k : 2 * JB - 1;
    const int row = 8 * au[k] + (lane >> 3);
    ao[k] = ((uint32_t)(row < rank ? row : rank - 1) * p.C + 8 * ((lane & 7) ^ mx_swz128(row))) * 2;
  }
  auto issue = [&](int s, int b) {
    const uint32_t st = base + b * kStage;
#pragma unroll
    for (int k = 0; k < 2; ++k) dma16(p.X + 64 * s, xo[k], st + (wave + 4 * k) * 1024);
#pragma unroll
    for (int k = 0; k < DA; ++k) dma16(A + 64 * s, ao[k], st + kX + au[k] * 1024);
  };
  f32x4 acc[JB];
#pragma unroll
  for (int j = 0; j < JB; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const bool mine = 16 * wave < n;
  const uint32_t row = i16 * 128, sw = mx_swz128(i16);
  issue(s0, 0);
  if (s0 + 1 < s1) issue(s0 + 1, 1);
  int b = 0;
  for (int s = s0; s < s1; ++s) {
    // this wave's loads of the stage have landed, then everybody's; all are done
    // with the stage before it, which the next loads go into
    mx_wait_loads<DL>(mx_less(s + 1, s1));
    __syncthreads();
    if (s + 2 < s1) issue(s + 2, b == 0 ? 2 : b - 1);
    if (mine) {
      const uint32_t st = base + b * kStage;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t c = ((4 * h + g) ^ sw) << 4;
        const u32x4 x = mx_read16(st + wave * 2048 + row + c);
#pragma unroll
        for (int j = 0; j < JB; ++j)
          acc[j] = mfma16(x, mx_read16(st + kX + j * 2048 + row + c), acc[j]);
      }
    }
    b = b == 2 ? 0 : b + 1;
  }
#pragma unroll
  for (int j = 0; j < JB; ++j)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int i = 16 * wave + 4 * g + v, k = 16 * j + i16;
      if (i < n && k < rank) out[(int64_t)rows_s[i] * p.rp + k] = acc[j][v];
    }
}

// FEW: no tile has more than kFew rows
template <int JB, bool FEW>
__global__ __launch_bounds__(256) void shrink_tiles_kernel(ShrinkParams p) {
  __shared__ int32_t rows_s[kTM];
  __shared__ __attribute__((aligned(1024))) char lds[FEW ? 4 * JB * 1024 : kStages * (kTM + 16 * JB) * 128];
  int part;
  const int tile = tile_of(p.a, blockIdx.x, p.splits, part);
  const Tile t = find_tile(p.a, tile, rows_s);
  if (t.n == 0 || t.rank == 0) return;
  __syncthreads();
  const int s0 = __builtin_amdgcn_readfirstlane(part * p.steps), all = p.C / 64;
  const int s1 = s0 + p.steps < all ? s0 + p.steps : all;
  const uint16_t* A = (const uint16_t*)uniform(p.A + (int64_t)t.slot * p.a.r * p.C);
  float* out = p.Tp + (int64_t)part * p.a.M * p.rp;
  if (FEW || t.n <= kFew)
    shrink_few<JB>(p, rows_s, t.n, A, t.rank, s0, s1, out, reinterpret_cast<f32x4*>(lds));
  else
    shrink_many<JB>(p, rows_s, t.n, A, t.rank, s0, s1, out, lds);
}

// -------------------------------------------------------------- expand

struct ExpandParams {
  RowArgs a;
  const float* Tp;    // splits x M x rp
  const uint16_t* B;  // slots x N x ldb
  const uint16_t* Yi;
  uint16_t* Yo;
  float* T_out;  // M x r or NULL
  int32_t splits, N, ldb, rp, parts, passes;
};

// chunk c (eight ranks) of row x of a wave's 64 rows of B in LDS sits at c ^
// b_swz(x), cpr chunks per row
__device__ __forceinline__ int b_swz(int x, int cpr) {
  return cpr & (cpr - 1) ? 0 : (x >> 2) & (cpr - 1);
}

// ranks 8 c .. 8 c + 7 of row x (zeros past r).  WHOLE: rows of whole chunks; else
// rows of r elements, one after another
template <bool WHOLE>
__device__ __forceinline__ u32x4 b_read(uint32_t lds, int x, int c, int r, int cpr) {
  if (8 * c >= r) return u32x4{0u, 0u, 0u, 0u};
  if (WHOLE) return mx_read16(lds + (x * cpr + (c ^ b_swz(x, cpr))) * 16);
  typedef __attribute__((address_space(3))) const uint16_t* lds_u16;
  uint16_t e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    e[i] = 8 * c + i < r ? *(lds_u16)(uintptr_t)(lds + (x * r + 8 * c + i) * 2) : (uint16_t)0;
  return mx_pack8(e);
}

// ... with zeros from ``rank`` on (whatever they were)
__device__ __forceinline__ void b_mask(u32x4& v, int j0, int rank) {
  const int left = rank - j0;
#pragma unroll
  for (int d = 0; d < 4; ++d)
    v[d] = 2 * d + 1 < left ? v[d] : 2 * d < left ? v[d] & 0xFFFFu : 0u;
}

// v as two bf16 parts: hi + lo is v to 2^-16 of it (lo 0 where hi is not finite)
__device__ __forceinline__ void split2(float v, uint16_t& hi, uint16_t& lo) {
  hi = f32_to_bf16(v);
  const float h = bf16_to_f32(hi);
  lo = (hi & 0x7F80u) == 0x7F80u ? (uint16_t)0 : f32_to_bf16(v - h);
}

// JC: 32-rank chunks; MB: 16-row blocks of a tile.  What does not depend on T (B,
// Y) is loaded before T's partial sums are waited for.
template <int JC, bool WHOLE, int MB>
__global__ __launch_bounds__(256, MB == 1 ? 6 : JC == 1 ? 4 : 3) void expand_tiles_kernel(ExpandParams p) {
  constexpr int LD = 32 * JC + 8;  // LDS row pitch of T in elements
  constexpr int VT = MB * JC / 2 > 0 ? MB * JC / 2 : 1;  // groups of four values of T per thread
  constexpr int kB = 64 * 64 * JC; // bytes of a wave's rows of B
  __shared__ int32_t rows_s[kTM];
  __shared__ __attribute__((aligned(16))) uint16_t t_hi[16 * MB * LD], t_lo[16 * MB * LD];
  __shared__ __attribute__((aligned(1024))) char bs[4 * kB];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, i16 = lane & 15;
  int part;
  const int tile = tile_of(p.a, blockIdx.x, p.parts, part);
  const Tile t = find_tile(p.a, tile, rows_s);
  const int n = t.n, rank = t.rank;
  if (n == 0) return;
  const bool store_t = p.T_out && part == 0;
  const bool same = !p.Yo || (rank == 0 && p.Yi == p.Yo);  // Y stays as it is
  if (same && !store_t) return;
  const bool has = t.slot < p.a.slots;
  const int r = p.a.r, M = p.a.M, N = p.N, ldb = p.ldb, cpr = ldb / 8;
  const float s = has ? p.a.scales[t.slot] : 0.0f;
  __syncthreads();
  const uint16_t* B = p.B + (int64_t)t.slot * N * ldb;
  const uint32_t mine = mx_lds_addr(bs) + wave * kB;
  // 64 rows of B are one run of 128 ldb bytes, 1024 per load (the last load's
  // lanes past the end: the last 16 bytes again)
  const int b_loads = (ldb + 7) / 8;
  u32x2 y[MB][4];
  int32_t at[MB][4];  // M N < 2^31
  auto load = [&](int n0) {
    if (has) {
      const char* run = uniform(B + (int64_t)n0 * ldb);
#pragma unroll
      for (int u = 0; u < 4 * JC; ++u) {
        if (u >= b_loads) break;
        const int q = 64 * u + lane;
        uint32_t off;
        if (WHOLE) {
          const int x = q / cpr;
          off = 16 * (x * cpr + ((q - x * cpr) ^ b_swz(x, cpr)));
        } else {
          off = 16 * (q < 8 * ldb ? q : 8 * ldb - 1);
        }
        dma16(run, off, mine + 1024 * u);
      }
    }
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      if (16 * m >= n) break;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int i = 16 * m + 4 * g + v;
        at[m][v] = rows_s[i < n ? i : n - 1] * N + n0 + 4 * i16;
        y[m][v] = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p.Yi + at[m][v]));
      }
    }
  };
  int n0 = part * p.passes * 256 + 64 * wave;
  if (!same && n0 < N) load(n0);
  {
    f32x4 v[VT];
    int32_t q[VT];
    bool in[VT];
#pragma unroll
    for (int u = 0; u < VT; ++u) {
      const int e = 256 * u + tid, i = e / (8 * JC), j = 4 * (e % (8 * JC));
      in[u] = i < n && j < r;
      q[u] = rows_s[in[u] ? i : 0] * p.rp + (in[u] ? j : 0);
      v[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    if (has) {  // (whatever lies past the rank)
      const int64_t part = (int64_t)M * p.rp;
      int k = 0;
      constexpr int D = MB == 1 ? 4 : 4 / JC;
      for (; k + D <= p.splits; k += D) {
        f32x4 x[D][VT];
#pragma unroll
        for (int d = 0; d < D; ++d)
#pragma unroll
          for (int u = 0; u < VT; ++u)
            x[d][u] = *reinterpret_cast<const f32x4*>(p.Tp + (k + d) * part + q[u]);
#pragma unroll
        for (int d = 0; d < D; ++d)
#pragma unroll
          for (int u = 0; u < VT; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) v[u][e] += x[d][u][e];
      }
      for (; k < p.splits; ++k)
#pragma unroll
        for (int u = 0; u < VT; ++u) {
          const f32x4 x = *reinterpret_cast<const f32x4*>(p.Tp + k * part + q[u]);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[u][e] += x[e];
        }
    }
#pragma unroll
    for (int u = 0; u < VT; ++u) {
      const int e = 256 * u + tid, i = e / (8 * JC), j = 4 * (e % (8 * JC));
      if (i >= 16 * MB) break;  // (one block of one chunk: half of the threads)
      uint16_t hi[4], lo[4];
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const float x = in[u] && j + d < rank ? v[u][d] : 0.0f;
        if (store_t && i < n && j + d < r) p.T_out[(int64_t)rows_s[i] * r + j + d] = x;
        split2(x * s, hi[d], lo[d]);
      }
      *reinterpret_cast<u32x2*>(t_hi + i * LD + j) =
          u32x2{hi[0] | ((uint32_t)hi[1] << 16), hi[2] | ((uint32_t)hi[3] << 16)};
      *reinterpret_cast<u32x2*>(t_lo + i * LD + j) =
          u32x2{lo[0] | ((uint32_t)lo[1] << 16), lo[2] | ((uint32_t)lo[3] << 16)};
    }
  }
  __syncthreads();
  if (same) return;
  for (int pass = 0; pass < p.passes && n0 < N; ++pass) {
    u32x4 bf[4][JC];
    mx_wait_loads();
    if (rank) {
#pragma unroll
      for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int jc = 0; jc < JC; ++jc) {
          bf[b][jc] = b_read<WHOLE>(mine, 4 * i16 + b, 4 * jc + g, WHOLE ? ldb : r, cpr);
          b_mask(bf[b][jc], 32 * jc + 8 * g, rank);
        }
    }
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      if (16 * m >= n) break;
      if (rank) {
        f32x4 acc[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          acc[0][v] = lo_bf16(y[m][v][0]);
          acc[1][v] = hi_bf16(y[m][v][0]);
          acc[2][v] = lo_bf16(y[m][v][1]);
          acc[3][v] = hi_bf16(y[m][v][1]);
        }
#pragma unroll
        for (int jc = 0; jc < JC; ++jc) {
          const int o = (16 * m + i16) * LD + 32 * jc + 8 * g;
          const u32x4 th = *reinterpret_cast<const u32x4*>(t_hi + o);
          const u32x4 tl = *reinterpret_cast<const u32x4*>(t_lo + o);
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            acc[b] = mfma16(tl, bf[b][jc], acc[b]);
            acc[b] = mfma16(th, bf[b][jc], acc[b]);
          }
        }
#pragma unroll
        for (int v = 0; v < 4; ++v)
          y[m][v] = u32x2{pack_bf16x2(acc[0][v], acc[1][v]), pack_bf16x2(acc[2][v], acc[3][v])};
      }
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (16 * m + 4 * g + v < n)
          __builtin_nontemporal_store(y[m][v], reinterpret_cast<u32x2*>(p.Yo + at[m][v]));
    }
    n0 += 256;
    if (pass + 1 < p.passes && n0 < N) load(n0);
  }
}

// ------------------------------------------------ few rows in one launch
// Up to kFew rows: every workgroup forms its tile's T itself, sixteen waves taking
// turns at the steps of the whole reduction, and then 256 columns of the expand.
// A is read again for every 256 columns (from L2), but there is one launch, no
// workspace, and no trip of T through memory.
struct FewParams {
  RowArgs a;
  const uint16_t* X;
  const uint16_t* A;
  const uint16_t* B;
  const uint16_t* Yi;
  uint16_t* Yo;
  float* T_out;
  int32_t K, N, parts;
};

template <int JB, bool WHOLE>
__global__ __launch_bounds__(1024) void few_rows_kernel(FewParams p) {
  constexpr int JC = (JB + 1) / 2, LD = 32 * JC + 8, kB = 64 * 64 * JC;
  __shared__ int32_t rows_s[kTM];
  __shared__ __attribute__((aligned(16))) uint16_t t_hi[16 * LD], t_lo[16 * LD];
  __shared__ f32x4 red[16 * JB * 64];
  __shared__ __attribute__((aligned(1024))) char bs[4 * kB];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, i16 = lane & 15;
  int part;
  const int tile = tile_of(p.a, blockIdx.x, p.parts, part);
  const Tile t = find_tile(p.a, tile, rows_s);
  const int n = t.n, rank = t.rank;
  const bool store_t = p.T_out && part == 0;
  if (n == 0 || (rank == 0 && p.Yi == p.Yo && !store_t)) return;
  const int r = p.a.r, N = p.N, K = p.K, cpr = r / 8;
  const bool has = t.slot < p.a.slots;
  const float s = has ? p.a.scales[t.slot] : 0.0f;
  for (int e = threadIdx.x; e < 16 * LD; e += 1024) t_hi[e] = t_lo[e] = 0;
  __syncthreads();
  // the expand's operands on their way
  const int n0 = part * 256 + 64 * wave;
  const bool mine = wave < 4 && n0 < N;
  const uint32_t b_lds = mx_lds_addr(bs) + (wave & 3) * kB;
  u32x2 y[4];
  int32_t at[4];
  if (mine) {
    if (has) {
      const char* run = uniform(p.B + ((int64_t)t.slot * N + n0) * r);
#pragma unroll
      for (int u = 0; u < 4 * JC; ++u) {
        if (u >= (r + 7) / 8) break;
        const int q = 64 * u + lane;
        dma16(run, WHOLE ? 16 * (q / cpr * cpr + ((q % cpr) ^ b_swz(q / cpr, cpr)))
                         : 16 * (q < 8 * r ? q : 8 * r - 1), b_lds + 1024 * u);
      }
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      at[v] = rows_s[4 * g + v < n ? 4 * g + v : n - 1] * N + n0 + 4 * i16;
      y[v] = *reinterpret_cast<const u32x2*>(p.Yi + at[v]);
    }
  }
  if (rank) {
    const uint16_t* A = p.A + (int64_t)t.slot * r * K;
    const uint16_t* xr = p.X + (int64_t)rows_s[i16 < n ? i16 : n - 1] * K + 8 * g;
    const uint16_t* ar[JB];
    f32x4 acc[JB];
#pragma unroll
    for (int j = 0; j < JB; ++j) {
      const int k = 16 * j + i16;
      ar[j] = A + (int64_t)(k < rank ? k : rank - 1) * K + 8 * g;
      acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    constexpr int D = JB == 1 ? 8 : 4;  // halves of steps in flight
    u32x4 x[D], a[D][JB];
    const int nw = (K / 64 - wave + 15) / 16;
    auto load = [&](int i, int b) {
      const int c = 64 * (wave + 16 * (i >> 1)) + 32 * (i & 1);
      x[b] = *reinterpret_cast<const u32x4*>(xr + c);
#pragma unroll
      for (int j = 0; j < JB; ++j) a[b][j] = *reinterpret_cast<const u32x4*>(ar[j] + c);
    };
#pragma unroll
    for (int b = 0; b < D; ++b)
      if (b < 2 * nw) load(b, b);
    for (int i = 0; i < 2 * nw; i += D)
#pragma unroll
      for (int b = 0; b < D; ++b) {
        if (i + b >= 2 * nw) break;
#pragma unroll
        for (int j = 0; j < JB; ++j) acc[j] = mfma16(x[b], a[b][j], acc[j]);
        if (i + b + D < 2 * nw) load(i + b + D, b);
      }
#pragma unroll
    for (int j = 0; j < JB; ++j) red[(wave * JB + j) * 64 + lane] = acc[j];
  }
  __syncthreads();
  if (wave < JB) {  // wave w finishes block w
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    const int j = 16 * wave + i16;
    if (j < rank) {
#pragma unroll
      for (int w = 0; w < 16; ++w)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += red[(w * JB + wave) * 64 + lane][e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = 4 * g + e;
      if (store_t && i < n && j < r) p.T_out[(int64_t)rows_s[i] * r + j] = v[e];
      uint16_t hi, lo;
      split2(i < n ? v[e] * s : 0.0f, hi, lo);
      t_hi[i * LD + j] = hi;
      t_lo[i * LD + j] = lo;
    }
  }
  __syncthreads();
  if (!mine || (rank == 0 && p.Yi == p.Yo)) return;
  mx_wait_loads();
  if (rank) {
    f32x4 acc[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      acc[0][v] = lo_bf16(y[v][0]);
      acc[1][v] = hi_bf16(y[v][0]);
      acc[2][v] = lo_bf16(y[v][1]);
      acc[3][v] = hi_bf16(y[v][1]);
    }
#pragma unroll
    for (int jc = 0; jc < JC; ++jc) {
      const u32x4 th = *reinterpret_cast<const u32x4*>(t_hi + i16 * LD + 32 * jc + 8 * g);
      const u32x4 tl = *reinterpret_cast<const u32x4*>(t_lo + i16 * LD + 32 * jc + 8 * g);
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        u32x4 bf = b_read<WHOLE>(b_lds, 4 * i16 + b, 4 * jc + g, r, cpr);
        b_mask(bf, 32 * jc + 8 * g, rank);
        acc[b] = mfma16(tl, bf, acc[b]);
        acc[b] = mfma16(th, bf, acc[b]);
      }
    }
#pragma unroll
    for (int v = 0; v < 4; ++v)
      y[v] = u32x2{pack_bf16x2(acc[0][v], acc[1][v]), pack_bf16x2(acc[2][v], acc[3][v])};
  }
#pragma unroll
  for (int v = 0; v < 4; ++v)
    if (4 * g + v < n) *reinterpret_cast<u32x2*>(p.Yo + at[v]) = y[v];
}

// ------------------------------------------------------------- gradients
// dA_a = s_a sum_i U[i]^T X[i] and dB_a = s_a sum_i dY[i]^T T[i] over one
// segment of the place's rows, 256 columns of X or dY per workgroup, 64 per
// wave.  Steps of 32 rows: their columns go row by row into LDS (rows 32 bytes
// off 512, so that the transposing reads of four rows meet different banks), U
// or T as three bf16 parts, transposed.
struct GradParams {
  RowArgs a;
  const uint16_t* X;   // M x K
  const uint16_t* dY;  // M x N
  const float* U;      // M x r
  const float* T;
  float* dA;    // slots x r x K
  float* dB;    // slots x N x r
  float* part;  // partial sums x (r K + N r)
  int32_t N, K, accumulate;
  int32_t by_place;  // no place has more rows than a segment: blockIdx.y is the place
};

constexpr int kZP = 256 + 16;  // LDS row pitch of a step's columns, in elements
constexpr int kVP = 32 + 8;    // ... of the parts of U or T
constexpr int kRowsLds = 512;  // row indices in LDS, two halves

typedef short s16x4g __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u32x2 read_turned(uint16_t* p) {
  typedef __attribute__((address_space(3))) s16x4g* lds_ptr;
  const s16x4g v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)p);
  return __builtin_bit_cast(u32x2, v);
}

template <int JB, bool DB>
__device__ __forceinline__ void grad_tile(const GradParams& p, int seg, int slot, int c0,
                                          uint16_t* zs, uint16_t* vs, int32_t* rows_s) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int g = lane >> 4, i16 = lane & 15;
  const int4 sg = seg < 0 ? make_int4(slot, 0, 0, 0) : p.a.segs[seg];
  const int n = sg.z, rank = sg.w, r = p.a.r, C = DB ? p.N : p.K;
  const int32_t* perm = p.a.perm + sg.y;
  const uint16_t* Z = DB ? p.dY : p.X;
  const float* V = DB ? p.T : p.U;
  constexpr int R = 16 * JB, VE = 32 * R / 256;  // values of U or T per thread
  f32x4 acc[4][JB];
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int j = 0; j < JB; ++j) acc[c][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  u32x4 z[2][4];
  float v[2][VE];
  // piece k of a thread: row 8 k + tid / 32, columns 8 (tid % 32)
  auto load = [&](int b, int buf) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = b + 8 * k + (tid >> 5), c = c0 + 8 * (tid & 31);
      z[buf][k] = u32x4{0u, 0u, 0u, 0u};
      if (i < n && c < C)
        z[buf][k] = *reinterpret_cast<const u32x4*>(Z + (int64_t)rows_s[i % kRowsLds] * C + c);
    }
#pragma unroll
    for (int k = 0; k < VE; ++k) {
      const int e = 256 * k + tid, i = b + e / R, j = e % R;
      v[buf][k] = 0.0f;
      if (i < n && j < rank) v[buf][k] = V[(int64_t)rows_s[i % kRowsLds] * r + j];
    }
  };
  // the indices of rows b0 .. b0 + kRowsLds / 2 - 1 into their half of the list
  auto rows = [&](int b0) {
    for (int i = b0 + tid; i < n && i < b0 + kRowsLds / 2; i += 256) rows_s[i % kRowsLds] = perm[i];
  };
  auto step = [&](int b, int buf) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k)
      *reinterpret_cast<u32x4*>(zs + (8 * k + (tid >> 5)) * kZP + 8 * (tid & 31)) = z[buf][k];
#pragma unroll
    for (int k = 0; k < VE; ++k) {
      const int e = 256 * k + tid, i = e / R, j = e % R;
      const uint16_t hi = f32_to_bf16(v[buf][k]);
      const bool fin = (hi & 0x7F80u) != 0x7F80u;
      const float r1 = fin ? v[buf][k] - bf16_to_f32(hi) : 0.0f;
      const uint16_t mid = f32_to_bf16(r1);
      vs[j * kVP + i] = hi;
      vs[(R + j) * kVP + i] = mid;
      vs[(2 * R + j) * kVP + i] = f32_to_bf16(r1 - bf16_to_f32(mid));
    }
    __syncthreads();
    if (b + 64 < n) {
      // (rows of steps b + 64 .. were listed before the barriers above)
      load(b + 64, buf);
      if ((b + 128) % (kRowsLds / 2) == 0) rows(b + 128);
    }
    u32x4 zf[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint16_t* q = zs + (8 * g + (i16 >> 2)) * kZP + 64 * wave + 16 * c + 4 * (i16 & 3);
      const u32x2 lo = read_turned(q), hi = read_turned(q + 4 * kZP);
      zf[c] = u32x4{lo[0], lo[1], hi[0], hi[1]};
    }
#pragma unroll
    for (int part = 2; part >= 0; --part)
#pragma unroll
      for (int j = 0; j < JB; ++j) {
        const u32x4 vf =
            *reinterpret_cast<const u32x4*>(vs + (part * R + 16 * j + i16) * kVP + 8 * g);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          acc[c][j] = DB ? mfma16(vf, zf[c], acc[c][j]) : mfma16(zf[c], vf, acc[c][j]);
      }
  };
  if (rank) {
    rows(0);
    rows(kRowsLds / 2);
    __syncthreads();
    load(0, 0);
    if (n > 32) load(32, 1);
    for (int b = 0; b < n; b += 64) {
      step(b, 0);
      if (b + 32 < n) step(b + 32, 1);
    }
  }
  const int first = p.a.seg0[slot];
  const bool whole = p.by_place || p.a.seg0[slot + 1] == first + 1;  // the place's only segment
  const float s = p.a.scales[slot];
  const int64_t size = (int64_t)r * p.K + (int64_t)p.N * r;
  float* out = whole ? (DB ? p.dB + (int64_t)slot * p.N * r : p.dA + (int64_t)slot * r * p.K)
                     : p.part + (p.a.part0[slot] + seg - first) * size + (DB ? (int64_t)r * p.K : 0);
  const bool add = whole && p.accumulate;
  const bool wide = !DB || r % 4 == 0;  // four results of a lane are one aligned group
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int j = 0; j < JB; ++j) {
      const int col = c0 + 64 * wave + 16 * c + (DB ? i16 : 4 * g);
      const int k = 16 * j + (DB ? 4 * g : i16);
      if (col >= C || k >= r) continue;
      float* o = DB ? out + (int64_t)col * r + k : out + (int64_t)k * C + col;
      f32x4 x;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = (DB ? k + e : k) < rank ? s * acc[c][j][e] : 0.0f;
      if (wide) {
        if (add) {
          const f32x4 y = *reinterpret_cast<const f32x4*>(o);
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] += y[e];
        }
        *reinterpret_cast<f32x4*>(o) = x;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (k + e < r) o[e] = add ? o[e] + x[e] : x[e];
      }
    }
}

template <int JB>
__global__ __launch_bounds__(256, JB <= 2 ? 4 : 3) void adapter_grads_kernel(GradParams p) {
  __shared__ __attribute__((aligned(16))) uint16_t zs[32 * kZP];
  __shared__ __attribute__((aligned(16))) uint16_t vs[3 * 16 * JB * kVP];
  __shared__ int32_t rows_s[kRowsLds];
  int seg = blockIdx.y, slot = blockIdx.y;
  if (p.by_place) {
    seg = p.a.seg0[slot];
    if (p.a.seg0[slot + 1] == seg) {  // no rows: zeros, or nothing to add
      if (p.accumulate) return;
      seg = -1;
    }
  } else {
    if (seg >= p.a.count[1]) return;
    slot = p.a.segs[seg].x;
  }
  const int ca = (p.K + 255) / 256;
  if ((int)blockIdx.x < ca)
    grad_tile<JB, false>(p, seg, slot, 256 * blockIdx.x, zs, vs, rows_s);
  else
    grad_tile<JB, true>(p, seg, slot, 256 * (blockIdx.x - ca), zs, vs, rows_s);
}

// Places of several segments: their sums in order; places without rows: zeros.
__global__ __launch_bounds__(256) void grads_finish_kernel(GradParams p) {
  const int slot = blockIdx.y;
  const int s0 = p.a.seg0[slot], s1 = p.a.seg0[slot + 1];
  if (s1 == s0 + 1 || (s1 == s0 && p.accumulate)) return;
  const int64_t na = (int64_t)p.a.r * p.K, size = na + (int64_t)p.N * p.a.r;
  const int64_t e = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x);  // both parts are multiples of 64
  if (e >= size) return;
  f32x4* o = reinterpret_cast<f32x4*>(e < na ? p.dA + slot * na + e
                                             : p.dB + (int64_t)slot * (size - na) + e - na);
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  const float* part = p.part + p.a.part0[slot] * size + e;
  for (int k = 0; k < s1 - s0; ++k) {
    const f32x4 x = *reinterpret_cast<const f32x4*>(part + k * size);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += x[i];
  }
  if (p.accumulate) {
    const f32x4 x = *o;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += x[i];
  }
  *o = v;
}

// ---------------------------------------------------------------- host

// row pitch of T's partial sums: groups of four
int t_pitch(int64_t r) { return (int)(r + 3) / 4 * 4; }

size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

// Tiles of a plan: every place may have one that is not full
int64_t max_tiles(int64_t M, int32_t slots) {
  const int64_t t = cdiv(M, kTM) + slots;
  return t < M ? t : M;
}
// a multiple of eight, so that a tile's workgroups of both launches run on one
// XCD and find T's partial sums in its L2
unsigned tile_grid(const RowArgs& a) {
  return (unsigned)(a.tiles ? cdiv(max_tiles(a.M, a.slots), 8) * 8 : a.M);
}

// Splits of the shrink's reduction over C columns: about 256 workgroups where
// tiles are full, each wave with four steps at least, so that they are in flight
// together
int shrink_splits(int64_t M, int64_t C) {
  const int64_t most = cdiv(C / 64, 16), want = cdiv(256, cdiv(M, kTM));
  const int64_t s = want < most ? want : most;
  return (int)(s < 16 ? s : 16);
}
// Rows of all splits of T's partial sums, of M rows or fewer: s splits need 256 / (s -
// 1) or more tiles to be too many
int64_t split_rows(int64_t M, int64_t C) {
  int64_t rows = M;
  for (int64_t s = shrink_splits(1, C); s > 1; --s) {
    const int64_t m = (cdiv(256, s - 1) - 1) * kTM;
    if (s * (m < M ? m : M) > rows) rows = s * (m < M ? m : M);
  }
  return rows;
}

// Rows of a segment of the gradients: about 768 workgroups where places have
// enough rows
int64_t segment_rows(int64_t M, int64_t N, int64_t K) {
  const int64_t cols = cdiv(N, 256) + cdiv(K, 256), want = cdiv(768, cols);
  const int64_t rows = cdiv(cdiv(M, want), 32) * 32;
  return rows < 128 ? 128 : rows;
}
int64_t max_segments(int64_t M, int64_t N, int64_t K, int32_t slots) {
  const int64_t s = cdiv(M, segment_rows(M, N, K)) + slots;
  return s < M ? s : M;
}

// The same for M rows or fewer: full segments are cdiv(M, 128) at most, and as many as
// segment_rows wants
int64_t most_full(int64_t M, int64_t N, int64_t K) {
  const int64_t want = cdiv(768, cdiv(N, 256) + cdiv(K, 256)), s = cdiv(M, 128);
  return s < want ? s : want;
}
int64_t most_segments(int64_t M, int64_t N, int64_t K, int32_t slots) {
  const int64_t s = most_full(M, N, K) + slots;
  return s < M ? s : M;
}

// Partial sums of the gradients, of M rows or fewer: of places with more rows than a
// segment, which have at most twice as many segments as their rows fill
int64_t most_parts(int64_t M, int64_t N, int64_t K, int32_t slots) {
  const int64_t p = 2 * most_full(M, N, K), s = most_segments(M, N, K, slots);
  return p < s ? p : s;
}

struct PlanLayout {
  size_t seg0, part0, count, tiles, segs, perm, end;
};
PlanLayout plan_layout(int64_t M, int32_t slots, int64_t segs) {
  PlanLayout l;
  l.seg0 = 0;
  l.part0 = l.seg0 + up256((size_t)(slots + 2) * 4);
  l.count = l.part0 + up256((size_t)(slots + 2) * 4);
  l.tiles = l.count + 256;
  l.segs = l.tiles + up256((size_t)(cdiv(max_tiles(M, slots), 8) * 8) * 16);  // tile_grid's
  l.perm = l.segs + up256((size_t)segs * 16);
  l.end = l.perm + up256((size_t)M * 4);
  return l;
}

// seg_rows 0: without segments (forward)
int launch_plan(RowArgs& a, const PlanLayout& l, char* ws, int64_t seg_rows, const TurnArgs& q,
                hipStream_t st) {
  PlanArgs p;
  p.rows = a.rows;
  p.ranks = a.ranks;
  p.r = a.r;
  p.seg0 = (int32_t*)(ws + l.seg0);
  p.part0 = (int32_t*)(ws + l.part0);
  p.count = (int32_t*)(ws + l.count);
  p.tiles = (int4*)(ws + l.tiles);
  p.segs = seg_rows ? (int4*)(ws + l.segs) : nullptr;
  p.perm = (int32_t*)(ws + l.perm);
  p.M = a.M;
  p.slots = a.slots;
  const int waves = kCnt / (a.slots + 1) - 3;
  p.waves = waves < 16 ? waves : 16;
  p.bits = 32 - __builtin_clz(a.slots);
  p.seg_rows = seg_rows ? (int32_t)seg_rows : kTM;
  a.seg0 = p.seg0;
  a.part0 = p.part0;
  a.count = p.count;
  a.tiles = p.tiles;
  a.segs = p.segs;
  a.perm = p.perm;
  const dim3 g((unsigned)(1 + (int64_t)a.slots * cdiv(q.chunks, 4)));
  const auto kernel = a.slots < 1024 ? plan_kernel<1> : plan_kernel<kPerThread>;
  hipLaunchKernelGGL(kernel, g, dim3(1024), 0, st, p, q);
  return hip_fail(hipGetLastError(), "adapters plan launch");
}

int launch_shrink(const RowArgs& a, const void* X, const void* A, int64_t C, float* Tp,
                  hipStream_t st) {
  const int splits = shrink_splits(a.M, C);
  ShrinkParams p;
  p.a = a;
  p.X = (const uint16_t*)X;
  p.A = (const uint16_t*)A;
  p.Tp = Tp;
  p.C = (int32_t)C;
  p.rp = t_pitch(a.r);
  p.splits = splits;
  p.steps = (int32_t)cdiv(C / 64, splits);
  const dim3 g(tile_grid(a) * (unsigned)splits), b(256);
  const auto kernel = a.tiles ? (a.r <= 16   ? shrink_tiles_kernel<1, false>
                                 : a.r <= 32 ? shrink_tiles_kernel<2, false>
                                 : a.r <= 48 ? shrink_tiles_kernel<3, false>
                                             : shrink_tiles_kernel<4, false>)
                              : (a.r <= 16   ? shrink_tiles_kernel<1, true>
                                 : a.r <= 32 ? shrink_tiles_kernel<2, true>
                                 : a.r <= 48 ? shrink_tiles_kernel<3, true>
                                             : shrink_tiles_kernel<4, true>);
  hipLaunchKernelGGL(kernel, g, b, 0, st, p);
  return hip_fail(hipGetLastError(), "adapters shrink launch");
}

// Yo NULL: only T_out
int launch_expand(const RowArgs& a, const float* Tp, int splits, const void* B, int64_t N, int ldb,
                  const void* Yi, void* Yo, float* T_out, hipStream_t st) {
  ExpandParams p;
  p.a = a;
  p.Tp = Tp;
  p.B = (const uint16_t*)B;
  p.Yi = (const uint16_t*)Yi;
  p.Yo = (uint16_t*)Yo;
  p.T_out = T_out;
  p.splits = splits;
  p.N = (int32_t)N;
  p.ldb = ldb;
  p.rp = t_pitch(a.r);
  // 256 columns per workgroup and pass; more than one pass where full tiles
  // alone are enough workgroups
  const int64_t chunks = Yo ? cdiv(N, 256) : 1, full = cdiv(a.M, kTM);
  int64_t passes = full * chunks / 4096;
  passes = passes < 1 ? 1 : passes > 8 ? 8 : passes;
  p.passes = (int32_t)passes;
  p.parts = (int32_t)cdiv(chunks, passes);
  const dim3 g(tile_grid(a) * (unsigned)p.parts), b(256);
  const bool whole = ldb % 8 == 0;
  const auto kernel =
      a.tiles ? (a.r <= 32 ? (whole ? expand_tiles_kernel<1, true, 4> : expand_tiles_kernel<1, false, 4>)
                           : (whole ? expand_tiles_kernel<2, true, 4> : expand_tiles_kernel<2, false, 4>))
              : (a.r <= 32 ? (whole ? expand_tiles_kernel<1, true, 1> : expand_tiles_kernel<1, false, 1>)
                           : (whole ? expand_tiles_kernel<2, true, 1> : expand_tiles_kernel<2, false, 1>));
  hipLaunchKernelGGL(kernel, g, b, 0, st, p);
  return hip_fail(hipGetLastError(), "adapters expand launch");
}

RowArgs row_args(int64_t M, const lq_adapter_pool& q, const int32_t* rows) {
  RowArgs a{};
  a.rows = rows;
  a.ranks = q.ranks;
  a.scales = q.scales;
  a.M = (int32_t)M;
  a.slots = q.slots;
  a.r = q.r;
  return a;
}

// Whether a forward takes one launch: few rows, one round of workgroups even if
// each row has an adapter of its own, and a factor A short enough for one
// workgroup.  In a captured graph, one launch against two: 8.4 us against 8.2 at
// 4096 x 4096 and rank 16 (1 to 16 rows), 5.0 against 7.7 at 1024 x 1024, but 19.5
// against 12.2 at rank 64 and 15.3 against 9.0 with 8 rows of 11008 columns; outside
// a graph it saves 4 us of launch and workspace.
bool few_rows(int64_t M, int64_t N, int64_t K, int64_t r) {
  return M <= kFew && M * cdiv(N, 256) <= 256 && r * K <= 65536;
}

int launch_few(const RowArgs& a, const void* X, const lq_adapter_pool& q, const void* Yi, void* Yo,
               float* T_out, hipStream_t st) {
  FewParams p;
  p.a = a;
  p.X = (const uint16_t*)X;
  p.A = (const uint16_t*)q.A;
  p.B = (const uint16_t*)q.B;
  p.Yi = (const uint16_t*)Yi;
  p.Yo = (uint16_t*)Yo;
  p.T_out = T_out;
  p.K = (int32_t)q.K;
  p.N = (int32_t)q.N;
  p.parts = (int32_t)cdiv(q.N, 256);
  const dim3 g((unsigned)(a.M * p.parts)), b(1024);
  const bool whole = q.r % 8 == 0;
  const auto kernel = q.r <= 16   ? (whole ? few_rows_kernel<1, true> : few_rows_kernel<1, false>)
                      : q.r <= 32 ? (whole ? few_rows_kernel<2, true> : few_rows_kernel<2, false>)
                      : q.r <= 48 ? (whole ? few_rows_kernel<3, true> : few_rows_kernel<3, false>)
                                  : (whole ? few_rows_kernel<4, true> : few_rows_kernel<4, false>);
  hipLaunchKernelGGL(kernel, g, b, 0, st, p);
  return hip_fail(hipGetLastError(), "adapters few-row launch");
}

// Workspace of the backward: [plan][B turned][A turned][U][T][partial sums of the
// shrinks][partial gradients]
struct BwdLayout {
  PlanLayout plan;
  size_t bt, at, u, t, tp, part, end;
};
BwdLayout bwd_layout(int64_t M, int64_t N, int64_t K, int64_t r, int32_t slots) {
  BwdLayout l;
  const int64_t r8 = cdiv(r, 8) * 8, sn = split_rows(M, N), sk = split_rows(M, K);
  l.plan = plan_layout(M, slots, most_segments(M, N, K, slots));
  l.bt = l.plan.end;
  l.at = l.bt + up256((size_t)slots * r * N * 2);
  l.u = l.at + up256((size_t)slots * r8 * K * 2);
  l.t = l.u + up256((size_t)M * r * 4);
  l.tp = l.t + up256((size_t)M * r * 4);
  l.part = l.tp + up256((size_t)(sn > sk ? sn : sk) * t_pitch(r) * 4);
  l.end = l.part + up256((size_t)most_parts(M, N, K, slots) * r * (N + K) * 4);
  return l;
}

}  // namespace

namespace dispatch {

size_t adapters_fwd_ws(int64_t M, int64_t N, int64_t K, int64_t r, int32_t slots) {
  if (few_rows(M, N, K, r)) return 0;
  const size_t plan = M <= kDirect ? 0 : plan_layout(M, slots, 0).end;
  return plan + (size_t)split_rows(M, K) * t_pitch(r) * 4;
}

size_t adapters_bwd_ws(int64_t M, int64_t N, int64_t K, int64_t r, int32_t slots) {
  return bwd_layout(M, N, K, r, slots).end;
}

int adapters_fwd(const void* X, int64_t M, const lq_adapter_pool& q, const int32_t* rows,
                 const void* Y_in, void* Y_out, float* T_out, void* ws, hipStream_t st) {
  RowArgs a = row_args(M, q, rows);
  if (few_rows(M, q.N, q.K, q.r)) return launch_few(a, X, q, Y_in, Y_out, T_out, st);
  char* base = (char*)ws;
  int rc;
  if (M > kDirect) {
    const PlanLayout l = plan_layout(M, q.slots, 0);  // (no segments)
    if ((rc = launch_plan(a, l, base, 0, TurnArgs{}, st))) return rc;
    base += l.end;
  }
  if ((rc = launch_shrink(a, X, q.A, q.K, (float*)base, st))) return rc;
  return launch_expand(a, (float*)base, shrink_splits(M, q.K), q.B, q.N, q.r, Y_in, Y_out, T_out,
                       st);
}

int adapters_bwd(const void* dY, const void* X, int64_t M, const lq_adapter_pool& q,
                 const int32_t* rows, const float* T_saved, const void* dX_in, void* dX_out,
                 float* dA, float* dB, int accumulate, void* ws, hipStream_t st) {
  const BwdLayout l = bwd_layout(M, q.N, q.K, q.r, q.slots);
  char* base = (char*)ws;
  RowArgs a = row_args(M, q, rows);
  TurnArgs t;
  t.A = (const uint16_t*)q.A;
  t.B = (const uint16_t*)q.B;
  t.At = (uint16_t*)(base + l.at);
  t.Bt = (uint16_t*)(base + l.bt);
  t.N = (int32_t)q.N;
  t.K = (int32_t)q.K;
  t.r = q.r;
  t.ld = (q.r + 7) / 8 * 8;
  t.inv = (uint32_t)cdiv(65536, t.ld / 8);
  t.chunks = (int32_t)(q.N / 64 + (dX_out ? q.K / 64 : 0));  // without dX only B is turned
  int rc = launch_plan(a, l.plan, base, segment_rows(M, q.N, q.K), t, st);
  if (rc) return rc;
  float *U = (float*)(base + l.u), *Tp = (float*)(base + l.tp), *T = (float*)(base + l.t);
  if ((rc = launch_shrink(a, dY, t.Bt, q.N, Tp, st))) return rc;
  if ((rc = launch_expand(a, Tp, shrink_splits(M, q.N), t.At, q.K, t.ld, dX_in, dX_out,
                          dA ? U : nullptr, st)))
    return rc;
  if (!dA) return LQ_OK;
  if (!T_saved) {
    if ((rc = launch_shrink(a, X, q.A, q.K, Tp, st))) return rc;
    if ((rc = launch_expand(a, Tp, shrink_splits(M, q.K), nullptr, 0, 8, nullptr, nullptr, T, st)))
      return rc;
  }
  GradParams p;
  p.a = a;
  p.X = (const uint16_t*)X;
  p.dY = (const uint16_t*)dY;
  p.U = U;
  p.T = T_saved ? T_saved : T;
  p.dA = dA;
  p.dB = dB;
  p.part = (float*)(base + l.part);
  p.N = (int32_t)q.N;
  p.K = (int32_t)q.K;
  p.accumulate = accumulate;
  p.by_place = M <= segment_rows(M, q.N, q.K);
  const dim3 g((unsigned)(cdiv(q.N, 256) + cdiv(q.K, 256)),
               (unsigned)(p.by_place ? q.slots : max_segments(M, q.N, q.K, q.slots)));
  switch ((q.r + 15) / 16) {
    case 1: hipLaunchKernelGGL(adapter_grads_kernel<1>, g, dim3(256), 0, st, p); break;
    case 2: hipLaunchKernelGGL(adapter_grads_kernel<2>, g, dim3(256), 0, st, p); break;
    case 3: hipLaunchKernelGGL(adapter_grads_kernel<3>, g, dim3(256), 0, st, p); break;
    default: hipLaunchKernelGGL(adapter_grads_kernel<4>, g, dim3(256), 0, st, p);
  }
  if ((rc = hip_fail(hipGetLastError(), "adapters gradient launch")) || p.by_place) return rc;
  const int64_t size = (int64_t)q.r * (q.N + q.K);
  hipLaunchKernelGGL(grads_finish_kernel, dim3((unsigned)cdiv(size, 1024), q.slots), dim3(256), 0,
                     st, p);
  return hip_fail(hipGetLastError(), "adapters gradient sums launch");
}

}  // namespace dispatch
}  // namespace lq
