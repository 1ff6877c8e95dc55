// Low-rank adapters of many requests at once beside a shared projection, and their gradients.
//
//   v[t] = A[a] x[t],  out[t] = bf16(base[t] + scale[a] B[a] v[t])          a: the row's adapter
//   backward: dv[t] = scale[a] B[a]^T dout[t],  dx[t] = bf16(dx_base[t] + A[a]^T dv[t]),
//   dA[a] = sum over its rows of dv[t] x[t]^T,  dB[a] = scale[a] sum of dout[t] v[t]^T.
//
// Rows of one adapter are worked on together: blocks of MB rows of a plan's tile (a plan with K = 1 groups rows by
// adapter as the layer's groups pairs by expert), or, for up to 64 rows, found by each workgroup
// from the rows' ids. Two products with the small dimension R between them:
//   down  (x -> v, dout -> dv): contraction over the long dimension, split over waves and, for few
//         rows, over workgroups, whose partial v the next kernel adds in order;
//   up    (v -> out, dv -> dx): contraction over R, v in LDS, the addition in the epilogue;
//   grad  (dA, dB): contraction over an adapter's rows, in chunks whose partial sums are added in order.
// All three are a few products for each byte of x, out or their gradients: memory bounds them.
//
// All products run on bf16 MFMA with fp32 sums. v and dv are fp32 and enter the next product as sums of bf16
// numbers: of two (off by 2^-18 at most, below the result's rounding to bf16), or of three (all of
// fp32's bits) in the gradients of the factors, whose results stay in fp32.
#include <algorithm>

#include "common.h"
#include "kernels.h"

namespace moe {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;

constexpr uint32_t kOutside = 0x80000000u;   // an offset past every buffer here: reads 0

__device__ inline f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }

// A 16 x 32 operand out of a row-major LDS tile whose rows are the contraction: lane l receives column l % 16
// (columns in fours, the lanes' own addresses choose which), rows 8 (l / 16) .. + 8. Each lane passes the address
// of row 8 (l / 16) + (l % 16) / 4, four columns l % 4; `pitch4` is four rows in bytes.
__device__ inline bf16x8 read_transposed(const uint8_t* at, uint32_t pitch4) {
  const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)at);
  const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(at + pitch4));
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// v as a sum of P bf16 numbers; what rounds to an infinity stays one
template <int P>
__device__ inline void split(float v, __bf16 (&o)[P]) {
#pragma unroll
  for (int p = 0; p < P; ++p) {
    o[p] = (__bf16)v;
    const float r = (float)o[p];
    v = __builtin_isinf(r) ? 0.f : v - r;
  }
}

struct RowArgs {
  const int32_t* src;          // plan
  const int32_t* tile_expert;
  const int32_t* num_tiles;
  const int32_t* pos;
  int32_t tile_shift;
  const int32_t* ids;          // or the rows' ids (at most 64), less `begin`
  int32_t begin;
  int32_t n, T;
  int32_t key_bits;
};

// The adapter and the rows of block mb (by the whole workgroup): false if there is no such block. rows[i] is -1
// where the block has fewer than MB.
template <int MB>
__device__ inline bool block_rows(const RowArgs& r, int mb, int& e, int* rows) {
  const int tid = threadIdx.x;
  if (!r.ids) {
    const int tile = (int)(((int64_t)mb * MB) >> r.tile_shift);
    if (tile >= r.num_tiles[0]) return false;
    e = r.tile_expert[tile];
    const int32_t* src = r.src + (int64_t)mb * MB;
    if ((uint32_t)e >= (uint32_t)r.n || src[0] < 0) return false;   // a tile's rows come first, its padding behind
    if (tid < MB) {
      const int t = src[tid];
      rows[tid] = (uint32_t)t < (uint32_t)r.T ? t : -1;
    }
    __syncthreads();
    return true;
  }
  // every wave for itself: a lane a row, the rows of one adapter one group, groups in order of their first rows
  const int lane = lane_id();
  const int id = lane < r.T ? r.ids[lane] - r.begin : -1;
  const bool valid = (uint32_t)id < (uint32_t)r.n;
  const uint64_t peers = match_key((uint32_t)id, valid, r.key_bits);
  const int rank = mask_rank(peers);
  const bool first = valid && rank == 0;
  const int blocks = first ? (__popcll(peers) + MB - 1) / MB : 0;
  const int end = wave_inclusive_scan(blocks);
  const uint64_t here = ballot(first && mb >= end - blocks && mb < end);
  if (!here) return false;
  const int lead = __builtin_ctzll(here);
  e = readlane(id, lead);
  const int j = mb - readlane(end - blocks, lead);
  if (tid < 64) {
    if (lane < MB) rows[lane] = -1;
    wave_sync();
    if (valid && id == e && rank / MB == j) rows[rank % MB] = lane;
  }
  __syncthreads();
  return true;
}

__device__ inline int adapter_rank(const int32_t* ranks, int e, int R) { return ranks ? min(max(ranks[e], 0), R) : R; }

// ---------------------------------------------------------------------------------------
// down: part[s][t][r] = f sum over slice s of z[t][k] m(r, k); TRANS: m is given as [k][r] (B for dv), else [r][k] (A)
// ---------------------------------------------------------------------------------------
struct DownArgs {
  RowArgs rows;
  const uint16_t* z;
  int64_t ldz;
  const uint16_t* m;
  const float* scale;      // of the result, or null
  const int32_t* ranks;
  int32_t K, R;
  int32_t splits;          // slices of K, whole groups of chunks each
  float* part;             // [splits][T][R]
};

constexpr int kChunk = 64;       // k of a wave's step: a 128-byte line of a row of z
constexpr int kDownWaves = 4;

template <int MB, int RF, bool TRANS>
__global__ __launch_bounds__(64 * kDownWaves) void adapter_down_kernel(DownArgs a) {
  constexpr int MF = MB / 16;
  constexpr int RP = RF * 16;
  constexpr int PITCH = RP * 2 + 16;         // bytes of a row of k in LDS (TRANS)
  constexpr int LOADS = RP / 8;              // 16-byte pieces of a chunk of m for each lane (TRANS)
  constexpr int SUMS = (kDownWaves - 1) * MB * RP * 4;
  constexpr int TILES = TRANS ? kDownWaves * kChunk * PITCH : 16;
  __shared__ __attribute__((aligned(16))) uint8_t s_mem[SUMS > TILES ? SUMS : TILES];
  __shared__ int s_rows[MB];
  const int slice = blockIdx.x % (uint32_t)a.splits;
  int e;
  if (!block_rows<MB>(a.rows, blockIdx.x / (uint32_t)a.splits, e, s_rows)) return;
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, lhi = lane >> 4;
  const int r0 = blockIdx.y * RP;
  const int rank = adapter_rank(a.ranks, e, a.R) - r0;       // ranks from r0 on
  const int nrf = rank <= 0 ? 0 : min(RF, (rank + 15) / 16);
  const int K = a.K;
  const int chunks = (K + kChunk - 1) / kChunk;
  const int per = (chunks + a.splits - 1) / a.splits;
  const int c1 = min(chunks, (slice + 1) * per);
  const uint16_t* mb = a.m + (int64_t)e * a.R * K;
  const __amdgpu_buffer_rsrc_t mr = make_rsrc(mb, (uint32_t)a.R * (uint32_t)K * 2u);
  const uint16_t* zp[MF];
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int t = s_rows[i * 16 + l16];
    zp[i] = a.z + (int64_t)(t < 0 ? max(s_rows[0], 0) : t) * a.ldz;   // rows that are not there: any, not written
  }
  f32x4 acc[MF][RF];
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int j = 0; j < RF; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  uint8_t* tile = s_mem + (TRANS ? wave * kChunk * PITCH : 0);

  u32x4 zv[2][MF];
  u32x4 mv[TRANS ? LOADS : 2 * RF];
  const auto load = [&](int c) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int k = c * kChunk + s * 32 + lhi * 8;
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        zv[s][i] = *reinterpret_cast<const u32x4*>(zp[i] + min(k, K - 8));
        if (k >= K) zv[s][i] = u32x4{0u, 0u, 0u, 0u};
      }
    }
    if constexpr (TRANS) {
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int at = lane + i * 64, row = c * kChunk + at / (RP / 8), col = (at % (RP / 8)) * 8;
        mv[i] = buf_load16(mr, row < K && col < rank ? ((uint32_t)row * (uint32_t)a.R + (uint32_t)(r0 + col)) * 2u : kOutside);
      }
    } else {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int k = c * kChunk + s * 32 + lhi * 8;
#pragma unroll
        for (int j = 0; j < RF; ++j)
          if (j < nrf) {
            const int r = j * 16 + l16;
            mv[s * RF + j] = buf_load16(mr, k < K && r < rank ? ((uint32_t)(r0 + r) * (uint32_t)K + (uint32_t)k) * 2u : kOutside);
          }
      }
    }
  };
  int c = slice * per + wave;
  if (nrf > 0 && c < c1) load(c);
  if (nrf > 0)
    for (; c < c1; c += kDownWaves) {
      bf16x8 zf[2][MF], mf[2][RF];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < MF; ++i) zf[s][i] = __builtin_bit_cast(bf16x8, zv[s][i]);
      if constexpr (TRANS) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
          const int at = lane + i * 64;
          *reinterpret_cast<u32x4*>(tile + (at / (RP / 8)) * PITCH + (at % (RP / 8)) * 16) = mv[i];
        }
        wave_sync();
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int j = 0; j < RF; ++j)
            mf[s][j] = read_transposed(tile + (s * 32 + 8 * lhi + (l16 >> 2)) * PITCH + j * 32 + (l16 & 3) * 8, 4 * PITCH);
        wave_sync();
      } else {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int j = 0; j < RF; ++j) mf[s][j] = __builtin_bit_cast(bf16x8, mv[s * RF + j]);
      }
      if (c + kDownWaves < c1) load(c + kDownWaves);
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < RF; ++j)
          if (j < nrf)
#pragma unroll
            for (int i = 0; i < MF; ++i) acc[i][j] = mfma(mf[s][j], zf[s][i], acc[i][j]);
    }
  // the waves' sums, in order; lane (l16, lhi) has row l16 and four ranks 4 lhi .. of each fragment
  __syncthreads();
  float* sums = reinterpret_cast<float*>(s_mem);
  if (wave > 0)
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int j = 0; j < RF; ++j)
        *reinterpret_cast<f32x4*>(sums + (((wave - 1) * MF + i) * RF + j) * 256 + lane * 4) = acc[i][j];
  __syncthreads();
  if (wave > 0) return;
  const float f = a.scale ? a.scale[e] : 1.f;
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int t = s_rows[i * 16 + l16];
#pragma unroll
    for (int j = 0; j < RF; ++j) {
      f32x4 v = acc[i][j];
#pragma unroll
      for (int w = 0; w < kDownWaves - 1; ++w) v += *reinterpret_cast<const f32x4*>(sums + ((w * MF + i) * RF + j) * 256 + lane * 4);
      const int r = j * 16 + lhi * 4;
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = r + q < rank ? v[q] * f : 0.f;
      if (t >= 0 && r0 + r < a.R)
        *reinterpret_cast<f32x4*>(a.part + ((int64_t)slice * a.rows.T + t) * a.R + r0 + r) = v;
    }
  }
}

// ---------------------------------------------------------------------------------------
// up: out[t][c] = bf16(base[t][c] + f sum over r of u[t][r] m(c, r)); TRANS: m is given as [r][c] (A for dx),
// else [c][r] (B). u is the sum of the down kernel's partial results.
// ---------------------------------------------------------------------------------------
struct UpArgs {
  RowArgs rows;
  const float* part;
  int32_t splits;
  const uint16_t* m;
  const float* scale;
  const int32_t* ranks;
  int32_t N, R;
  const uint16_t* base;    // null: zeros
  int64_t ld_base;
  uint16_t* out;
  int64_t ld_out;
  float* u_out;            // the sums themselves, where there are several partial results, or null
  int32_t blocks;          // blocks of rows; workgroups behind them copy rows without an adapter
  int32_t slab;            // columns of a workgroup, a multiple of 128
};

constexpr int kUpWaves = 4;
constexpr int kCopyRows = 64;

template <int MB, bool TRANS>
__global__ __launch_bounds__(64 * kUpWaves) void adapter_up_kernel(UpArgs a) {
  constexpr int MF = MB / 16;
  constexpr int MAXR = 256;
  constexpr int UP = MAXR * 2 + 16;            // bytes of a row of u in LDS
  constexpr int AP = 64 + 16;                  // bytes of a row of 32 columns of m in LDS (TRANS)
  __shared__ __attribute__((aligned(16))) uint8_t s_u[2][MB * UP];
  __shared__ __attribute__((aligned(16))) uint8_t s_m[TRANS ? kUpWaves * 32 * AP : 16];
  __shared__ int s_rows[MB];
  const int tid = threadIdx.x;
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int slabs = (a.N + a.slab - 1) / a.slab;
  const int slab = blockIdx.x % (uint32_t)slabs, block = blockIdx.x / (uint32_t)slabs;
  const int n0 = slab * a.slab, n1 = min(a.N, n0 + a.slab);
  if (block >= a.blocks) {                     // rows without an adapter
    const int t0 = (block - a.blocks) * kCopyRows;
    for (int t = t0 + wave; t < min(a.rows.T, t0 + kCopyRows); t += kUpWaves) {
      const bool has = a.rows.ids ? (uint32_t)(a.rows.ids[t] - a.rows.begin) < (uint32_t)a.rows.n : a.rows.pos[t] >= 0;
      if (has) continue;
      for (int c = n0 + lane * 8; c < n1; c += 512)
        *reinterpret_cast<u32x4*>(a.out + t * a.ld_out + c) =
            a.base ? *reinterpret_cast<const u32x4*>(a.base + t * a.ld_base + c) : u32x4{0u, 0u, 0u, 0u};
    }
    return;
  }
  int e;
  if (!block_rows<MB>(a.rows, block, e, s_rows)) return;
  const int l16 = lane & 15, lhi = lane >> 4;
  const int R = a.R, rank = adapter_rank(a.ranks, e, R);
  const int steps = (rank + 31) / 32;
  // u: partial results added in order, as two bf16 numbers each
  for (int at = tid; at < MB * steps * 8; at += 64 * kUpWaves) {
    const int row = at / (steps * 8), r = (at % (steps * 8)) * 4, t = s_rows[row];
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (t >= 0 && r < R) {
      const float* p = a.part + (int64_t)t * R + r;
      v = *reinterpret_cast<const f32x4*>(p);
#pragma unroll 4
      for (int s = 1; s < a.splits; ++s) v += *reinterpret_cast<const f32x4*>(p + (int64_t)s * a.rows.T * R);
      if (a.u_out && slab == 0) *reinterpret_cast<f32x4*>(a.u_out + (int64_t)t * R + r) = v;
    }
    bf16x4 hi, lo;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      __bf16 b[2];
      split<2>(v[q], b);
      hi[q] = b[0];
      lo[q] = b[1];
    }
    *reinterpret_cast<bf16x4*>(&s_u[0][row * UP + r * 2]) = hi;
    *reinterpret_cast<bf16x4*>(&s_u[1][row * UP + r * 2]) = lo;
  }
  // ranks past the adapter's own are zeros in u's sums as well
  if (a.u_out && slab == 0)
    for (int at = tid; at < MB * (R / 4); at += 64 * kUpWaves) {
      const int row = at / (R / 4), r = (at % (R / 4)) * 4, t = s_rows[row];
      if (t >= 0 && r >= steps * 32) *reinterpret_cast<f32x4*>(a.u_out + (int64_t)t * R + r) = f32x4{0.f, 0.f, 0.f, 0.f};
    }
  __syncthreads();
  const float f = a.scale ? a.scale[e] : 1.f;
  const uint16_t* mb = a.m + (int64_t)e * a.N * R;
  const __amdgpu_buffer_rsrc_t mr = make_rsrc(mb, (TRANS ? (uint32_t)rank : (uint32_t)R) * (uint32_t)a.N * 2u);
  uint8_t* tile = s_m + (TRANS ? wave * 32 * AP : 0);
  int tok[MF];
#pragma unroll
  for (int i = 0; i < MF; ++i) tok[i] = s_rows[i * 16 + l16];
  for (int c0 = n0 + wave * 32; c0 < n1; c0 += 32 * kUpWaves) {
    const int c = c0 + lhi * 8;                // this lane's 8 columns of the result
    u32x4 b[MF];
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      b[i] = u32x4{0u, 0u, 0u, 0u};
      if (a.base && tok[i] >= 0 && c < n1) b[i] = *reinterpret_cast<const u32x4*>(a.base + tok[i] * a.ld_base + c);
    }
    f32x4 acc[MF][2];
#pragma unroll
    for (int i = 0; i < MF; ++i) acc[i][0] = acc[i][1] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < steps; ++s) {
      bf16x8 mf[2];
      if constexpr (TRANS) {
        // rows s 32 .. of m, this wave's 32 columns
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int at = lane + i * 64, r = s * 32 + (at >> 2), col = c0 + (at & 3) * 8;
          const u32x4 v = buf_load16(mr, r < rank && col < a.N ? ((uint32_t)r * (uint32_t)a.N + (uint32_t)col) * 2u : kOutside);
          *reinterpret_cast<u32x4*>(tile + (at >> 2) * AP + (at & 3) * 16) = v;
        }
        wave_sync();
#pragma unroll
        for (int h = 0; h < 2; ++h) mf[h] = read_transposed(tile + (8 * lhi + (l16 >> 2)) * AP + (l16 & 3) * 16 + h * 8, 4 * AP);
        wave_sync();
      } else {
        const int r = s * 32 + lhi * 8;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int col = c0 + (l16 >> 2) * 8 + h * 4 + (l16 & 3);
          u32x4 v = buf_load16(mr, r < rank && col < a.N ? ((uint32_t)col * (uint32_t)R + (uint32_t)r) * 2u : kOutside);
          if (r + 8 > rank) {                  // columns past the adapter's rank hold anything
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int left = rank - (r + 2 * q);
              v[q] = left >= 2 ? v[q] : left == 1 ? v[q] & 0xffffu : 0u;
            }
          }
          mf[h] = __builtin_bit_cast(bf16x8, v);
        }
      }
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        const int at = (i * 16 + l16) * UP + (s * 32 + lhi * 8) * 2;
        const bf16x8 hi = *reinterpret_cast<const bf16x8*>(&s_u[0][at]);
        const bf16x8 lo = *reinterpret_cast<const bf16x8*>(&s_u[1][at]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          acc[i][h] = mfma(mf[h], lo, acc[i][h]);
          acc[i][h] = mfma(mf[h], hi, acc[i][h]);
        }
      }
    }
    if (c < n1)
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        if (tok[i] < 0) continue;
        u32x4 o;
        o.x = pack_bf16x2(bf16_lo(b[i].x) + f * acc[i][0][0], bf16_hi(b[i].x) + f * acc[i][0][1]);
        o.y = pack_bf16x2(bf16_lo(b[i].y) + f * acc[i][0][2], bf16_hi(b[i].y) + f * acc[i][0][3]);
        o.z = pack_bf16x2(bf16_lo(b[i].z) + f * acc[i][1][0], bf16_hi(b[i].z) + f * acc[i][1][1]);
        o.w = pack_bf16x2(bf16_lo(b[i].w) + f * acc[i][1][2], bf16_hi(b[i].w) + f * acc[i][1][3]);
        *reinterpret_cast<u32x4*>(a.out + tok[i] * a.ld_out + c) = o;
      }
  }
}

// ---------------------------------------------------------------------------------------
// grad: C[e] = sum over the adapter's rows of z[t] (columns) times u[t] (ranks)
// ---------------------------------------------------------------------------------------
// Chunks of `rows` pool rows: an adapter with one chunk has its result from it; those with more have a place in
// `part` for each chunk, added by the join kernel, which also clears those without rows.
struct GradSide {
  const uint16_t* z;
  int64_t ldz;
  const float* u;        // [splits][T][R]
  int32_t splits;
  int32_t N;             // columns
  const float* scale;    // or null
  float* out;            // dA: [n][R][N], dB: [n][N][R]; null: not wanted
  int64_t part;          // first place of `part`
};
struct GradArgs {
  const int32_t* src;
  const int32_t* offsets;
  const int32_t* counts;
  const int32_t* ranks;
  int32_t n, T, R;
  int32_t rows;          // rows of a chunk
  GradSide side[2];      // 0: dA (x, dv), 1: dB (dout, v)
  int32_t slabs0, slabs; // column slabs of side 0, and of both
  float* part;
};

constexpr int kGradCols = 128;
constexpr int kGradStep = 32;
constexpr int kGradMaxRows = 1024;

// Chunk c: its adapter and place in that; `slot` its place in part (-1: written straight). False past the last.
__device__ inline bool find_chunk(const int32_t* counts, int n, int rows, int c, int& e, int& at, int& slot) {
  const int lane = lane_id();
  int before = 0, slots = 0;
  for (int e0 = 0; e0 < n; e0 += 64) {
    const int cnt = e0 + lane < n ? counts[e0 + lane] : 0;
    const int k = (cnt + rows - 1) / rows;
    const int end = wave_inclusive_scan(k);
    const int send = wave_inclusive_scan(k > 1 ? k : 0);
    const uint64_t here = ballot(c >= before + end - k && c < before + end);
    if (here) {
      const int l = __builtin_ctzll(here);
      e = e0 + l;
      at = c - before - readlane(end - k, l);
      slot = readlane(k, l) > 1 ? slots + readlane(send - k, l) + at : -1;
      return true;
    }
    before += readlane(end, 63);
    slots += readlane(send, 63);
  }
  return false;
}

template <int RF>
__global__ __launch_bounds__(256) void adapter_grad_kernel(GradArgs a) {
  constexpr int RP = RF * 16;
  constexpr int ZP = kGradCols * 2 + 16, UP = RP * 2 + 16;
  __shared__ __attribute__((aligned(16))) uint8_t s_z[2][kGradStep * ZP];
  __shared__ __attribute__((aligned(16))) uint8_t s_u[2][3][kGradStep * UP];
  __shared__ int s_src[kGradMaxRows];
  const int tid = threadIdx.x;
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, lhi = lane >> 4;
  const int slab = blockIdx.x % (uint32_t)a.slabs;
  const bool db = slab >= a.slabs0;
  const GradSide& g = a.side[db ? 1 : 0];
  const int n0 = (slab - (db ? a.slabs0 : 0)) * kGradCols;
  const int r0 = blockIdx.y * RP;
  int e, at, slot;
  if (!find_chunk(a.counts, a.n, a.rows, blockIdx.x / (uint32_t)a.slabs, e, at, slot)) return;
  e = __builtin_amdgcn_readfirstlane(e);
  const int cnt = min(a.rows, a.counts[e] - at * a.rows);
  const int rank = adapter_rank(a.ranks, e, a.R) - r0;
  const int32_t* src = a.src + a.offsets[e] + (int64_t)at * a.rows;
  for (int i = tid; i < cnt; i += 256) {
    const int t = src[i];
    s_src[i] = (uint32_t)t < (uint32_t)a.T ? t : -1;
  }
  __syncthreads();
  const int steps = (cnt + kGradStep - 1) / kGradStep;
  // a thread's part of a step: two 16-byte pieces of z, 8 values of u
  u32x4 zv[2];
  f32x4 uv[2];
  const int urow = tid / (RP / 8), ucol = (tid % (RP / 8)) * 8;
  const auto load = [&](int s) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int p = tid + i * 256, row = s * kGradStep + (p >> 4), col = n0 + (p & 15) * 8;
      const int t = row < cnt ? s_src[row] : -1;
      zv[i] = u32x4{0u, 0u, 0u, 0u};
      if (t >= 0 && col < g.N) zv[i] = *reinterpret_cast<const u32x4*>(g.z + t * g.ldz + col);
    }
    uv[0] = uv[1] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (urow < kGradStep) {
      const int row = s * kGradStep + urow;
      const int t = row < cnt ? s_src[row] : -1;
      if (t >= 0 && ucol < rank && r0 + ucol < a.R) {
        const float* p = g.u + (int64_t)t * a.R + r0 + ucol;
        for (int q = 0; q < g.splits; ++q, p += (int64_t)a.T * a.R) {
          uv[0] += *reinterpret_cast<const f32x4*>(p);
          uv[1] += *reinterpret_cast<const f32x4*>(p + 4);
        }
      }
    }
  };
  const auto store = [&](int buf) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int p = tid + i * 256;
      *reinterpret_cast<u32x4*>(&s_z[buf][(p >> 4) * ZP + (p & 15) * 16]) = zv[i];
    }
    if (urow < kGradStep) {
      bf16x8 o[3];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        __bf16 b[3];
        split<3>(uv[q >> 2][q & 3], b);
#pragma unroll
        for (int p = 0; p < 3; ++p) o[p][q] = b[p];
      }
#pragma unroll
      for (int p = 0; p < 3; ++p) *reinterpret_cast<bf16x8*>(&s_u[buf][p][urow * UP + ucol * 2]) = o[p];
    }
  };
  f32x4 acc[2][RF];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < RF; ++j) acc[h][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  load(0);
  store(0);
  if (steps > 1) load(1);
  __syncthreads();
  const int trow = 8 * lhi + (l16 >> 2), tcol = l16 & 3;
  for (int s = 0; s < steps; ++s) {
    const int buf = s & 1;
    bf16x8 zf[2];
    // dA: a lane's columns are to be 8 neighbours (over both fragments), dB: 16 neighbours a fragment
#pragma unroll
    for (int h = 0; h < 2; ++h)
      zf[h] = read_transposed(&s_z[buf][trow * ZP + wave * 64 + (db ? h * 32 + tcol * 8 : tcol * 16 + h * 8)], 4 * ZP);
#pragma unroll
    for (int j = 0; j < RF; ++j)
#pragma unroll
      for (int p = 2; p >= 0; --p) {
        const bf16x8 uf = read_transposed(&s_u[buf][p][trow * UP + j * 32 + tcol * 8], 4 * UP);
#pragma unroll
        for (int h = 0; h < 2; ++h) acc[h][j] = db ? mfma(uf, zf[h], acc[h][j]) : mfma(zf[h], uf, acc[h][j]);
      }
    if (s + 1 < steps) {
      store(buf ^ 1);
      if (s + 2 < steps) load(s + 2);
    }
    __syncthreads();
  }
  const float f = g.scale ? g.scale[e] : 1.f;
  const int64_t size = (int64_t)a.R * g.N;
  float* out = slot < 0 ? g.out + e * size : a.part + g.part + slot * size;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < RF; ++j) {
      f32x4 v = acc[h][j];
      if (db) {
        const int col = n0 + wave * 32 + h * 16 + l16, r = j * 16 + lhi * 4;
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = r + q < rank ? v[q] * f : 0.f;
        if (col < g.N && r0 + r < a.R) *reinterpret_cast<f32x4*>(out + (int64_t)col * a.R + r0 + r) = v;
      } else {
        const int col = n0 + wave * 32 + lhi * 8 + h * 4, r = j * 16 + l16;
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = r < rank ? v[q] * f : 0.f;
        if (col < g.N && r0 + r < a.R) *reinterpret_cast<f32x4*>(out + (int64_t)(r0 + r) * g.N + col) = v;
      }
    }
}

constexpr int kJoinValues = 2048;    // values of a workgroup of the join kernel

// Adapters with several chunks: their partial results added in order; those without rows: zeros.
__global__ __launch_bounds__(256) void adapter_join_kernel(GradArgs a) {
  const int lane = lane_id();
  const int e = blockIdx.y;
  int slot = 0;
  if (a.counts)
    for (int e0 = 0; e0 <= e; e0 += 64) {     // slots of the adapters before this one
      const int cnt = e0 + lane < e ? a.counts[e0 + lane] : 0;
      const int k = (cnt + a.rows - 1) / a.rows;
      slot += readlane(wave_inclusive_scan(k > 1 ? k : 0), 63);
    }
  const int k = a.counts ? (a.counts[e] + a.rows - 1) / a.rows : 0;
  if (k == 1) return;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const GradSide& g = a.side[q];
    const int64_t size = (int64_t)a.R * g.N;
    if (!g.out) continue;
    for (int64_t i = (int64_t)blockIdx.x * kJoinValues + threadIdx.x * 4; i < min(size, ((int64_t)blockIdx.x + 1) * kJoinValues); i += 1024) {
      f32x4 v = {0.f, 0.f, 0.f, 0.f};
      const float* p = a.part + g.part + (int64_t)slot * size + i;
#pragma unroll 4
      for (int s = 0; s < k; ++s, p += size) v += *reinterpret_cast<const f32x4*>(p);
      *reinterpret_cast<f32x4*>(g.out + e * size + i) = v;
    }
  }
}

// ---------------------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------------------
constexpr int64_t kMaxGrid = (1 << 24) - 1;      // workgroups of 256 threads: fewer than 2^32 threads

// Slices of the long dimension: enough workgroups for few rows, each wave a chunk at least.
int32_t adapter_splits(int32_t T, int32_t K) {
  const int blocks = std::max(1, (T + 15) / 16), most = std::max(1, K / (kChunk * kDownWaves));
  return std::max(1, std::min(most, 512 / blocks));
}
int32_t adapter_grad_rows(int32_t T) { return T <= 2048 ? 256 : 1024; }
int32_t adapter_grad_slots(int32_t T) { return T <= adapter_grad_rows(T) ? 0 : 2 * (T / adapter_grad_rows(T)); }

static RowArgs row_args(const AdapterLaunch& l) {
  RowArgs r{};
  if (l.ids) {
    r.ids = l.ids;
    r.begin = l.begin;
    r.key_bits = l.n > 1 ? 32 - __builtin_clz((unsigned)(l.n - 1)) : 1;
  } else {
    r.src = l.plan->src;
    r.tile_expert = l.plan->tile_expert;
    r.num_tiles = l.plan->num_tiles;
    r.pos = l.plan->pos;
    r.tile_shift = __builtin_ctz((unsigned)l.plan->tile);
  }
  r.n = l.n;
  r.T = l.T;
  return r;
}
// blocks of MB rows that a grouping can have: a tile of a plan has a row at least
static int block_rows_of(const AdapterLaunch& l) { return l.ids || l.plan->tile == 16 ? 16 : 32; }
static int block_count(const AdapterLaunch& l, int mb) {
  if (l.ids) return l.T;
  const int64_t tiles = std::min<int64_t>(l.T, l.plan->rows_cap / l.plan->tile);
  return (int)(tiles * (l.plan->tile / mb));
}

static int copy_blocks(int32_t T) { return (T + kCopyRows - 1) / kCopyRows; }
static int up_slab(int32_t T) { return T <= 256 ? 128 : 512; }
static int grad_chunks(int32_t T, int32_t n) { return T / adapter_grad_rows(T) + std::min(n, T); }

// whether every launch of a forward (K to N) or backward pass has a grid that can be launched
static bool fits(const AdapterLaunch& l, int32_t K, int32_t N, bool grads) {
  if (l.T == 0) return true;
  const int64_t blocks = block_count(l, block_rows_of(l)), slab = up_slab(l.T);
  if (blocks * adapter_splits(l.T, K) > kMaxGrid || (blocks + copy_blocks(l.T)) * ((N + slab - 1) / slab) > kMaxGrid) return false;
  return !grads || (int64_t)((K + kGradCols - 1) / kGradCols + (N + kGradCols - 1) / kGradCols) * grad_chunks(l.T, l.n) <= kMaxGrid;
}

template <int MB, bool TRANS>
static void launch_down(const DownArgs& a, int blocks, hipStream_t s) {
  const int rp = a.R <= 16 ? 16 : a.R <= 32 ? 32 : a.R <= 64 ? 64 : 128;
  const dim3 grid((unsigned)(a.splits * blocks), (a.R + rp - 1) / rp), block(64 * kDownWaves);
  if (rp == 16) hipLaunchKernelGGL((adapter_down_kernel<MB, 1, TRANS>), grid, block, 0, s, a);
  else if (rp == 32) hipLaunchKernelGGL((adapter_down_kernel<MB, 2, TRANS>), grid, block, 0, s, a);
  else if (rp == 64) hipLaunchKernelGGL((adapter_down_kernel<MB, 4, TRANS>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((adapter_down_kernel<MB, 8, TRANS>), grid, block, 0, s, a);
}

template <bool TRANS>
static int down(const AdapterLaunch& l, const void* z, int64_t ldz, const void* m, const float* scale, int32_t K, float* part,
                hipStream_t stream) {
  DownArgs a;
  a.rows = row_args(l);
  a.z = static_cast<const uint16_t*>(z);
  a.ldz = ldz;
  a.m = static_cast<const uint16_t*>(m);
  a.scale = scale;
  a.ranks = l.ranks;
  a.K = K;
  a.R = l.R;
  a.splits = adapter_splits(l.T, K);
  a.part = part;
  const int mb = block_rows_of(l), blocks = block_count(l, mb);
  if (mb == 16) launch_down<16, TRANS>(a, blocks, stream);
  else launch_down<32, TRANS>(a, blocks, stream);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

template <bool TRANS>
static int up(const AdapterLaunch& l, const float* part, int32_t splits, const void* m, const float* scale, int32_t N,
              const void* base, int64_t ld_base, void* out, int64_t ld_out, float* u_out, hipStream_t stream) {
  UpArgs a;
  a.rows = row_args(l);
  a.part = part;
  a.splits = splits;
  a.m = static_cast<const uint16_t*>(m);
  a.scale = scale;
  a.ranks = l.ranks;
  a.N = N;
  a.R = l.R;
  a.base = static_cast<const uint16_t*>(base);
  a.ld_base = ld_base;
  a.out = static_cast<uint16_t*>(out);
  a.ld_out = ld_out;
  a.u_out = u_out;
  const int mb = block_rows_of(l);
  a.blocks = block_count(l, mb);
  const int copies = base == out ? 0 : copy_blocks(l.T);   // in place they stay as they are
  a.slab = up_slab(l.T);
  const dim3 grid((unsigned)((N + a.slab - 1) / a.slab * (a.blocks + copies))), block(64 * kUpWaves);
  if (mb == 16) hipLaunchKernelGGL((adapter_up_kernel<16, TRANS>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((adapter_up_kernel<32, TRANS>), grid, block, 0, stream, a);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int launch_adapter(const AdapterLaunch& l, hipStream_t stream) {
  if (!fits(l, l.K, l.N, false)) return MOE_ERR_UNSUPPORTED;
  const int splits = adapter_splits(l.T, l.K);
  float* part = splits == 1 && l.v ? l.v : static_cast<float*>(l.ws);
  int rc = down<false>(l, l.x, l.ldx, l.a, nullptr, l.K, part, stream);
  if (rc != MOE_OK) return rc;
  return up<false>(l, part, splits, l.b, l.scale, l.N, l.base, l.ld_base, l.out, l.ld_out, splits > 1 ? l.v : nullptr, stream);
}

int launch_adapter_backward(const AdapterLaunch& l, const AdapterGrads& g, hipStream_t stream) {
  if (!fits(l, l.N, l.K, true)) return MOE_ERR_UNSUPPORTED;
  const int splits = adapter_splits(l.T, l.N);
  float* dv = static_cast<float*>(l.ws);
  if (l.T > 0 && (g.dx || g.da)) {
    int rc = down<true>(l, g.dout, g.ld_dout, l.b, l.scale, l.N, dv, stream);
    if (rc == MOE_OK && g.dx)
      rc = up<true>(l, dv, splits, l.a, nullptr, l.K, g.dx_base, g.ld_base, g.dx, g.ld_dx, nullptr, stream);
    if (rc != MOE_OK) return rc;
  }
  if (!g.da && !g.db) return MOE_OK;
  GradArgs a{};
  a.ranks = l.ranks;
  a.n = l.n;
  a.T = l.T;
  a.R = l.R;
  a.rows = adapter_grad_rows(l.T);
  a.part = dv + (int64_t)splits * l.T * l.R;
  a.side[0] = {static_cast<const uint16_t*>(l.x), l.ldx, dv, splits, l.K, nullptr, g.da, 0};
  a.side[1] = {static_cast<const uint16_t*>(g.dout), g.ld_dout, l.v, 1, l.N, l.scale, g.db,
               (int64_t)adapter_grad_slots(l.T) * l.R * l.K};
  if (l.T > 0) {
    a.src = l.plan->src;
    a.offsets = l.plan->offsets;
    a.counts = l.plan->counts;
    a.slabs0 = g.da ? (l.K + kGradCols - 1) / kGradCols : 0;
    a.slabs = a.slabs0 + (g.db ? (l.N + kGradCols - 1) / kGradCols : 0);
    const int rp = l.R <= 16 ? 16 : l.R <= 32 ? 32 : 64;
    const dim3 grid((unsigned)(a.slabs * grad_chunks(l.T, l.n)), (l.R + rp - 1) / rp);
    if (rp == 16) hipLaunchKernelGGL(adapter_grad_kernel<1>, grid, dim3(256), 0, stream, a);
    else if (rp == 32) hipLaunchKernelGGL(adapter_grad_kernel<2>, grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL(adapter_grad_kernel<4>, grid, dim3(256), 0, stream, a);
    if (hipGetLastError() != hipSuccess) return MOE_ERR_HIP;
  }
  const int64_t most = (int64_t)l.R * std::max(g.da ? l.K : 0, g.db ? l.N : 0);
  hipLaunchKernelGGL(adapter_join_kernel, dim3((unsigned)((most + kJoinValues - 1) / kJoinValues), l.n), dim3(256), 0, stream, a);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe
