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
// All three are a few products for each byte of x, out or their gradients: memory bounds them. 8192 x 4096 in bf16,
// rank 64, one adapter (a copy of 1 GiB runs at 5.06 TB/s): down 17 us (x at 3.9 TB/s), v into parts 5.5, up 35 (base and
// out, 134 MB, and v's parts: 4.3 TB/s), dv 19, parts of both 6, the factors' gradients 35 + 7 (134 MB: 3.8 TB/s), dx 35. One
// row, rank 16: 4.1 + 4.9 us, two launches.
//
// All products run on bf16 MFMA with fp32 sums. v and dv are fp32 and enter the next product as sums of bf16
// numbers: of two (off by 2^-17 at most, far below the result's rounding to bf16, 2^-8; a third in out and dx costs 8 % of the
// forward pass with 64 ranks, 8192 rows, and 60 % with 256), or of three (all of fp32's bits) in the gradients of the
// factors, whose results stay in fp32.
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
// of row 8 (l / 16) + (l % 16) / 4, four columns l % 4, in bytes of the tile; `pitch4` is four rows.
// The offset is one number: through a longer chain of sums the compiler loses whose LDS it is, and waits for every
// load in flight.
__device__ inline bf16x8 read_transposed(const uint8_t* tile, uint32_t at, uint32_t pitch4) {
  const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(tile + at));
  const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(tile + at + pitch4));
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

__device__ inline float cut_bf16(float v) { return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, v) & 0xffff0000u); }

// v as a sum of two bf16 numbers, each rounded: off by 2^-17 of v at most (the first leaves 2^-8 of v's power of two, 8 bits of which
// the second has). The first is infinite where v is and not else, and the second 0 there.
__device__ inline void split(float v, __bf16 (&o)[2]) {
  o[0] = (__bf16)v;
  if (__builtin_isinf((float)o[0])) o[0] = (__bf16)cut_bf16(v);
  const float r = (float)o[0];
  o[1] = (__bf16)(__builtin_isinf(r) ? 0.f : v - r);
}

// v as a sum of three, all of its 24 bits: cut off and not rounded, so that the three are of one sign, none of them 0 unless v is,
// and all infinite where it is. So their products with an infinity or 0 add up to what v's would be, which no sum with parts
// of 0 or of both signs does. (In a part that v has no bits for stands 2^-32 of v, which is 0 below 2^-101.)
__device__ inline void split(float v, __bf16 (&o)[3]) {
  const bool finite = __builtin_fabsf(v) < __builtin_inff();
  const float none = cut_bf16(v * 0x1p-32f);
  const float p0 = cut_bf16(v), r = v - p0;
  const float p1 = cut_bf16(r), q = r - p1;
  o[0] = (__bf16)(finite ? p0 : v);
  o[1] = (__bf16)(!finite ? v : r == 0.f ? none : p1);
  o[2] = (__bf16)(!finite ? v : q == 0.f ? none : q);
}

struct RowArgs {
  const int32_t* src;          // plan
  const int32_t* tile_expert;
  const int32_t* pos;
  int32_t tile_shift;
  const int32_t* ids;          // or the rows' ids (at most 64), less `begin`
  int32_t begin;
  int32_t n, T;
  int32_t key_bits;
};

// the adapter of row t, told by its id: -1 for none (id - begin itself may leave 32 bits)
__device__ inline int id_of(const RowArgs& r, int t) {
  const int id = r.ids[t], x = (int)((uint32_t)id - (uint32_t)r.begin);
  return id >= r.begin && (uint32_t)x < (uint32_t)r.n ? x : -1;
}

// The adapter and the rows of block mb (by the whole workgroup): false if there is no such block. rows[i] is -1
// where the block has fewer than MB.
template <int MB>
__device__ inline bool block_rows(const RowArgs& r, int mb, int& e, int* rows) {
  const int tid = threadIdx.x;
  if (!r.ids) {
    // tiles past the last have no expert, src ends with its padding: both are loaded at once
    const int64_t at = (int64_t)mb * MB;
    e = r.tile_expert[at >> r.tile_shift];
    const int t = tid < MB ? r.src[at + tid] : -1;
    if ((uint32_t)e >= (uint32_t)r.n) return false;
    if (tid < MB) rows[tid] = (uint32_t)t < (uint32_t)r.T ? t : -1;
    __syncthreads();
    return rows[0] >= 0;                         // a tile's rows come first, its padding behind
  }
  // every wave for itself: a lane a row, the rows of one adapter one group, groups in order of their first rows
  const int lane = lane_id();
  const int id = lane < r.T ? id_of(r, lane) : -1;
  const bool valid = id >= 0;
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
  int32_t blocks;          // blocks of rows
  int32_t splits;          // slices of K, whole groups of chunks each
  float* part;             // [splits][T][R]
};

// Both operands come by LDS-DMA, so that every load is of whole 128-byte lines (straight into MFMA registers a load
// would touch 16 rows, 64 bytes of each, and a CU gets 10 bytes a clock that way). A stage is kc columns of the
// block's rows and of m; three stages, two of them in flight while one is multiplied, its steps of 32 columns by a wave
// each. In a stage, 16-byte pieces are permuted within their rows so that fragments are read without bank conflicts;
// the DMA writes lane after lane, so the permutation is in the source addresses.
constexpr int kDownWaves = 8;
// columns of a stage: three of them have to fit, and with more than 32 ranks two workgroups on a CU are worth more than
// longer stages (300 rows of 16 adapters, 4096 to 4096, rank 64: 17.9 us with 256, 14.3 with 128)
constexpr int down_kc(int mb, int rf) { return mb > 32 || rf > 2 ? 128 : 256; }

__device__ u32x4 adapter_zeros[1];              // never written: what is loaded for columns and rows that are not there

typedef const __attribute__((address_space(1))) void* global_ptr;
typedef __attribute__((address_space(3))) void* lds_ptr;

// 16 bytes a lane from anywhere to LDS, lane after lane from `to` on; NT: to be read once. (The host's pass, which has no
// use for it, refuses 16.)
template <bool NT = false>
__device__ inline void load_to_lds(const void* from, void* to) {
#ifdef __HIP_DEVICE_COMPILE__
  __builtin_amdgcn_global_load_lds((global_ptr)from, (lds_ptr)to, 16, 0, NT ? 2 : 0);
#endif
}
__device__ inline void load_to_lds(__amdgpu_buffer_rsrc_t from, uint32_t at, void* to) {
#ifdef __HIP_DEVICE_COMPILE__
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_ptr)to, 16, at, 0, 0, 0);
#endif
}

// A barrier behind which the wave's LDS reads are done, and all but its last N loads to LDS. (A __syncthreads
// would wait for all of them.)
template <int N>
__device__ inline void stage_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(vmcnt_enc(N) & kLgkm0);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// permutation of the 16-byte pieces of row k of transposed m, RP / 8 of them: the rows that a transposing read
// touches at once (4 neighbours of two groups of 8) land on distinct banks
template <int RP>
__device__ inline int piece_swz(int k) {
  if constexpr (RP == 32) return ((k >> 3) & 1) << 1;
  if constexpr (RP == 64) return (((k >> 1) & 1) | (((k >> 3) & 1) << 1)) << 1;
  if constexpr (RP == 128) return ((k & 3) | (((k >> 3) & 1) << 2)) << 1;
  return 0;
}

template <int MB, int RF, bool TRANS>
__global__ __launch_bounds__(64 * kDownWaves) void adapter_down_kernel(DownArgs a) {
  constexpr int MF = MB / 16, RP = RF * 16, KC = down_kc(MB, RF), PIECES = KC / 8;
  constexpr int KS = KC / 32;                    // steps of a stage
  // Few rows: a wave has a step of the stage (two waves half the rows, or half the ranks, of one), and the waves' sums
  // are added at the end. Many: a wave has rows and ranks of its own, and all steps.
  constexpr int KG = MB > 32 ? 1 : KS;           // waves among which the steps are dealt
  constexpr int JW = kDownWaves / KG;            // waves that share a step
  constexpr int IW = JW == 8 ? (RF > 1 ? 4 : 8) : MF % JW == 0 ? JW : 1;     // of them by rows
  constexpr int MW = MF / IW, RW = RF / (JW / IW);                           // fragments of z and of m of a wave
  constexpr int ZB = MB * KC * 2 / 1024, MBK = RP * KC * 2 / 1024;   // DMA blocks of 1 KiB
  constexpr int ZN = (ZB + kDownWaves - 1) / kDownWaves, MN = (MBK + kDownWaves - 1) / kDownWaves;
  constexpr int STAGE = (MB + RP) * KC * 2;
  constexpr bool NT = MB >= 64 && !TRANS;        // many rows of x pass the caches by: 20.7 us without, 16.7 so (8192 x 4096, rank 64);
                                                 // of dout they are read once more soon, by the gradients
  constexpr int JG = RW < 4 ? RW : 4;            // fragments that are summed over the waves at a time
  // every wave has the same number of loads; with fewer blocks than waves some load the same
  static_assert((ZB % kDownWaves == 0 || kDownWaves % ZB == 0) && (MBK % kDownWaves == 0 || kDownWaves % MBK == 0));
  static_assert(KG == 1 || kDownWaves / 2 * MW * JG * 1024 <= STAGE, "sums fit a stage");
  __shared__ __attribute__((aligned(16))) uint8_t s_t0[STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t s_t1[STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t s_t2[STAGE];
  __shared__ int s_rows[MB];
  const int slice = blockIdx.x % (uint32_t)a.splits;
  // one slice: neighbouring blocks, which mostly share an adapter, on one XCD
  const int block = a.splits > 1 ? blockIdx.x / (uint32_t)a.splits : (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
  int e;
  if (block >= a.blocks || !block_rows<MB>(a.rows, block, e, s_rows)) return;
  e = __builtin_amdgcn_readfirstlane(e);
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, lhi = lane >> 4;
  const int r0 = blockIdx.y * RP;
  const int rank = adapter_rank(a.ranks, e, a.R) - r0;       // ranks from r0 on
  const int K = a.K;
  const int chunks = rank > 0 ? (K + KC - 1) / KC : 0;
  const int per = (chunks + a.splits - 1) / a.splits;
  const int c0 = slice * per, c1 = min(chunks, c0 + per), n = c1 - c0, k1 = min(K, c1 * KC);
  const __amdgpu_buffer_rsrc_t mr = make_rsrc(a.m + (int64_t)e * a.R * K, (uint32_t)a.R * (uint32_t)K * 2u);
  // this lane's piece of each of its wave's blocks: of z a pointer to its row and the column, of m an offset
  const uint16_t* zrow[ZN];
  int zcol[ZN], zend[ZN], mcol[MN];
  uint32_t moff[MN];
#pragma unroll
  for (int i = 0; i < ZN; ++i) {
    const int at = (wave + i * kDownWaves) % ZB * 64 + lane, row = at / PIECES;
    const int t = s_rows[row];
    zcol[i] = ((at % PIECES) ^ (row & 15)) * 8;
    zrow[i] = a.z + max(t, 0) * a.ldz;
    zend[i] = t < 0 ? 0 : k1 - zcol[i];          // stages that begin before have the column
  }
#pragma unroll
  for (int i = 0; i < MN; ++i) {
    const int at = (wave + i * kDownWaves) % MBK * 64 + lane;
    if constexpr (TRANS) {
      const int k = at / (RP / 8), col = ((at % (RP / 8)) ^ piece_swz<RP>(k)) * 8;
      mcol[i] = col < rank ? k : K;
      moff[i] = ((uint32_t)k * (uint32_t)a.R + (uint32_t)(r0 + col)) * 2u;
    } else {
      const int r = at / PIECES;
      mcol[i] = r < rank ? ((at % PIECES) ^ (r & 15)) * 8 : K;
      moff[i] = ((uint32_t)(r0 + r) * (uint32_t)K + (uint32_t)mcol[i]) * 2u;
    }
  }
  const auto dma = [&](int c, uint8_t* stage) {
    const int k0 = (c0 + c) * KC;
#pragma unroll
    for (int i = 0; i < ZN; ++i) {
      const uint64_t there = reinterpret_cast<uint64_t>(zrow[i] + k0 + zcol[i]), none = reinterpret_cast<uint64_t>(adapter_zeros);
      load_to_lds<NT>(reinterpret_cast<const void*>(k0 < zend[i] ? there : none), stage + (wave + i * kDownWaves) % ZB * 1024);
    }
    const uint32_t step = (uint32_t)k0 * (TRANS ? (uint32_t)a.R : 1u) * 2u;
#pragma unroll
    for (int i = 0; i < MN; ++i)
      load_to_lds(mr, k0 + mcol[i] < k1 ? moff[i] + step : kOutside, stage + MB * KC * 2 + (wave + i * kDownWaves) % MBK * 1024);
  };
  f32x4 acc[MW][RW];
#pragma unroll
  for (int i = 0; i < MW; ++i)
#pragma unroll
    for (int j = 0; j < RW; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int kg = wave % KG, i0 = wave / KG % IW * MW, j0 = wave / KG / IW * RW;
  // where m begins in a stage: not to be known, else the compiler sees that reads of m miss the stage's first load, which
  // it takes for all of them, and waits for every load in flight
  int m_at = MB * KC * 2;
  asm volatile("" : "+s"(m_at));
  const auto step = [&](int c, const uint8_t* cur, uint8_t* next) {
    dma(c + 2, next);      // the stage that everybody was done with at the last barrier
#pragma unroll
    for (int q = 0; q < KS / KG; ++q) {
      const int ks = KG == 1 ? q : kg;
      bf16x8 zf[MW];
#pragma unroll
      for (int i = 0; i < MW; ++i)
        zf[i] = *reinterpret_cast<const bf16x8*>(cur + (((i0 + i) * 16 + l16) * (KC * 2) + (((ks * 4 + lhi) ^ l16) << 4)));
#pragma unroll
      for (int j = 0; j < RW; ++j) {
        bf16x8 mf;
        if constexpr (TRANS) {
          const int k = ks * 32 + 8 * lhi + (l16 >> 2);      // + 4 has the same permutation
          const int piece = ((j0 + j) * 2 + ((l16 >> 1) & 1)) ^ piece_swz<RP>(k);
          mf = read_transposed(cur, m_at + k * (RP * 2) + piece * 16 + (l16 & 1) * 8, 4 * RP * 2);
        } else {
          mf = *reinterpret_cast<const bf16x8*>(cur + (m_at + ((j0 + j) * 16 + l16) * (KC * 2) + (((ks * 4 + lhi) ^ l16) << 4)));
        }
#pragma unroll
        for (int i = 0; i < MW; ++i) acc[i][j] = mfma(mf, zf[i], acc[i][j]);
      }
    }
    // this wave's loads of stage c + 1 have landed (those of c + 2 are behind them), then everybody's. Stages past the
    // last are loaded as zeros, without traffic, so that the counts hold.
    stage_barrier<ZN + MN>();
  };
  if (n > 0) {
    dma(0, s_t0);
    dma(1, s_t1);
    stage_barrier<ZN + MN>();
    int c = 0;
    for (; c + 3 <= n; c += 3) {
      step(c, s_t0, s_t2);
      step(c + 1, s_t1, s_t0);
      step(c + 2, s_t2, s_t1);
    }
    if (c < n) step(c, s_t0, s_t2);
    if (c + 1 < n) step(c + 1, s_t1, s_t0);
    wait_vm0();
  }
  // Lane (l16, lhi) has row l16 and four ranks 4 lhi .. of each fragment. The waves' sums of a step each are halved until
  // one wave has them.
  if constexpr (KG > 1) {
    float* sums = reinterpret_cast<float*>(s_t0);
#pragma unroll
    for (int g = 0; g < RW; g += JG)
#pragma unroll
      for (int half = KG / 2; half > 0; half /= 2) {
        __syncthreads();
        const int at = wave / KG * half;
        if (kg >= half && kg < 2 * half)
#pragma unroll
          for (int i = 0; i < MW; ++i)
#pragma unroll
            for (int j = 0; j < JG; ++j)
              *reinterpret_cast<f32x4*>(sums + (((at + kg - half) * MW + i) * JG + j) * 256 + lane * 4) = acc[i][g + j];
        __syncthreads();
        if (kg < half)
#pragma unroll
          for (int i = 0; i < MW; ++i)
#pragma unroll
            for (int j = 0; j < JG; ++j)
              acc[i][g + j] += *reinterpret_cast<const f32x4*>(sums + (((at + kg) * MW + i) * JG + j) * 256 + lane * 4);
      }
    if (kg > 0) return;
  }
  const float f = a.scale ? a.scale[e] : 1.f;
#pragma unroll
  for (int i = 0; i < MW; ++i) {
    const int t = s_rows[(i0 + i) * 16 + l16];
#pragma unroll
    for (int j = 0; j < RW; ++j) {
      f32x4 v = acc[i][j];
      const int r = (j0 + j) * 16 + lhi * 4;
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
// Row t, one without an adapter: out = base. By a wave, a row's loads in flight together.
struct CopyArgs {
  const uint16_t* base;    // null: zeros
  int64_t ld_base;
  uint16_t* out;
  int64_t ld_out;
  int32_t N;
};
__device__ inline void copy_row(const CopyArgs& a, const RowArgs& rows, int t) {
  if ((rows.ids ? id_of(rows, t) : rows.pos[t]) >= 0) return;
  const uint16_t* from = a.base + t * a.ld_base;
  uint16_t* to = a.out + t * a.ld_out;
  for (int c = lane_id() * 8; c < a.N; c += 8 * 512) {
    u32x4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = a.base ? *reinterpret_cast<const u32x4*>(from + min(c + i * 512, a.N - 8)) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i * 512 < a.N) *reinterpret_cast<u32x4*>(to + c + i * 512) = v[i];
  }
}

struct UpArgs {
  RowArgs rows;
  const float* part;       // u as partial results,
  int32_t splits;
  const uint16_t* parts;   // or (not null) as two bf16 numbers: the first [T][R], the second behind them
  const uint16_t* m;
  const float* scale;
  const int32_t* ranks;
  int32_t N, R;
  CopyArgs io;             // base and out
  float* u_out;            // the sums themselves, where there are several partial results, or null
  int32_t copies;          // workgroups in front that copy rows without an adapter, kCopyRows each
};

constexpr int kCopyRows = 4;     // of a workgroup, a row a wave
constexpr int kUpWaves = 4;
constexpr int up_cols(int rs) { return rs > 4 ? 32 : 64; }    // columns of a wave
constexpr int kRowsAhead = 2;

// A wave has CW columns of m in registers and makes them for the block's rows, 16 at a time, with base of the next ones
// in flight. A CU's address unit takes 64 neighbouring bytes of neighbouring lanes a clock, so u is the first operand of
// the product and fragment j has columns 4 i + j (CW = 64): a lane has 4 neighbours of a row, 16 lanes a whole line
// (with the rows along the lanes, each lane's 16 bytes were a clock of their own: 44 us for 8192 x 4096 in bf16, rank 64).
// RS: steps of 32 ranks that u has at most.
template <int MB, int RS, bool TRANS>
__global__ __launch_bounds__(64 * kUpWaves, RS <= 2 ? 4 : 2) void adapter_up_kernel(UpArgs a) {
  constexpr int NW = kUpWaves, CW = up_cols(RS), CF = CW / 16;
  constexpr int CD = CF / 2;                             // 4-byte words of a row for each lane
  typedef uint32_t words __attribute__((ext_vector_type(CD)));
  constexpr int UP = RS * 64 + 16;                       // bytes of a row of u in LDS,
  constexpr int MP = TRANS ? CW * 2 + 16 : 64 + 16;      // of 32 ranks of m: a rank's columns (TRANS), else a column's ranks
  constexpr int MR = TRANS ? 32 : CW;                    // rows of that
  constexpr int MPC = TRANS ? CW / 8 : 4;                // 16-byte pieces of such a row,
  constexpr int MN = MR * MPC / 64;                      // of all of it for each lane
  __shared__ __attribute__((aligned(16))) uint8_t s_mem[2 * MB * UP > NW * MR * MP ? 2 * MB * UP : NW * MR * MP];   // m, then u
  __shared__ __attribute__((aligned(16))) int s_rows[MB];
  const int tid = threadIdx.x;
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  if ((int)blockIdx.x < a.copies) {            // rows without an adapter
    const int t = blockIdx.x * kCopyRows + wave;
    if (t < a.rows.T) copy_row(a.io, a.rows, t);
    return;
  }
  const int slabs = (a.N + CW * NW - 1) / (CW * NW);
  const int slab = (blockIdx.x - a.copies) % (uint32_t)slabs, block = (blockIdx.x - a.copies) / (uint32_t)slabs;
  const int n0 = slab * (CW * NW), n1 = min(a.N, n0 + CW * NW);
  int e;
  if (!block_rows<MB>(a.rows, block, e, s_rows)) return;
  e = __builtin_amdgcn_readfirstlane(e);
  const int l16 = lane & 15, lhi = lane >> 4;
  const int R = a.R, rank = adapter_rank(a.ranks, e, R);
  const int steps = (rank + 31) / 32;
  const __amdgpu_buffer_rsrc_t mr = make_rsrc(a.m + (int64_t)e * a.N * R, (uint32_t)R * (uint32_t)a.N * 2u);
  const int c0 = n0 + wave * CW;               // this wave's columns,
  const int lc = c0 + l16 * CF;                // this lane's CF of them

  u32x4 mv[RS][MN];
#pragma unroll
  for (int s = 0; s < RS; ++s)
#pragma unroll
    for (int i = 0; i < MN; ++i) {
      const int at = lane + i * 64, row = at / MPC, piece = at % MPC;
      const int r = s * 32 + (TRANS ? row : piece * 8), col = c0 + (TRANS ? piece * 8 : row);
      const uint32_t off = TRANS ? (uint32_t)r * (uint32_t)a.N + (uint32_t)col : (uint32_t)col * (uint32_t)R + (uint32_t)r;
      mv[s][i] = buf_load16(mr, r < rank && col < a.N ? off * 2u : kOutside);
    }
  // u, where it is there in parts
  constexpr int UN = MB * RS * 4 / (64 * NW) > 0 ? MB * RS * 4 / (64 * NW) : 1;     // 16-byte pieces of a part for each lane
  u32x4 uv[UN][2];
  if (a.parts) {
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      const int at = tid + i * 64 * NW, row = at / (RS * 4), r = (at % (RS * 4)) * 8, t = row < MB ? s_rows[row] : -1;
      const bool has = t >= 0 && r < R;
      const uint16_t* p = a.parts + (has ? (int64_t)t * R + r : 0);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uv[i][k] = *reinterpret_cast<const u32x4*>(p + k * (int64_t)a.rows.T * R);
        if (!has) uv[i][k] = u32x4{0u, 0u, 0u, 0u};
      }
    }
  }
  words base[kRowsAhead][4];
  const auto load_base = [&](int i, words (&b)[4]) {
    const int4 t = *reinterpret_cast<const int4*>(&s_rows[i * 16 + lhi * 4]);
    const int ts[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int q = 0; q < 4; ++q)
      b[q] = a.io.base ? *reinterpret_cast<const words*>(a.io.base + max(ts[q], 0) * a.io.ld_base + min(lc, a.N - CF)) : words{};
  };
#pragma unroll
  for (int i = 0; i < kRowsAhead; ++i) load_base(min(i, MB / 16 - 1), base[i]);

  // m's fragments: lane (l16, lhi) has ranks 8 lhi .. of column CF l16 + j. Transposed, the tile holds column CF i + j
  // at place 16 j + i, which is where the transposing read looks for lane i's.
  bf16x8 mf[RS][CF];
  uint8_t* tile = s_mem + wave * (MR * MP);
#pragma unroll
  for (int s = 0; s < RS; ++s) {
#pragma unroll
    for (int i = 0; i < MN; ++i) {
      const int at = lane + i * 64, row = at / MPC, piece = at % MPC;
      u32x4 v = mv[s][i];
      if constexpr (!TRANS) {
        if (rank & 7) {                        // columns past the adapter's rank hold anything
          const int left = rank - (s * 32 + piece * 8);
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] = left >= 2 * q + 2 ? v[q] : left == 2 * q + 1 ? v[q] & 0xffffu : 0u;
        }
        *reinterpret_cast<u32x4*>(tile + row * MP + piece * 16) = v;
      } else if constexpr (CF == 4) {          // columns k and 4 + k of the piece are neighbours
        uint8_t* to = tile + row * MP + piece * 4;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<uint32_t*>(to + k * 32) = k & 1 ? (v[k >> 1] >> 16) | (v[2 + (k >> 1)] & 0xffff0000u)
                                                            : (v[k >> 1] & 0xffffu) | (v[2 + (k >> 1)] << 16);
      } else {                                 // columns k, 2 + k, 4 + k and 6 + k are
        uint8_t* to = tile + row * MP + piece * 8;
        *reinterpret_cast<u32x2*>(to) = u32x2{(v[0] & 0xffffu) | (v[1] << 16), (v[2] & 0xffffu) | (v[3] << 16)};
        *reinterpret_cast<u32x2*>(to + 32) = u32x2{(v[0] >> 16) | (v[1] & 0xffff0000u), (v[2] >> 16) | (v[3] & 0xffff0000u)};
      }
    }
    wave_sync();
#pragma unroll
    for (int j = 0; j < CF; ++j) {
      if constexpr (TRANS) mf[s][j] = read_transposed(tile, (8 * lhi + (l16 >> 2)) * MP + j * 32 + (l16 & 3) * 8, 4 * MP);
      else mf[s][j] = *reinterpret_cast<const bf16x8*>(tile + ((l16 * CF + j) * MP + lhi * 16));
    }
    wave_sync();
  }

  // Whether m holds an infinity or NaN: a product with zeros shows it. Where u's second part is 0 or of the other sign, an
  // infinity times both parts is NaN, so what is not finite of such a wave's results is made of the first part alone.
  bool odd;
  {
    f32x4 z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < RS; ++s)
#pragma unroll
      for (int j = 0; j < CF; ++j) z = mfma(bf16x8{}, mf[s][j], z);
    odd = ballot(z[0] != 0.f) != 0;
  }

  // u as two bf16 numbers each: as they are, or of partial results added in order
  uint8_t* s_u = s_mem;
  __syncthreads();
  if (a.parts) {
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      const int at = tid + i * 64 * NW, row = at / (RS * 4), r = (at % (RS * 4)) * 8;
      if (row >= MB) break;
#pragma unroll
      for (int k = 0; k < 2; ++k) *reinterpret_cast<u32x4*>(&s_u[k * (MB * UP) + row * UP + r * 2]) = uv[i][k];
    }
  } else {
    for (int at = tid; at < MB * RS * 8; at += 64 * NW) {
      const int row = at / (RS * 8), r = (at % (RS * 8)) * 4, t = s_rows[row];
      f32x4 v = {0.f, 0.f, 0.f, 0.f};
      if (t >= 0 && r < R) {
        const float* p = a.part + (int64_t)t * R + r;
        v = *reinterpret_cast<const f32x4*>(p);
#pragma unroll 8
        for (int s = 1; s < a.splits; ++s) v += *reinterpret_cast<const f32x4*>(p + (int64_t)s * a.rows.T * R);
        if (a.u_out && slab == 0) *reinterpret_cast<f32x4*>(a.u_out + (int64_t)t * R + r) = v;
      }
      bf16x4 hi, lo;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        __bf16 o[2];
        split(v[q], o);
        hi[q] = o[0];
        lo[q] = o[1];
      }
      *reinterpret_cast<bf16x4*>(&s_u[row * UP + r * 2]) = hi;
      *reinterpret_cast<bf16x4*>(&s_u[MB * UP + row * UP + r * 2]) = lo;
    }
  }
  __syncthreads();
  const float f = a.scale ? a.scale[e] : 1.f;
  const auto rows16 = [&](int i, words (&b)[4]) {
    f32x4 acc[CF];
#pragma unroll
    for (int j = 0; j < CF; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < RS; ++s)
      if (s < steps) {
        const int at = (i * 16 + l16) * UP + (s * 32 + lhi * 8) * 2;
        const bf16x8 hi = *reinterpret_cast<const bf16x8*>(&s_u[at]);
        const bf16x8 lo = *reinterpret_cast<const bf16x8*>(&s_u[MB * UP + at]);
#pragma unroll
        for (int j = 0; j < CF; ++j) acc[j] = mfma(lo, mf[s][j], acc[j]);
#pragma unroll
        for (int j = 0; j < CF; ++j) acc[j] = mfma(hi, mf[s][j], acc[j]);
      }
    if (odd)
#pragma unroll
      for (int j = 0; j < CF; ++j) {
        f32x4 one = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < RS; ++s)
          if (s < steps) one = mfma(*reinterpret_cast<const bf16x8*>(&s_u[(i * 16 + l16) * UP + (s * 32 + lhi * 8) * 2]), mf[s][j], one);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (!(__builtin_fabsf(acc[j][q]) < __builtin_inff())) acc[j][q] = one[q];
      }
    words o[4];                                  // row 4 lhi + q
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int k = 0; k < CD; ++k) {
        const uint32_t w = b[q][k];
        o[q][k] = pack_bf16x2(bf16_lo(w) + f * acc[2 * k][q], bf16_hi(w) + f * acc[2 * k + 1][q]);
      }
    if (i + kRowsAhead < MB / 16) load_base(i + kRowsAhead, b);
    const int4 t = *reinterpret_cast<const int4*>(&s_rows[i * 16 + lhi * 4]);
    const int ts[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (ts[q] >= 0 && lc < n1) {
        words* to = reinterpret_cast<words*>(a.io.out + ts[q] * a.io.ld_out + lc);
        // many rows are written past the caches, whose lines the next kernel would have to wait for: 20.5 us
        // instead of 24.2 for the down kernel behind it, and as long here
        if constexpr (MB >= 64) __builtin_nontemporal_store(o[q], to);
        else *to = o[q];
      }
  };
#pragma unroll
  for (int i = 0; i < MB / 16; ++i) {
    if (i > 0 && s_rows[i * 16] < 0) break;      // padding behind the adapter's rows
    rows16(i, base[i % kRowsAhead]);
  }
}

// ---------------------------------------------------------------------------------------
// grad: C[e] = sum over the adapter's rows of z[t] (columns) times u[t] (ranks)
// ---------------------------------------------------------------------------------------
// Each of x and dout is read once more than the formulas need (by the down kernel before): dA waits for all of dv, and
// dB in the down kernel's order, rows outside and columns inside, would leave a partial result for every 128 rows.
// Chunks of `rows` pool rows: an adapter with one chunk has its result from it; those with more have a place in
// `part` for each chunk, added by the join kernel, which also clears those without rows.
struct GradSide {
  const uint16_t* z;
  int64_t ldz;
  const uint16_t* u;     // three bf16 numbers a value: [3][T][R]
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
  int32_t slots;         // places of `part`, for each side
  int32_t rows_cap;      // of src
  GradSide side[2];      // 0: dA (x, dv), 1: dB (dout, v)
  int32_t slabs0, slabs; // column slabs of side 0, and of both
  float* part;
};

constexpr int kGradCols = 256;
constexpr int kGradStep = 32;
constexpr int kGradMaxRows = 1024;
constexpr int kGradWaves = 8;

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

// A step is 32 rows: 512 bytes of each row of z and its three parts of u, by LDS-DMA as in the down kernel, four stages
// of which three are in flight. The rows are the contraction, so both operands are read transposed. A wave
// has 64 columns and half the ranks (32 columns with one fragment of ranks).
template <int RF>
__global__ __launch_bounds__(64 * kGradWaves) void adapter_grad_kernel(GradArgs a) {
  constexpr int RP = RF * 16;
  constexpr int RG = RF > 1 ? 2 : 1, CG = kGradWaves / RG;   // waves by ranks and by columns
  constexpr int CF = kGradCols / 16 / CG, RW = RF / RG;      // fragments of a wave
  constexpr int ZBYTES = kGradStep * kGradCols * 2, UBYTES = kGradStep * RP * 2;
  constexpr int ZN = ZBYTES / 1024 / kGradWaves;             // loads of a wave
  constexpr int UB = 3 * UBYTES / 1024, UN = (UB + kGradWaves - 1) / kGradWaves;
  constexpr int STAGE = ZBYTES + 3 * UBYTES;
  __shared__ __attribute__((aligned(16))) uint8_t s_t0[STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t s_t1[STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t s_t2[STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t s_t3[STAGE];
  __shared__ int s_src[kGradMaxRows + 8 * kGradStep];
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
  if (!find_chunk(a.counts, a.n, a.rows, blockIdx.x / (uint32_t)a.slabs, e, at, slot) || slot >= a.slots) return;
  e = __builtin_amdgcn_readfirstlane(e);
  const int cnt = min(a.rows, a.counts[e] - at * a.rows);
  const int rank = adapter_rank(a.ranks, e, a.R) - r0;
  const int steps = (cnt + kGradStep - 1) / kGradStep;
  const int64_t first = a.offsets[e] + (int64_t)at * a.rows;
  for (int i = tid; i < (steps + 8) * kGradStep; i += 64 * kGradWaves) {      // steps past the last: no rows
    const int t = i < cnt && (uint64_t)(first + i) < (uint64_t)a.rows_cap ? a.src[first + i] : -1;
    s_src[i] = (uint32_t)t < (uint32_t)a.T ? t : -1;
  }
  __syncthreads();
  // this lane's pieces of a step: row and column. The 16-byte pieces of a row of z are permuted so that the 16 rows
  // of a transposing read land on distinct banks (u: piece_swz).
  const uint16_t* zc[ZN];
  const uint16_t* uc[UN];
  int urow[UN];
#pragma unroll
  for (int i = 0; i < ZN; ++i) {
    const int p = (wave + i * kGradWaves) * 64 + lane, row = p >> 5;
    const int swz = ((row & 3) | (((row >> 3) & 3) << 2)) << 1;
    zc[i] = g.z + min(n0 + ((p & 31) ^ swz) * 8, g.N - 8);     // columns past the last are never written
  }
#pragma unroll
  for (int i = 0; i < UN; ++i) {
    const int p = (wave + i * kGradWaves) % UB * 64 + lane, plane = p / (UBYTES / 16), q = p % (UBYTES / 16);
    urow[i] = q / (RP / 8);
    const int r = r0 + ((q % (RP / 8)) ^ piece_swz<RP>(urow[i])) * 8;
    uc[i] = r < a.R ? g.u + (int64_t)plane * a.T * a.R + r : nullptr;
  }
  const int64_t ldz = g.ldz;
  const auto dma = [&](int s, uint8_t* stage) {
    const uint64_t none = reinterpret_cast<uint64_t>(adapter_zeros);
#pragma unroll
    for (int i = 0; i < ZN; ++i) {
      const int t = s_src[s * kGradStep + (((wave + i * kGradWaves) * 64 + lane) >> 5)];
      const uint64_t there = reinterpret_cast<uint64_t>(zc[i] + t * ldz);
      load_to_lds(reinterpret_cast<const void*>(t >= 0 ? there : none), stage + (wave + i * kGradWaves) * 1024);
    }
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      const int t = s_src[s * kGradStep + urow[i]];
      const uint64_t there = reinterpret_cast<uint64_t>(uc[i] + (int64_t)t * a.R);
      load_to_lds(reinterpret_cast<const void*>(((t >= 0) & (uc[i] != nullptr)) ? there : none), stage + ZBYTES + (wave + i * kGradWaves) % UB * 1024);
    }
  };
  f32x4 acc[CF][RW];
#pragma unroll
  for (int h = 0; h < CF; ++h)
#pragma unroll
    for (int j = 0; j < RW; ++j) acc[h][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int h0 = wave % CG * CF, j0 = wave / CG * RW;
  // this lane's places in a stage (the rows of a fragment's second half have the same permutation)
  const int trow = 8 * lhi + (l16 >> 2);
  const int tswz = ((trow & 3) | (((trow >> 3) & 3) << 2)) << 1;
  uint32_t zat[CF], uat[RW];
#pragma unroll
  for (int h = 0; h < CF; ++h) zat[h] = trow * (kGradCols * 2) + ((((h0 + h) * 2 + ((l16 >> 1) & 1)) ^ tswz) << 4) + (l16 & 1) * 8;
#pragma unroll
  for (int j = 0; j < RW; ++j)
    uat[j] = ZBYTES + trow * (RP * 2) + ((((j0 + j) * 2 + ((l16 >> 1) & 1)) ^ piece_swz<RP>(trow)) << 4) + (l16 & 1) * 8;
  const auto step = [&](int s, const uint8_t* cur, uint8_t* next) {
    dma(s + 3, next);      // the stage that everybody was done with at the last barrier
    bf16x8 zf[CF];
#pragma unroll
    for (int h = 0; h < CF; ++h) zf[h] = read_transposed(cur, zat[h], 4 * kGradCols * 2);
#pragma unroll
    for (int j = 0; j < RW; ++j)
#pragma unroll
      for (int p = 2; p >= 0; --p) {
        const bf16x8 uf = read_transposed(cur, uat[j] + p * UBYTES, 4 * RP * 2);
#pragma unroll
        for (int h = 0; h < CF; ++h) acc[h][j] = mfma(zf[h], uf, acc[h][j]);
      }
    stage_barrier<2 * (ZN + UN)>();
  };
  dma(0, s_t0);
  dma(1, s_t1);
  dma(2, s_t2);
  stage_barrier<2 * (ZN + UN)>();
  for (int s = 0; s < steps; s += 4) {      // whole rounds: steps past the last add zeros
    step(s, s_t0, s_t3);
    step(s + 1, s_t1, s_t0);
    step(s + 2, s_t2, s_t1);
    step(s + 3, s_t3, s_t2);
  }
  wait_vm0();
  const float f = g.scale ? g.scale[e] : 1.f;
  const int64_t size = (int64_t)a.R * g.N;
  float* out = slot < 0 ? g.out + e * size : a.part + g.part + slot * size;
#pragma unroll
  for (int h = 0; h < CF; ++h) {
    const int col = n0 + (h0 + h) * 16 + lhi * 4;
#pragma unroll
    for (int j = 0; j < RW; ++j) {
      const int r = (j0 + j) * 16 + l16;
      f32x4 v = acc[h][j];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = r < rank ? v[q] * f : 0.f;
      if (col >= g.N || r0 + r >= a.R) continue;
      if (db) {
#pragma unroll
        for (int q = 0; q < 4; ++q) out[(int64_t)(col + q) * a.R + r0 + r] = v[q];
      } else {
        *reinterpret_cast<f32x4*>(out + (int64_t)(r0 + r) * g.N + col) = v;
      }
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
  if (k == 1 || (k > 1 && slot + k > a.slots)) return;
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

// u[i], the sum of `splits` partial results in order, in bf16 numbers n apart: two for the up kernel and three for the
// gradients (each null: not wanted); of two arrays
struct PartsArgs {
  const float* part[2];
  int32_t splits[2];
  uint16_t* two[2];
  uint16_t* three[2];
  int64_t n;
  float* sum;            // the first array's sums themselves, or null
  int32_t R;
  int32_t blocks;        // workgroups of that; those behind them copy rows without an adapter
  RowArgs rows;
  CopyArgs io;
};
__global__ __launch_bounds__(256) void adapter_parts_kernel(PartsArgs a) {
  if ((int)blockIdx.x >= a.blocks) {
    const int t = ((int)blockIdx.x - a.blocks) * kCopyRows + (threadIdx.x >> 6);
    if (t < a.rows.T && blockIdx.y == 0) copy_row(a.io, a.rows, t);
    return;
  }
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  const int k = blockIdx.y;
  if (i >= a.n || !(a.two[k] || a.three[k])) return;
  const float* part = a.part[k];
  f32x4 v = *reinterpret_cast<const f32x4*>(part + i);
#pragma unroll 8
  for (int s = 1; s < a.splits[k]; ++s) v += *reinterpret_cast<const f32x4*>(part + s * a.n + i);
  if (a.sum && k == 0 && a.rows.pos[i / a.R] >= 0) *reinterpret_cast<f32x4*>(a.sum + i) = v;   // R % 4 == 0: one row's
  const auto write = [&]<int P>(uint16_t* out, std::integral_constant<int, P>) {
    bf16x4 o[P];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      __bf16 b[P];
      split(v[q], b);
#pragma unroll
      for (int p = 0; p < P; ++p) o[p][q] = b[p];
    }
#pragma unroll
    for (int p = 0; p < P; ++p) *reinterpret_cast<bf16x4*>(out + p * a.n + i) = o[p];
  };
  if (a.two[k]) write(a.two[k], std::integral_constant<int, 2>{});
  if (a.three[k]) write(a.three[k], std::integral_constant<int, 3>{});
}

// ---------------------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------------------
constexpr int64_t kMaxGrid = (1 << 23) - 8;      // workgroups of up to 512 threads: fewer than 2^32 threads

// rows of a block: 128 for many rows in tiles of 128, so that an adapter's factors are read for more rows at once; 64 with
// more than 64 ranks, of which three stages would not fit (8192 rows of one adapter, 4096 to 4096: rank 128 85 us in blocks of
// 32, 63 of 64; rank 256 194 and 144)
static int block_rows_of(int32_t T, int32_t tile, int32_t R) { return tile == 16 ? 16 : tile < 128 || T < 256 ? 32 : R <= 64 ? 128 : 64; }
// Slices of the long dimension: so many that there are about as many workgroups as CUs, all in one round. Down alone in us, with
// 2, 3, 4 and 8 slices: 64 rows of nearly as many adapters (rule: 4) 10.3, 8.1, 7.5, 7.6; 1021 rows in tiles of 16 (3) 9.1,
// 8.6, 8.2, 10.9; 8192 rows of 16 adapters (3) 21.5, 20.0, 25.0, 26.3; of one (4) 21.8, 17.8, 16.7, 22.3.
static int32_t splits_of(int32_t T, int32_t K, int32_t n, int mb) {
  const int blocks = std::max(1, T <= 64 ? T : (T + mb - 1) / mb + std::min(n, T) / 2);    // half a block more for each adapter
  return std::max(1, std::min((K + 255) / 256, 256 / blocks));
}
int32_t adapter_splits(int32_t T, int32_t K, int32_t R) { return splits_of(T, K, 0, block_rows_of(T, 128, R)); }
// rows of a chunk of the factors' gradients (8192 rows of one adapter: 33 us in chunks of 1024, 42 of 512; few rows have
// too few workgroups otherwise)
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
    r.pos = l.plan->pos;
    r.tile_shift = __builtin_ctz((unsigned)l.plan->tile);
  }
  r.n = l.n;
  r.T = l.T;
  return r;
}
// blocks of MB rows that a grouping can have: a tile of a plan has a row at least
static int block_rows_of(const AdapterLaunch& l) { return block_rows_of(l.T, l.ids ? 16 : l.plan->tile, l.R); }
static int block_count(const AdapterLaunch& l, int mb) {
  if (l.ids) return l.T;
  const int64_t tiles = std::min<int64_t>(l.T, l.plan->rows_cap / l.plan->tile);
  return (int)(tiles * (l.plan->tile / mb));
}

static int copy_blocks(int32_t T) { return (T + kCopyRows - 1) / kCopyRows; }
static int up_slabs(int32_t N, int32_t R) { const int c = up_cols(R > 128 ? 8 : 4) * kUpWaves; return (N + c - 1) / c; }
// rows of a block of the up kernel
static int up_rows_of(const AdapterLaunch& l) { return l.ids ? 16 : l.R > 64 ? std::min(l.plan->tile, 64) : l.plan->tile; }
static int grad_chunks(int32_t T, int32_t n) { return T / adapter_grad_rows(T) + std::min(n, T); }

// whether every launch of a forward (K to N) or backward pass has a grid that can be launched
static bool fits(const AdapterLaunch& l, int32_t K, int32_t N, bool grads) {
  if (l.T == 0) return true;
  const int mb = block_rows_of(l);
  if ((int64_t)block_count(l, mb) * splits_of(l.T, K, l.n, mb) > kMaxGrid) return false;
  if ((int64_t)block_count(l, up_rows_of(l)) * up_slabs(N, l.R) + copy_blocks(l.T) > kMaxGrid) return false;
  if (((int64_t)l.T * l.R / 4 + 255) / 256 + copy_blocks(l.T) > kMaxGrid) return false;
  return !grads || (int64_t)((K + kGradCols - 1) / kGradCols + (N + kGradCols - 1) / kGradCols) * grad_chunks(l.T, l.n) <= kMaxGrid;
}

template <int MB, bool TRANS>
static void launch_down(const DownArgs& a, hipStream_t s) {
  const int rp = a.R <= 16 ? 16 : a.R <= 32 ? 32 : a.R <= 64 ? 64 : 128;
  const int x = a.splits > 1 ? a.splits * a.blocks : (a.blocks + 7) / 8 * 8;
  const dim3 grid((unsigned)x, (a.R + rp - 1) / rp), block(64 * kDownWaves);
  if constexpr (MB != 64) {
    if (rp == 16) hipLaunchKernelGGL((adapter_down_kernel<MB, 1, TRANS>), grid, block, 0, s, a);
    else if (rp == 32) hipLaunchKernelGGL((adapter_down_kernel<MB, 2, TRANS>), grid, block, 0, s, a);
    else if (rp == 64) hipLaunchKernelGGL((adapter_down_kernel<MB, 4, TRANS>), grid, block, 0, s, a);
  }
  if constexpr (MB <= 64)
    if (rp == 128) hipLaunchKernelGGL((adapter_down_kernel<MB, 8, TRANS>), grid, block, 0, s, a);
}

template <int MB, bool TRANS>
static void launch_up(const UpArgs& a, dim3 grid, hipStream_t s) {
  const dim3 block(64 * kUpWaves);
  if (a.R <= 32) hipLaunchKernelGGL((adapter_up_kernel<MB, 1, TRANS>), grid, block, 0, s, a);
  else if (a.R <= 64) hipLaunchKernelGGL((adapter_up_kernel<MB, 2, TRANS>), grid, block, 0, s, a);
  else if constexpr (MB <= 64) {
    if (a.R <= 128) hipLaunchKernelGGL((adapter_up_kernel<MB, 4, TRANS>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((adapter_up_kernel<MB, 8, TRANS>), grid, block, 0, s, a);
  }
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
  a.part = part;
  const int mb = block_rows_of(l);
  a.blocks = block_count(l, mb);
  a.splits = splits_of(l.T, K, l.n, mb);
  if (mb == 16) launch_down<16, TRANS>(a, stream);
  else if (mb == 128) launch_down<128, TRANS>(a, stream);
  else if (mb == 64) launch_down<64, TRANS>(a, stream);
  else launch_down<32, TRANS>(a, stream);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

template <bool TRANS>
static int up(const AdapterLaunch& l, const float* part, int32_t splits, const uint16_t* parts, const void* m, const float* scale, int32_t N,
              const void* base, int64_t ld_base, void* out, int64_t ld_out, float* u_out, hipStream_t stream) {
  UpArgs a;
  a.rows = row_args(l);
  a.part = part;
  a.splits = splits;
  a.parts = parts;
  a.m = static_cast<const uint16_t*>(m);
  a.scale = scale;
  a.ranks = l.ranks;
  a.N = N;
  a.R = l.R;
  a.io = {static_cast<const uint16_t*>(base), ld_base, static_cast<uint16_t*>(out), ld_out, N};
  a.u_out = u_out;
  const int mb = up_rows_of(l);
  a.copies = parts || base == out ? 0 : copy_blocks(l.T);   // with parts they are copied already; in place they stay as they are
  const dim3 grid((unsigned)(a.copies + up_slabs(N, l.R) * block_count(l, mb)));
  if (mb == 16) launch_up<16, TRANS>(a, grid, stream);
  else if (mb == 32) launch_up<32, TRANS>(a, grid, stream);
  else if (mb == 64) launch_up<64, TRANS>(a, grid, stream);
  else launch_up<128, TRANS>(a, grid, stream);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

// u (and another array) in parts, and the rows without an adapter copied (unless nothing is written, or in place)
static int make_parts(const AdapterLaunch& l, PartsArgs p, const CopyArgs& io, hipStream_t stream) {
  p.R = l.R;
  p.blocks = (int)((p.n / 4 + 255) / 256);
  p.rows = row_args(l);
  p.io = io;
  const int copies = io.out && io.out != io.base ? copy_blocks(l.T) : 0;
  hipLaunchKernelGGL(adapter_parts_kernel, dim3((unsigned)(p.blocks + copies), p.three[1] ? 2 : 1), dim3(256), 0, stream, p);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int launch_adapter(const AdapterLaunch& l, hipStream_t stream) {
  if (!fits(l, l.K, l.N, false)) return MOE_ERR_UNSUPPORTED;
  const int64_t size = (int64_t)l.T * l.R;
  const int splits = splits_of(l.T, l.K, l.n, block_rows_of(l));
  float* part = splits == 1 && l.v ? l.v : static_cast<float*>(l.ws);
  int rc = down<false>(l, l.x, l.ldx, l.a, nullptr, l.K, part, stream);
  if (rc != MOE_OK) return rc;
  // many rows: v once, in parts, rather than the partial results by every workgroup
  uint16_t* parts = nullptr;
  if (block_rows_of(l) >= 64) {
    parts = reinterpret_cast<uint16_t*>(static_cast<float*>(l.ws) + splits * size);
    const int rc = make_parts(l, {{part, nullptr}, {splits, 0}, {parts, nullptr}, {}, size, splits > 1 ? l.v : nullptr},
                              {static_cast<const uint16_t*>(l.base), l.ld_base, static_cast<uint16_t*>(l.out), l.ld_out, l.N}, stream);
    if (rc != MOE_OK) return rc;
  }
  return up<false>(l, part, splits, parts, l.b, l.scale, l.N, l.base, l.ld_base, l.out, l.ld_out,
                   splits > 1 && !parts ? l.v : nullptr, stream);
}

// dA and dB; dv and v in three bf16 numbers each
static int factor_grads(const AdapterLaunch& l, const AdapterGrads& g, const uint16_t* dv, const uint16_t* v, float* part,
                        hipStream_t stream) {
  GradArgs a{};
  a.ranks = l.ranks;
  a.n = l.n;
  a.T = l.T;
  a.R = l.R;
  a.rows = adapter_grad_rows(l.T);
  a.slots = adapter_grad_slots(l.T);
  a.part = part;
  a.side[0] = {static_cast<const uint16_t*>(l.x), l.ldx, dv, l.K, nullptr, g.da, 0};
  a.side[1] = {static_cast<const uint16_t*>(g.dout), g.ld_dout, v, l.N, l.scale, g.db,
               (int64_t)a.slots * l.R * l.K};
  if (l.T > 0) {
    a.src = l.plan->src;
    a.rows_cap = (int32_t)l.plan->rows_cap;
    a.offsets = l.plan->offsets;
    a.counts = l.plan->counts;
    a.slabs0 = g.da ? (l.K + kGradCols - 1) / kGradCols : 0;
    a.slabs = a.slabs0 + (g.db ? (l.N + kGradCols - 1) / kGradCols : 0);
    const int rp = l.R <= 16 ? 16 : l.R <= 32 ? 32 : 64;
    const dim3 grid((unsigned)(a.slabs * grad_chunks(l.T, l.n)), (l.R + rp - 1) / rp), block(64 * kGradWaves);
    if (rp == 16) hipLaunchKernelGGL(adapter_grad_kernel<1>, grid, block, 0, stream, a);
    else if (rp == 32) hipLaunchKernelGGL(adapter_grad_kernel<2>, grid, block, 0, stream, a);
    else hipLaunchKernelGGL(adapter_grad_kernel<4>, grid, block, 0, stream, a);
    if (hipGetLastError() != hipSuccess) return MOE_ERR_HIP;
  }
  const int64_t most = (int64_t)l.R * std::max(g.da ? l.K : 0, g.db ? l.N : 0);
  hipLaunchKernelGGL(adapter_join_kernel, dim3((unsigned)((most + kJoinValues - 1) / kJoinValues), l.n), dim3(256), 0, stream, a);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int launch_adapter_backward(const AdapterLaunch& l, const AdapterGrads& g, hipStream_t stream) {
  if (!fits(l, l.N, l.K, true)) return MOE_ERR_UNSUPPORTED;
  // dv's partial results, dv in two bf16 numbers, dv and v in three each, partial results of dA and dB
  const int splits = l.T > 0 ? splits_of(l.T, l.N, l.n, block_rows_of(l)) : 1;
  const int64_t size = (int64_t)l.T * l.R;
  float* const part = static_cast<float*>(l.ws);
  uint16_t* const dv2 = reinterpret_cast<uint16_t*>(part + splits * size);
  uint16_t* const dv = dv2 + 2 * size;
  uint16_t* const v = dv + 3 * size;
  const bool rows = g.dx || g.da;
  int rc = MOE_OK;
  if (l.T > 0) {
    if (rows) rc = down<true>(l, g.dout, g.ld_dout, l.b, l.scale, l.N, part, stream);
    if (rc != MOE_OK) return rc;
    rc = make_parts(l, {{part, l.v}, {splits, 1}, {g.dx ? dv2 : nullptr, nullptr}, {g.da ? dv : nullptr, g.db ? v : nullptr}, size, nullptr},
                    {static_cast<const uint16_t*>(g.dx_base), g.ld_base, static_cast<uint16_t*>(g.dx), g.ld_dx, l.K}, stream);
  }
  // the factors' gradients first: dout is in the Infinity Cache yet
  if (rc == MOE_OK && (g.da || g.db)) rc = factor_grads(l, g, dv, v, reinterpret_cast<float*>(v + 3 * size), stream);
  if (rc == MOE_OK && l.T > 0 && g.dx)
    rc = up<true>(l, nullptr, 0, dv2, l.a, nullptr, l.K, g.dx_base, g.ld_base, g.dx, g.ld_dx, nullptr, stream);
  return rc;
}

}  // namespace moe
