// A2 -- dispatch: copy every local (token, k) pair's activation row into its
// pool row and raise the per-tile ready flags.
//
// StreamEP README, "How it works": received pairs land directly in the
// expert-major, tile-padded pool (pool-layout dispatch), and dispatch signals
// each pool tile as it fills (per-tile streaming).
//
// Each token's row is read once (16-byte lanes) and stored to each of its
// local pairs' rows, so x is read T*H*2 bytes once and the pool written once per
// pair. In fp8 mode each 1x128 group (16 lanes x 8 values) is quantised on the
// way: scale = amax/448 in fp32 (1 for an all-zero group), code = e4m3(x /
// scale) with IEEE division, round to nearest even, saturating. In mxfp4 mode
// the activations become MXFP8 (OCP MX): each 1x32 block (4 lanes x 8 values)
// gets the E8M0 scale 2^e, e = floor(log2(amax)) - 8, and codes e4m3(x * 2^-e),
// exact scaling then the same rounding. Scales go to their tile-major words
// (scale_word: one K step of a pool tile reads them as consecutive words). A wave handles
// a run of 64/K tokens; a workgroup's runs are published with a single
// device-scope release (an L2 write-back on this chip, so it is paid per
// workgroup, not per row or per wave); each stored pair then bumps its tile's
// fill counter, and the lane that completes a tile's real rows stores the epoch
// into tile_ready with release ordering.
#include "common.h"
#include "kernels.h"

#include <algorithm>

namespace moe {

struct DispatchArgs {
  const uint16_t* x;
  int32_t T, K, H;
  int32_t tile, tile_shift;
  const int32_t* pos;
  const int32_t* tile_expert;
  const int32_t* offsets;
  const int32_t* counts;
  uint8_t* pool;
  void* pool_s;                // scale words, tile-major (scale_word): fp8 float, mxfp4 4 E8M0 bytes
  int32_t pool_rows;
  uint32_t* tile_fill;
  uint32_t* tile_ready;
  uint32_t* tiles_done;     // count of raised flags: equal to num_tiles once every tile is in
  uint32_t epoch;
  uint32_t* err;
  int32_t tokens_per_wave;  // tokens_per_wave * K <= 64
};

// max over the 4 lanes of a DPP quad (quad_perm [1,0,3,2] then [2,3,0,1])
__device__ inline float quad_max(float v) {
  v = fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0xB1, 0xf, 0xf, false)));
  v = fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x4E, 0xf, 0xf, false)));
  return v;
}

// One token's row: read once, stored to each of its local pairs' rows.
// FMT: 0 bf16 copy, 1 fp8 1x128 groups, 2 MXFP8 1x32 blocks.
template <int CPL, int FMT>
__device__ inline void dispatch_token(const DispatchArgs& a, int t, int p, uint64_t dest, int lane) {
  constexpr bool FP8 = FMT != 0;
  const int H = a.H;
  const int nch = H >> 3;  // 16-byte chunks of 8 bf16 in a row
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x + (int64_t)t * H, (uint32_t)H * 2u);
  const int64_t out_row_bytes = FP8 ? H : (int64_t)H * 2;
  for (int c0 = 0; c0 < nch; c0 += kWave * CPL) {
    u32x4 v[CPL];
#pragma unroll
    for (int i = 0; i < CPL; ++i) v[i] = buf_load16_nt(xr, (uint32_t)(c0 + i * kWave + lane) * 16u);  // x is read once
    if constexpr (FMT == 0) {
      for (int k = 0; k < a.K; ++k) {
        if (!((dest >> k) & 1ull)) continue;
        const int pk = readlane(p, k);
        const __amdgpu_buffer_rsrc_t pr = make_rsrc(a.pool + (int64_t)pk * out_row_bytes, (uint32_t)out_row_bytes);
#pragma unroll
        for (int i = 0; i < CPL; ++i) buf_store16(v[i], pr, (uint32_t)(c0 + i * kWave + lane) * 16u);
      }
    } else if constexpr (FMT == 2) {
      u32x2 q[CPL];
      uint32_t sb[CPL];
#pragma unroll
      for (int i = 0; i < CPL; ++i) {
        float f[8];
        f[0] = bf16_lo(v[i].x); f[1] = bf16_hi(v[i].x);
        f[2] = bf16_lo(v[i].y); f[3] = bf16_hi(v[i].y);
        f[4] = bf16_lo(v[i].z); f[5] = bf16_hi(v[i].z);
        f[6] = bf16_lo(v[i].w); f[7] = bf16_hi(v[i].w);
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(f[j]));
        m = quad_max(m);                       // the 4 lanes of a DPP quad hold one block
        const int e = mx_e4m3_shared_exp(m);
        const float inv = mx_inv_scale(e);
        sb[i] = (uint32_t)(e + 127);
        q[i].x = pack_e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
        q[i].y = pack_e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv);
      }
      const int words = (H + 127) >> 7;
      for (int k = 0; k < a.K; ++k) {
        if (!((dest >> k) & 1ull)) continue;
        const int pk = readlane(p, k);
        const __amdgpu_buffer_rsrc_t pr = make_rsrc(a.pool + (int64_t)pk * out_row_bytes, (uint32_t)out_row_bytes);
        // byte (c >> 2) & 3 of the row's scale word for group c >> 4 (chunk c: 8 elements)
        uint8_t* srow = static_cast<uint8_t*>(a.pool_s) + scale_word(pk, 0, words, a.tile_shift) * 4;
#pragma unroll
        for (int i = 0; i < CPL; ++i) {
          const int c = c0 + i * kWave + lane;
          buf_store8(q[i], pr, (uint32_t)c * 8u);
          if ((lane & 3) == 0 && c < nch)
            srow[((int64_t)(c >> 4) << a.tile_shift) * 4 + ((c >> 2) & 3)] = (uint8_t)sb[i];
        }
      }
    } else {
      u32x2 q[CPL];
      float s[CPL];
#pragma unroll
      for (int i = 0; i < CPL; ++i) {
        float f[8];
        f[0] = bf16_lo(v[i].x); f[1] = bf16_hi(v[i].x);
        f[2] = bf16_lo(v[i].y); f[3] = bf16_hi(v[i].y);
        f[4] = bf16_lo(v[i].z); f[5] = bf16_hi(v[i].z);
        f[6] = bf16_lo(v[i].w); f[7] = bf16_hi(v[i].w);
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(f[j]));
        m = row16_max(m);                      // the 16 lanes of a DPP row hold one group
        const float sc = m > 0.f ? m / 448.0f : 1.0f;
        s[i] = sc;
        q[i].x = pack_e4m3x4(f[0] / sc, f[1] / sc, f[2] / sc, f[3] / sc);
        q[i].y = pack_e4m3x4(f[4] / sc, f[5] / sc, f[6] / sc, f[7] / sc);
      }
      const int groups = H >> 7;
      for (int k = 0; k < a.K; ++k) {
        if (!((dest >> k) & 1ull)) continue;
        const int pk = readlane(p, k);
        const __amdgpu_buffer_rsrc_t pr = make_rsrc(a.pool + (int64_t)pk * out_row_bytes, (uint32_t)out_row_bytes);
        float* srow = static_cast<float*>(a.pool_s) + scale_word(pk, 0, groups, a.tile_shift);
#pragma unroll
        for (int i = 0; i < CPL; ++i) {
          const int c = c0 + i * kWave + lane;
          buf_store8(q[i], pr, (uint32_t)c * 8u);
          if ((lane & 15) == 0 && c < nch) srow[(int64_t)(c >> 4) << a.tile_shift] = s[i];
        }
      }
    }
  }
}

// A wave dispatches a run of `tpw` consecutive tokens (tpw * K <= 64). The block's
// WPB waves then publish together: a barrier (every store of the block has reached
// L2), one device-scope release by wave 0 (an L2 write-back on this chip, which is
// what makes the rows visible to the other XCDs -- paid once per block rather than
// once per wave: a write-back by every wave costs as much as before even when the
// L2 is mostly clean), then wave 0 bumps the fill count of every stored pair's tile
// (relaxed), and the lane whose count completes a tile acquires and stores the
// epoch into tile_ready (release). The host picks the largest WPB (up to 16) that
// still gives every CU a block.
template <int CPL, int FMT, int WPB>
__global__ __launch_bounds__(64 * WPB) void dispatch_kernel(DispatchArgs a) {
  const int lane = lane_id();
  const int w = threadIdx.x >> 6;
  const int tpw = a.tokens_per_wave;
  const int tb = blockIdx.x * WPB * tpw;  // the block's first token
  const int t0 = tb + w * tpw;
  const int ntok = t0 < a.T ? min(tpw, a.T - t0) : 0;
  for (int i = 0; i < ntok; ++i) {
    const int t = t0 + i;
    int p = lane < a.K ? a.pos[(int64_t)t * a.K + lane] : -1;
    if (p >= a.pool_rows) {
      record_error(a.err, MOE_ERR_INVALID);
      p = -1;
    }
    const uint64_t dest = ballot(p >= 0);
    if (dest != 0) dispatch_token<CPL, FMT>(a, t, p, dest, lane);
  }

  __syncthreads();
  if (w != 0) return;
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
  const int npairs = (min(a.T, tb + WPB * tpw) - tb) * a.K;
  for (int q = lane; q < npairs; q += 64) {
    int p = a.pos[(int64_t)tb * a.K + q];
    if (p >= a.pool_rows) p = -1;
    if (p >= 0) {
      const int ti = p >> a.tile_shift;
      const uint32_t old = __hip_atomic_fetch_add(&a.tile_fill[ti], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      const int e = a.tile_expert[ti];
      const int real = min(a.tile, a.offsets[e] + a.counts[e] - (ti << a.tile_shift));
      if ((int)old + 1 == real) {
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
        __hip_atomic_store(&a.tile_ready[ti], a.epoch, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_fetch_add(a.tiles_done, 1u, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
  }
}

template <int FMT, int WPB>
static void launch_cpl(int cpl, dim3 grid, hipStream_t s, const DispatchArgs& a) {
  switch (cpl) {
    case 1: hipLaunchKernelGGL((dispatch_kernel<1, FMT, WPB>), grid, dim3(64 * WPB), 0, s, a); break;
    case 2: hipLaunchKernelGGL((dispatch_kernel<2, FMT, WPB>), grid, dim3(64 * WPB), 0, s, a); break;
    case 4: hipLaunchKernelGGL((dispatch_kernel<4, FMT, WPB>), grid, dim3(64 * WPB), 0, s, a); break;
    default: hipLaunchKernelGGL((dispatch_kernel<8, FMT, WPB>), grid, dim3(64 * WPB), 0, s, a); break;
  }
}

template <int FMT>
static void launch_wpb(int wpb, int cpl, int waves, hipStream_t s, const DispatchArgs& a) {
  const dim3 grid((waves + wpb - 1) / wpb);
  switch (wpb) {
    case 1: launch_cpl<FMT, 1>(cpl, grid, s, a); break;
    case 2: launch_cpl<FMT, 2>(cpl, grid, s, a); break;
    case 4: launch_cpl<FMT, 4>(cpl, grid, s, a); break;
    case 8: launch_cpl<FMT, 8>(cpl, grid, s, a); break;
    default: launch_cpl<FMT, 16>(cpl, grid, s, a); break;
  }
}

int launch_dispatch(const void* x, int32_t H, int32_t dtype, const moe_plan_t& p, int32_t pool_rows,
                    void* pool, void* pool_s, uint32_t epoch, const WsLayout& L, char* ws,
                    hipStream_t stream) {
  DispatchArgs a;
  a.x = static_cast<const uint16_t*>(x);
  a.T = p.T;
  a.K = p.K;
  a.H = H;
  a.tile = p.tile;
  a.tile_shift = __builtin_ctz((unsigned)p.tile);
  a.pos = p.pos;
  a.tile_expert = p.tile_expert;
  a.offsets = p.offsets;
  a.counts = p.counts;
  a.pool = static_cast<uint8_t*>(pool);
  a.pool_s = pool_s;
  a.pool_rows = pool_rows;
  a.tile_fill = reinterpret_cast<uint32_t*>(ws + L.fill);
  a.tile_ready = p.tile_ready;
  a.tiles_done = reinterpret_cast<uint32_t*>(ws + L.tiles_done);
  a.epoch = epoch;
  a.err = reinterpret_cast<uint32_t*>(ws + L.err);
  const int nch = H / 8;
  const int cpl = nch <= 64 ? 1 : nch <= 128 ? 2 : nch <= 256 ? 4 : 8;
  const int cus = std::max(1, device_cu_count());
  // tokens per wave: up to 64/K (one pos load per wave and token run), fewer when that
  // leaves under two waves per CU -- a wave walks its tokens one after another, so a
  // small batch wants one or two tokens per wave
  a.tokens_per_wave = std::max(1, std::min(64 / p.K, p.T / (2 * cus)));
  const int waves = (p.T + a.tokens_per_wave - 1) / a.tokens_per_wave;
  // waves per block: the largest power of two up to 16 that leaves a block per CU
  int wpb = 1;
  while (wpb < 16 && waves / (2 * wpb) >= cus) wpb *= 2;
  if (dtype == MOE_FP8_E4M3_G128)
    launch_wpb<1>(wpb, cpl, waves, stream, a);
  else if (dtype == MOE_MXFP4)
    launch_wpb<2>(wpb, cpl, waves, stream, a);
  else
    launch_wpb<0>(wpb, cpl, waves, stream, a);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

// ---------------------------------------------------------------------------------------
// rows that are codes with scale words already
// ---------------------------------------------------------------------------------------
// Both formats move H bytes and a 4-byte word for 128 columns a row, so the same kernels serve them. The
// first `scale_blocks` workgroups fill the scale words tile by tile, consecutive words at a time (stored
// beside the rows, a word of each 128 columns lands alone in its line of the tile-major array: 20 of 92
// us at 8192 x 4096, top-8). The others have the codes, by token or by tile:
//   by token, as above: a wave reads a row once and stores it to each of its pool rows. Few steps
//     one after another, so the faster one for small batches; but the pool's rows are then written
//     all over it (8192 x 4096, top-8: 79 us, 3.9 TB/s).
//   by tile: a workgroup has every so many tiles, so the pool is written nearly in order, and one of up
//     to 8 slices of the columns. Workgroups go to the 8 XCDs in turn, so an XCD reads one slice of x
//     alone (4 MB at 8192 x 4096, its L2's size) and a row's K readings come from there; the pool's
//     stores pass the caches by to keep it so (67 us, 4.6 TB/s; with ordinary stores a fifth more, with
//     whole rows, each read from memory K times, 122; 4 slices 86, two tiles' loads at once 70).
struct DispatchQArgs {
  DispatchArgs d;               // x: the codes
  const uint32_t* x_s;          // [T][ceil(H / 128)]
  const int32_t* src;
  const int32_t* num_tiles;
  int32_t max_tiles;            // that pool and plan have room for
  int32_t scale_blocks;
  int32_t slices;               // by tile: of the columns
  int32_t slice_blocks;         // and workgroups of a slice
};
// Few, large workgroups, since each pays an L2 write-back to publish: 16 waves (4 at 8192 x 4096 by token:
// 125 us, 16: 89 on that machine); 16 workgroups for the scales (8: 112 us; more: no gain), and by tile
// as many in all as there are CUs. So the flags rise at the end, nearly all at once. A workgroup that publishes as it goes pays more than
// an FFN on another stream gains: plan and dispatch of 8192 x 4096 fp8 rows 85 us at the end, 117 every 8 tiles, 156 every 4; the
// layer on two streams 1872, 1908 and 1945 us (1926 from bf16 rows), on one 1643.
constexpr int kQWaves = 16;
constexpr int kQScaleBlocks = 16;
constexpr int kQWords = 8;   // scale words of a row in an item
constexpr int kQSlices = 8;
constexpr int kQTileTokens = 4096;
constexpr int kQSliceChunks = 16;   // 256 bytes, at least

// a tile's real rows
__device__ inline int tile_rows(const DispatchArgs& a, int ti) {
  const int e = a.tile_expert[ti];
  return min(a.tile, a.offsets[e] + a.counts[e] - (ti << a.tile_shift));
}
// one more of the `all` parts of tile ti is in
__device__ inline void count_tile(const DispatchArgs& a, int ti, int all) {
  const uint32_t old = __hip_atomic_fetch_add(&a.tile_fill[ti], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if ((int)old + 1 == all) {
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    __hip_atomic_store(&a.tile_ready[ti], a.epoch, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_fetch_add(a.tiles_done, 1u, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_AGENT);
  }
}
// the token of pool row `row`, -1: none
__device__ inline int row_token(const DispatchQArgs& b, int64_t row) {
  const int q = b.src[row];
  return q < 0 || q >= (int64_t)b.d.T * b.d.K ? -1 : (int)((uint32_t)q / (uint32_t)b.d.K);
}

// The scale words, by the first workgroups. An item is eight of a tile's words a row: read along the
// rows, written along the tile. Each counts as one part of its tile, beside what `parts(tile)` says.
template <typename PARTS>
__device__ inline void dispatch_scales(const DispatchQArgs& b, int tiles, PARTS parts) {
  const DispatchArgs& a = b.d;
  const int lane = lane_id();
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int words = (a.H + 127) >> 7;
  const int per_tile = (words + kQWords - 1) / kQWords;
  __shared__ uint32_t s_word[kQWaves][128][kQWords + 1];
  __shared__ int s_token[kQWaves][128];
  const int items = tiles * per_tile;
  const int first = (int)blockIdx.x * kQWaves, step = b.scale_blocks * kQWaves;
  for (int it = first + w; it < items; it += step) {
    const int ti = it / per_tile;
    const int g0 = (it - ti * per_tile) * kQWords;
    const int64_t row0 = (int64_t)ti << a.tile_shift;
    for (int r = lane; r < a.tile; r += kWave) s_token[w][r] = row_token(b, row0 + r);
    wave_sync();
    // two lanes a row, four words each
    const int g = g0 + 4 * (lane & 1);
    u32x4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = (lane >> 1) + 32 * j;
      const int t = r < a.tile ? s_token[w][r] : -1;
      v[j] = u32x4{0u, 0u, 0u, 0u};
      if (t >= 0) {
        const uint32_t* from = b.x_s + (int64_t)t * words;
        if (g + 4 <= words) {
          __builtin_memcpy(&v[j], from + g, 16);
        } else {
          for (int k = 0; k < 4; ++k)
            if (g + k < words) v[j][k] = from[g + k];
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = (lane >> 1) + 32 * j;
      if (r < a.tile)
        for (int k = 0; k < 4; ++k) s_word[w][r][4 * (lane & 1) + k] = v[j][k];
    }
    wave_sync();
    uint32_t* to = static_cast<uint32_t*>(a.pool_s) + row0 * words;
    for (int r = lane; r < a.tile; r += kWave) {
      if (s_token[w][r] < 0) continue;   // padding rows' words are left alone
#pragma unroll
      for (int k = 0; k < kQWords; ++k)
        if (g0 + k < words) to[((int64_t)(g0 + k) << a.tile_shift) + r] = s_word[w][r][k];
    }
    wave_sync();
  }
  __syncthreads();
  if (w != 0) return;
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
  // this workgroup's items: kQWaves at `first`, then every `step`
  for (int n = lane;; n += 64) {
    const int it = first + n / kQWaves * step + n % kQWaves;
    if (first + n / kQWaves * step >= items) break;
    if (it < items) count_tile(a, it / per_tile, per_tile + parts(it / per_tile));
  }
}

template <int CPL>
__global__ __launch_bounds__(64 * kQWaves) void dispatch_quantized_kernel(DispatchQArgs b) {
  const DispatchArgs& a = b.d;
  const int lane = lane_id();
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int per_tile = (((a.H + 127) >> 7) + kQWords - 1) / kQWords;
  if ((int)blockIdx.x < b.scale_blocks) {
    dispatch_scales(b, min(b.num_tiles[0], b.max_tiles), [&](int ti) { return tile_rows(a, ti); });
    return;
  }

  const int tb = ((int)blockIdx.x - b.scale_blocks) * kQWaves;   // the block's first token
  const int t = tb + w;
  const int nch = a.H >> 4;   // 16-byte chunks of 16 codes
  if (t < a.T) {
    int p = lane < a.K ? a.pos[(int64_t)t * a.K + lane] : -1;
    if (p >= a.pool_rows) {
      record_error(a.err, MOE_ERR_INVALID);
      p = -1;
    }
    const uint64_t dest = ballot(p >= 0);
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(reinterpret_cast<const uint8_t*>(a.x) + (int64_t)t * a.H, (uint32_t)a.H);
    for (int c0 = 0; dest != 0 && c0 < nch; c0 += kWave * CPL) {
      u32x4 v[CPL];
#pragma unroll
      for (int j = 0; j < CPL; ++j) v[j] = buf_load16_nt(xr, (uint32_t)(c0 + j * kWave + lane) * 16u);
      for (uint64_t m = dest; m != 0; m &= m - 1) {
        const int pk = readlane(p, __builtin_ctzll(m));
        const __amdgpu_buffer_rsrc_t pr = make_rsrc(a.pool + (int64_t)pk * a.H, (uint32_t)a.H);
#pragma unroll
        for (int j = 0; j < CPL; ++j) buf_store16(v[j], pr, (uint32_t)(c0 + j * kWave + lane) * 16u);
      }
    }
  }
  // published as above, once a workgroup
  __syncthreads();
  if (w != 0) return;
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
  const int npairs = (min(a.T, tb + kQWaves) - tb) * a.K;
  for (int q = lane; q < npairs; q += 64) {
    const int p = a.pos[(int64_t)tb * a.K + q];
    if (p >= 0 && p < a.pool_rows) count_tile(a, p >> a.tile_shift, per_tile + tile_rows(a, p >> a.tile_shift));
  }
}

__global__ __launch_bounds__(64 * kQWaves) void dispatch_quantized_tiles_kernel(DispatchQArgs b) {
  const DispatchArgs& a = b.d;
  const int lane = lane_id();
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int all = b.num_tiles[0], tiles = min(all, b.max_tiles);
  if ((int)blockIdx.x < b.scale_blocks) {
    dispatch_scales(b, tiles, [&](int) { return b.slices; });
    return;
  }
  if (all > tiles && threadIdx.x == 0) record_error(a.err, MOE_ERR_INVALID);
  const int n = (int)blockIdx.x - b.scale_blocks;
  const int slice = n % b.slices, wg = n / b.slices;
  const int nch = a.H >> 4;   // 16-byte chunks of 16 codes
  const int first = nch * slice / b.slices, cn = nch * (slice + 1) / b.slices - first;
  constexpr int kRows = 128 / kQWaves;                 // a wave's rows of a tile, at most
  const int rows = a.tile / kQWaves;                   // 1 .. kRows
  const int rpi = cn >= kWave ? 1 : kWave / cn;        // rows of an instruction, if a slice's row fits
  const int ro = cn >= kWave ? 0 : lane / cn, co = cn >= kWave ? lane : lane - ro * cn;
  // lane r: the token of the wave's row r
  const auto tokens = [&](int ti) {
    return ti < tiles ? row_token(b, ((int64_t)ti << a.tile_shift) + w * rows + min(lane, rows - 1)) : -1;
  };
  int next = tokens(wg);
  for (int ti = wg; ti < tiles; ti += b.slice_blocks) {
    const int tok = next;
    next = tokens(ti + b.slice_blocks);
    const int64_t row0 = ((int64_t)ti << a.tile_shift) + w * rows;
    for (int c0 = 0; c0 < cn; c0 += kWave) {
      const int c = c0 + co;
      const int64_t col = (int64_t)(first + min(c, cn - 1)) * 16;
      u32x4 v[kRows];
      int t[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        if (i * rpi >= rows) break;
        const int r = i * rpi + ro;
        t[i] = __shfl(tok, min(r, rows - 1), 64);
        if (c >= cn || ro >= rpi || r >= rows) t[i] = -1;
        // rows without a token read token 0's: all loads are in flight together
        v[i] = *reinterpret_cast<const u32x4*>(reinterpret_cast<const uint8_t*>(a.x) + (int64_t)max(t[i], 0) * a.H + col);
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i)
        if (i * rpi < rows && t[i] >= 0)
          __builtin_nontemporal_store(v[i], reinterpret_cast<u32x4*>(a.pool + (row0 + i * rpi + ro) * a.H + col));
    }
  }
  __syncthreads();
  if (w != 0) return;
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
  const int per_tile = (((a.H + 127) >> 7) + kQWords - 1) / kQWords;
  for (int ti = wg + lane * b.slice_blocks; ti < tiles; ti += kWave * b.slice_blocks) count_tile(a, ti, per_tile + b.slices);
}

int launch_dispatch_quantized(const void* q, const void* q_s, int32_t H, const moe_plan_t& p, int32_t pool_rows,
                              void* pool, void* pool_s, uint32_t epoch, const WsLayout& L, char* ws,
                              hipStream_t stream) {
  DispatchQArgs b;
  DispatchArgs& a = b.d;
  a.x = static_cast<const uint16_t*>(q);
  a.T = p.T;
  a.K = p.K;
  a.H = H;
  a.tile = p.tile;
  a.tile_shift = __builtin_ctz((unsigned)p.tile);
  a.pos = p.pos;
  a.tile_expert = p.tile_expert;
  a.offsets = p.offsets;
  a.counts = p.counts;
  a.pool = static_cast<uint8_t*>(pool);
  a.pool_s = pool_s;
  a.pool_rows = pool_rows;
  a.tile_fill = reinterpret_cast<uint32_t*>(ws + L.fill);
  a.tile_ready = p.tile_ready;
  a.tiles_done = reinterpret_cast<uint32_t*>(ws + L.tiles_done);
  a.epoch = epoch;
  a.err = reinterpret_cast<uint32_t*>(ws + L.err);
  b.x_s = static_cast<const uint32_t*>(q_s);
  b.src = p.src;
  b.num_tiles = p.num_tiles;
  b.max_tiles = std::min(pool_rows, p.rows_cap) / p.tile;
  const int cus = std::max(1, device_cu_count());
  b.scale_blocks = std::min(p.rows_cap / p.tile, kQScaleBlocks);
  const int nch = H / 16;
  const dim3 block(64 * kQWaves);
  // By tile from 4096 tokens on, and from 2048 pairs on where the experts are few, whose tiles' counters the
  // tokens of all workgroups share. By token / by tile, us: H 4096, 128 experts, top-8 27.6 / 30.2 (2048 tokens), 47 / 39
  // (4096), 79 / 67 (8192); 32 of 256 experts at H 7168 16.1 / 16.6 (2560), 25 / 24 (4096), 81 / 51 (16384); 8
  // experts, top-8 20.9 / 17.6 (512), 55 / 28 (2048)
  if (p.T >= kQTileTokens || (p.E_local <= 16 && (int64_t)p.T * p.K > 2048)) {
    b.slices = kQSlices;
    while (b.slices > 1 && nch / b.slices < kQSliceChunks) b.slices /= 2;
    b.slice_blocks = std::max(1, (cus - b.scale_blocks) / b.slices);
    hipLaunchKernelGGL(dispatch_quantized_tiles_kernel, dim3(b.scale_blocks + b.slices * b.slice_blocks), block, 0, stream, b);
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
  }
  const dim3 grid((unsigned)(b.scale_blocks + (p.T + kQWaves - 1) / kQWaves));   // a token a wave
  if (nch <= 64) hipLaunchKernelGGL((dispatch_quantized_kernel<1>), grid, block, 0, stream, b);
  else if (nch <= 128) hipLaunchKernelGGL((dispatch_quantized_kernel<2>), grid, block, 0, stream, b);
  else hipLaunchKernelGGL((dispatch_quantized_kernel<4>), grid, block, 0, stream, b);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe
