// The expert FFN of a few tokens with MXFP4 weights: matrix-vector products, straight from
// the routing.
//
//   h[t,k] = mxfp8(silu(W1[e] gate . x[t]) * (W1[e] up . x[t])),
//   out[t] = sum_k topk_weights[t,k] * (W2[e] . h[t,k]).
//
// Every reached expert's 3 * H * I * (1/2 + 1/32) bytes are read once and hardly anything
// else moves: the memory's rate bounds it. The products run on the matrix cores all the same, 16
// weight rows by 16 token columns, in bf16: a 16 x 128 weight tile of the layer's load-time layout is one
// 16-byte load a lane, and up to 16 tokens cost what one does.
//
// The pooled path's plan, dispatch and combine launches are not needed: with at most 64 * 16
// pairs each workgroup finds the reached experts itself (a bitmap in LDS), the h kernel's
// workgroup (slot, block of 32 columns of h) takes the slot-th of them, and the out kernel's
// workgroup sums all experts' shares of its 16 columns in LDS, each wave for itself and then
// the waves in order, so out needs no second pass and no atomics.
//
// H 4096, I 1536, 128 experts, top-8 (h and out kernel, MXFP8 rows): one token 14 + 9 us (80 MB),
// 64 tokens 124 + 79 us (1.27 GB: 6.8 and 5.4 TB/s). The pooled path takes 110 and 379 us.
#include "common.h"
#include "kernels.h"

#include <algorithm>
#include <type_traits>

namespace moe {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kDecodeTokens = 64;                     // at most
constexpr int kDecodePairs = kDecodeTokens * 16;

struct DecodeArgs {
  const uint8_t* x;
  const uint8_t* x_s;
  int32_t T, H, I, K, begin, E;
  const int32_t* idx;
  const float* weights;
  const uint8_t* w1;
  const uint8_t* w1_s;
  const uint8_t* w2;
  const uint8_t* w2_s;
  uint8_t* h;     // [T * K][I] codes
  uint8_t* h_s;   // [T * K][I / 32] E8M0 bytes
  uint16_t* out;
};

__device__ inline uint32_t buf_load1(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(r, off, 0, 0);
}
constexpr uint32_t kNowhere = 0x7fffff00u;   // past every buffer: reads 0

// 16 weight rows times 16 token columns over 128 K: lane (l16, lhi) has of row l16 the 32 e2m1 codes K = 32 lhi .. + 32, of
// column l16 the 32 e4m3 codes of the same K, and both sides' E8M0 scale of that block. The products are formed in
// bf16, which holds codes with their scales exactly (values from 2^-133 to 2^128): four instructions of 32 K, the j-th of
// every lane's codes 8 j .. + 8, with exact products and fp32 sums. One v_mfma_scale_f32_16x16x128_f8f6f4 takes
// the codes as they are, but it lines its 128 products up on the largest and drops what is too small beside it, up to 2e-4 of
// the sum of their magnitudes. h's sums decide between neighbouring e4m3 codes, and 4 in 10000 went to the wrong one; out's
// can be small beside their terms, and then that is far more than out's rounding to bf16. It costs 24 conversions a
// tile for h and 32 for out (the call, one token 21.2 -> 23.1 us, 13 tokens at H 7168 48 -> 52, 64 tokens 194 -> 199).
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
struct Bf16Block {
  bf16x8 v[4];
};
__device__ inline float e8m0_scale(uint32_t byte) { return __builtin_bit_cast(float, byte << 23); }
__device__ inline bf16x8 join(bf16x2 a, bf16x2 b, bf16x2 c, bf16x2 d) {
  return __builtin_shufflevector(__builtin_shufflevector(a, b, 0, 1, 2, 3), __builtin_shufflevector(c, d, 0, 1, 2, 3), 0, 1, 2, 3, 4, 5, 6, 7);
}
__device__ inline Bf16Block from_e2m1(u32x4 codes, float s) {
  Bf16Block r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t c = codes[j];
    r.v[j] = join(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1),
                  __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3));
  }
  return r;
}
__device__ inline Bf16Block from_e4m3(u32x4 lo, u32x4 hi, float s) {
  Bf16Block r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t c = j < 2 ? lo[2 * j] : hi[2 * j - 4], d = j < 2 ? lo[2 * j + 1] : hi[2 * j - 3];
    r.v[j] = join(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, s, false), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, s, true),
                  __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, s, false), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, s, true));
  }
  return r;
}

// ---------------------------------------------------------------------------------------
// the reached experts: local ids of all pairs and a bit for each reached one
// ---------------------------------------------------------------------------------------
struct Reached {
  int16_t id[kDecodePairs];   // local expert of a pair, or -1
  uint32_t bits[32];
};

template <int THREADS>
__device__ inline void find_reached(const DecodeArgs& a, Reached& r) {
  if (threadIdx.x < 32) r.bits[threadIdx.x] = 0;
  __syncthreads();
  for (int q = threadIdx.x; q < a.T * a.K; q += THREADS) {
    const int64_t e = (int64_t)a.idx[q] - a.begin;
    const bool local = e >= 0 && e < a.E;
    r.id[q] = local ? (int16_t)e : (int16_t)-1;
    if (local) atomicOr(&r.bits[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
}

// the slot-th reached expert (ascending), or -1; by every wave for itself
__device__ inline int reached_expert(const Reached& r, int slot) {
  const int lane = lane_id();
  const uint32_t word = lane < 32 ? r.bits[lane] : 0u;
  const int n = __popc(word);
  const int upto = wave_inclusive_scan(n);
  const uint64_t after = ballot(upto > slot);
  if (after == 0) return -1;
  const int at = __builtin_ctzll(after);
  uint32_t w = (uint32_t)readlane((int)word, at);
  for (int i = slot - (readlane(upto, at) - readlane(n, at)); i > 0; --i) w &= w - 1;
  return at * 32 + __builtin_ctz(w);
}

// All reached experts, ascending, into `list`: thread e has experts e, e + THREADS, ...
// Returns their number; a barrier follows.
template <int THREADS>
__device__ inline int list_reached(const Reached& r, int16_t* list) {
  const int lane = lane_id();
  const int n = lane < 32 ? __popc(r.bits[lane]) : 0;
  const int upto = wave_inclusive_scan(n);
  for (int e = threadIdx.x; e < 1024; e += THREADS) {
    const uint32_t word = r.bits[e >> 5];
    const int before = __shfl(upto - n, e >> 5, 64) + __popc(word & ((1u << (e & 31)) - 1u));
    if ((word >> (e & 31)) & 1u) list[before] = (int16_t)e;
  }
  return readlane(upto, 63);
}

// ---------------------------------------------------------------------------------------
// bf16 rows to MXFP8: a lane has 8 values, four lanes a block
// ---------------------------------------------------------------------------------------
__global__ __launch_bounds__(256) void decode_quantise_kernel(const uint16_t* x, int32_t chunks, uint8_t* q, uint8_t* q_s) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= chunks) return;                            // chunks % 16 == 0: whole blocks
  const u32x4 v = reinterpret_cast<const u32x4*>(x)[c];
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(v[i]);
    f[2 * i + 1] = bf16_hi(v[i]);
  }
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __builtin_bit_cast(uint32_t, f[j]) & 0x7fffffffu);
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xf, 0xf, false));
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xf, 0xf, false));
  const bool bad = m >= 0x7f800000u;                  // NaN or infinity: the block is NaN
  const int e = mx_e4m3_shared_exp(__builtin_bit_cast(float, m));
  const float inv = mx_inv_scale(e);
  u32x2 o = {pack_e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
             pack_e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv)};
  if (bad) o = u32x2{0u, 0u};
  reinterpret_cast<u32x2*>(q)[c] = o;
  if ((threadIdx.x & 3) == 0) q_s[c >> 2] = (uint8_t)(bad ? 255 : e + 127);
}

// ---------------------------------------------------------------------------------------
// h: grid (I / 32 column blocks, slots); the waves share K. An expert of more than 16 C tokens takes
// them 16 C at a time and reads its weights again (from the caches) for every 16 C.
// ---------------------------------------------------------------------------------------
template <int NW, int U, int C>
__global__ __launch_bounds__(64 * NW, C == 2 ? 3 : 1) void decode_h_kernel(DecodeArgs a) {
  __shared__ Reached reached;
  __shared__ int16_t s_q[kDecodeTokens];              // the expert's pairs, one of each of its tokens
  __shared__ f32x4 s_red[NW][4][64];
  const int lane = lane_id(), l16 = lane & 15, lhi = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  find_reached<64 * NW>(a, reached);
  const int e = reached_expert(reached, blockIdx.y);
  if (e < 0) return;                                  // the same in every wave
  // lane t: token t's first pair with this expert (h of a later one would be the same)
  int q = -1;
  if (lane < a.T)
    for (int k = a.K - 1; k >= 0; --k)
      if (reached.id[lane * a.K + k] == e) q = lane * a.K + k;
  const uint64_t has = ballot(q >= 0);
  const int n = __popcll(has);
  if (wave == 0 && q >= 0) s_q[mask_rank(has)] = (int16_t)q;
  __syncthreads();

  const int KB = a.H >> 7;
  const int nb = blockIdx.x;
  const uint32_t tiles = (uint32_t)KB * 1024u, tscales = (uint32_t)KB * 64u;
  const uint8_t* w = a.w1 + (int64_t)e * a.I * a.H;
  const uint8_t* ws = a.w1_s + (int64_t)e * a.I * (a.H >> 4);
  __amdgpu_buffer_rsrc_t wr[4], sr[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {                       // gate, gate, up, up
    const int rb = nb * 2 + (i & 1) + (i >> 1) * (a.I >> 4);
    wr[i] = make_rsrc(w + (int64_t)rb * tiles, tiles);
    sr[i] = make_rsrc(ws + (int64_t)rb * tscales, tscales);
  }
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x, (uint32_t)a.T * (uint32_t)a.H);
  const __amdgpu_buffer_rsrc_t xsr = make_rsrc(a.x_s, (uint32_t)a.T * (uint32_t)KB * 4u);

  // C times 16 tokens from c0 on
  const auto pass = [&](auto columns, int c0) {
    constexpr int N = columns;
    // tokens past the last: past the buffers, zeros
    uint32_t xo[N], xso[N];
    bool on[N];
    f32x4 acc[N][4];
#pragma unroll
    for (int g = 0; g < N; ++g) {
      const int c = c0 + g * 16 + l16;
      on[g] = c < n;
      const uint32_t t = on[g] ? (uint32_t)s_q[c] / (uint32_t)a.K : 0u;
      xo[g] = t * (uint32_t)a.H + (uint32_t)lhi * 32u;
      xso[g] = t * (uint32_t)KB * 4u + (uint32_t)lhi;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[g][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    // K blocks wave, wave + NW, ...: at every moment the waves read neighbouring tiles
    for (int kb0 = wave; kb0 < KB; kb0 += NW * U) {
      u32x4 wt[U][4], b0[U][N], b1[U][N];
      uint32_t wsc[U][4], sb[U][N];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t kb = (uint32_t)(kb0 + u * NW);   // past KB: weights past the buffer, zeros
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          wt[u][i] = buf_load16_nt(wr[i], kb * 1024u + (uint32_t)lane * 16u);
          wsc[u][i] = buf_load1(sr[i], kb * 64u + (uint32_t)lane);
        }
#pragma unroll
        for (int g = 0; g < N; ++g) {
          const bool in = kb < (uint32_t)KB && on[g];
          b0[u][g] = buf_load16(xr, in ? xo[g] + kb * 128u : kNowhere);
          b1[u][g] = buf_load16(xr, in ? xo[g] + kb * 128u + 16u : kNowhere);
          sb[u][g] = buf_load1(xsr, in ? xso[g] + kb * 4u : kNowhere);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
      {
        Bf16Block b[N];
#pragma unroll
        for (int g = 0; g < N; ++g) b[g] = from_e4m3(b0[u][g], b1[u][g], e8m0_scale(sb[u][g]));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const Bf16Block w = from_e2m1(wt[u][i], e8m0_scale(wsc[u][i]));
#pragma unroll
          for (int g = 0; g < N; ++g)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              acc[g][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[j], b[g].v[j], acc[g][i], 0, 0, 0);
        }
      }
    }

    // the waves' sums, then SwiGLU and the MXFP8 of 32 columns: lane (l16, lhi) has token column
    // l16 and columns 4 lhi .. + 4 of both tiles of 16. expf, since __expf is off by |gate| 2^-24 (one token 23.0 -> 23.3 us)
#pragma unroll
    for (int g = 0; g < N; ++g) {
      if (c0 + g > 0) __syncthreads();                // wave 0 has read the sums before
#pragma unroll
      for (int i = 0; i < 4; ++i) s_red[wave][i][lane] = acc[g][i];
      __syncthreads();
      if (wave != 0) continue;
      f32x4 s[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[i] = s_red[0][i][lane];
#pragma unroll
        for (int v = 1; v < NW; ++v) s[i] += s_red[v][i][lane];
      }
      float h[8];
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float gate = s[j >> 2][j & 3], up = s[2 + (j >> 2)][j & 3];
        h[j] = gate / (1.0f + expf(-gate)) * up;
        m = max(m, __builtin_bit_cast(uint32_t, h[j]) & 0x7fffffffu);
      }
      m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
      m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
      const bool bad = m >= 0x7f800000u;
      const int ex = mx_e4m3_shared_exp(__builtin_bit_cast(float, m));
      const float inv = mx_inv_scale(ex);
      if (on[g]) {
        const int64_t p = s_q[c0 + g * 16 + l16];
        uint32_t* d = reinterpret_cast<uint32_t*>(a.h + p * a.I + nb * 32 + lhi * 4);
        d[0] = bad ? 0u : pack_e4m3x4(h[0] * inv, h[1] * inv, h[2] * inv, h[3] * inv);
        d[4] = bad ? 0u : pack_e4m3x4(h[4] * inv, h[5] * inv, h[6] * inv, h[7] * inv);
        if (lhi == 0) a.h_s[p * (a.I >> 5) + nb] = (uint8_t)(bad ? 255 : ex + 127);
      }
    }
  };
  for (int c0 = 0; c0 < n; c0 += 16 * C)
    if (C > 1 && n - c0 > 16) pass(std::integral_constant<int, C>(), c0);
    else pass(std::integral_constant<int, 1>(), c0);
}

// A token's experts in a lane's registers, two in one, so that finding its pair with an expert reads no memory where it
// has none. (Sixteen and their weights leave too few registers for the products: 10 spilled, 64 tokens 215 us, so 199.)
struct TokenPairs {
  uint32_t id[8];
  __device__ void load(const DecodeArgs& a, const Reached& r, int t) {
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const bool on = k < a.K && t < a.T;
      const uint32_t v = on ? (uint16_t)r.id[t * a.K + k] : 0xffffu;
      id[k >> 1] = k & 1 ? id[k >> 1] | v << 16 : v;
    }
  }
  // the places of expert e, a bit each
  __device__ uint32_t find(int e) const {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 16; ++k) m |= ((k & 1 ? id[k >> 1] >> 16 : id[k >> 1] & 0xffffu) == (uint32_t)e ? 1u : 0u) << k;
    return m;
  }
};

// ---------------------------------------------------------------------------------------
// out: a workgroup has 16 columns of out for all tokens; its waves share the (expert, K block)
// pairs evenly. An expert's tokens are gathered into the columns of the product, eight at a time, or
// sixteen where it has more (8 experts with 64 tokens each at H 5120, eight at a time: 76 us, so 51),
// and the columns' sums go to their tokens' sums in the wave's part of LDS.
//
// A weight tile is one load, and what belongs to it must not cost several: the address unit
// takes as long for a scattered load of 16 bytes a lane as for a weight tile, and with two of
// those for h, one for its scale and one for the weight's it was busy 77% of the time (64 tokens:
// 96 us, products and all). So h comes in whole lines, several K blocks a load, and goes to the lanes that want it by way
// of LDS, and the scales of four K blocks come as words (70 us then; 80 with the latter alone).
// ---------------------------------------------------------------------------------------
// 4 waves a SIMD: two workgroups of 8 waves a CU, or one of 16 (13 tokens at H 7168: 26 us; 35 with 2)
template <int NW, int TOK>
__global__ __launch_bounds__(64 * NW, 4) void decode_out_kernel(DecodeArgs a) {
  constexpr int U = 4;                                // K blocks at a time
  constexpr int COLS = 8;
  __shared__ Reached reached;
  __shared__ float s_w[TOK * 16];
  __shared__ int16_t s_expert[TOK * 16];              // the reached experts
  __shared__ f32x4 s_sum[NW][4][TOK];                 // [wave][columns 4 lhi ..][token]
  __shared__ int16_t s_pair[NW][TOK];
  __shared__ float s_weight[NW][TOK];
  __shared__ u32x4 s_h[NW][U * COLS][8];              // a column's 128 codes, 16-byte chunk k at k ^ column % 8
  __shared__ uint32_t s_scale[NW][U * 16];            // weight scales, 64 bytes a tile
  const int lane = lane_id(), l16 = lane & 15, lhi = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int q = threadIdx.x; q < a.T * a.K; q += 64 * NW) s_w[q] = a.weights[q];
  find_reached<64 * NW>(a, reached);
  const int slots = list_reached<64 * NW>(reached, s_expert);
  TokenPairs pairs;                                   // lane t: token t
  pairs.load(a, reached, lane);
  __syncthreads();
  if (lane < TOK)
#pragma unroll
    for (int i = 0; i < 4; ++i) s_sum[wave][i][lane] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int KB = a.I >> 7;
  const int rb = blockIdx.x;
  const uint32_t tiles = (uint32_t)KB * 1024u, tscales = (uint32_t)KB * 64u;
  const uint32_t rows = (uint32_t)a.T * (uint32_t)a.K;
  const __amdgpu_buffer_rsrc_t hr = make_rsrc(a.h, rows * (uint32_t)a.I);
  const __amdgpu_buffer_rsrc_t hsr = make_rsrc(a.h_s, rows * (uint32_t)(a.I >> 5));
  const int64_t items = (int64_t)slots * KB;
  const int first = (int)(items * wave / NW), last = (int)(items * (wave + 1) / NW);
  for (int it = first; it < last;) {
    const int slot = it / KB, kb_first = it - slot * KB;
    const int kb_last = min(KB, kb_first + last - it);
    it += kb_last - kb_first;
    const int e = __builtin_amdgcn_readfirstlane(s_expert[slot]);
    const uint32_t places = pairs.find(e);
    const uint64_t has = ballot(places != 0);
    const int n = __popcll(has);
    if (places != 0) {
      const int at = mask_rank(has);
      float s = 0.f;                                  // h of a later place is the first one's
      for (uint32_t m = places; m != 0; m &= m - 1) s += s_w[lane * a.K + __builtin_ctz(m)];
      s_pair[wave][at] = (int16_t)(lane * a.K + __builtin_ctz(places));
      s_weight[wave][at] = s;
    }
    wave_sync();
    const __amdgpu_buffer_rsrc_t wr = make_rsrc(a.w2 + ((int64_t)e * (a.H >> 4) + rb) * tiles, tiles);
    const __amdgpu_buffer_rsrc_t sr = make_rsrc(a.w2_s + ((int64_t)e * (a.H >> 4) + rb) * tscales, tscales);
    // G times 8 columns from c0 on
    const auto pass = [&](auto groups, int c0) {
      constexpr int G = groups;
      constexpr int R = U / G;                        // K blocks that LDS holds at a time
      // loading: 2^p >= the columns, eight lanes a column's 128 codes, 8 >> p K blocks a load
      const int cols = min(COLS * G, n - c0);
      const int p = G > 1 || cols > 4 ? 3 : cols > 2 ? 2 : cols > 1 ? 1 : 0;
      const int lc = (lane >> 3) & ((1 << p) - 1), chunk = lane & 7, lu = lane >> (3 + p);
      uint32_t from[G];
#pragma unroll
      for (int g = 0; g < G; ++g)
        from[g] = g * COLS + lc < cols ? (uint32_t)s_pair[wave][c0 + g * COLS + lc] * (uint32_t)a.I + (uint32_t)chunk * 16u : kNowhere;
      // computing: column l16
      const bool mine = l16 < cols;
      const uint32_t hso = mine ? (uint32_t)s_pair[wave][c0 + l16] * (uint32_t)(a.I >> 5) : 0u;
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
      for (int kb0 = kb_first; kb0 < kb_last; kb0 += U) {
        u32x4 w[U], h[G][U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          w[u] = buf_load16_nt(wr, kb0 + u < kb_last ? (uint32_t)(kb0 + u) * 1024u + (uint32_t)lane * 16u : kNowhere);
        const uint32_t ws = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(sr, (uint32_t)kb0 * 64u + (uint32_t)lane * 4u, 0, 0);
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int i = 0; i < U; ++i)
            if (i == 0 || G > 1 || i < (1 << p) / 2) {  // (1 << p) * U columns of K blocks, 8 a load
              const int u = i * (8 >> p) + lu;
              h[g][i] = buf_load16(hr, u < U && kb0 + u < kb_last && from[g] != kNowhere ? from[g] + (uint32_t)(kb0 + u) * 128u : kNowhere);
            }
        const u32x4 hs = buf_load16(hsr, mine ? hso + (uint32_t)kb0 * 4u : kNowhere);
        s_scale[wave][lane] = ws;
#pragma unroll
        for (int r = 0; r < G; ++r) {
#pragma unroll
          for (int g = 0; g < G; ++g)
#pragma unroll
            for (int i = r * R; i < (r + 1) * R; ++i)
              if (i == 0 || G > 1 || i < (1 << p) / 2) {
                const int u = i * (8 >> p) + lu;
                if (u < U) s_h[wave][((u - r * R) * G + g) * COLS + lc][chunk ^ lc] = h[g][i];
              }
          wave_sync();
#pragma unroll
          for (int u = r * R; u < (r + 1) * R; ++u) {
            // K blocks past the last have zero weights and codes, and no NaN for a scale
            const bool in = kb0 + u < kb_last;
            const int c = l16 & (COLS * G - 1), x = c & (COLS - 1);
            const u32x4* col = s_h[wave][(u - r * R) * G * COLS + c];
            u32x4 b0 = col[(2 * lhi) ^ x], b1 = col[(2 * lhi + 1) ^ x];
            if (!mine) b0 = b1 = u32x4{0u, 0u, 0u, 0u};
            const uint32_t wb = reinterpret_cast<const uint8_t*>(s_scale[wave])[u * 64 + lane];
            const Bf16Block wv = from_e2m1(w[u], e8m0_scale(in ? wb : 0u));
            const Bf16Block hv = from_e4m3(b0, b1, e8m0_scale(in ? (hs[u] >> (8 * lhi)) & 255u : 0u));
#pragma unroll
            for (int j = 0; j < 4; ++j) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv.v[j], hv.v[j], acc, 0, 0, 0);
          }
          wave_sync();
        }
      }
      if (mine) s_sum[wave][lhi][s_pair[wave][c0 + l16] / a.K] += s_weight[wave][c0 + l16] * acc;   // a token has one column
    };
    for (int c0 = 0; c0 < n; c0 += 2 * COLS)
      if (n - c0 > COLS) pass(std::integral_constant<int, 2>(), c0);
      else pass(std::integral_constant<int, 1>(), c0);
    wave_sync();
  }

  __syncthreads();
  if (wave >= 4) return;
  if (lane < a.T) {
    f32x4 s = s_sum[0][wave][lane];
#pragma unroll
    for (int v = 1; v < NW; ++v) s += s_sum[v][wave][lane];
    const u32x2 o = {pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3])};
    *reinterpret_cast<u32x2*>(a.out + (int64_t)lane * a.H + rb * 16 + wave * 4) = o;
  }
}

// ---------------------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------------------
size_t decode_scales_at(int32_t T, int32_t K, int32_t I) { return align_up((size_t)T * K * I, 256); }
size_t decode_ws_bytes(int32_t T, int32_t K, int32_t I) { return decode_scales_at(T, K, I) + (size_t)T * K * (I / 32); }

int launch_expert_ffn_decode(const void* x, const void* x_s, int32_t T, int32_t H, int32_t I, int32_t K, int32_t begin,
                             int32_t E, const int32_t* idx, const float* weights, const void* w1, const void* w1_s,
                             const void* w2, const void* w2_s, void* ws, void* out, hipStream_t stream) {
  DecodeArgs a;
  a.x = static_cast<const uint8_t*>(x);
  a.x_s = static_cast<const uint8_t*>(x_s);
  a.T = T;
  a.H = H;
  a.I = I;
  a.K = K;
  a.begin = begin;
  a.E = E;
  a.idx = idx;
  a.weights = weights;
  a.w1 = static_cast<const uint8_t*>(w1);
  a.w1_s = static_cast<const uint8_t*>(w1_s);
  a.w2 = static_cast<const uint8_t*>(w2);
  a.w2_s = static_cast<const uint8_t*>(w2_s);
  a.h = static_cast<uint8_t*>(ws);
  a.h_s = a.h + decode_scales_at(T, K, I);
  a.out = static_cast<uint16_t*>(out);
  const dim3 gh(I / 32, std::min(T * K, E)), go(H / 16);
  if (!x_s) {
    // bf16 rows are quantised into out, which has room for them and is written only after h is done
    uint8_t* q = static_cast<uint8_t*>(out);
    uint8_t* q_s = q + (size_t)T * H;
    const int chunks = T * (H / 8);
    hipLaunchKernelGGL(decode_quantise_kernel, dim3((chunks + 255) / 256), dim3(256), 0, stream,
                       static_cast<const uint16_t*>(x), chunks, q, q_s);
    if (hipGetLastError() != hipSuccess) return MOE_ERR_HIP;
    a.x = q;
    a.x_s = q_s;
  }
  const int cus = std::max(1, device_cu_count());
  // 8 waves a workgroup for up to 8 pairs, 4 for more: from 16 on there may be three workgroups a CU, and
  // registers admit two of 8 waves. 8 against 4, of 128 experts at H 4096: 13.3 / 13.8 us (8 pairs), 23.6 / 18.9
  // (16), 37.1 / 33.1 (32); 6 of them on one of 8 ranks at H 7168 14.2 / 15.1
  if (T * K <= 8) hipLaunchKernelGGL((decode_h_kernel<8, 2, 1>), gh, dim3(512), 0, stream, a);
  // 32 tokens for one read of the weights where there are more than 8 pairs for each local expert and so, if all pairs
  // are local, some experts with more than 16 tokens; it leaves room for 3 waves a SIMD instead of 4. 32 against 16: 52 / 70 us (8
  // experts with 64 tokens each, H 5120), 25 / 34 (16 with up to 24, H 4096), 49 / 49 (64 with 8), 145 / 139 (127 with 4). T K counts the
  // pairs of all ranks; on one of several, where few of them are local, 32 is no slower (whole call, 64 tokens, top-8): 108 / 111 us
  // (32 of 256 experts, up to 7 tokens each, H 7168), 37.4 / 38.4 (8 of 256), 59 / 60 (32 of 128, H 4096), 34.6 / 34.6 (16 of 128)
  else if (T > 16 && T * K > 8 * E) hipLaunchKernelGGL((decode_h_kernel<4, 2, 2>), gh, dim3(256), 0, stream, a);
  else hipLaunchKernelGGL((decode_h_kernel<4, 2, 1>), gh, dim3(256), 0, stream, a);
  if (hipGetLastError() != hipSuccess) return MOE_ERR_HIP;
  // 16 waves a workgroup where that is one workgroup a CU at most and each wave has a dozen tiles and more
  // (16 against 8 waves: 11.0 / 9.5 us at 96 tiles a workgroup, 14.5 / 15.7 and 18.9 / 20.6 at 192, 22 / 24 at 384, 85 / 100 at 1536)
  const bool wide = H / 16 <= cus && (int64_t)gh.y * (I / 128) >= 192;
  if (T > 16) {
    if (wide) hipLaunchKernelGGL((decode_out_kernel<16, 64>), go, dim3(1024), 0, stream, a);
    else hipLaunchKernelGGL((decode_out_kernel<8, 64>), go, dim3(512), 0, stream, a);
  } else {
    if (wide) hipLaunchKernelGGL((decode_out_kernel<16, 16>), go, dim3(1024), 0, stream, a);
    else hipLaunchKernelGGL((decode_out_kernel<8, 16>), go, dim3(512), 0, stream, a);
  }
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe
