// The expert FFN of a few tokens with MXFP4 weights: matrix-vector products, straight from
// the routing.
//
//   h[t,k] = mxfp8(silu(W1[e] gate . x[t]) * (W1[e] up . x[t])),
//   out[t] = sum_k topk_weights[t,k] * (W2[e] . h[t,k]).
//
// Every reached expert's 3 * H * I * (1/2 + 1/32) bytes are read once and hardly anything
// else moves: the memory's rate bounds it. The products run on the matrix cores all the same
// (v_mfma_scale_f32_16x16x128_f8f6f4, 16 weight rows by 16 token columns): a 16 x 128 weight
// tile of the layer's load-time layout is one 16-byte load a lane, taken as it is, scales
// included, so no value is unpacked, and up to 16 tokens cost what one does.
//
// The pooled path's plan, dispatch and combine launches are not needed: with at most 64 * 16
// pairs each workgroup finds the reached experts itself (a bitmap in LDS), the h kernel's
// workgroup (slot, block of 32 columns of h) takes the slot-th of them, and the out kernel's
// workgroup sums all experts' shares of its 16 columns in registers, so out needs no second
// pass and no atomics.
#include "common.h"
#include "kernels.h"

#include <algorithm>

namespace moe {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kDecodeTokens = 64;                     // at most
constexpr int kDecodePairs = kDecodeTokens * 16;
constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;

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

// 16 weight rows times 16 tokens over 128 K. Lane (l16, lhi) has of row l16 the 32 e2m1 codes
// K = 32 lhi .. + 32 (a), of column l16 the 16 e4m3 codes K = 16 lhi .. + 16 (b0) and the 16 from
// K = 64 + 16 lhi (b1), and the E8M0 scales of both sides' block K = 32 lhi .. + 32 (sa, sb)
__device__ inline f32x4 mfma_mx(u32x4 a, uint32_t sa, u32x4 b0, u32x4 b1, uint32_t sb, f32x4 acc) {
  const i32x8 av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i32x8 bv = {(int)b0.x, (int)b0.y, (int)b0.z, (int)b0.w, (int)b1.x, (int)b1.y, (int)b1.z, (int)b1.w};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, acc, 4, 0, 0, (int)sa, 0, (int)sb);
}

// ---------------------------------------------------------------------------------------
// the reached experts: local ids of all pairs and a bit for each reached one
// ---------------------------------------------------------------------------------------
struct Reached {
  int16_t id[kDecodePairs];   // local expert of a pair, or -1
  uint32_t bits[32];
};

__device__ inline void find_reached(const DecodeArgs& a, Reached& r) {
  if (threadIdx.x < 32) r.bits[threadIdx.x] = 0;
  __syncthreads();
  for (int q = threadIdx.x; q < a.T * a.K; q += kThreads) {
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

// bf16 values of column l16 to MXFP8, laid out as mfma_mx takes them: f has the lane's 16 values of
// K = 16 lhi .. and of K = 64 + 16 lhi .., so a block of 32 is half in this lane and half in lane
// lhi ^ 1, and the scale of block lhi is found in lanes lhi ^ 2 for lhi 1 and 2. By the whole wave.
__device__ inline uint32_t quantise_column(const float (&f)[32], int lhi, u32x4& b0, u32x4& b1) {
  uint32_t m[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 32; ++j) m[j >> 4] = max(m[j >> 4], __builtin_bit_cast(uint32_t, f[j]) & 0x7fffffffu);
  u32x4 c[2];
  uint32_t byte[2];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    m[p] = max(m[p], (uint32_t)__shfl_xor((int)m[p], 16, 64));
    const bool bad = m[p] >= 0x7f800000u;   // NaN or infinity: the block is NaN
    const int e = mx_e4m3_shared_exp(__builtin_bit_cast(float, m[p]));
    const float inv = mx_inv_scale(e);
    const float* v = f + 16 * p;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c[p][j] = bad ? 0u : pack_e4m3x4(v[4 * j] * inv, v[4 * j + 1] * inv, v[4 * j + 2] * inv, v[4 * j + 3] * inv);
    byte[p] = bad ? 255u : (uint32_t)(e + 127);
  }
  b0 = c[0];
  b1 = c[1];
  const uint32_t other = (uint32_t)__shfl_xor((int)(lhi >= 2 ? byte[0] : byte[1]), 32, 64);
  return lhi == 0 ? byte[0] : lhi == 3 ? byte[1] : other;
}

// ---------------------------------------------------------------------------------------
// h: grid (I / 32 column blocks, slots); the waves share K, NG groups of 16 token columns
// ---------------------------------------------------------------------------------------
template <bool XBF16, int NG, int U>
__global__ __launch_bounds__(kThreads) void decode_h_kernel(DecodeArgs a) {
  __shared__ Reached reached;
  __shared__ int16_t s_q[kDecodeTokens];              // the expert's pairs, one of each of its tokens
  __shared__ f32x4 s_red[kWaves][4][64];
  const int lane = lane_id(), l16 = lane & 15, lhi = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  find_reached(a, reached);
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
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x, (uint32_t)a.T * (uint32_t)a.H * (XBF16 ? 2u : 1u));
  const __amdgpu_buffer_rsrc_t xsr = make_rsrc(a.x_s, XBF16 ? 0u : (uint32_t)a.T * (uint32_t)KB * 4u);
  uint32_t xo[NG], xso[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const int c = g * 16 + l16;
    const uint32_t t = c < n ? (uint32_t)s_q[c] / (uint32_t)a.K : 0u;
    xo[g] = c < n ? t * (uint32_t)a.H * (XBF16 ? 2u : 1u) + (uint32_t)lhi * (XBF16 ? 32u : 16u) : kNowhere;
    xso[g] = c < n ? t * (uint32_t)KB * 4u + (uint32_t)lhi : kNowhere;
  }

  f32x4 acc[NG][4];
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[g][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  // K blocks wave, wave + 8, ...: at every moment the waves read neighbouring tiles
  for (int kb0 = wave; kb0 < KB; kb0 += kWaves * U) {
    u32x4 wt[U][4];
    uint32_t wsc[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t kb = (uint32_t)(kb0 + u * kWaves);   // past KB: past the buffer, zeros
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        wt[u][i] = buf_load16_nt(wr[i], kb * 1024u + (uint32_t)lane * 16u);
        wsc[u][i] = buf_load1(sr[i], kb * 64u + (uint32_t)lane);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t kb = (uint32_t)(kb0 + u * kWaves);
      const bool in = kb < (uint32_t)KB;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if (NG > 1 && g * 16 >= n) break;
        u32x4 b0, b1;
        uint32_t sb;
        if constexpr (XBF16) {
          float f[32];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const u32x4 v = buf_load16(xr, in && xo[g] != kNowhere ? xo[g] + kb * 256u + (uint32_t)(j & 1) * 16u + (uint32_t)(j >> 1) * 128u : kNowhere);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              f[8 * j + 2 * i] = bf16_lo(v[i]);
              f[8 * j + 2 * i + 1] = bf16_hi(v[i]);
            }
          }
          sb = quantise_column(f, lhi, b0, b1);
        } else {
          const uint32_t o = in && xo[g] != kNowhere ? xo[g] + kb * 128u : kNowhere;
          b0 = buf_load16(xr, o);
          b1 = buf_load16(xr, o == kNowhere ? kNowhere : o + 64u);
          sb = buf_load1(xsr, in && xso[g] != kNowhere ? xso[g] + kb * 4u : kNowhere);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[g][i] = mfma_mx(wt[u][i], wsc[u][i], b0, b1, sb, acc[g][i]);
      }
    }
  }

  // the waves' sums, then SwiGLU and the MXFP8 of 32 columns: lane (l16, lhi) has token column
  // l16 and columns 4 lhi .. + 4 of both tiles of 16
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    if (g * 16 >= n) break;
    if (g > 0) __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) s_red[wave][i][lane] = acc[g][i];
    __syncthreads();
    if (wave != g) continue;
    f32x4 s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[i] = s_red[0][i][lane];
#pragma unroll
      for (int v = 1; v < kWaves; ++v) s[i] += s_red[v][i][lane];
    }
    float h[8];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float gate = s[j >> 2][j & 3], up = s[2 + (j >> 2)][j & 3];
      h[j] = gate / (1.0f + __expf(-gate)) * up;
      m = max(m, __builtin_bit_cast(uint32_t, h[j]) & 0x7fffffffu);
    }
    m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
    const bool bad = m >= 0x7f800000u;
    const int ex = mx_e4m3_shared_exp(__builtin_bit_cast(float, m));
    const float inv = mx_inv_scale(ex);
    const int c = g * 16 + l16;
    if (c < n) {
      const int64_t p = s_q[c];
      uint32_t* d = reinterpret_cast<uint32_t*>(a.h + p * a.I + nb * 32 + lhi * 4);
      d[0] = bad ? 0u : pack_e4m3x4(h[0] * inv, h[1] * inv, h[2] * inv, h[3] * inv);
      d[4] = bad ? 0u : pack_e4m3x4(h[4] * inv, h[5] * inv, h[6] * inv, h[7] * inv);
      if (lhi == 0) a.h_s[p * (a.I >> 5) + nb] = (uint8_t)(bad ? 255 : ex + 127);
    }
  }
}

// ---------------------------------------------------------------------------------------
// out: a workgroup has 16 columns of out for all tokens; its waves share the (expert, K block)
// pairs evenly, token t is column t % 16 of group t / 16
// ---------------------------------------------------------------------------------------
template <int NG, int U>
__global__ __launch_bounds__(kThreads) void decode_out_kernel(DecodeArgs a) {
  __shared__ Reached reached;
  __shared__ float s_w[kDecodePairs];
  __shared__ f32x4 s_red[kWaves][NG][64];
  const int lane = lane_id(), l16 = lane & 15, lhi = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int q = threadIdx.x; q < a.T * a.K; q += kThreads) s_w[q] = a.weights[q];
  find_reached(a, reached);
  const int slots = readlane(wave_inclusive_scan(lane < 32 ? __popc(reached.bits[lane]) : 0), 63);

  const int KB = a.I >> 7;
  const int rb = blockIdx.x;
  const uint32_t tiles = (uint32_t)KB * 1024u, tscales = (uint32_t)KB * 64u;
  const uint32_t rows = (uint32_t)a.T * (uint32_t)a.K;
  const __amdgpu_buffer_rsrc_t hr = make_rsrc(a.h, rows * (uint32_t)a.I);
  const __amdgpu_buffer_rsrc_t hsr = make_rsrc(a.h_s, rows * (uint32_t)(a.I >> 5));
  f32x4 sum[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) sum[g] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int64_t items = (int64_t)slots * KB;
  const int first = (int)(items * wave / kWaves), last = (int)(items * (wave + 1) / kWaves);
  for (int it = first; it < last;) {
    const int slot = it / KB, kb_first = it - slot * KB;
    const int kb_last = min(KB, kb_first + last - it);
    it += kb_last - kb_first;
    const int e = reached_expert(reached, slot);
    // this lane's token in every group: its pair with the expert and the pairs' weight
    uint32_t ho[NG], hso[NG];
    float wt[NG];
    bool mine[NG], any[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const int t = g * 16 + l16;
      int q = -1;
      float s = 0.f;
      if (t < a.T)
        for (int k = 0; k < a.K; ++k)
          if (reached.id[t * a.K + k] == e) {
            if (q < 0) q = t * a.K + k;
            s += s_w[t * a.K + k];
          }
      mine[g] = q >= 0;
      any[g] = ballot(q >= 0) != 0;
      wt[g] = s;
      ho[g] = q >= 0 ? (uint32_t)q * (uint32_t)a.I + (uint32_t)lhi * 16u : kNowhere;
      hso[g] = q >= 0 ? (uint32_t)q * (uint32_t)(a.I >> 5) + (uint32_t)lhi : kNowhere;
    }
    const __amdgpu_buffer_rsrc_t wr = make_rsrc(a.w2 + ((int64_t)e * (a.H >> 4) + rb) * tiles, tiles);
    const __amdgpu_buffer_rsrc_t sr = make_rsrc(a.w2_s + ((int64_t)e * (a.H >> 4) + rb) * tscales, tscales);
    f32x4 acc[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) acc[g] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int kb0 = kb_first; kb0 < kb_last; kb0 += U) {
      u32x4 w[U];
      uint32_t wsc[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool in = kb0 + u < kb_last;
        const uint32_t kb = (uint32_t)(kb0 + u);
        w[u] = buf_load16_nt(wr, in ? kb * 1024u + (uint32_t)lane * 16u : kNowhere);
        wsc[u] = buf_load1(sr, in ? kb * 64u + (uint32_t)lane : kNowhere);
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if (!any[g]) continue;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const bool in = mine[g] && kb0 + u < kb_last;
          const uint32_t kb = (uint32_t)(kb0 + u);
          const u32x4 b0 = buf_load16(hr, in ? ho[g] + kb * 128u : kNowhere);
          const u32x4 b1 = buf_load16(hr, in ? ho[g] + kb * 128u + 64u : kNowhere);
          const uint32_t sb = buf_load1(hsr, in ? hso[g] + kb * 4u : kNowhere);
          acc[g] = mfma_mx(w[u], wsc[u], b0, b1, sb, acc[g]);
        }
      }
    }
    // a token without this expert takes nothing of it, a NaN of its weights neither
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[g][i] += mine[g] ? wt[g] * acc[g][i] : 0.f;
  }

#pragma unroll
  for (int g = 0; g < NG; ++g) s_red[wave][g][lane] = sum[g];
  __syncthreads();
  if (wave >= NG) return;
  f32x4 s = s_red[0][wave][lane];
#pragma unroll
  for (int v = 1; v < kWaves; ++v) s += s_red[v][wave][lane];
  const int t = wave * 16 + l16;
  if (t < a.T) {
    const u32x2 o = {pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3])};
    *reinterpret_cast<u32x2*>(a.out + (int64_t)t * a.H + rb * 16 + lhi * 4) = o;
  }
}

// ---------------------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------------------
size_t decode_scales_at(int32_t T, int32_t K, int32_t I) { return align_up((size_t)T * K * I, 256); }
size_t decode_ws_bytes(int32_t T, int32_t K, int32_t I) { return decode_scales_at(T, K, I) + (size_t)T * K * (I / 32); }

template <bool XBF16, int NG, int U>
static void launch_h(dim3 grid, hipStream_t s, const DecodeArgs& a) {
  hipLaunchKernelGGL((decode_h_kernel<XBF16, NG, U>), grid, dim3(kThreads), 0, s, a);
}

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
  if (x_s) {
    if (T <= 16) launch_h<false, 1, 4>(gh, stream, a);
    else launch_h<false, 4, 2>(gh, stream, a);
  } else {
    if (T <= 16) launch_h<true, 1, 4>(gh, stream, a);
    else launch_h<true, 4, 2>(gh, stream, a);
  }
  if (hipGetLastError() != hipSuccess) return MOE_ERR_HIP;
  if (T <= 16) hipLaunchKernelGGL((decode_out_kernel<1, 4>), go, dim3(kThreads), 0, stream, a);
  else hipLaunchKernelGGL((decode_out_kernel<4, 4>), go, dim3(kThreads), 0, stream, a);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe
