// The router's choice: the K experts of every token with their weights, from the logits, and
// the backward pass.
//
// A token's keys are held by L lanes, expert j * L + l in register j of lane l, and the K
// largest are taken one after another: the lanes' largest, then the row's (the same on every
// lane after log2(L) exchanges). Keys are unsigned integers in the order of the numbers, 0 for
// an expert that is switched off. What the picks compare is short: the key's leading bits with
// the expert's index behind them, so that one maximum names both; whole keys are looked at only
// where picks share their leading bits, so ties are exact. The K dependent steps bound a single
// token and, with the scores' 64-bit arithmetic, the grouped choice; a large batch by logits is
// half latency, half its one read of them.
//
// 16384 tokens, 128 experts by logits 7.9 us (8.4 MB) and its backward 5.4; 8192 tokens, 256
// experts by scores in groups 16.5 and 4.8; one token 3.1.
//
// Keys are the logits (32 bits) where their order is the scores'. With a bias or with groups
// ranked by two keys the scores themselves are compared: in 64 bits, since a 32-bit sum would
// put experts in another order, or make a tie of two, when they differ by less than 2^-24.
#include "common.h"
#include "kernels.h"

#include <algorithm>
#include <cfloat>

namespace moe {

constexpr int kRouterWaves = 4;
constexpr int kNarrowTokens = 4096;   // more: 16 lanes a token, else 64

struct RouterArgs {
  const void* logits;
  int32_t bf16;
  const float* bias;
  int32_t T, E, K;
  int32_t score, normalize, groups, topk_groups, group_top;
  int32_t group_size;
  int32_t group_lanes_log2;   // P: the power of two of a token's L lanes that a group gets
  uint32_t group_magic;   // ceil(2^32 / group_size): e / group_size = umulhi(e, magic); 0 for size 1
  float scale;
  int32_t* idx;
  float* weights;
};

// keys in the order of the numbers; 0 is below every one of them
__device__ inline uint32_t order32(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ inline uint64_t order64(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return (b >> 63) ? ~b : (b | (1ull << 63));
}
__device__ inline double from_order64(uint64_t k) {
  return __builtin_bit_cast(double, (k >> 63) ? (k & ~(1ull << 63)) : ~k);
}

// an expert that is switched off reads as -infinity; +infinity as the largest finite value.
// -0 becomes +0 (they are equal, and equal keys are ties).
__device__ inline float clean_logit(float v) {
  if (!(v > -__builtin_inff())) return -__builtin_inff();
  return fminf(v, FLT_MAX) + 0.0f;
}
__device__ inline float load_logit(const RouterArgs& a, int64_t at) {
  if (a.bf16) return clean_logit(bf16_lo(static_cast<const uint16_t*>(a.logits)[at]));
  return clean_logit(static_cast<const float*>(a.logits)[at]);
}

// The logits of `rows` tokens from t0 on, expert j * L + l of token `sub` in v[j]. Buffer loads,
// whatever lies past the last expert or token masked afterwards, so that they can be in flight at once (a
// load behind a condition waits for the one before, 0.6 us each). The compiler does not know that t0 is the
// wave's: it puts a loop over the lanes' different buffers around each load, which runs once (a sixth of the code of
// the kernel by scores with 16 experts a lane).
template <int L, int EPL>
__device__ inline void load_logits(const RouterArgs& a, int64_t t0, int sub, int l, float (&v)[EPL]) {
  const int rows = (int)min((int64_t)(64 / L), a.T - t0);
  const uint32_t first = (uint32_t)(sub * a.E + l);
  uint32_t r[EPL];
  if (a.bf16) {
    const __amdgpu_buffer_rsrc_t b =
        make_rsrc(static_cast<const uint16_t*>(a.logits) + t0 * a.E, (uint32_t)(rows * a.E) * 2u);
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      r[j] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(b, (first + (uint32_t)(j * L)) * 2u, 0, 0) << 16;
  } else {
    const __amdgpu_buffer_rsrc_t b =
        make_rsrc(static_cast<const float*>(a.logits) + t0 * a.E, (uint32_t)(rows * a.E) * 4u);
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      r[j] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(b, (first + (uint32_t)(j * L)) * 4u, 0, 0);
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const float f = clean_logit(__builtin_bit_cast(float, r[j]));
    v[j] = j * L + l < a.E && sub < rows ? f : -__builtin_inff();
  }
}

// ---------------------------------------------------------------------------------------
// reductions over the L lanes of a token (16: a DPP row, 64: the wave)
// ---------------------------------------------------------------------------------------
struct MaxU { __device__ static uint32_t f(uint32_t a, uint32_t b) { return a > b ? a : b; } };
struct MinU { __device__ static uint32_t f(uint32_t a, uint32_t b) { return a < b ? a : b; } };
struct MaxF {
  __device__ static uint32_t f(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)));
  }
};
struct AddF {
  __device__ static uint32_t f(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
  }
};
template <int CTRL>
__device__ inline uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
}
template <typename OP, int L>
__device__ inline uint32_t token_reduce(uint32_t v) {
  v = OP::f(v, dpp<0x128>(v));
  v = OP::f(v, dpp<0x124>(v));
  v = OP::f(v, dpp<0x122>(v));
  v = OP::f(v, dpp<0x121>(v));
  if constexpr (L == 64)
    v = OP::f(OP::f((uint32_t)readlane((int)v, 0), (uint32_t)readlane((int)v, 16)),
              OP::f((uint32_t)readlane((int)v, 32), (uint32_t)readlane((int)v, 48)));
  return v;
}
template <int L>
__device__ inline float token_max(float v) { return __builtin_bit_cast(float, token_reduce<MaxF, L>(__builtin_bit_cast(uint32_t, v))); }
template <int L>
__device__ inline float token_sum(float v) { return __builtin_bit_cast(float, token_reduce<AddF, L>(__builtin_bit_cast(uint32_t, v))); }
template <int L>
__device__ inline uint32_t token_umax(uint32_t k) { return token_reduce<MaxU, L>(k); }
template <int L>
__device__ inline uint64_t token_umax(uint64_t k) {
  const uint32_t hi = token_reduce<MaxU, L>((uint32_t)(k >> 32));
  const uint32_t lo = token_reduce<MaxU, L>((uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
  return ((uint64_t)hi << 32) | lo;
}
// 64-bit sum over the token's lanes, the same on all of them
template <int L>
__device__ inline double token_sum(double v) {
#pragma unroll
  for (int o = 1; o < L; o *= 2) v += __shfl_xor(v, o, 64);
  return v;
}

// the two largest of (first, second) and k; equal keys count twice
template <typename KEY>
__device__ inline void add_top2(KEY& first, KEY& second, KEY k) {
  const KEY low = k > first ? first : k;
  first = k > first ? k : first;
  second = low > second ? low : second;
}
__device__ inline uint32_t lane_xor(uint32_t v, int o) { return (uint32_t)__shfl_xor((int)v, o, 64); }
__device__ inline uint64_t lane_xor(uint64_t v, int o) {
  return ((uint64_t)lane_xor((uint32_t)(v >> 32), o) << 32) | lane_xor((uint32_t)v, o);
}

// the value of lane k of token `sub`
template <int L>
__device__ inline uint32_t token_lane(uint32_t v, int sub, int k) { return (uint32_t)__shfl((int)v, sub * L + k, 64); }
template <int L>
__device__ inline uint64_t token_lane(uint64_t v, int sub, int k) {
  return ((uint64_t)token_lane<L>((uint32_t)(v >> 32), sub, k) << 32) | token_lane<L>((uint32_t)v, sub, k);
}

__device__ inline float sigmoidf(float v) { return 1.0f / (1.0f + expf(-v)); }
// sigmoid(v) e^-c for c <= 0, and c = 0 for v > 0: with c = min(0, the largest of some logits) their ratios are those of the
// sigmoids, also where these are no fp32 numbers (v below -88). What is 0 in 64 bits, 1 / (1 + e^-v) for v below
// -709.78, is 0.
__device__ inline float sigmoid_over(float v, float c) {
  const float top = v > 0.0f ? 1.0f : v < -709.78266f ? 0.0f : expf(v - c);
  return top / (1.0f + expf(-fabsf(v)));
}
// c of a token: chosen logits, -infinity for none
template <int L>
__device__ inline float sigmoid_shift(float z, int normalize) { return normalize ? fminf(token_max<L>(z), 0.0f) : 0.0f; }

// ---------------------------------------------------------------------------------------
// forward: 64 / L tokens a wave, EPL experts a lane. SCORES: keys are scores (64 bits, in LDS),
// else the logits. Only what is done for every pick is unrolled over the lane's experts, the rest
// loops over LDS: the kernel runs once through its code, and fetching it costs more than the
// loops do (8192 tokens, 256 experts by scores: 18.2 us with 25 KB of unrolled code, 15.6 so).
// ---------------------------------------------------------------------------------------
template <bool SCORES>
struct RouterKey { typedef uint32_t type; };
template <>
struct RouterKey<true> { typedef uint64_t type; };

template <bool SCORES, int L, int EPL>
__global__ __launch_bounds__(64 * kRouterWaves) void router_topk_kernel(RouterArgs a) {
  typedef typename RouterKey<SCORES>::type KEY;
  constexpr int TPW = 64 / L;
  constexpr int N = L * EPL;
  __shared__ float s_logit[kRouterWaves][TPW][N];
  __shared__ uint64_t s_key[SCORES ? kRouterWaves : 1][TPW][SCORES ? N : 1];
  __shared__ float s_bias[SCORES ? N : 1];
  __shared__ KEY s_rank[kRouterWaves][TPW][L];
  __shared__ int s_order[kRouterWaves][TPW][L];
  const int lane = lane_id();
  const int wave = threadIdx.x >> 6;
  const int l = lane & (L - 1), sub = lane / L;
  float* logits = s_logit[wave][sub];
  uint64_t* keys = s_key[SCORES ? wave : 0][SCORES ? sub : 0];
  if constexpr (SCORES) {
    for (int e = threadIdx.x; e < N; e += 64 * kRouterWaves) s_bias[e] = a.bias && e < a.E ? a.bias[e] : 0.0f;
    __syncthreads();
  }
  // the whole key of expert e, 0: switched off
  const auto key_of = [&](int e) -> KEY {
    if constexpr (SCORES) return keys[e];
    else return logits[e] > -__builtin_inff() ? order32(logits[e]) : 0u;
  };
  const int64_t per_grid = (int64_t)gridDim.x * kRouterWaves * TPW;
  // whole waves loop: a wave's last tokens may be past T and are then not stored
  for (int64_t t0 = ((int64_t)blockIdx.x * kRouterWaves + wave) * TPW; t0 < a.T; t0 += per_grid) {
    const int64_t t = t0 + sub;
    const bool live = t < a.T;
    float v[EPL];
    load_logits<L, EPL>(a, t0, sub, l, v);
    float m = v[0];
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      logits[j * L + l] = v[j];
      m = fmaxf(m, v[j]);
    }
    m = token_max<L>(m);

    if constexpr (SCORES) {
      const bool sigmoid = a.score == MOE_SCORE_SIGMOID;
      double sum = 0.0;
#pragma unroll 4
      for (int e = l; e < N; e += L) {
        const float z = logits[e];
        const double x = exp(sigmoid ? -(double)z : (double)z - (double)m);
        const double p = sigmoid ? 1.0 / (1.0 + x) : z > -__builtin_inff() ? x : 0.0;
        sum += p;
        keys[e] = __builtin_bit_cast(uint64_t, p);
      }
      const double factor = sigmoid ? 1.0 : 1.0 / token_sum<L>(sum);
#pragma unroll 4
      for (int e = l; e < N; e += L) {
        const double p = __builtin_bit_cast(double, keys[e]) * factor + (double)s_bias[e];
        const bool on = logits[e] > -__builtin_inff() && p > -__builtin_inf();
        keys[e] = on ? order64(p + 0.0) : 0ull;
      }
    }

    // ---- groups: P lanes find a group's two largest keys, then every group is ranked ----
    uint64_t kept = ~0ull;
    if (a.groups > 1) {
      wave_sync();
      const int g = l >> a.group_lanes_log2, P = 1 << a.group_lanes_log2;
      KEY first = 0, second = 0;
      if (g < a.groups) {
#pragma unroll 4
        for (int i = l & (P - 1); i < a.group_size; i += P) add_top2(first, second, key_of(g * a.group_size + i));
      }
      for (int o = 1; o < P; o *= 2) {
        const KEY f = lane_xor(first, o), s = lane_xor(second, o);
        add_top2(first, second, f);
        add_top2(first, second, s);
      }
      KEY rank = first;
      if constexpr (SCORES)
        if (a.group_top == 2 && second != 0) rank = order64(from_order64(first) + from_order64(second) + 0.0);
      KEY* ranks = s_rank[wave][sub];
      if (g < a.groups) ranks[g] = rank;   // the same from all P lanes
      wave_sync();
      const KEY own = l < a.groups ? ranks[l] : 0;
      int before = 0;
#pragma unroll 4
      for (int i = 0; i < a.groups; ++i) {
        const KEY o = ranks[i];
        before += o > own || (o == own && i < l);
      }
      kept = ballot(l < a.groups && own != 0 && before < a.topk_groups);
      if constexpr (L < 64) kept = (kept >> (sub * L)) & ((1ull << (L & 63)) - 1);
    }
    const auto in_kept = [&](uint32_t e) {
      const uint32_t g = a.group_magic ? __umulhi(e, a.group_magic) : e;
      return a.groups == 1 || ((kept >> (g & 63)) & 1ull) != 0;
    };

    // ---- the K largest, one after another; lane k keeps the k-th ----
    // By short keys: the key as an fp32 number without its last bits, which hold the expert (lower
    // is larger), so that one maximum names the expert and its key. One pick more than K is taken
    // (where a lane is left for it) and the next one looked at: if that is below the K-th, the K
    // largest are among the picks, and only the order of picks with the same short number is open.
    constexpr uint32_t M = N - 1;
    uint32_t quick[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const uint32_t e = (uint32_t)(j * L + l);
      bool on;
      float f;
      if constexpr (SCORES) {
        const uint64_t k = keys[e];
        on = k != 0;
        f = (float)from_order64(k);
      } else {
        on = v[j] > -__builtin_inff();
        f = v[j];
      }
      quick[j] = on && in_kept(e) ? (order32(f) & ~M) | (M - e) : 0u;
    }
    const int picks = min(a.K + 1, L);
    uint32_t my = 0, best = 0;
#pragma unroll 1
    for (int k = 0; k <= picks; ++k) {
      best = quick[0];
#pragma unroll
      for (int j = 1; j < EPL; ++j) best = MaxU::f(best, quick[j]);
      best = token_umax<L>(best);
      if (k == picks) break;
#pragma unroll
      for (int j = 0; j < EPL; ++j) quick[j] = quick[j] == best ? 0u : quick[j];
      my = l == k ? best : my;
    }
    int my_e = my != 0 ? (int)(M - (my & M)) : -1;
    wave_sync();
    // bf16 logits have nothing in the bits that were dropped
    if (SCORES || !a.bf16) {
      const uint32_t next = (uint32_t)__shfl_down((int)my, 1, L);
      const bool same = l + 1 < picks && my != 0 && (my & ~M) == (next & ~M);
      const bool open = l == a.K - 1 && my != 0 && (my & ~M) == (best & ~M);
      if (ballot(open) != 0) {
        // three in a row at the K-th place: whole keys, in order
        my_e = -1;
        KEY last = 0;
        int last_e = -1;
#pragma unroll 1
        for (int k = 0; k < a.K; ++k) {
          KEY top = 0;
          int at = -1;
#pragma unroll 4
          for (int e = l; e < N; e += L) {
            const KEY c = in_kept((uint32_t)e) ? key_of(e) : 0;
            const bool after = k == 0 || c < last || (c == last && e > last_e);   // not picked yet
            if (after && c > top) {
              top = c;
              at = e;
            }
          }
          last = token_umax<L>(top);
          last_e = (int)token_reduce<MinU, L>(top == last && at >= 0 ? (uint32_t)at : 0xffffffffu);
          if (l == k) my_e = last != 0 ? last_e : -1;
        }
      } else if (ballot(same) != 0) {
        // the picks' order by whole keys: each counts those before it
        const KEY c = my_e >= 0 ? key_of(my_e) : 0;
        const uint32_t tie = my_e >= 0 ? (uint32_t)my_e : (uint32_t)(N + l);
        int rank = 0;
        for (int k = 0; k < picks; ++k) {
          const KEY o = token_lane<L>(c, sub, k);
          const uint32_t ot = token_lane<L>(tie, sub, k);
          rank += o > c || (o == c && ot < tie);
        }
        int* order = s_order[wave][sub];
        if (l < picks) order[rank] = my_e;
        wave_sync();
        my_e = order[l];   // past the picks: not used
      }
    }

    // ---- weights ----
    const bool got = l < a.K && my_e >= 0;
    const float z = got ? logits[my_e] : -__builtin_inff();
    float w, total = 1.0f;
    if (a.score == MOE_SCORE_SOFTMAX) {
      if (a.normalize) m = token_max<L>(z);
      w = got ? expf(z - m) : 0.0f;
      float sum = w;
      if (!a.normalize) {
        sum = 0.0f;
#pragma unroll 4
        for (int e = l; e < N; e += L) sum += logits[e] > -__builtin_inff() ? expf(logits[e] - m) : 0.0f;
      }
      total = token_sum<L>(sum);
    } else {
      const float c = sigmoid_shift<L>(z, a.normalize);
      w = got ? sigmoid_over(z, c) : 0.0f;
      if (a.normalize) total = token_sum<L>(w);
    }
    if (live && l < a.K) {
      a.idx[t * a.K + l] = my_e;
      a.weights[t * a.K + l] = total > 0.0f ? w / total * a.scale : 0.0f;
    }
    wave_sync();   // the next tokens' logits go where these are read
  }
}

// ---------------------------------------------------------------------------------------
// backward: 64 / L tokens a wave. Lane k < K of a token has the k-th place's part; the wave's
// rows are put together in LDS (all experts' share of the softmax, then the places' parts) and
// written as one run.
// ---------------------------------------------------------------------------------------
struct RouterBwdArgs {
  RouterArgs r;
  const float* d_weights;
  void* d_logits;
  int32_t wide;   // d_logits is 16-byte aligned and E % 4 == 0
};

template <int L, int EPL>
__global__ __launch_bounds__(64 * kRouterWaves) void router_topk_backward_kernel(RouterBwdArgs b) {
  constexpr int TPW = 64 / L;
  __shared__ float s_row[kRouterWaves][TPW * L * EPL];
  const RouterArgs& a = b.r;
  const int lane = lane_id();
  const int l = lane & (L - 1), sub = lane / L;
  const int wave = threadIdx.x >> 6;
  float* rows = s_row[wave];            // TPW rows of E
  float* mine = rows + sub * a.E;
  const bool dense = a.score == MOE_SCORE_SOFTMAX && !a.normalize;   // every expert has a share
  const int64_t per_grid = (int64_t)gridDim.x * kRouterWaves * TPW;
  for (int64_t t0 = ((int64_t)blockIdx.x * kRouterWaves + wave) * TPW; t0 < a.T; t0 += per_grid) {
    const int64_t t = t0 + sub;
    const bool live = t < a.T;
    const int64_t row = (live ? t : 0) * a.E;
    int e = -1;
    float d = 0.0f, z = -__builtin_inff();
    if (live && l < a.K) {
      e = a.idx[t * a.K + l];
      const float dw = b.d_weights[t * a.K + l];
      if ((uint32_t)e < (uint32_t)a.E) {
        z = load_logit(a, row + e);
        if (z > -__builtin_inff()) d = dw * a.scale;
      }
    }
    const bool got = z > -__builtin_inff();
    float m, w, total = 1.0f;
    float p[EPL];
    if (dense) {
      float v[EPL];
      load_logits<L, EPL>(a, t0, sub, l, v);
      m = v[0];
#pragma unroll
      for (int j = 1; j < EPL; ++j) m = fmaxf(m, v[j]);
      m = token_max<L>(m);
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        p[j] = v[j] > -__builtin_inff() ? expf(v[j] - m) : 0.0f;
        sum += p[j];
      }
      total = token_sum<L>(sum);
      w = got ? expf(z - m) : 0.0f;
    } else if (a.score == MOE_SCORE_SOFTMAX) {
      m = token_max<L>(z);
      w = got ? expf(z - m) : 0.0f;
      total = token_sum<L>(w);
    } else {
      const float c = sigmoid_shift<L>(z, a.normalize);
      w = got ? sigmoid_over(z, c) : 0.0f;
      if (a.normalize) total = token_sum<L>(w);
    }
    // every part is the weight, at most 1, times a difference of d, so none passes fp32's end before the result does
    w = total > 0.0f ? w / total : 0.0f;
    const float inv = total > 0.0f ? 1.0f / total : 0.0f;   // of the dense share alone, whose total is 1 at least
    const float mean = token_sum<L>(w * d);
    float part;
    if (dense) part = w * d;
    else if (a.score == MOE_SCORE_SOFTMAX) part = w * (d - mean);
    else part = w * (a.normalize ? d - mean : d) * sigmoidf(-z);
    const int n = (int)min((int64_t)TPW, a.T - t0) * a.E;   // the run
    if (dense) {
#pragma unroll
      for (int j = 0; j < EPL; ++j)
        if (j * L + l < a.E) mine[j * L + l] = -p[j] * inv * mean;
    } else {
      for (int i = lane; i < n; i += 64) rows[i] = 0.0f;
    }
    wave_sync();
    if (got) atomicAdd(&mine[e], part);
    wave_sync();
    const int64_t at = t0 * a.E;
    if (b.wide) {
      for (int i = lane * 4; i < n; i += 256) {
        const float o0 = rows[i], o1 = rows[i + 1], o2 = rows[i + 2], o3 = rows[i + 3];
        if (a.bf16) {
          const u32x2 o = {pack_bf16x2(o0, o1), pack_bf16x2(o2, o3)};
          *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(b.d_logits) + at + i) = o;
        } else {
          typedef float f32x4 __attribute__((ext_vector_type(4)));
          *reinterpret_cast<f32x4*>(static_cast<float*>(b.d_logits) + at + i) = f32x4{o0, o1, o2, o3};
        }
      }
    } else {
      for (int i = lane; i < n; i += 64) {
        if (a.bf16) static_cast<uint16_t*>(b.d_logits)[at + i] = (uint16_t)pack_bf16x2(rows[i], 0.0f);
        else static_cast<float*>(b.d_logits)[at + i] = rows[i];
      }
    }
    wave_sync();
  }
}

// ---------------------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------------------
static RouterArgs router_args(const void* logits, bool bf16, const float* bias, int32_t T, int32_t E, int32_t K,
                              const moe_router_config& c) {
  RouterArgs a{};
  a.logits = logits;
  a.bf16 = bf16;
  a.bias = bias;
  a.T = T;
  a.E = E;
  a.K = K;
  a.score = c.score;
  a.normalize = c.normalize;
  a.groups = c.groups;
  a.topk_groups = c.topk_groups;
  a.group_top = c.group_top;
  a.group_size = E / c.groups;
  a.group_magic = a.group_size > 1 ? (uint32_t)(((1ull << 32) + a.group_size - 1) / a.group_size) : 0u;
  a.scale = c.scale;
  return a;
}

static dim3 router_grid(int32_t T, int tokens_per_block) {
  return dim3((unsigned)std::min<int64_t>(((int64_t)T + tokens_per_block - 1) / tokens_per_block, 1 << 16));
}

template <bool SCORES, int L, int EPL>
static void launch_topk_as(RouterArgs a, hipStream_t s) {
  a.group_lanes_log2 = 31 - __builtin_clz((unsigned)(L / a.groups));
  const dim3 grid = router_grid(a.T, kRouterWaves * (64 / L)), block(64 * kRouterWaves);
  hipLaunchKernelGGL((router_topk_kernel<SCORES, L, EPL>), grid, block, 0, s, a);
}

template <bool SCORES>
static void launch_topk(const RouterArgs& a, hipStream_t s) {
  // 16 lanes a token where the tokens fill the CUs so, else (and for many experts or groups) 64.
  // 64 against 16 lanes: 128 experts by logits 2.8 / 3.9 us (one token), 4.1 / 4.8 (1024), 5.7 / 5.6
  // (4096), 13.1 / 7.3 (16384); 256 experts by scores, grouped: 5.0 / 10.0, 7.0 / 12.7, 11.3 / 13.6, 32.4 / 29.2
  const bool narrow = a.groups <= 16 && a.T > kNarrowTokens;
  if (narrow && a.E <= 64) launch_topk_as<SCORES, 16, 4>(a, s);
  else if (narrow && a.E <= 128) launch_topk_as<SCORES, 16, 8>(a, s);
  else if (narrow && a.E <= 256) launch_topk_as<SCORES, 16, 16>(a, s);
  else if (a.E <= 128) launch_topk_as<SCORES, 64, 2>(a, s);
  else if (a.E <= 256) launch_topk_as<SCORES, 64, 4>(a, s);
  else if (a.E <= 512) launch_topk_as<SCORES, 64, 8>(a, s);
  else launch_topk_as<SCORES, 64, 16>(a, s);
}

int launch_router_topk(const void* logits, bool bf16, const float* bias, int32_t T, int32_t E, int32_t K,
                       const moe_router_config& c, int32_t* idx, float* weights, hipStream_t stream) {
  RouterArgs a = router_args(logits, bf16, bias, T, E, K, c);
  a.idx = idx;
  a.weights = weights;
  if (bias || (c.groups > 1 && c.group_top == 2)) launch_topk<true>(a, stream);
  else launch_topk<false>(a, stream);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int launch_router_topk_backward(const float* d_weights, const void* logits, bool bf16, const int32_t* idx, int32_t T,
                                int32_t E, int32_t K, const moe_router_config& c, void* d_logits, hipStream_t stream) {
  RouterBwdArgs b;
  b.r = router_args(logits, bf16, nullptr, T, E, K, c);
  b.r.idx = const_cast<int32_t*>(idx);
  b.r.weights = nullptr;
  b.d_weights = d_weights;
  b.d_logits = d_logits;
  b.wide = E % 4 == 0 && reinterpret_cast<uintptr_t>(d_logits) % 16 == 0;
  const dim3 block(64 * kRouterWaves);
  const dim3 g16 = router_grid(T, kRouterWaves * 4), g64 = router_grid(T, kRouterWaves);
  if (E <= 128) hipLaunchKernelGGL((router_topk_backward_kernel<16, 8>), g16, block, 0, stream, b);
  else if (E <= 256) hipLaunchKernelGGL((router_topk_backward_kernel<16, 16>), g16, block, 0, stream, b);
  else if (E <= 512) hipLaunchKernelGGL((router_topk_backward_kernel<64, 8>), g64, block, 0, stream, b);
  else hipLaunchKernelGGL((router_topk_backward_kernel<64, 16>), g64, block, 0, stream, b);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe
