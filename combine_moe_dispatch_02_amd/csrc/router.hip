// The router's choice: the K experts of every token with their weights, from the logits, and
// the backward pass.
//
// A token's keys are held by L lanes, expert j * L + l in register j of lane l, and the K
// largest are taken one after another: the lanes' largest, the row's largest (the same on
// every lane after log2(L) exchanges), the lowest index that has it. Keys are unsigned
// integers in the order of the numbers, 0 for an expert that is switched off, so that one
// comparison decides and ties are exact. Reading the logits once bounds a large batch
// (T * E * 4 bytes); the K dependent steps bound a single token.
//
// Keys are the logits (32 bits) where their order is the scores'. With a bias or with groups
// ranked by two keys the scores themselves are compared: in 64 bits, since a 32-bit sum would
// put experts in another order, or make a tie of two, when they differ by less than 2^-24.
#include "common.h"
#include "kernels.h"

#include <algorithm>
#include <cfloat>

namespace moe {

constexpr int kTokensPerBlockWaves = 4;

struct RouterArgs {
  const void* logits;
  int32_t bf16;
  const float* bias;
  int32_t T, E, K;
  int32_t score, normalize, groups, topk_groups, group_top;
  int32_t group_size;
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

// ---------------------------------------------------------------------------------------
// reductions over the L lanes of a token (L = 16: a DPP row; L = 64: the wave)
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

// LDS written by lanes of a wave is read by others of the same wave
__device__ inline void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ inline float sigmoidf(float v) { return 1.0f / (1.0f + expf(-v)); }

// ---------------------------------------------------------------------------------------
// forward: 64 / L tokens a wave, EPL experts a lane; KEY uint32_t (logits) or uint64_t (scores)
// ---------------------------------------------------------------------------------------
template <typename KEY, int L, int EPL>
__global__ __launch_bounds__(64 * kTokensPerBlockWaves) void router_topk_kernel(RouterArgs a) {
  constexpr int TPW = 64 / L;
  __shared__ KEY s_key[kTokensPerBlockWaves][TPW][L * EPL];   // groups only
  const int lane = lane_id();
  const int wave = threadIdx.x >> 6;
  const int l = lane & (L - 1), sub = lane / L;
  const int64_t per_grid = (int64_t)gridDim.x * kTokensPerBlockWaves * TPW;
  // whole waves loop: a wave's last tokens may be past T and are then not stored
  for (int64_t t0 = ((int64_t)blockIdx.x * kTokensPerBlockWaves + wave) * TPW; t0 < a.T; t0 += per_grid) {
    const int64_t t = t0 + sub;
    const bool live = t < a.T;
    const int64_t row = (live ? t : 0) * a.E;
    float v[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const int e = j * L + l;
      v[j] = e < a.E ? load_logit(a, row + e) : -__builtin_inff();
    }
    float m = v[0];
#pragma unroll
    for (int j = 1; j < EPL; ++j) m = fmaxf(m, v[j]);
    m = token_max<L>(m);

    // ---- keys ----
    KEY key[EPL];
    if constexpr (sizeof(KEY) == 4) {
#pragma unroll
      for (int j = 0; j < EPL; ++j) key[j] = v[j] > -__builtin_inff() ? order32(v[j]) : 0u;
    } else {
      double p[EPL];
      double sum = 0.0;
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        const double d = (double)v[j];
        if (a.score == MOE_SCORE_SIGMOID) {
          p[j] = 1.0 / (1.0 + exp(-d));
        } else {
          p[j] = v[j] > -__builtin_inff() ? exp(d - (double)m) : 0.0;
          sum += p[j];
        }
      }
      if (a.score == MOE_SCORE_SOFTMAX) {
        sum = token_sum<L>(sum);
#pragma unroll
        for (int j = 0; j < EPL; ++j) p[j] /= sum;
      }
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        const int e = j * L + l;
        if (a.bias) p[j] += e < a.E ? (double)a.bias[e] : 0.0;
        const bool on = v[j] > -__builtin_inff() && p[j] > -__builtin_inf();
        key[j] = on ? order64(p[j] + 0.0) : 0ull;
      }
    }

    // ---- groups: lane g of the token ranks group g ----
    if (a.groups > 1) {
      KEY* mine = s_key[wave][sub];
#pragma unroll
      for (int j = 0; j < EPL; ++j) mine[j * L + l] = key[j];
      wave_sync();
      KEY first = 0, second = 0;
      if (l < a.groups)
        for (int i = 0; i < a.group_size; ++i) {
          const KEY k = mine[l * a.group_size + i];
          if (k > first) {
            second = first;
            first = k;
          } else if (k > second) {
            second = k;
          }
        }
      KEY rank = first;
      if constexpr (sizeof(KEY) == 8)
        if (a.group_top == 2 && second != 0) rank = order64(from_order64(first) + from_order64(second) + 0.0);
      wave_sync();
      mine[l] = rank;
      wave_sync();
      int before = 0;
      for (int g = 0; g < a.groups; ++g) {
        const KEY o = mine[g];
        before += o > rank || (o == rank && g < l);
      }
      const uint64_t kept64 = ballot(l < a.groups && rank != 0 && before < a.topk_groups);
      const uint64_t kept = L == 64 ? kept64 : (kept64 >> (sub * L)) & ((1ull << (L & 63)) - 1);
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        const uint32_t e = (uint32_t)(j * L + l);
        const uint32_t g = a.group_magic ? __umulhi(e, a.group_magic) : e;
        if (!((kept >> (g & 63)) & 1ull)) key[j] = 0;
      }
      wave_sync();
    }

    // ---- the K largest, one after another; lane k keeps the k-th ----
    int my_e = -1;
    for (int k = 0; k < a.K; ++k) {
      KEY best = key[0];
#pragma unroll
      for (int j = 1; j < EPL; ++j) best = key[j] > best ? key[j] : best;
      best = token_umax<L>(best);
      uint32_t e = 0xffffffffu;
#pragma unroll
      for (int j = EPL - 1; j >= 0; --j)
        if (key[j] == best) e = (uint32_t)(j * L + l);
      e = token_reduce<MinU, L>(e);
#pragma unroll
      for (int j = 0; j < EPL; ++j)
        if ((uint32_t)(j * L + l) == e) key[j] = 0;
      if (l == k) my_e = best != 0 ? (int)e : -1;
    }

    // ---- weights ----
    const bool got = l < a.K && my_e >= 0;
    const float z = got ? load_logit(a, row + my_e) : -__builtin_inff();
    float w, total = 1.0f;
    if (a.score == MOE_SCORE_SOFTMAX) {
      if (a.normalize) {
        m = token_max<L>(z);
        w = got ? expf(z - m) : 0.0f;
        total = token_sum<L>(w);
      } else {
        w = got ? expf(z - m) : 0.0f;
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) sum += v[j] > -__builtin_inff() ? expf(v[j] - m) : 0.0f;
        total = token_sum<L>(sum);
      }
    } else {
      w = got ? sigmoidf(z) : 0.0f;
      if (a.normalize) total = token_sum<L>(w);
    }
    if (live && l < a.K) {
      a.idx[t * a.K + l] = my_e;
      a.weights[t * a.K + l] = total > 0.0f ? w / total * a.scale : 0.0f;
    }
  }
}

// ---------------------------------------------------------------------------------------
// backward: a token a wave. Lane k < K has the k-th place's part; the row is put together in
// LDS (all experts' share of the softmax, then the places' parts) and written in order.
// ---------------------------------------------------------------------------------------
struct RouterBwdArgs {
  RouterArgs r;
  const float* d_weights;
  void* d_logits;
};

template <int EPL>
__global__ __launch_bounds__(64 * kTokensPerBlockWaves) void router_topk_backward_kernel(RouterBwdArgs b) {
  __shared__ float s_row[kTokensPerBlockWaves][64 * EPL];
  const RouterArgs& a = b.r;
  const int l = lane_id();
  const int wave = threadIdx.x >> 6;
  float* mine = s_row[wave];
  const bool dense = a.score == MOE_SCORE_SOFTMAX && !a.normalize;   // every expert has a share
  for (int64_t t = (int64_t)blockIdx.x * kTokensPerBlockWaves + wave; t < a.T;
       t += (int64_t)gridDim.x * kTokensPerBlockWaves) {
    const int64_t row = t * a.E;
    int e = -1;
    float d = 0.0f, z = -__builtin_inff();
    if (l < a.K) {
      e = a.idx[t * a.K + l];
      if ((uint32_t)e < (uint32_t)a.E) {
        z = load_logit(a, row + e);
        if (z > -__builtin_inff()) d = b.d_weights[t * a.K + l] * a.scale;
      }
    }
    const bool got = z > -__builtin_inff();
    float p[EPL];
    float m, w, total = 1.0f;
    if (dense) {
      float v[EPL];
      m = -__builtin_inff();
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        const int i = j * 64 + l;
        v[j] = i < a.E ? load_logit(a, row + i) : -__builtin_inff();
        m = fmaxf(m, v[j]);
      }
      m = token_max<64>(m);
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        p[j] = v[j] > -__builtin_inff() ? expf(v[j] - m) : 0.0f;
        sum += p[j];
      }
      total = token_sum<64>(sum);
      w = got ? expf(z - m) : 0.0f;
    } else if (a.score == MOE_SCORE_SOFTMAX) {
      m = token_max<64>(z);
      w = got ? expf(z - m) : 0.0f;
      total = token_sum<64>(w);
    } else {
      w = got ? sigmoidf(z) : 0.0f;
      if (a.normalize) total = token_sum<64>(w);
    }
    const float s = w;                           // sigmoid: the score itself
    const float inv = total > 0.0f ? 1.0f / total : 0.0f;
    w *= inv;
    const float mean = token_sum<64>(w * d);
    float part;
    if (dense) part = w * d;
    else if (a.score == MOE_SCORE_SOFTMAX) part = w * (d - mean);
    else part = (a.normalize ? (d - mean) * inv : d) * s * sigmoidf(-z);
#pragma unroll
    for (int j = 0; j < EPL; ++j) mine[j * 64 + l] = dense ? -p[j] * inv * mean : 0.0f;
    wave_sync();
    if (got) atomicAdd(&mine[e], part);
    wave_sync();
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const int i = j * 64 + l;
      if (i >= a.E) continue;
      const float o = mine[i];
      if (a.bf16) static_cast<uint16_t*>(b.d_logits)[row + i] = (uint16_t)pack_bf16x2(o, 0.0f);
      else static_cast<float*>(b.d_logits)[row + i] = o;
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

template <typename KEY>
static void launch_topk(const RouterArgs& a, hipStream_t s) {
  const dim3 block(64 * kTokensPerBlockWaves);
  const dim3 g16 = router_grid(a.T, kTokensPerBlockWaves * 4), g64 = router_grid(a.T, kTokensPerBlockWaves);
  if (a.E <= 64 && a.groups <= 16) hipLaunchKernelGGL((router_topk_kernel<KEY, 16, 4>), g16, block, 0, s, a);
  else if (a.E <= 128 && a.groups <= 16) hipLaunchKernelGGL((router_topk_kernel<KEY, 16, 8>), g16, block, 0, s, a);
  else if (a.E <= 256) hipLaunchKernelGGL((router_topk_kernel<KEY, 64, 4>), g64, block, 0, s, a);
  else if (a.E <= 512) hipLaunchKernelGGL((router_topk_kernel<KEY, 64, 8>), g64, block, 0, s, a);
  else hipLaunchKernelGGL((router_topk_kernel<KEY, 64, 16>), g64, block, 0, s, a);
}

int launch_router_topk(const void* logits, bool bf16, const float* bias, int32_t T, int32_t E, int32_t K,
                       const moe_router_config& c, int32_t* idx, float* weights, hipStream_t stream) {
  RouterArgs a = router_args(logits, bf16, bias, T, E, K, c);
  a.idx = idx;
  a.weights = weights;
  if (bias || (c.groups > 1 && c.group_top == 2)) launch_topk<uint64_t>(a, stream);
  else launch_topk<uint32_t>(a, stream);
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
  const dim3 block(64 * kTokensPerBlockWaves), grid = router_grid(T, kTokensPerBlockWaves);
  if (E <= 128) hipLaunchKernelGGL((router_topk_backward_kernel<2>), grid, block, 0, stream, b);
  else if (E <= 256) hipLaunchKernelGGL((router_topk_backward_kernel<4>), grid, block, 0, stream, b);
  else if (E <= 512) hipLaunchKernelGGL((router_topk_backward_kernel<8>), grid, block, 0, stream, b);
  else hipLaunchKernelGGL((router_topk_backward_kernel<16>), grid, block, 0, stream, b);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe
