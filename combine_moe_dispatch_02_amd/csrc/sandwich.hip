// The norms behind a block and in front of the next one, with the block's gate, the scales of both
// branches and the residual's addition between them, and the backward pass.
//
//   r1 = fp32(1 / sqrt(mean(x^2) + eps1)), p = (x r1) wp      (without a post-norm: p = x)
//   f = act(gate) branch_scale, s = bf16(res_scale res + p f)
//   r2 = fp32(1 / sqrt(mean(s^2) + eps2)), y = bf16((s r2) w), (q, q_s) = y in 8 bits;
//   backward, with xs = s r2, xh = x r1, g = dy w:
//   ds = d_s + r2 (g - xs mean(g xs)), d_res = res_scale ds, dp = f ds,
//   dx = r1 (dp wp - xh mean(dp wp xh)), d_gate = branch_scale act'(gate) ds p, summed over what
//   the gate is broadcast to, dw = sum over rows of dy xs, dwp = sum over rows of dp xh.
//
// Both passes move a few bytes for every value and compute some tens of operations on it: the memory's
// rate bounds them (16384 x 4096 with a channel gate: forward 97 us, 5.6 TB/s, backward 137 + 7, 5.9 TB/s; 1021 x 7168
// with a gate a value: 21, 30 + 5), and for one row the launch (4.0 us). As in the single norm a row lives in the registers
// of the W waves that share it, and only sums cross lanes. The two sums of squares are in 64
// bits, so that both statistics are the same fp32 numbers in whatever order they are summed, and
// products and sums are rounded one by one (no contraction), so that the stream, y and the codes do
// not hang on how the compiler pairs them.
#include "norm.h"

#include <algorithm>

#include "kernels.h"

namespace moe {

// 2^S e^c within 2 units in the last place, where that is no denormal and S is 0 or t + S exact: 2^t (1 + ln 2 d) with t = c log2 e
// as fp32 rounds it and d what that leaves out; the hardware's exp2 is good to a unit.
template <int S = 0>
__device__ inline float exp_of(float c) {
#pragma clang fp contract(off)      // t is to be the rounded one in both places
  const float t = c * 0x1.715476p+0f;
  const float d = __builtin_fmaf(c, 0x1.4ae0bep-26f, __builtin_fmaf(c, 0x1.715476p+0f, -t));
  const float e = __builtin_amdgcn_exp2f(t + (float)S);
  return __builtin_fmaf(e * d, 0x1.62e430p-1f, e);
}
// A gate's factor f in the backward pass, without branch_scale, and its slope, each within 6 units in the last place. Both are made
// of one exponential: f (1 - f) of a sigmoid and 1 - f^2 of a tanh would have few or no digits left where the gate is
// saturated. expf and a division take 13 instructions more a value, 9 us of 43 (1021 x 7168 backward, a
// gate for each value, before its rows were loaded ahead).
struct Gate {
  float f, slope;
};
// e = e^-|z|: f = 1 / (1 + e), below zero e / (1 + e), the slope e / (1 + e)^2; e below e^-87 is taken as 0
__device__ inline Gate sigmoid(float z) {
  const float x = __builtin_fabsf(z);
  float e = exp_of(-__builtin_fminf(x, 87.0f));
  e = z != z ? z : x > 87.0f ? 0.0f : e;
  const float r = __builtin_amdgcn_rcpf(1.0f + e), er = e * r;
  return {z < 0.0f ? er : r, er * r};
}
// u = e^-2|z|: f = (1 - u) / (1 + u), the slope 4 u / (1 + u)^2, taken as 0 below e^-87. Below 0.6, where 1 - u cancels, f is
// five terms of the continued fraction z / (1 + z^2 / (3 + z^2 / (5 + ...))), which leave out 1e-9 of it, and 1 - f^2 is above 0.7.
__device__ inline Gate tanh_of(float z) {
  const float x = __builtin_fabsf(z), s = z * z;
  const float u4 = x > 44.19f ? 0.0f : exp_of<2>(-2.0f * __builtin_fminf(x, 44.19f)), u = 0.25f * u4;   // t <= -1 (else small): t + 2 is exact
  const bool small = x < 0.6f;
  const float num = small ? z * __builtin_fmaf(s, s + 105.0f, 945.0f) : __builtin_copysignf(1.0f - u, z);
  const float den = small ? __builtin_fmaf(s, __builtin_fmaf(15.0f, s, 420.0f), 945.0f) : z != z ? z : 1.0f + u;
  const float r = __builtin_amdgcn_rcpf(den), f = num * r;
  return {f, small ? __builtin_fmaf(-f, f, 1.0f) : (u4 * r) * r};
}
// The forward's gate: by the math library's functions and a full division, a unit or two off. What the stream is rounded to hangs on
// it: with the functions above 40 of 7 million values (1021 x 7168) are rounded to their other neighbour, which
// the norm weight's gradient shows (3e-6 of it instead of 1e-7). They cost 1.5 of 21 us there.
__device__ inline float gate_value(int act, float z) {
  if (act == MOE_GATE_SIGMOID) return 1.0f / (1.0f + expf(-z));
  if (act == MOE_GATE_TANH) return tanhf(z);
  return z;
}
__device__ inline Gate gate_act(int act, float z) {
  if (act == MOE_GATE_SIGMOID) return sigmoid(z);
  if (act == MOE_GATE_TANH) return tanh_of(z);
  return {z, 1.0f};
}
__device__ inline float load_scalar(const void* p, bool f32, int64_t i) {
  return f32 ? static_cast<const float*>(p)[i] : bf16_lo(static_cast<const uint16_t*>(p)[i]);
}
__device__ inline uint32_t val_bytes(bool f32, int H) { return (uint32_t)H * (f32 ? 4u : 2u); }

struct SandwichArgs {
  const uint16_t* x;
  const uint16_t* res;
  const void* wp;      // null: no post-norm
  const void* w;       // null: no norm behind the addition
  const void* gate;
  int32_t w_f32, gate_f32, gate_kind, act;
  float res_scale, branch_scale;
  int32_t T, H;
  double eps1, eps2;
  uint16_t* s;
  uint16_t* y;
  float* r1;
  float* r2;
  uint8_t* q;
  void* q_s;
};

__device__ inline float inverse_rms(double ss, int H, double eps) { return (float)(1.0 / __builtin_sqrt(ss / (double)H + eps)); }

// W waves a row, W = 1: four rows a workgroup; CPL chunks of 8 values a lane. With an 8-bit output the
// rows in 16 bits pass the caches by, as in the single norm. COLS: the gate is one for each column or value. Gate and weights
// are loaded before the sums that they wait for (333 x 5120: 7.9 us without, 6.0 so), but with the widest rows, which have no
// registers for them.
template <int W, int CPL, int QF, bool COLS>
__global__ __launch_bounds__(W == 16 ? 1024 : 64 * (W == 1 ? 4 : W)) void sandwich_kernel(SandwichArgs a) {
#pragma clang fp contract(off)
  constexpr int ROWS = W == 1 ? 4 : 1;
  constexpr bool NT = QF != 0, EARLY = CPL < 4;
  __shared__ double red[2 * W];
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int sub = W == 1 ? 0 : wave;
  const int H = a.H, nch = H >> 3, words = (H + 127) >> 7;
  const int c0 = sub * (kWave * CPL) + lane;
  const uint32_t row_bytes = (uint32_t)H * 2u;
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(a.w, a.w ? val_bytes(a.w_f32, H) : 0u);
  const __amdgpu_buffer_rsrc_t wpr = make_rsrc(a.wp, a.wp ? val_bytes(a.w_f32, H) : 0u);
  int odd = 0;
  for (int64_t t = (int64_t)blockIdx.x * ROWS + (W == 1 ? wave : 0); t < a.T; t += (int64_t)gridDim.x * ROWS) {
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x + t * H, row_bytes);
    const __amdgpu_buffer_rsrc_t rr = make_rsrc(a.res ? a.res + t * H : nullptr, a.res ? row_bytes : 0u);
    u32x4 v[CPL], r[CPL];
#pragma unroll
    for (int i = 0; i < CPL; ++i) v[i] = load_row<NT>(xr, (uint32_t)(c0 + i * kWave) * 16u);
#pragma unroll
    for (int i = 0; i < CPL; ++i) r[i] = load_row<NT>(rr, (uint32_t)(c0 + i * kWave) * 16u);
    float row_f = a.branch_scale;
    if (a.gate_kind == MOE_GATE_ROW) row_f = gate_value(a.act, load_scalar(a.gate, a.gate_f32, t)) * a.branch_scale;
    const uint32_t gb = val_bytes(a.gate_f32, H);
    const __amdgpu_buffer_rsrc_t gr =
        make_rsrc(COLS ? static_cast<const char*>(a.gate) + (a.gate_kind == MOE_GATE_FULL ? t * gb : 0) : nullptr, COLS ? gb : 0u);
    Raw8 z[CPL], w[CPL];
    if constexpr (EARLY)
#pragma unroll
      for (int i = 0; i < CPL; ++i) {
        if constexpr (COLS) z[i] = load_raw(gr, a.gate_f32, c0 + i * kWave);
        w[i] = load_raw(wpr, a.w_f32, c0 + i * kWave);
      }
    float r1 = 0.f;
    if (a.wp) {
      double ss = 0.0;
#pragma unroll
      for (int i = 0; i < CPL; ++i) {
        float f[8];
        unpack8(v[i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = __builtin_fma((double)f[j], (double)f[j], ss);
      }
      ss = row_sum<W>(ss, red, sub, odd);
      odd ^= 1;
      r1 = inverse_rms(ss, H, a.eps1);
      if (a.r1 && sub == 0 && lane == 0) a.r1[t] = r1;
    }
    const __amdgpu_buffer_rsrc_t sr = make_rsrc(a.s + t * H, row_bytes);
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const int c = c0 + i * kWave;
      if constexpr (!EARLY) {
        if constexpr (COLS) z[i] = load_raw(gr, a.gate_f32, c);
        w[i] = load_raw(wpr, a.w_f32, c);
      }
      float p[8], b[8];
      unpack8(v[i], p);
      unpack8(r[i], b);
      if (a.wp) {
        float wf[8];
        unpack_raw(w[i], a.w_f32, wf);
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = (p[j] * r1) * wf[j];
      }
      if constexpr (COLS) {
        float zf[8];
        unpack_raw(z[i], a.gate_f32, zf);
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = p[j] * (gate_value(a.act, zf[j]) * a.branch_scale);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = p[j] * row_f;
      }
      if (a.res) {
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = b[j] * a.res_scale + p[j];
      }
      v[i] = pack8(p);
      store_row<NT>(v[i], sr, (uint32_t)c * 16u);
      if (c < nch) {       // chunks past the row: a gate of theirs may have made anything of their zeros
        unpack8(v[i], p);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = __builtin_fma((double)p[j], (double)p[j], ss);
      }
    }
    if (!a.w) continue;
    if constexpr (EARLY)
#pragma unroll
      for (int i = 0; i < CPL; ++i) w[i] = load_raw(wr, a.w_f32, c0 + i * kWave);
    ss = row_sum<W>(ss, red, sub, odd);
    odd ^= 1;
    const float r2 = inverse_rms(ss, H, a.eps2);
    if (a.r2 && sub == 0 && lane == 0) a.r2[t] = r2;
    const __amdgpu_buffer_rsrc_t yr = make_rsrc(a.y ? a.y + t * H : nullptr, a.y ? row_bytes : 0u);
    const __amdgpu_buffer_rsrc_t qr = make_rsrc(QF ? a.q + t * H : nullptr, QF ? (uint32_t)H : 0u);
    uint8_t* q_s = static_cast<uint8_t*>(a.q_s) + t * words * 4;
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const int c = c0 + i * kWave;
      if constexpr (!EARLY) w[i] = load_raw(wr, a.w_f32, c);
      float f[8], wf[8];
      unpack8(v[i], f);
      unpack_raw(w[i], a.w_f32, wf);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = (f[j] * r2) * wf[j];
      u32x4 o = pack8(f);
      if (QF == 2 && c >= nch) o = u32x4{0u, 0u, 0u, 0u};
      store_row<NT>(o, yr, (uint32_t)c * 16u);
      if constexpr (QF != 0) store_quantised<QF>(o, c, nch, words, qr, q_s);
    }
  }
}

// ---------------------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------------------
struct SandwichBwdArgs {
  const uint16_t* dy;
  const uint16_t* d_s;
  const uint16_t* x;
  const uint16_t* s;
  const void* wp;
  const void* w;
  const void* gate;
  int32_t w_f32, gate_f32, gate_kind, act;
  float res_scale, branch_scale;
  const float* r1;
  const float* r2;
  int32_t T, H;
  uint16_t* dx;
  uint16_t* d_res;
  void* d_gate;          // row and full: in the gate's type (channel: through part_gate)
  float* part_w;         // [gridDim.x][H] partial sums of dw, dwp and d_gate, or null
  float* part_wp;
  float* part_gate;
};

// value j of 8 bf16 values
__device__ inline float value(u32x4 v, int j) { return j & 1 ? bf16_hi(v[j >> 1]) : bf16_lo(v[j >> 1]); }

// three sums over a row at once
template <int W>
__device__ inline void row_sum3(float (&v)[3], float* red, int sub, int odd) {
#pragma unroll
  for (int k = 0; k < 3; ++k) v[k] = wave_sum(v[k]);
  if constexpr (W > 1) {
    float* r = red + odd * 3 * W;
    if (lane_id() == 0) {
#pragma unroll
      for (int k = 0; k < 3; ++k) r[sub * 3 + k] = v[k];
    }
    __syncthreads();
    // a wave's sum a lane, and 16 lanes' by rotations: read one after another by every lane, 16 waves' would take 48 registers
    const int w = lane_id() & 15;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      float s = w < W ? r[w * 3 + k] : 0.f;
      s = row_add<0x128>(s);
      s = row_add<0x124>(s);
      s = row_add<0x122>(s);
      v[k] = row_add<0x121>(s);
    }
  }
}

// A row's two means need one exchange: with k = p f (its column sums over the row) the second mean is linear in
// the first, mean(dp wp xh) = (sum k (d_s + r2 g) - r2 mean(g xs) sum k xs) / H. GK: 0 no gate or one a row (k = p:
// f leaves the sums), 1 a gate for each column, 2 (bf16) and 3 (fp32) for each value.
template <int W, int CPL, bool POST, int GK>
__global__ __launch_bounds__(W == 16 ? 1024 : 64 * (W == 1 ? 4 : W)) void sandwich_backward_kernel(SandwichBwdArgs a) {
  constexpr int ROWS = W == 1 ? 4 : 1;
  constexpr bool HELD = CPL == 1;         // weights, a channel gate and rows stay in registers
  // The next row is loaded while one is worked on where a CU has but one workgroup (8192 x 7168, a gate a value, both
  // launches: 188 us with, 191 without; 1021 rows, four a workgroup with the last loaded once more, 36.1 and 35.0). With workgroups of 8
  // waves it costs (16384 x 4096: 154 with, 149 without).
  constexpr bool AHEAD = HELD && W == 16;
  constexpr int NACC = 1 + (POST ? 1 : 0) + (GK == 1 ? 1 : 0);
  __shared__ float red[2 * 3 * W];
  __shared__ float s_acc[W == 1 ? 3 : 1][W == 1 ? 64 * 8 : 1];
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int sub = W == 1 ? 0 : wave;
  const int H = a.H;
  const int c0 = sub * (kWave * CPL) + lane;
  const uint32_t row_bytes = (uint32_t)H * 2u;
  const bool pre = a.w != nullptr;
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(a.w, pre ? val_bytes(a.w_f32, H) : 0u);
  const __amdgpu_buffer_rsrc_t wpr = make_rsrc(a.wp, POST ? val_bytes(a.w_f32, H) : 0u);
  const uint32_t gb = val_bytes(a.gate_f32, H);
  float acc[NACC][CPL][8];
  constexpr int AW = 0, AP = 1, AG = POST ? 2 : 1;
#pragma unroll
  for (int k = 0; k < NACC; ++k)
#pragma unroll
    for (int i = 0; i < CPL; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[k][i][j] = 0.f;
  float w[8], wp[8], z[8], slope[8];
  const __amdgpu_buffer_rsrc_t gcr = make_rsrc(GK == 1 ? a.gate : nullptr, GK == 1 ? gb : 0u);
  const auto weights = [&](int c) {
    load_weight(wr, a.w_f32, c, w);
    if constexpr (POST) load_weight(wpr, a.w_f32, c, wp);
  };
  const auto channel = [&](int c) {
    if constexpr (GK == 1) {
      load_weight(gcr, a.gate_f32, c, z);
#pragma unroll
      for (int j = 0; j < 8; ++j) z[j] = gate_act(a.act, z[j]).f;
    }
  };
  if constexpr (HELD) {
    channel(c0);
    weights(c0);
  }
  struct Chunk {
    u32x4 d, e, x, s;
    Raw8 z;
  };
  struct Stats {
    float r1, r2, z;
  };
  const auto load = [&](int64_t t, int c) {
    const auto row = [&](const uint16_t* p) { return make_rsrc(p ? p + t * H : nullptr, p ? row_bytes : 0u); };
    const uint32_t o = (uint32_t)c * 16u;
    Chunk k;
    k.d = load_row<HELD>(row(a.dy), o);
    k.e = load_row<HELD>(row(a.d_s), o);
    k.x = load_row<HELD>(row(a.x), o);
    k.s = load_row<HELD>(row(a.s), o);
    if constexpr (GK >= 2) k.z = load_raw(make_rsrc(static_cast<const char*>(a.gate) + t * gb, gb), GK == 3, c);
    return k;
  };
  const auto stats = [&](int64_t t) {
    Stats r = {0.f, 0.f, 1.f};
    if (pre) r.r2 = a.r2[t];
    if (POST) r.r1 = a.r1[t];
    if (GK == 0 && a.gate_kind == MOE_GATE_ROW) r.z = load_scalar(a.gate, a.gate_f32, t);
    return r;
  };
  // the gate of a chunk's values, and its slopes
  const auto gates = [&](const Chunk& k) {
    if constexpr (GK >= 2) {
      unpack_raw(k.z, GK == 3, z);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const Gate g = gate_act(a.act, z[j]);
        z[j] = g.f;
        slope[j] = g.slope;
      }
    }
  };
  int odd = 0;
  const int64_t stride = (int64_t)gridDim.x * ROWS;
  int64_t t = blockIdx.x + (W == 1 ? (int64_t)wave * gridDim.x : 0);
  Chunk next;
  Stats st;
  if constexpr (AHEAD) {
    next = load(t, c0);
    st = stats(t);
  }
  for (; t < a.T; t += stride) {
    Chunk cur, ahead;
    Stats now;
    if constexpr (AHEAD) {
      cur = next;
      // Behind the last row the last once more. (With a range of no bytes chosen there, t < T ? gb : 0, the compiler took
      // the choice from the carry of the address's addition, and gates were read from past their end.)
      const int64_t tn = min(t + stride, (int64_t)a.T - 1);
      ahead = load(tn, c0);
      now = st;
      st = stats(tn);
    } else {
      if constexpr (HELD) cur = load(t, c0);
      now = stats(t);
    }
    const float r1 = now.r1, r2 = now.r2;
    Gate row = {1.f, 0.f};
    if (GK == 0 && a.gate_kind == MOE_GATE_ROW) row = gate_act(a.act, now.z);
    const float zr = row.f;
    float sum[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const int c = c0 + i * kWave;
      if constexpr (!HELD) {
        cur = load(t, c);
        channel(c);
        weights(c);
      }
      gates(cur);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = value(cur.d, j), e = value(cur.e, j), x = value(cur.x, j), s = value(cur.s, j);
        float k = x;
        if constexpr (POST) k = (x * r1) * wp[j];
        if constexpr (GK != 0) k *= z[j];
        float de = e;
        if (pre) {
          const float xs = s * r2, dxs = d * xs;
          acc[AW][i][j] += dxs;
          sum[0] += dxs * w[j];
          sum[2] += k * xs;
          de += r2 * (d * w[j]);
        }
        sum[1] += k * de;
      }
    }
    row_sum3<W>(sum, red, sub, odd);
    odd ^= 1;
    const float c2 = sum[0] / (float)H;
    const float kds = sum[1] - (r2 * c2) * sum[2];       // of ds with p, times the gate where that is not one a row
    const float c1 = a.branch_scale * (GK == 0 ? zr : 1.f) * kds / (float)H;
    if (GK == 0 && a.gate_kind == MOE_GATE_ROW && a.d_gate && sub == 0 && lane == 0) {
      const float dg = a.branch_scale * row.slope * kds;
      if (a.gate_f32) static_cast<float*>(a.d_gate)[t] = dg;
      else static_cast<uint16_t*>(a.d_gate)[t] = (uint16_t)pack_bf16x2(dg, 0.f);
    }
    const __amdgpu_buffer_rsrc_t dxr = make_rsrc(a.dx + t * H, row_bytes);
    const __amdgpu_buffer_rsrc_t drr = make_rsrc(a.d_res ? a.d_res + t * H : nullptr, a.d_res ? row_bytes : 0u);
    const bool write_gate = GK >= 2 && a.d_gate;
    const __amdgpu_buffer_rsrc_t dgr =
        make_rsrc(write_gate ? static_cast<char*>(a.d_gate) + t * gb : nullptr, write_gate ? gb : 0u);
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const int c = c0 + i * kWave;
      if constexpr (!HELD) {
        cur = load(t, c);
        channel(c);
        weights(c);
        gates(cur);
      } else {
        // unpacked anew: what the first pass unpacked would not fit the registers
        asm volatile("" : "+v"(cur.d), "+v"(cur.e), "+v"(cur.x), "+v"(cur.s));
      }
      u32x4 o, ro, dg;
      float odd_o = 0.f, odd_r = 0.f, odd_g = 0.f;      // values that wait for their neighbours
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = value(cur.d, j), e = value(cur.e, j), x = value(cur.x, j), s = value(cur.s, j);
        float ds = e;
        if (pre) ds += r2 * (d * w[j] - (s * r2) * c2);
        const float r = a.res_scale * ds;
        const float f = a.branch_scale * (GK == 0 ? zr : z[j]);
        const float dp = f * ds;
        const float xh = POST ? x * r1 : x;
        float g = 0.f, v = dp;
        if constexpr (GK != 0) {
          const float p = POST ? xh * wp[j] : xh;
          if constexpr (GK == 1) acc[AG][i][j] += ds * p;
          else g = a.branch_scale * slope[j] * ds * p;
        }
        if constexpr (POST) {
          acc[AP][i][j] += dp * xh;
          v = r1 * (dp * wp[j] - xh * c1);
        }
        if (j & 1) {
          o[j >> 1] = pack_bf16x2(odd_o, v);
          ro[j >> 1] = pack_bf16x2(odd_r, r);
          if constexpr (GK == 2) dg[j >> 1] = pack_bf16x2(odd_g, g);
        } else {
          odd_o = v;
          odd_r = r;
          odd_g = g;
        }
        if constexpr (GK == 3) {
          dg[j & 3] = __builtin_bit_cast(uint32_t, g);
          if ((j & 3) == 3) store_row<true>(dg, dgr, (uint32_t)c * 32u + (j >> 2) * 16u);
        }
      }
      store_row<true>(o, dxr, (uint32_t)c * 16u);
      store_row<true>(ro, drr, (uint32_t)c * 16u);
      if constexpr (GK == 2) store_row<true>(dg, dgr, (uint32_t)c * 16u);
    }
    if constexpr (AHEAD) next = ahead;
  }
  // a channel's slope is the same for all rows
  if constexpr (GK == 1) {
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      load_weight(gcr, a.gate_f32, c0 + i * kWave, z);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[AG][i][j] *= a.branch_scale * gate_act(a.act, z[j]).slope;
    }
  }
  float* const parts[3] = {a.part_w, POST ? a.part_wp : a.part_gate, a.part_gate};
#pragma unroll
  for (int k = 0; k < NACC; ++k) {
    if (!parts[k]) continue;
    if constexpr (W == 1) {              // four waves' sums joined before they are written
      __syncthreads();
      if (wave > 0)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          s_acc[wave - 1][j * 64 + lane] = acc[k][0][j];
      __syncthreads();
      if (wave > 0) continue;
#pragma unroll
      for (int v = 0; v < 3; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[k][0][j] += s_acc[v][j * 64 + lane];
    }
    const __amdgpu_buffer_rsrc_t pr = make_rsrc(parts[k] + (int64_t)blockIdx.x * H, (uint32_t)H * 4u);
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const uint32_t o = (uint32_t)(c0 + i * kWave) * 32u;
      u32x4 p, q;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        p[j] = __builtin_bit_cast(uint32_t, acc[k][i][j]);
        q[j] = __builtin_bit_cast(uint32_t, acc[k][i][4 + j]);
      }
      buf_store16(p, pr, o);
      buf_store16(q, pr, o + 16u);
    }
  }
}

struct ColumnSums {
  const float* part[3];
  float* out[3];
  int32_t n, H;
};
// out[h] = sum of the n partial rows, always in the same order; as the single norm's (32 columns a workgroup)
__global__ __launch_bounds__(1024) void sandwich_columns_kernel(ColumnSums a) {
  typedef float f32x4 __attribute__((ext_vector_type(4)));
  __shared__ f32x4 red[16][8];
  const float* part = a.part[blockIdx.y];
  const int lane = lane_id(), wave = threadIdx.x >> 6;
  const int c = lane & 7, r = lane >> 3;
  const int h = blockIdx.x * 32 + c * 4;   // H % 8 == 0: four columns are in or out together
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  if (h < a.H)
#pragma unroll 8
    for (int i = wave * 8 + r; i < a.n; i += 128) v += *reinterpret_cast<const f32x4*>(part + (int64_t)i * a.H + h);
#pragma unroll
  for (int o = 8; o < 64; o *= 2)
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] += __shfl_xor(v[j], o, 64);
  if (r == 0) red[wave][c] = v;
  __syncthreads();
  if (wave == 0 && r == 0 && h < a.H) {
#pragma unroll
    for (int i = 1; i < 16; ++i) v += red[i][c];
#pragma unroll
    for (int j = 0; j < 4; ++j) a.out[blockIdx.y][h + j] = v[j];
  }
}

// ---------------------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------------------
constexpr int kSandwichMaxBlocks = 1 << 16;

template <int W, int CPL>
static void launch_q(int qf, int64_t rows, hipStream_t s, const SandwichArgs& a) {
  const dim3 block(64 * (W == 1 ? 4 : W));
  const dim3 grid((unsigned)std::min<int64_t>((rows + (W == 1 ? 3 : 0)) / (W == 1 ? 4 : 1), kSandwichMaxBlocks));
  if (a.gate_kind == MOE_GATE_CHANNEL || a.gate_kind == MOE_GATE_FULL) {
    if (qf == 1) hipLaunchKernelGGL((sandwich_kernel<W, CPL, 1, true>), grid, block, 0, s, a);
    else if (qf == 2) hipLaunchKernelGGL((sandwich_kernel<W, CPL, 2, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((sandwich_kernel<W, CPL, 0, true>), grid, block, 0, s, a);
  } else {
    if (qf == 1) hipLaunchKernelGGL((sandwich_kernel<W, CPL, 1, false>), grid, block, 0, s, a);
    else if (qf == 2) hipLaunchKernelGGL((sandwich_kernel<W, CPL, 2, false>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((sandwich_kernel<W, CPL, 0, false>), grid, block, 0, s, a);
  }
}

int launch_sandwich_norm(const SandwichLaunch& l, hipStream_t stream) {
  SandwichArgs a;
  a.x = static_cast<const uint16_t*>(l.x);
  a.res = static_cast<const uint16_t*>(l.res);
  a.wp = l.post_weight;
  a.w = l.weight;
  a.gate = l.gate;
  a.w_f32 = l.w_f32;
  a.gate_f32 = l.cfg.gate_dtype == MOE_F32;
  a.gate_kind = l.cfg.gate;
  a.act = l.cfg.gate_act;
  a.res_scale = l.cfg.res_scale;
  a.branch_scale = l.cfg.branch_scale;
  a.T = l.T;
  a.H = l.H;
  a.eps1 = l.cfg.post_eps;
  a.eps2 = l.cfg.eps;
  a.s = static_cast<uint16_t*>(l.s);
  a.y = static_cast<uint16_t*>(l.y);
  a.r1 = l.post_rstd;
  a.r2 = l.rstd;
  a.q = static_cast<uint8_t*>(l.q);
  a.q_s = l.q_s;
  const int qf = l.q_dtype == MOE_FP8_E4M3_G128 ? 1 : l.q_dtype == MOE_MXFP4 ? 2 : 0;
  const int nch = ((l.H + 127) / 128) * 16;   // chunks, the last scale word's whole
  if (nch <= 64) launch_q<1, 1>(qf, l.T, stream, a);
  else if (nch <= 128) launch_q<1, 2>(qf, l.T, stream, a);
  else if (nch <= 256) launch_q<4, 1>(qf, l.T, stream, a);
  else if (nch <= 512) launch_q<4, 2>(qf, l.T, stream, a);
  else if (nch <= 1024) launch_q<8, 2>(qf, l.T, stream, a);
  else if (nch <= 2048) launch_q<16, 2>(qf, l.T, stream, a);
  else launch_q<16, 4>(qf, l.T, stream, a);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

// Waves that share a row of the backward pass, and its workgroups (4096 waves, 16 a CU): rows of
// partial sums that the workspace holds. Both depend on T and H alone, and so does the order of the sums.
static int backward_waves(int32_t H) {
  const int nch = H / 8;
  return nch <= 64 ? 1 : nch <= 256 ? 4 : nch <= 512 ? 8 : 16;
}
int32_t sandwich_backward_blocks(int32_t T, int32_t H) { return std::min(T, 4096 / std::max(4, backward_waves(H))); }

template <bool POST, int GK>
static void launch_backward(const SandwichBwdArgs& a, int n, hipStream_t s) {
  const int nch = a.H / 8;
  const dim3 grid(n);
  if (nch <= 64) hipLaunchKernelGGL((sandwich_backward_kernel<1, 1, POST, GK>), grid, dim3(256), 0, s, a);
  else if (nch <= 256) hipLaunchKernelGGL((sandwich_backward_kernel<4, 1, POST, GK>), grid, dim3(256), 0, s, a);
  else if (nch <= 512) hipLaunchKernelGGL((sandwich_backward_kernel<8, 1, POST, GK>), grid, dim3(512), 0, s, a);
  else if (nch <= 1024) hipLaunchKernelGGL((sandwich_backward_kernel<16, 1, POST, GK>), grid, dim3(1024), 0, s, a);
  else if (nch <= 2048) hipLaunchKernelGGL((sandwich_backward_kernel<16, 2, POST, GK>), grid, dim3(1024), 0, s, a);
  else hipLaunchKernelGGL((sandwich_backward_kernel<16, 4, POST, GK>), grid, dim3(1024), 0, s, a);
}

template <bool POST>
static void launch_backward(const SandwichBwdArgs& a, int gk, int n, hipStream_t s) {
  if (gk == 1) launch_backward<POST, 1>(a, n, s);
  else if (gk == 2) launch_backward<POST, 2>(a, n, s);
  else if (gk == 3) launch_backward<POST, 3>(a, n, s);
  else launch_backward<POST, 0>(a, n, s);
}

int launch_sandwich_norm_backward(const SandwichBwdLaunch& l, hipStream_t stream) {
  SandwichBwdArgs a;
  a.dy = static_cast<const uint16_t*>(l.dy);
  a.d_s = static_cast<const uint16_t*>(l.d_s);
  a.x = static_cast<const uint16_t*>(l.x);
  a.s = static_cast<const uint16_t*>(l.s);
  a.wp = l.post_weight;
  a.w = l.weight;
  a.gate = l.gate;
  a.w_f32 = l.w_f32;
  a.gate_f32 = l.cfg.gate_dtype == MOE_F32;
  a.gate_kind = l.cfg.gate;
  a.act = l.cfg.gate_act;
  a.res_scale = l.cfg.res_scale;
  a.branch_scale = l.cfg.branch_scale;
  a.r1 = l.post_rstd;
  a.r2 = l.rstd;
  a.T = l.T;
  a.H = l.H;
  a.dx = static_cast<uint16_t*>(l.dx);
  a.d_res = static_cast<uint16_t*>(l.d_res);
  const bool channel = l.cfg.gate == MOE_GATE_CHANNEL;
  a.d_gate = channel ? nullptr : l.d_gate;
  const int n = l.T > 0 ? sandwich_backward_blocks(l.T, l.H) : 0;
  // the sums over rows that the caller wants, their partial rows one array behind another
  ColumnSums c{};
  c.n = n;
  c.H = l.H;
  int arrays = 0;
  const auto sums = [&](void* out) -> float* {
    if (!out) return nullptr;
    float* part = static_cast<float*>(l.ws) + (int64_t)arrays * n * l.H;
    c.part[arrays] = part;
    c.out[arrays++] = static_cast<float*>(out);
    return part;
  };
  a.part_w = sums(l.dweight);
  a.part_wp = sums(l.d_post_weight);
  a.part_gate = channel ? sums(l.d_gate) : nullptr;
  if (n > 0) {
    const int gk = channel ? 1 : l.cfg.gate == MOE_GATE_FULL ? (a.gate_f32 ? 3 : 2) : 0;
    if (a.wp) launch_backward<true>(a, gk, n, stream);
    else launch_backward<false>(a, gk, n, stream);
    if (hipGetLastError() != hipSuccess) return MOE_ERR_HIP;
  }
  if (arrays > 0) {
    hipLaunchKernelGGL(sandwich_columns_kernel, dim3((l.H + 31) / 32, arrays), dim3(1024), 0, stream, c);
    if (hipGetLastError() != hipSuccess) return MOE_ERR_HIP;
  }
  return MOE_OK;
}

}  // namespace moe
