// What the norm kernels share: sums over the waves of a row, 8 consecutive values, and the 8-bit
// copy of a row in the layer's activation formats.
#pragma once

#include "common.h"

namespace moe {

// ---------------------------------------------------------------------------------------
// sums over a wave, and over the W waves that share a row
// ---------------------------------------------------------------------------------------
template <int CTRL>
__device__ inline float row_add(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
}
template <int CTRL>
__device__ inline double row_add(double v) {
  const u32x2 b = __builtin_bit_cast(u32x2, v);
  const u32x2 r = {(uint32_t)__builtin_amdgcn_update_dpp(0, (int)b.x, CTRL, 0xf, 0xf, false),
                   (uint32_t)__builtin_amdgcn_update_dpp(0, (int)b.y, CTRL, 0xf, 0xf, false)};
  return v + __builtin_bit_cast(double, r);
}
__device__ inline float lane_value(float v, int lane) {
  return __builtin_bit_cast(float, readlane(__builtin_bit_cast(int, v), lane));
}
__device__ inline double lane_value(double v, int lane) {
  const u32x2 b = __builtin_bit_cast(u32x2, v);
  return __builtin_bit_cast(double, u32x2{(uint32_t)readlane((int)b.x, lane), (uint32_t)readlane((int)b.y, lane)});
}
// rotations inside the 16-lane rows, then the four rows' sums by readlane: every lane gets it
template <typename F>
__device__ inline F wave_sum(F v) {
  v = row_add<0x128>(v);
  v = row_add<0x124>(v);
  v = row_add<0x122>(v);
  v = row_add<0x121>(v);
  return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}
// `red` holds W values of two consecutive rows (parity `odd`), so that one barrier a row is enough
template <int W, typename F>
__device__ inline F row_sum(F v, F* red, int sub, int odd) {
  v = wave_sum(v);
  if constexpr (W > 1) {
    F* r = red + odd * W;
    if (lane_id() == 0) r[sub] = v;
    __syncthreads();
    v = r[0];
#pragma unroll
    for (int i = 1; i < W; ++i) v += r[i];
  }
  return v;
}

// ---------------------------------------------------------------------------------------
// 8 consecutive values
// ---------------------------------------------------------------------------------------
__device__ inline void unpack8(u32x4 v, float (&f)[8]) {
  f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x);
  f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
  f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z);
  f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
}
__device__ inline u32x4 pack8(const float (&f)[8]) {
  return u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
}
// 8 values, bf16 or fp32, as they are loaded (the second half for fp32 alone) ...
struct Raw8 {
  u32x4 lo, hi;
};
__device__ inline Raw8 load_raw(__amdgpu_buffer_rsrc_t r, bool f32, int c) {
  Raw8 v;
  v.lo = buf_load16(r, (uint32_t)c * (f32 ? 32u : 16u));
  if (f32) v.hi = buf_load16(r, (uint32_t)c * 32u + 16u);
  return v;
}
// ... and what they are
__device__ inline void unpack_raw(const Raw8& v, bool f32, float (&w)[8]) {
  if (f32) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = v.lo[j], hi = v.hi[j];   // a bit cast of a vector's element would take its first
      w[j] = __builtin_bit_cast(float, lo);
      w[4 + j] = __builtin_bit_cast(float, hi);
    }
  } else {
    unpack8(v.lo, w);
  }
}
// the norm's weight, bf16 or fp32 (chunks past the row read as 0)
__device__ inline void load_weight(__amdgpu_buffer_rsrc_t r, bool f32, int c, float (&w)[8]) {
  unpack_raw(load_raw(r, f32, c), f32, w);
}

__device__ inline uint32_t umax_dpp(uint32_t v, uint32_t o) { return v > o ? v : o; }
template <int CTRL>
__device__ inline uint32_t row_umax(uint32_t v) {
  return umax_dpp(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false));
}

// NT: with the non-temporal cache policy, for rows that are not read again soon
template <bool NT>
__device__ inline u32x4 load_row(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return NT ? buf_load16_nt(r, off) : buf_load16(r, off);
}
template <bool NT>
__device__ inline void store_row(u32x4 v, __amdgpu_buffer_rsrc_t r, uint32_t off) {
  __builtin_amdgcn_raw_buffer_store_b128(v, r, off, 0, NT ? 2 : 0);
}

// v = f / sc, rounded as IEEE division rounds it. With the correctly rounded reciprocal i, f * i is
// within a unit of the quotient, the fused remainder f - (f * i) * sc is exact and the corrected
// quotient rounds right (Markstein's theorem); what could underflow on the way (`plain` false:
// sc below 2^-99) is divided in full. The remainder is taken with its sign turned, so that a zero's correction is a zero of
// its own sign and -0 stays -0.
__device__ inline void divide8(const float (&f)[8], float sc, bool plain, float (&v)[8]) {
  if (plain) {
    const float i = 1.0f / sc;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float q = f[j] * i;
      v[j] = __builtin_fmaf(-__builtin_fmaf(q, sc, -f[j]), i, q);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = f[j] / sc;
  }
}

// QF: 0 none, 1 fp8 (1x128 groups), 2 MXFP8 (1x32 blocks); formats and rounding as in dispatch.
// The group's largest magnitude is taken over bit patterns: those of NaN and infinity are the
// largest, so a group that holds one shows it.
template <int QF>
__device__ inline void store_quantised(u32x4 v, int c, int nch, int words, __amdgpu_buffer_rsrc_t qr, uint8_t* q_s) {
  float f[8];
  unpack8(v, f);
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = umax_dpp(m, __builtin_bit_cast(uint32_t, f[j]) & 0x7fffffffu);
  const int lane = lane_id();
  u32x2 q;
  if constexpr (QF == 1) {
    m = row_umax<0x128>(m);
    m = row_umax<0x124>(m);
    m = row_umax<0x122>(m);
    m = row_umax<0x121>(m);
    const bool bad = m >= 0x7f800000u;
    const float amax = __builtin_bit_cast(float, m);
    const float sc = amax > 0.f ? amax / 448.0f : 1.0f;
    float v[8];
    divide8(f, sc, amax >= 0x1p-90f, v);
    q.x = pack_e4m3x4(v[0], v[1], v[2], v[3]);
    q.y = pack_e4m3x4(v[4], v[5], v[6], v[7]);
    if (bad) q = u32x2{0u, 0u};
    buf_store8(q, qr, (uint32_t)c * 8u);
    if ((lane & 15) == 0 && c < nch)
      reinterpret_cast<uint32_t*>(q_s)[c >> 4] = bad ? 0x7fc00000u : __builtin_bit_cast(uint32_t, sc);
  } else {
    m = row_umax<0xB1>(m);   // quad_perm [1,0,3,2], then [2,3,0,1]: the 4 lanes that hold a block
    m = row_umax<0x4E>(m);
    const bool bad = m >= 0x7f800000u;
    const int e = mx_e4m3_shared_exp(__builtin_bit_cast(float, m));
    const float inv = mx_inv_scale(e);
    q.x = pack_e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
    q.y = pack_e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv);
    if (bad) q = u32x2{0u, 0u};
    buf_store8(q, qr, (uint32_t)c * 8u);
    // blocks of the last word that the row does not have (zeros here): byte 0
    if ((lane & 3) == 0 && c < words * 16) q_s[c >> 2] = (uint8_t)(c >= nch ? 0 : bad ? 255 : e + 127);
  }
}

}  // namespace moe
