// RMS norm with the residual's addition and an 8-bit output, and its backward pass.
//
//   s = bf16(x + res), rstd = fp32(1 / sqrt(mean(s^2) + eps)), y = bf16((s * rstd) * w),
//   (q, q_s) = y in the layer's fp8 or MXFP8 activation format;
//   backward: g = dy w, xhat = s rstd, dx = rstd (g - xhat mean(g xhat)) + d_res,
//   dweight = sum over rows of dy xhat.
//
// Both passes move a few bytes for every value and compute about ten operations on it: the
// memory's rate bounds them, and for one row the launch. A row lives in the registers of the
// waves that share it (W of them, CPL chunks of 8 values a lane): it is read once, and nothing
// but the row's sum crosses lanes.
//
// The sum of squares and the root are in 64 bits: the squares of bf16 values and their sums
// are then exact enough that rstd is the same fp32 number in whatever order they are summed,
// and with it y, the scales and the codes are, to the last bit, functions of the inputs alone
// (W, CPL and the plain formula agree). It costs two 64-bit operations a value, hidden behind
// the loads.
#include "norm.h"

#include <algorithm>

#include "kernels.h"

namespace moe {

struct NormArgs {
  const uint16_t* x;
  const uint16_t* res;
  const void* w;
  int32_t w_f32;
  int32_t T, H;
  double eps;
  uint16_t* s_out;
  uint16_t* y;
  float* rstd;
  uint8_t* q;
  void* q_s;
};

// W waves a row, W = 1: four rows a workgroup. With an 8-bit output, the codes are what the next
// kernel reads: x, res, s_out and y pass the caches by (norm, plan and dispatch of 8192 x 4096 fp8 rows:
// 223 us without, 186 with; 2048: 81.6 and 77.0; 256: no difference). Without one, y is read next.
template <int W, int CPL, int QF>
__global__ __launch_bounds__(W == 16 ? 1024 : 256) void rmsnorm_kernel(NormArgs a) {
  constexpr int ROWS = W == 1 ? 4 : 1;
  constexpr bool NT = QF != 0;
  __shared__ double red[2 * W];
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int sub = W == 1 ? 0 : wave;
  const int H = a.H, nch = H >> 3, words = (H + 127) >> 7;
  const int c0 = sub * (kWave * CPL) + lane;
  const uint32_t row_bytes = (uint32_t)H * 2u;
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(a.w, a.w_f32 ? (uint32_t)H * 4u : row_bytes);
  int odd = 0;
  for (int64_t t = (int64_t)blockIdx.x * ROWS + (W == 1 ? wave : 0); t < a.T; t += (int64_t)gridDim.x * ROWS) {
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x + t * H, row_bytes);
    u32x4 v[CPL];
#pragma unroll
    for (int i = 0; i < CPL; ++i) v[i] = load_row<NT>(xr, (uint32_t)(c0 + i * kWave) * 16u);
    if (a.res) {
      const __amdgpu_buffer_rsrc_t rr = make_rsrc(a.res + t * H, row_bytes);
      u32x4 r[CPL];
#pragma unroll
      for (int i = 0; i < CPL; ++i) r[i] = load_row<NT>(rr, (uint32_t)(c0 + i * kWave) * 16u);
#pragma unroll
      for (int i = 0; i < CPL; ++i) {
        float f[8], g[8];
        unpack8(v[i], f);
        unpack8(r[i], g);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] += g[j];
        v[i] = pack8(f);
      }
      if (a.s_out) {
        const __amdgpu_buffer_rsrc_t sr = make_rsrc(a.s_out + t * H, row_bytes);
#pragma unroll
        for (int i = 0; i < CPL; ++i) store_row<NT>(v[i], sr, (uint32_t)(c0 + i * kWave) * 16u);
      }
    }
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
    const float rstd = (float)(1.0 / __builtin_sqrt(ss / (double)H + a.eps));
    if (a.rstd && sub == 0 && lane == 0) a.rstd[t] = rstd;
    const __amdgpu_buffer_rsrc_t yr = make_rsrc(a.y ? a.y + t * H : nullptr, a.y ? row_bytes : 0u);
    const __amdgpu_buffer_rsrc_t qr = make_rsrc(QF ? a.q + t * H : nullptr, QF ? (uint32_t)H : 0u);
    uint8_t* q_s = static_cast<uint8_t*>(a.q_s) + t * words * 4;
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const int c = c0 + i * kWave;
      float f[8], w[8];
      unpack8(v[i], f);
      load_weight(wr, a.w_f32, c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = (f[j] * rstd) * w[j];
      const u32x4 o = pack8(f);
      store_row<NT>(o, yr, (uint32_t)c * 16u);
      if constexpr (QF != 0) store_quantised<QF>(o, c, nch, words, qr, q_s);
    }
  }
}

// ---------------------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------------------
struct NormBwdArgs {
  const uint16_t* dy;
  const uint16_t* s;
  const void* w;
  int32_t w_f32;
  const float* rstd;
  const uint16_t* d_res;
  int32_t T, H;
  uint16_t* dx;
  float* part;   // [gridDim.x][H] partial sums of dweight, or null
};

// One row at a time by the W waves of a workgroup (W = 1: four, by a wave each); dweight's sums of the
// lane's columns stay in its registers over all of the workgroup's rows, and four waves' are
// added before they are written (4333 x 472: 8.2 us and 11.3 for dweight with a partial row a wave, 4.5 and 4.8 so).
template <int W, int CPL>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void rmsnorm_backward_kernel(NormBwdArgs a) {
  constexpr int ROWS = W == 1 ? 4 : 1;
  __shared__ float red[2 * W];
  __shared__ float s_dw[W == 1 ? 3 : 1][W == 1 ? 64 * 8 : 1];
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int sub = W == 1 ? 0 : wave;
  const int H = a.H;
  const int c0 = sub * (kWave * CPL) + lane;
  const uint32_t row_bytes = (uint32_t)H * 2u;
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(a.w, a.w_f32 ? (uint32_t)H * 4u : row_bytes);
  // the weight stays in registers too, except with the widest rows, which have none left for it
  // (1024 x 32768: 155 us with it, 61 so; 12 registers are spilled even so)
  constexpr bool HELD = CPL < 4;
  float w[HELD ? CPL : 1][8], dw[CPL][8];
#pragma unroll
  for (int i = 0; i < CPL; ++i) {
    if constexpr (HELD) load_weight(wr, a.w_f32, c0 + i * kWave, w[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
  }
  int odd = 0;
  for (int64_t t = blockIdx.x + (W == 1 ? (int64_t)wave * gridDim.x : 0); t < a.T; t += (int64_t)gridDim.x * ROWS) {
    const __amdgpu_buffer_rsrc_t dr = make_rsrc(a.dy + t * H, row_bytes);
    const __amdgpu_buffer_rsrc_t sr = make_rsrc(a.s + t * H, row_bytes);
    const __amdgpu_buffer_rsrc_t rr = make_rsrc(a.d_res ? a.d_res + t * H : nullptr, a.d_res ? row_bytes : 0u);
    u32x4 vd[CPL], vs[CPL], vr[CPL];
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const uint32_t o = (uint32_t)(c0 + i * kWave) * 16u;
      vd[i] = buf_load16_nt(dr, o);
      vs[i] = buf_load16_nt(sr, o);
      if constexpr (HELD) vr[i] = buf_load16_nt(rr, o);
    }
    const float rstd = a.rstd[t];
    int cw = c0;
    if constexpr (!HELD) asm volatile("" : "+v"(cw));   // else the compiler holds what it loads and unpacks after all
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      float d[8], s[8];
      unpack8(vd[i], d);
      unpack8(vs[i], s);
      if constexpr (!HELD) load_weight(wr, a.w_f32, cw + i * kWave, w[0]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float dxh = d[j] * (s[j] * rstd);
        dw[i][j] += dxh;
        dot += dxh * w[HELD ? i : 0][j];
      }
    }
    const float c = row_sum<W>(dot, red, sub, odd) / (float)H;
    odd ^= 1;
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.dx + t * H, row_bytes);
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      float d[8], s[8], r[8], o[8];
      if constexpr (!HELD) asm volatile("" : "+v"(vd[i]), "+v"(vs[i]));
      unpack8(vd[i], d);
      unpack8(vs[i], s);
      unpack8(HELD ? vr[i] : buf_load16_nt(rr, (uint32_t)(c0 + i * kWave) * 16u), r);
      if constexpr (!HELD) load_weight(wr, a.w_f32, cw + i * kWave, w[0]);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = rstd * (d[j] * w[HELD ? i : 0][j] - (s[j] * rstd) * c) + r[j];
      store_row<true>(pack8(o), xr, (uint32_t)(c0 + i * kWave) * 16u);
    }
  }
  if (a.part) {
    if constexpr (W == 1) {                            // CPL is 1
      if (wave > 0)
#pragma unroll
        for (int j = 0; j < 8; ++j) s_dw[wave - 1][j * 64 + lane] = dw[0][j];
      __syncthreads();
      if (wave > 0) return;
#pragma unroll
      for (int v = 0; v < 3; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[0][j] += s_dw[v][j * 64 + lane];
    }
    const __amdgpu_buffer_rsrc_t pr = make_rsrc(a.part + (int64_t)blockIdx.x * H, (uint32_t)H * 4u);
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const uint32_t o = (uint32_t)(c0 + i * kWave) * 32u;
      u32x4 p, q;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        p[j] = __builtin_bit_cast(uint32_t, dw[i][j]);
        q[j] = __builtin_bit_cast(uint32_t, dw[i][4 + j]);
      }
      buf_store16(p, pr, o);
      buf_store16(q, pr, o + 16u);
    }
  }
}

// dweight[h] = sum of the n partial rows, always in the same order. A workgroup has 32 columns,
// lane (r, c) of wave v sums rows 8 v + r, + 128, ... of columns 4 c .. + 4, eight loads in flight
// (n = 512, H = 4096: 4.8 us; with 8 row groups of a column a thread 18).
__global__ __launch_bounds__(1024) void rmsnorm_dweight_kernel(const float* part, int n, int H, float* dweight) {
  typedef float f32x4 __attribute__((ext_vector_type(4)));
  __shared__ f32x4 red[16][8];
  const int lane = lane_id(), wave = threadIdx.x >> 6;
  const int c = lane & 7, r = lane >> 3;
  const int h = blockIdx.x * 32 + c * 4;   // H % 8 == 0: four columns are in or out together
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  if (h < H)
#pragma unroll 8
    for (int i = wave * 8 + r; i < n; i += 128) v += *reinterpret_cast<const f32x4*>(part + (int64_t)i * H + h);
#pragma unroll
  for (int o = 8; o < 64; o *= 2)
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] += __shfl_xor(v[j], o, 64);
  if (r == 0) red[wave][c] = v;
  __syncthreads();
  if (wave == 0 && r == 0 && h < H) {
#pragma unroll
    for (int i = 1; i < 16; ++i) v += red[i][c];
#pragma unroll
    for (int j = 0; j < 4; ++j) dweight[h + j] = v[j];
  }
}

// ---------------------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------------------
constexpr int kNormMaxBlocks = 1 << 16;

template <int W, int CPL>
static void launch_norm_q(int qf, dim3 grid, hipStream_t s, const NormArgs& a) {
  const dim3 block(W == 16 ? 1024 : 256);
  if (qf == 1) hipLaunchKernelGGL((rmsnorm_kernel<W, CPL, 1>), grid, block, 0, s, a);
  else if (qf == 2) hipLaunchKernelGGL((rmsnorm_kernel<W, CPL, 2>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((rmsnorm_kernel<W, CPL, 0>), grid, block, 0, s, a);
}

int launch_rmsnorm(const void* x, const void* res, const void* weight, bool w_f32, int32_t T, int32_t H, double eps,
                   void* s_out, void* y, float* rstd, int32_t q_dtype, void* q, void* q_s, hipStream_t stream) {
  NormArgs a;
  a.x = static_cast<const uint16_t*>(x);
  a.res = static_cast<const uint16_t*>(res);
  a.w = weight;
  a.w_f32 = w_f32;
  a.T = T;
  a.H = H;
  a.eps = eps;
  a.s_out = static_cast<uint16_t*>(s_out);
  a.y = static_cast<uint16_t*>(y);
  a.rstd = rstd;
  a.q = static_cast<uint8_t*>(q);
  a.q_s = q_s;
  const int qf = q_dtype == MOE_FP8_E4M3_G128 ? 1 : q_dtype == MOE_MXFP4 ? 2 : 0;
  const int nch = ((H + 127) / 128) * 16;   // chunks, the last scale word's whole
  const auto blocks = [&](int rows) { return dim3((unsigned)std::min<int64_t>(((int64_t)T + rows - 1) / rows, kNormMaxBlocks)); };
  if (nch <= 64) launch_norm_q<1, 1>(qf, blocks(4), stream, a);
  else if (nch <= 128) launch_norm_q<1, 2>(qf, blocks(4), stream, a);
  else if (nch <= 256) launch_norm_q<4, 1>(qf, blocks(1), stream, a);
  else if (nch <= 512) launch_norm_q<4, 2>(qf, blocks(1), stream, a);
  else if (nch <= 1024) launch_norm_q<4, 4>(qf, blocks(1), stream, a);
  else if (nch <= 2048) launch_norm_q<16, 2>(qf, blocks(1), stream, a);
  else launch_norm_q<16, 4>(qf, blocks(1), stream, a);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

// Waves that share a row of the backward pass, and its workgroups (4096 waves, 16 a CU): rows of
// partial sums that the workspace holds. Both depend on T and H alone, and so does the order of
// the sums.
static int backward_waves(int32_t H) {
  const int nch = H / 8;
  return nch <= 64 ? 1 : nch <= 256 ? 4 : nch <= 1024 ? 8 : 16;
}
int32_t rmsnorm_backward_blocks(int32_t T, int32_t H) {
  return std::min(T, 4096 / std::max(4, backward_waves(H)));
}

int launch_rmsnorm_backward(const void* dy, const void* s, const void* weight, bool w_f32, const float* rstd,
                            const void* d_res, int32_t T, int32_t H, void* dx, float* dweight, void* ws,
                            hipStream_t stream) {
  NormBwdArgs a;
  a.dy = static_cast<const uint16_t*>(dy);
  a.s = static_cast<const uint16_t*>(s);
  a.w = weight;
  a.w_f32 = w_f32;
  a.rstd = rstd;
  a.d_res = static_cast<const uint16_t*>(d_res);
  a.T = T;
  a.H = H;
  a.dx = static_cast<uint16_t*>(dx);
  a.part = dweight ? static_cast<float*>(ws) : nullptr;
  const int n = T > 0 ? rmsnorm_backward_blocks(T, H) : 0;
  if (n > 0) {
    const int nch = H / 8;
    const dim3 grid(n);
    if (nch <= 64) hipLaunchKernelGGL((rmsnorm_backward_kernel<1, 1>), grid, dim3(256), 0, stream, a);
    else if (nch <= 256) hipLaunchKernelGGL((rmsnorm_backward_kernel<4, 1>), grid, dim3(256), 0, stream, a);
    else if (nch <= 512) hipLaunchKernelGGL((rmsnorm_backward_kernel<8, 1>), grid, dim3(512), 0, stream, a);
    else if (nch <= 1024) hipLaunchKernelGGL((rmsnorm_backward_kernel<8, 2>), grid, dim3(512), 0, stream, a);
    else if (nch <= 2048) hipLaunchKernelGGL((rmsnorm_backward_kernel<16, 2>), grid, dim3(1024), 0, stream, a);
    else hipLaunchKernelGGL((rmsnorm_backward_kernel<16, 4>), grid, dim3(1024), 0, stream, a);
    if (hipGetLastError() != hipSuccess) return MOE_ERR_HIP;
  }
  if (dweight) {
    hipLaunchKernelGGL(rmsnorm_dweight_kernel, dim3((H + 31) / 32), dim3(1024), 0, stream, a.part, n, H, dweight);
    if (hipGetLastError() != hipSuccess) return MOE_ERR_HIP;
  }
  return MOE_OK;
}

}  // namespace moe
