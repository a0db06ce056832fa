// Root-mean-square norm with the residual's addition and an 8-bit output (sm_103a), and its
// backward pass.
//
//   s = x + r,  h = bf16(s),  rstd = 1 / sqrt(mean(s^2) + eps),  y = s * rstd * w
//   codes: cast(y * scale), scale = fp8_max / max(amax, 1e-12) of the row or of each 1 x 128 block,
//          or the power-of-two scales of blocks of 32 (MX)
//   g = dy * w,  xhat = h * rstd,  dx = rstd * (g - xhat * mean(g * xhat)) + dh,
//   dw = sum over rows of dy * xhat
//
// Everything between the loads and the stores is fp32: s is not rounded to bf16 on its way into
// the statistics or into y, and y is rounded once, into each of its outputs.
#include "common.cuh"
#include "internal.h"

namespace fp8lin {

namespace {

FP8_DEVI float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
FP8_DEVI float bf_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }
FP8_DEVI uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// max that keeps a NaN, so that a NaN reaches the scale as it does in fp8_quantize
FP8_DEVI float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// 16 bytes through L2 only: each row is read once. Not ld.nc: an output may be one of the inputs.
FP8_DEVI uint4 ld_stream(const uint4* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

FP8_DEVI void unpack8(uint4 v, float* f) {
  f[0] = bf_lo(v.x), f[1] = bf_hi(v.x), f[2] = bf_lo(v.y), f[3] = bf_hi(v.y);
  f[4] = bf_lo(v.z), f[5] = bf_hi(v.z), f[6] = bf_lo(v.w), f[7] = bf_hi(v.w);
}
FP8_DEVI uint4 pack8(const float* f) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}
// 8 weights from bf16 or fp32
FP8_DEVI void load_w(const void* w, int w_f32, int c, float* f) {
  if (w_f32) {
    const float4 a = __ldg(static_cast<const float4*>(w) + 2 * c), b = __ldg(static_cast<const float4*>(w) + 2 * c + 1);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
    unpack8(__ldg(static_cast<const uint4*>(w) + c), f);
  }
}

struct NormArgs {
  const uint4* x;
  const uint4* res;  // may be null
  const void* w;
  int w_f32;
  float eps;
  float H;
  int64_t T;
  int nvec;          // 16-byte vectors of a row
  uint4* h;          // the outputs may be null
  uint4* y;
  uint2* q;
  void* inv;
  float* rstd;
};

constexpr int kNone = -1;  // no 8-bit output

// One row per team: one warp (WARP; eight rows a CTA, no barrier), or the whole CTA. A thread holds
// VPT vectors of its row, vector t + i * team, as fp32 sums. The sum of squares and the largest
// |s * w| are reduced together, behind one barrier: y = (s * w) * rstd, and rounding keeps order,
// so rstd * max |s * w| is the largest |y| exactly and the scale needs no second pass.
template <int VPT, int GRAN, int FMT, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 512) add_rmsnorm_kernel(const NormArgs p) {
  constexpr float FMAX = FmtMax<FMT>::v;
  __shared__ float red_s[16], red_m[16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = WARP ? (int64_t)blockIdx.x * 8 + warp : (int64_t)blockIdx.x;
  const int t = WARP ? lane : threadIdx.x;
  const int team = WARP ? 32 : blockDim.x;
  if (WARP && row >= p.T) return;
  const uint4* xr = p.x + row * p.nvec;
  const uint4* rr = p.res ? p.res + row * p.nvec : nullptr;

  uint4 vx[VPT], vr[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = t + i * team;
    vx[i] = c < p.nvec ? ld_stream(xr + c) : make_uint4(0, 0, 0, 0);
    vr[i] = rr && c < p.nvec ? ld_stream(rr + c) : make_uint4(0, 0, 0, 0);
  }
  float s[VPT][8];
  float sum = 0.f, mx = 0.f;
  float bm[VPT];  // block scales: the block's largest |s * w|
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = t + i * team;
    float r8[8], w8[8];
    unpack8(vx[i], s[i]);
    if (rr) {
      unpack8(vr[i], r8);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[i][j] += r8[j];
    }
    if (p.h && c < p.nvec) p.h[row * p.nvec + c] = pack8(s[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) w8[j] = 0.f;
    if (c < p.nvec) load_w(p.w, p.w_f32, c, w8);
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sum = fmaf(s[i][j], s[i][j], sum);
      s[i][j] *= w8[j];
      m = max_nan(m, fabsf(s[i][j]));
    }
    if (GRAN == FP8_GRAN_ROW) mx = max_nan(mx, m);
    if (GRAN == FP8_GRAN_BLOCK_1x128 || GRAN == FP8_GRAN_MX) {
      // a block is 16 (128 elements) or 4 (32 elements) consecutive lanes' vectors
#pragma unroll
      for (int o = 1; o < (GRAN == FP8_GRAN_MX ? 4 : 16); o <<= 1)
        m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
      bm[i] = m;
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (GRAN == FP8_GRAN_ROW) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  if (!WARP) {
    if (lane == 0) {
      red_s[warp] = sum;
      red_m[warp] = mx;
    }
    __syncthreads();
    sum = 0.f;
    mx = 0.f;
    for (int w = 0; w < team / 32; ++w) {
      sum += red_s[w];
      if (GRAN == FP8_GRAN_ROW) mx = max_nan(mx, red_m[w]);
    }
  }
  const float rstd = 1.0f / sqrtf(sum / p.H + p.eps);
  if (p.rstd && t == 0) p.rstd[row] = rstd;
  float scale = 1.f;
  if (GRAN == FP8_GRAN_ROW) {
    float a = mx * rstd;
    a = a < 1e-12f ? 1e-12f : a;  // a NaN stays
    scale = FMAX / a;
    if (t == 0) static_cast<float*>(p.inv)[row] = a / FMAX;
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = t + i * team;
    if (c >= p.nvec) continue;
#pragma unroll
    for (int j = 0; j < 8; ++j) s[i][j] *= rstd;
    if (p.y) p.y[row * p.nvec + c] = pack8(s[i]);
    if (GRAN == kNone) continue;
    if (GRAN == FP8_GRAN_BLOCK_1x128) {
      float a = bm[i] * rstd;
      a = a < 1e-12f ? 1e-12f : a;
      scale = FMAX / a;
      if ((t & 15) == 0) static_cast<float*>(p.inv)[row * (p.nvec / 16) + c / 16] = a / FMAX;
    }
    if (GRAN == FP8_GRAN_MX) {
      // the block's exponent field, as the rule takes it from a bf16 amax, here from the fp32 one
      const uint32_t code = mx_code<FMT>(__float_as_uint(bm[i] * rstd) >> 16);
      scale = mx_inv(code);
      const int j = c / 4;  // block of 32 along the row
      if ((t & 3) == 0)
        static_cast<uint8_t*>(p.inv)[((row >> 7) * (p.nvec / 16) + (j >> 2)) * 512 + (row & 31) * 16 +
                                     ((row >> 5) & 3) * 4 + (j & 3)] = (uint8_t)code;
    }
    uint2 o;
    o.x = cvt_fp8x2<FMT>(s[i][0] * scale, s[i][1] * scale) | (cvt_fp8x2<FMT>(s[i][2] * scale, s[i][3] * scale) << 16);
    o.y = cvt_fp8x2<FMT>(s[i][4] * scale, s[i][5] * scale) | (cvt_fp8x2<FMT>(s[i][6] * scale, s[i][7] * scale) << 16);
    p.q[row * p.nvec + c] = o;
  }
}

template <int VPT, int GRAN, int FMT>
int run_norm(const NormArgs& a, const Ctx& c) {
  if (a.nvec <= 32 * VPT) {
    add_rmsnorm_kernel<VPT, GRAN, FMT, true><<<(unsigned)ceil_div64(a.T, 8), 256, 0, c.stream>>>(a);
  } else {
    const int team = (int)round_up64(ceil_div64(a.nvec, VPT), 32);
    add_rmsnorm_kernel<VPT, GRAN, FMT, false><<<(unsigned)a.T, team, 0, c.stream>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
}

template <int GRAN, int FMT>
int norm_dispatch(const NormArgs& a, const Ctx& c) {
  // two vectors a thread while a CTA of 512 threads covers the row, four for the widest rows
  if (a.nvec <= 1024) return run_norm<2, GRAN, FMT>(a, c);
  return run_norm<4, GRAN, FMT>(a, c);
}

}  // namespace

int launch_add_rmsnorm(const void* x, const void* res, const void* w, int w_f32, float eps, int64_t T, int64_t H,
                       int gran, int fmt, void* h, void* y, void* q, void* inv, float* rstd, const Ctx& c) {
  if (T == 0 || H == 0) return FP8_OK;
  NormArgs a;
  a.x = static_cast<const uint4*>(x);
  a.res = static_cast<const uint4*>(res);
  a.w = w;
  a.w_f32 = w_f32;
  a.eps = eps;
  a.H = (float)H;
  a.T = T;
  a.nvec = (int)(H / 8);
  a.h = static_cast<uint4*>(h);
  a.y = static_cast<uint4*>(y);
  a.q = static_cast<uint2*>(q);
  a.inv = inv;
  a.rstd = rstd;
  if (!q) return norm_dispatch<kNone, FP8_DT_E4M3>(a, c);
  const bool e4 = fmt == FP8_DT_E4M3;
  switch (gran) {
    case FP8_GRAN_ROW:
      return e4 ? norm_dispatch<FP8_GRAN_ROW, FP8_DT_E4M3>(a, c) : norm_dispatch<FP8_GRAN_ROW, FP8_DT_E5M2>(a, c);
    case FP8_GRAN_BLOCK_1x128:
      return e4 ? norm_dispatch<FP8_GRAN_BLOCK_1x128, FP8_DT_E4M3>(a, c)
                : norm_dispatch<FP8_GRAN_BLOCK_1x128, FP8_DT_E5M2>(a, c);
    case FP8_GRAN_MX:
      return e4 ? norm_dispatch<FP8_GRAN_MX, FP8_DT_E4M3>(a, c) : norm_dispatch<FP8_GRAN_MX, FP8_DT_E5M2>(a, c);
    default:
      return FP8_ERR_UNSUPPORTED;
  }
}

// ==========================================================================================
// Backward. A CTA walks rows with a grid stride; a thread owns VPT vectors of every row, so its
// share of dw stays in registers from row to row and leaves once, as one of `parts` partial rows
// in the workspace. A second kernel adds the partial rows in a fixed order: no atomics, the same
// bits on every run.
namespace {

struct NormBwdArgs {
  const uint4* dy;
  const uint4* h;
  const void* w;
  int w_f32;
  const float* rstd;
  const uint4* dh;  // may be null
  uint4* dx;
  float* part;      // [grid][H], null without dw
  int64_t T;
  int nvec;
  float H;
};

template <int VPT>
__global__ void __launch_bounds__(512) rmsnorm_bwd_kernel(const NormBwdArgs p) {
  __shared__ float red[2][16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = threadIdx.x, team = blockDim.x;
  float dw[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
  int par = 0;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x, par ^= 1) {
    const float rstd = __ldg(p.rstd + row);
    uint4 vdy[VPT], vh[VPT], vdh[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = t + i * team;
      const bool in = c < p.nvec;
      vdy[i] = in ? ld_stream(p.dy + row * p.nvec + c) : make_uint4(0, 0, 0, 0);
      vh[i] = in ? ld_stream(p.h + row * p.nvec + c) : make_uint4(0, 0, 0, 0);
      vdh[i] = p.dh && in ? ld_stream(p.dh + row * p.nvec + c) : make_uint4(0, 0, 0, 0);
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = t + i * team;
      float d8[8], h8[8], w8[8];
      unpack8(vdy[i], d8);
      unpack8(vh[i], h8);
#pragma unroll
      for (int j = 0; j < 8; ++j) w8[j] = 0.f;
      if (c < p.nvec) load_w(p.w, p.w_f32, c, w8);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xhat = h8[j] * rstd;
        const float dyx = d8[j] * xhat;
        dw[i][j] += dyx;
        sum = fmaf(dyx, w8[j], sum);
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) red[par][warp] = sum;  // two buffers: a row's values are read while the next row's are written
    __syncthreads();
    sum = 0.f;
    for (int w = 0; w < team / 32; ++w) sum += red[par][w];
    const float mean = sum / p.H;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = t + i * team;
      if (c >= p.nvec) continue;
      float d8[8], h8[8], w8[8], g8[8];
      unpack8(vdy[i], d8);
      unpack8(vh[i], h8);
      unpack8(vdh[i], g8);
      load_w(p.w, p.w_f32, c, w8);
#pragma unroll
      for (int j = 0; j < 8; ++j) d8[j] = rstd * (d8[j] * w8[j] - h8[j] * rstd * mean) + g8[j];
      if (p.dx) p.dx[row * p.nvec + c] = pack8(d8);
    }
  }
  if (p.part) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = t + i * team;
      if (c >= p.nvec) continue;
      float4* o = reinterpret_cast<float4*>(p.part) + ((int64_t)blockIdx.x * p.nvec + c) * 2;
      o[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
      o[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
    }
  }
}

// dw[c] = sum of `parts` partial rows: 32 float4 columns a CTA, the rows split over 16 thread rows
// that are then added in order.
__global__ void __launch_bounds__(512) dw_sum_kernel(const float4* __restrict__ part, int parts, int n4, void* dw,
                                                     int dw_bf16) {
  __shared__ float4 sh[16][32];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < n4) {
#pragma unroll 4
    for (int r = threadIdx.y; r < parts; r += 16) {
      const float4 v = part[(int64_t)r * n4 + c];
      a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
    }
  }
  sh[threadIdx.y][threadIdx.x] = a;
  __syncthreads();
  if (threadIdx.y || c >= n4) return;
  for (int r = 1; r < 16; ++r) {
    const float4 v = sh[r][threadIdx.x];
    a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
  }
  if (dw_bf16)
    static_cast<uint2*>(dw)[c] = make_uint2(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w));
  else
    static_cast<float4*>(dw)[c] = a;
}

template <int VPT>
int run_norm_bwd(const NormBwdArgs& a, int grid, const Ctx& c) {
  rmsnorm_bwd_kernel<VPT><<<grid, (int)round_up64(ceil_div64(a.nvec, VPT), 32), 0, c.stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
}

constexpr int64_t kBwdParts = 304;  // partial rows of dw at most: two CTAs on each of 152 SMs

}  // namespace

int64_t rmsnorm_bwd_ws_bytes(int64_t T, int64_t H) { return (T < kBwdParts ? T : kBwdParts) * H * 4; }

int launch_rmsnorm_bwd(const void* dy, const void* h, const void* w, int w_f32, const float* rstd, const void* dh,
                       int64_t T, int64_t H, void* dx, void* dw, int dw_bf16, float* ws, const Ctx& c) {
  if (H == 0) return FP8_OK;
  const int64_t grid = T < kBwdParts ? T : kBwdParts;
  if (grid > 0) {
    NormBwdArgs a;
    a.dy = static_cast<const uint4*>(dy);
    a.h = static_cast<const uint4*>(h);
    a.w = w;
    a.w_f32 = w_f32;
    a.rstd = rstd;
    a.dh = static_cast<const uint4*>(dh);
    a.dx = static_cast<uint4*>(dx);
    a.part = dw ? ws : nullptr;
    a.T = T;
    a.nvec = (int)(H / 8);
    a.H = (float)H;
    const int rc = a.nvec <= 1024 ? run_norm_bwd<2>(a, (int)grid, c) : run_norm_bwd<4>(a, (int)grid, c);
    if (rc != FP8_OK) return rc;
  }
  if (dw) {  // no rows: an empty sum
    const int n4 = (int)(H / 4);
    dw_sum_kernel<<<(unsigned)ceil_div64(n4, 32), dim3(32, 16), 0, c.stream>>>(reinterpret_cast<const float4*>(ws),
                                                                              (int)grid, n4, dw, dw_bf16);
    if (cudaGetLastError() != cudaSuccess) return FP8_ERR_CUDA;
  }
  return FP8_OK;
}

}  // namespace fp8lin
