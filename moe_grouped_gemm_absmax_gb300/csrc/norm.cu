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
#include <atomic>

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
// Backward. Persistent CTAs walk groups of `rows` rows with a grid stride, a team of threads a row. A
// group's inputs arrive by bulk copies into a ring in shared memory, several groups ahead, so memory
// never waits for a row's reduction and its barrier. A thread owns VPT vectors of every row of its team,
// so its share of dw stays in registers from row to row; a CTA's teams add theirs up at the end, and it
// leaves as one of `grid` partial rows in the workspace. A second kernel adds the partial rows in a
// fixed order: no atomics, the same bits on every run.
namespace {

constexpr int kBwdStages = 5;

struct NormBwdArgs {
  const uint4* dy;
  const uint4* h;
  const void* w;
  int w_f32;
  const float* rstd;
  const uint4* dh;  // may be null
  uint4* dx;        // may be null
  float* part;      // [grid][H], null without dw
  int64_t T;
  int nvec;
  float H;
  int rows, stages;
  uint64_t wait_ns;
};

FP8_DEVI void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

template <int VPT>
__global__ void __launch_bounds__(512) rmsnorm_bwd_kernel(const NormBwdArgs p) {
  extern __shared__ uint4 ring[];  // [stages][dy, h, dh][rows][nvec]
  __shared__ float red[2][16];
  __shared__ uint64_t full[kBwdStages];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int team_size = blockDim.x / p.rows, team = threadIdx.x / team_size, t = threadIdx.x % team_size;
  const int team_warps = team_size / 32, warp0 = team * team_warps;
  const int tensors = p.dh ? 3 : 2;
  const int slab = p.rows * p.nvec;  // vectors of a tensor in a stage
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
  }
  __syncthreads();
  const int64_t groups = ceil_div64(p.T, p.rows);
  auto load = [&](int64_t g, int s) {
    const int64_t row = g * p.rows;
    const uint32_t bytes = (uint32_t)min((int64_t)p.rows, p.T - row) * (uint32_t)p.nvec * 16;
    uint4* d = ring + s * tensors * slab;
    mbar_arrive_expect_tx(&full[s], bytes * tensors);
    bulk_load(d, p.dy + row * p.nvec, bytes, &full[s]);
    bulk_load(d + slab, p.h + row * p.nvec, bytes, &full[s]);
    if (p.dh) bulk_load(d + 2 * slab, p.dh + row * p.nvec, bytes, &full[s]);
  };
  if (threadIdx.x == 0)
    for (int s = 0; s < p.stages; ++s) {
      const int64_t g = blockIdx.x + (int64_t)s * gridDim.x;
      if (g < groups) load(g, s);
    }
  float dw[VPT][8], w8[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = w8[i][j] = 0.f;
    if (t + i * team_size < p.nvec) load_w(p.w, p.w_f32, t + i * team_size, w8[i]);
  }
  int s = 0, prev = 0, par = 0;
  uint32_t phase = 0;
  auto row_rstd = [&](int64_t g) {
    const int64_t row = g * p.rows + team;
    return row < p.T ? __ldg(p.rstd + row) : 0.f;
  };
  float rstd_next = row_rstd(blockIdx.x);
  for (int64_t g = blockIdx.x; g < groups; g += gridDim.x, par ^= 1) {
    const int64_t row = g * p.rows + team;
    const bool active = row < p.T;
    float rstd = rstd_next;
    rstd_next = row_rstd(g + gridDim.x);
    // a wait that ran out would show as NaN in everything that the row reaches
    if (!mbar_wait(&full[s], phase, nullptr, p.wait_ns)) rstd = __uint_as_float(0x7FC00000u);
    const uint4* d = ring + s * tensors * slab + team * p.nvec;
    float sum = 0.f;
    if (active) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = t + i * team_size;
        if (c >= p.nvec) continue;
        float d8[8], h8[8];
        unpack8(d[c], d8);
        unpack8(d[slab + c], h8);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float dyx = d8[j] * (h8[j] * rstd);
          dw[i][j] += dyx;
          sum = fmaf(dyx, w8[i][j], sum);
        }
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) red[par][warp] = sum;  // two buffers: a row's values are read while the next row's are written
    __syncthreads();
    // every thread is done with the group before this one: its stage takes the group `stages` further on
    if (threadIdx.x == 0 && g != blockIdx.x) {
      const int64_t next = g + (int64_t)(p.stages - 1) * gridDim.x;
      if (next < groups) load(next, prev);
    }
    if (p.dx && active) {
      sum = 0.f;
      for (int w = 0; w < team_warps; ++w) sum += red[par][warp0 + w];
      const float mean = sum / p.H;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = t + i * team_size;
        if (c >= p.nvec) continue;
        float d8[8], h8[8], g8[8];
        unpack8(d[c], d8);
        unpack8(d[slab + c], h8);
        unpack8(p.dh ? d[2 * slab + c] : make_uint4(0, 0, 0, 0), g8);
#pragma unroll
        for (int j = 0; j < 8; ++j) d8[j] = rstd * (d8[j] * w8[i][j] - h8[j] * rstd * mean) + g8[j];
        p.dx[row * p.nvec + c] = pack8(d8);
      }
    }
    prev = s;
    if (++s == p.stages) s = 0, phase ^= 1;
  }
  if (p.part) {
    float4* out = reinterpret_cast<float4*>(p.part) + (int64_t)blockIdx.x * p.nvec * 2;
    float4* sh = reinterpret_cast<float4*>(ring);  // [rows][2 nvec], after the last group
    if (p.rows > 1) __syncthreads();
    if (p.rows > 1) out = sh + team * p.nvec * 2;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = t + i * team_size;
      if (c >= p.nvec) continue;
      out[2 * c] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
      out[2 * c + 1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
    }
    if (p.rows > 1) {
      __syncthreads();
      out = reinterpret_cast<float4*>(p.part) + (int64_t)blockIdx.x * p.nvec * 2;
      for (int c = threadIdx.x; c < 2 * p.nvec; c += blockDim.x) {
        float4 a = sh[c];
        for (int r = 1; r < p.rows; ++r) {
          const float4 v = sh[r * 2 * p.nvec + c];
          a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
        }
        out[c] = a;
      }
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// dw[c] = sum of `parts` partial rows: 32 float4 columns a CTA, the rows split over 16 thread rows
// that are then added in order.
__global__ void __launch_bounds__(512) dw_sum_kernel(const float4* part, int parts, int n4, void* dw, int dw_bf16) {
  __shared__ float4 sh[16][32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x * 32 + threadIdx.x;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < n4) {
#pragma unroll 8
    for (int r = threadIdx.y; r < parts; r += 16) {
      const float4 v = __ldcg(part + (int64_t)r * n4 + c);
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

// Shape of the backward kernel for rows of nvec vectors: two vectors a thread up to 8192 columns, four
// beyond; teams for several short rows, up to 512 threads a CTA; two CTAs an SM where each then has a ring of three
// groups, else one with as many as fit (two for the widest rows).
struct BwdShape {
  int vpt, team, rows, ctas, stages;
};
BwdShape bwd_shape(int nvec, bool dh) {
  constexpr int kRoom = 220 * 1024;
  BwdShape b;
  b.vpt = nvec <= 1024 ? 2 : 4;
  b.team = (int)round_up64(ceil_div64(nvec, b.vpt), 32);
  b.rows = 512 / b.team;
  const int group = (dh ? 3 : 2) * b.rows * nvec * 16;
  b.ctas = kRoom / 2 / group >= 3 ? 2 : 1;
  const int fit = kRoom / b.ctas / group;
  b.stages = fit < kBwdStages ? fit : kBwdStages;
  return b;
}
constexpr int64_t kBwdSms = 152;
int64_t bwd_grid(int64_t T, const BwdShape& b) {
  const int64_t groups = ceil_div64(T, b.rows);
  return groups < kBwdSms * b.ctas ? groups : kBwdSms * b.ctas;
}

template <int VPT>
int run_norm_bwd(const NormBwdArgs& a, const BwdShape& b, int grid, const Ctx& c) {
  const size_t smem = (size_t)b.stages * (a.dh ? 3 : 2) * b.rows * a.nvec * 16;
  static std::atomic<uint64_t> done{0};
  const uint64_t bit = 1ull << (c.device & 63);
  if (!(done.load(std::memory_order_acquire) & bit)) {
    if (cudaFuncSetAttribute(rmsnorm_bwd_kernel<VPT>, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024) != cudaSuccess)
      return FP8_ERR_CUDA;
    done.fetch_or(bit, std::memory_order_release);
  }
  rmsnorm_bwd_kernel<VPT><<<grid, b.team * b.rows, smem, c.stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
}

}  // namespace

int64_t rmsnorm_bwd_ws_bytes(int64_t T, int64_t H) {
  // without dh the ring is shorter and more CTAs may fit: room for those
  return bwd_grid(T, bwd_shape((int)(H / 8), false)) * H * 4;
}

int launch_rmsnorm_bwd(const void* dy, const void* h, const void* w, int w_f32, const float* rstd, const void* dh,
                       int64_t T, int64_t H, void* dx, void* dw, int dw_bf16, float* ws, const Ctx& c) {
  const BwdShape b = bwd_shape((int)(H / 8), dh != nullptr);
  const int64_t grid = bwd_grid(T, b);
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
    a.rows = b.rows;
    a.stages = b.stages;
    a.wait_ns = c.wait_ns;
    const int rc = b.vpt == 2 ? run_norm_bwd<2>(a, b, (int)grid, c) : run_norm_bwd<4>(a, b, (int)grid, c);
    if (rc != FP8_OK) return rc;
  }
  if (!dw) return FP8_OK;
  if (grid == 0)  // no rows: an empty sum
    return cudaMemsetAsync(dw, 0, (size_t)H * (dw_bf16 ? 2 : 4), c.stream) == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
  const int n4 = (int)(H / 4);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)ceil_div64(n4, 32));
  cfg.blockDim = dim3(32, 16);
  cfg.stream = c.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, dw_sum_kernel, static_cast<const float4*>(static_cast<const void*>(ws)), (int)grid, n4,
                            dw, dw_bf16) == cudaSuccess
             ? FP8_OK
             : FP8_ERR_CUDA;
}

}  // namespace fp8lin
