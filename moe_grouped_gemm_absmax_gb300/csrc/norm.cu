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

// Two fp32 operations in one instruction, each rounded as the scalar one. The kernels here move 7 to 8
// bytes an element and run into the issue rate before the memory's with scalar arithmetic (221
// instructions for 8 elements forward, 266 backward, at 2.5-2.9 of 4 a cycle), so all of it is paired.
FP8_DEVI float2 fadd2_rn(float2 a, float2 b) {
  uint64_t ra, rb, rd;
  asm("mov.b64 %0, {%1, %2};" : "=l"(ra) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(rb) : "f"(b.x), "f"(b.y));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(rd) : "l"(ra), "l"(rb));
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(rd));
  return d;
}
FP8_DEVI float2 ffma2_rn(float2 a, float2 b, float2 c) {
  uint64_t ra, rb, rc, rd;
  asm("mov.b64 %0, {%1, %2};" : "=l"(ra) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(rb) : "f"(b.x), "f"(b.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(rc) : "f"(c.x), "f"(c.y));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(rd) : "l"(ra), "l"(rb), "l"(rc));
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(rd));
  return d;
}
FP8_DEVI float2 both(float v) { return make_float2(v, v); }
FP8_DEVI uint32_t pack_bf16(float2 v) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(v.y), "f"(v.x));
  return r;
}
// Maxima that keep a NaN, so that a NaN reaches the scale as it does in fp8_quantize.
FP8_DEVI float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
FP8_DEVI float absmax3_nan(float m, float2 v) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(v.x), "f"(v.y));
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

FP8_DEVI float2 unpack2(uint32_t w) { return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }
FP8_DEVI uint32_t word(uint4 v, int j) { return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w; }
// 8 elements as 4 pairs
FP8_DEVI void unpack8(uint4 v, float2* f) {
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = unpack2(word(v, j));
}
FP8_DEVI uint4 pack8(const float2* f) {
  return make_uint4(pack_bf16(f[0]), pack_bf16(f[1]), pack_bf16(f[2]), pack_bf16(f[3]));
}
// 8 weights from bf16 (one vector) or fp32 (two)
FP8_DEVI void unpack_w(const uint4* v, bool f32, float2* f) {
  if (f32) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f[i] = make_float2(__uint_as_float(i & 1 ? v[i / 2].z : v[i / 2].x), __uint_as_float(i & 1 ? v[i / 2].w : v[i / 2].y));
  } else {
    unpack8(v[0], f);
  }
}
FP8_DEVI void load_w(const void* w, int f32, int c, float2* f) {
  const uint4* v = static_cast<const uint4*>(w);
  uint4 a[2];
  if (f32)
    a[0] = v[2 * c], a[1] = v[2 * c + 1];
  else
    a[0] = v[c];
  unpack_w(a, f32, f);
}

// A team's values from its warps, 32 slots; the slots past its warps hold zeros. Written by the team's first warp
// and by each warp's lane 0, before the barrier.
FP8_DEVI void team_put(float* slots, int t, int warps, float v) {
  if ((t & 31) == 0) slots[t >> 5] = v;
  if (t < 32 && t >= warps) slots[t] = 0.f;
}
// The same sum with two additions an instruction (PAIRS) or one: the backward kernels with several vectors a thread have
// no registers to pair (3000 x 16384 77 us instead of 73); with one vector it is worth 1 us of 75.
template <bool PAIRS>
FP8_DEVI float team_sum(const float* slots, int warps) {
  const float4 v = *reinterpret_cast<const float4*>(slots);
  float2 a = make_float2(v.x, v.y), b = make_float2(v.z, v.w);
  for (int i = 4; i < warps; i += 4) {
    const float4 u = *reinterpret_cast<const float4*>(slots + i);
    if (PAIRS)
      a = fadd2_rn(a, make_float2(u.x, u.y)), b = fadd2_rn(b, make_float2(u.z, u.w));
    else
      a.x += u.x, a.y += u.y, b.x += u.z, b.y += u.w;
  }
  return (a.x + a.y) + (b.x + b.y);
}
FP8_DEVI float team_max(const float* slots, int warps) {
  float m = 0.f;
  for (int i = 0; i < warps; i += 4) {
    const float4 b = *reinterpret_cast<const float4*>(slots + i);
    m = absmax3_nan(absmax3_nan(m, make_float2(b.x, b.y)), make_float2(b.z, b.w));
  }
  return m;
}

struct NormArgs {
  const uint4* x;
  const uint4* res;  // may be null
  const void* w;
  int w_f32;
  float eps;
  float inv_H;
  int64_t T;
  int nvec;          // 16-byte vectors of a row
  uint4* h;          // the outputs may be null
  uint4* y;
  uint2* q;
  void* inv;
  float* rstd;
};

constexpr int kNone = -1;  // no 8-bit output

// ------------------------------------------------------------------------------------------
// Forward, 8 elements at a time. y = (s * w) * rstd, and rounding keeps order, so rstd times the largest
// |s * w| is the largest |y| exactly: both reductions of a row meet at one barrier.

// s = x + r, its part of the sum of squares, then s * w in its place; returns the largest |s * w|
FP8_DEVI float norm_in(uint4 x, uint4 r, bool has_r, const float2* w, uint4* h, float2* s, float2* sum) {
  unpack8(x, s);
  if (has_r) {
    float2 r8[4];
    unpack8(r, r8);
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = fadd2_rn(s[j], r8[j]);
  }
  if (h) *h = pack8(s);
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    *sum = ffma2_rn(s[j], s[j], *sum);
    s[j] = fmul2_rn(s[j], w[j]);
    m = absmax3_nan(m, s[j]);
  }
  return m;
}
// the block's maximum: 16 (128 elements) or 4 (32 elements) consecutive lanes' vectors
template <int GRAN>
FP8_DEVI float block_max(float m) {
#pragma unroll
  for (int o = 1; o < (GRAN == FP8_GRAN_MX ? 4 : 16); o <<= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}
FP8_DEVI float amax_floor(float a) { return a < 1e-12f ? 1e-12f : a; }  // a NaN stays
// What brings s * w to the codes' range: FMAX * rstd / (m * rstd), for the largest |s * w| m. Where the amax m * rstd
// is neither below the floor nor infinite or NaN, rstd cancels and one quotient is left. It is rounded exactly, since its
// error moves all codes of the row or block the same way: over 137 calls of 1x128 e4m3 codes their distance from the exact ones
// is 1.1e-4 of the 2-norm, with an approximate quotient 2.6e-4, of fp32 arithmetic in the formula's order 3.8e-4 (14336 x 4096
// 37.1 us, approximate 36.3).
template <int FMT>
FP8_DEVI float code_scale(float m, float a, float rstd) {
  const bool cancels = a >= 1e-12f && a <= 3.4e38f;
  const float q = __fdiv_rn(FmtMax<FMT>::v, cancels ? m : amax_floor(a));
  return cancels ? q : rstd * q;
}
// y and its codes of vector c of a row; f: rstd times the row's scale, with row scales
template <int GRAN, int FMT>
FP8_DEVI void norm_out(const NormArgs& p, int64_t row, int c, const float2* s, float rstd, float f, float bm) {
  constexpr float FMAX = FmtMax<FMT>::v;
  if (p.y) {
    float2 y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = fmul2_rn(s[j], both(rstd));
    p.y[row * p.nvec + c] = pack8(y);
  }
  if (GRAN == kNone) return;
  if (GRAN == FP8_GRAN_BLOCK_1x128) {
    const float a = bm * rstd;
    f = code_scale<FMT>(bm, a, rstd);
    if ((c & 15) == 0) static_cast<float*>(p.inv)[row * (p.nvec / 16) + c / 16] = amax_floor(a) * (1.0f / FMAX);
  }
  if (GRAN == FP8_GRAN_MX) {
    // the block's exponent field, as the rule takes it from a bf16 amax, here from the fp32 one
    const uint32_t code = mx_code<FMT>(__float_as_uint(bm * rstd) >> 16);
    const int j = c / 4;  // block of 32 along the row
    if ((c & 3) == 0)
      static_cast<uint8_t*>(p.inv)[((row >> 7) * (p.nvec / 16) + (j >> 2)) * 512 + (row & 31) * 16 +
                                   ((row >> 5) & 3) * 4 + (j & 3)] = (uint8_t)code;
    f = rstd * mx_inv(code);
  }
  float2 v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = fmul2_rn(s[j], both(f));
  uint2 o;
  o.x = cvt_fp8x2<FMT>(v[0].x, v[0].y) | (cvt_fp8x2<FMT>(v[1].x, v[1].y) << 16);
  o.y = cvt_fp8x2<FMT>(v[2].x, v[2].y) | (cvt_fp8x2<FMT>(v[3].x, v[3].y) << 16);
  p.q[row * p.nvec + c] = o;
}

// One row per team: one warp (WARP; eight rows a CTA, no barrier) or the whole CTA, VPT vectors a thread.
// A CTA ends with its row: while some of an SM's CTAs reduce or store, others load. Persistent CTAs that
// asked for the next row ahead had fewer warps an SM and took 43 us instead of 40 for 8192 x 4096 at the time; one
// that took rows through shared memory 53 us. 36 us now, 96% of the copy rate; without a residual and with block
// scales the instructions bound it instead (14336 x 4096 37 us; the bytes are 26 us; 43 us at 77% of the issue slots
// with one kernel for every residual and weight type). The weights' type is known at compile time except in a CTA a
// row with four vectors a thread: there all weights loaded ahead take registers that cost CTAs (4778 x 12288 68 us
// instead of 64). Registers: 48 keep five CTAs of 256 threads an SM (8192 x 4096 35.8 us, with 52 37.4), 80 three
// of 224 or 256 (8192 x 7168 with block scales and no residual 48 us, with 91 63), 64 four of eight warps.
template <int VPT, int GRAN, int FMT, bool WARP, bool RES, bool WF32>
__global__ void __maxnreg__(VPT == 2 ? 48 : WARP ? 64 : 80) add_rmsnorm_kernel(const NormArgs p) {
  constexpr float FMAX = FmtMax<FMT>::v;
  __shared__ __align__(16) float red_s[32], red_m[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = WARP ? (int64_t)blockIdx.x * 8 + warp : (int64_t)blockIdx.x;
  const int t = WARP ? lane : threadIdx.x;
  const int team = WARP ? 32 : blockDim.x;
  pdl_wait();
  pdl_trigger();
  if (WARP && row >= p.T) return;
  uint4 vx[VPT], vr[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = t + i * team;
    vx[i] = c < p.nvec ? ld_stream(p.x + row * p.nvec + c) : make_uint4(0, 0, 0, 0);
    vr[i] = RES && c < p.nvec ? ld_stream(p.res + row * p.nvec + c) : make_uint4(0, 0, 0, 0);
  }
  constexpr bool kTyped = WARP || VPT == 2;  // the weights' type is WF32; they are loaded ahead of h's stores
  uint4 vw[VPT][2];
#pragma unroll
  for (int i = 0; kTyped && i < VPT; ++i) {
    const int c = t + i * team;
    const uint4* w = static_cast<const uint4*>(p.w) + (WF32 ? 2 * c : c);
    vw[i][0] = c < p.nvec ? w[0] : make_uint4(0, 0, 0, 0);
    vw[i][1] = WF32 && c < p.nvec ? w[1] : make_uint4(0, 0, 0, 0);
  }
  float2 s[VPT][4];
  float2 sum2 = both(0.f);
  float mx = 0.f;
  float bm[VPT];  // block scales: the block's largest |s * w|
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = t + i * team;
    float2 w8[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w8[j] = both(0.f);
    if (kTyped)
      unpack_w(vw[i], WF32, w8);
    else if (c < p.nvec)
      load_w(p.w, p.w_f32, c, w8);
    const float m = norm_in(vx[i], vr[i], RES, w8, p.h && c < p.nvec ? p.h + row * p.nvec + c : nullptr,
                            s[i], &sum2);
    if (GRAN == FP8_GRAN_ROW) mx = max_nan(mx, m);
    if (GRAN == FP8_GRAN_BLOCK_1x128 || GRAN == FP8_GRAN_MX) bm[i] = block_max<GRAN>(m);
  }
  float sum = sum2.x + sum2.y;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (GRAN == FP8_GRAN_ROW) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  if (!WARP) {
    team_put(red_s, t, team / 32, sum);
    if (GRAN == FP8_GRAN_ROW) team_put(red_m, t, team / 32, mx);
    __syncthreads();
    sum = team_sum<true>(red_s, team / 32);
    if (GRAN == FP8_GRAN_ROW) mx = team_max(red_m, team / 32);
  }
  const float rstd = rsqrtf(fmaf(sum, p.inv_H, p.eps));
  if (p.rstd && t == 0) p.rstd[row] = rstd;
  float f = 1.f;
  if (GRAN == FP8_GRAN_ROW) {
    const float a = mx * rstd;
    f = code_scale<FMT>(mx, a, rstd);
    if (t == 0) static_cast<float*>(p.inv)[row] = amax_floor(a) * (1.0f / FMAX);
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = t + i * team;
    if (c < p.nvec) norm_out<GRAN, FMT>(p, row, c, s[i], rstd, f, bm[i]);
  }
}

template <int VPT, int GRAN, int FMT, bool WARP>
int run_norm(const NormArgs& a, int threads, const Ctx& c) {
  constexpr bool F32 = WARP || VPT == 2;
  const auto kern = a.res ? (F32 && a.w_f32 ? add_rmsnorm_kernel<VPT, GRAN, FMT, WARP, true, F32>
                                            : add_rmsnorm_kernel<VPT, GRAN, FMT, WARP, true, false>)
                          : (F32 && a.w_f32 ? add_rmsnorm_kernel<VPT, GRAN, FMT, WARP, false, F32>
                                            : add_rmsnorm_kernel<VPT, GRAN, FMT, WARP, false, false>);
  return launch_dependent(kern, dim3((unsigned)ceil_div64(a.T, WARP ? 8 : 1)), dim3(threads), 0, c.stream, a);
}

template <int GRAN, int FMT>
int norm_dispatch(const NormArgs& a, const Ctx& c) {
  // A warp a row for the shortest rows, and with four vectors a thread up to 1024 columns where there are so many
  // rows that the start of a CTA for each (17 us for 16384) is what a call takes: 16384 x 768 10 us instead of
  // 17, with a residual 15.6 instead of 17.6; 16384 x 1024 11 instead of 17, 19.4 instead of 19.1.
  // Fewer rows end sooner with a CTA each (1024 x 1024 2.3 and 2.8 us).
  // A CTA a row else, two vectors a thread: with few rows a row's latency counts (1024 x 5120 4.2 us, with four
  // 5.6). Four for rows above 8192 columns, which 512 threads with two do not cover, and above 5120 for many
  // rows, where CTAs with two leave a third of an SM's threads empty (8192 x 7168 63 us, with two 70; but 11468 x
  // 5120 64 us, with two 61, and without a residual 50 and 40).
  if (a.nvec <= 64) return run_norm<2, GRAN, FMT, true>(a, 256, c);
  if (a.nvec <= 128 && a.T >= 8192) return run_norm<4, GRAN, FMT, true>(a, 256, c);
  if (a.nvec <= 640 || (a.nvec <= 1024 && a.T < 2048))
    return run_norm<2, GRAN, FMT, false>(a, (int)round_up64(ceil_div64(a.nvec, 2), 32), c);
  return run_norm<4, GRAN, FMT, false>(a, (int)round_up64(ceil_div64(a.nvec, 4), 32), c);
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
  a.inv_H = 1.0f / (float)H;
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
// Backward. Rows pass in order through shared memory. A persistent CTA takes groups of `rows` consecutive rows
// with a grid stride, a team of threads a row. A group's inputs arrive by bulk copies, a tensor each, a group
// or more ahead, so that memory does not wait for a row's reduction and its barrier; a thread has its
// vectors in registers before the group's barrier, behind which the stage is loaded anew. A thread owns VPT vectors of every row of its team, so its share of dw stays
// in registers from row to row; a CTA's teams add theirs up at the end, and it leaves as one of `grid`
// partial rows in the workspace. A second kernel adds the partial rows in a fixed order: no atomics, the
// same bits on every run.
namespace {

constexpr int kRingStages = 3;
constexpr int kRingRoom = 220 * 1024;  // of an SM, for its CTAs' rings together

FP8_DEVI void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

struct RingShape {
  int vpt, team, rows, ctas, stages, tensors;
};
// One vector a thread up to 8192 columns, two up to 12288 (4096 x 12288 70 us; with four, on 384 threads, 79), four
// beyond; teams for several short rows up to 512 threads a CTA, as many CTAs an SM as make 1024 threads with one vector
// each (one CTA with more: it needs the registers), and up to three groups in a CTA's ring. Measured for 8192 x
// 7168, 470 MB: 74 us, 94% of the copy rate; with the weights read from L1 row by row instead of kept in registers
// 93 us, with two vectors a thread and two CTAs an SM (spills) 91 us, with a ring of five groups 2 us more. Without
// dh (353 MB) 68 us: there the ~250 instructions a warp and row and the barrier bound it.
inline RingShape ring_shape(int nvec, int tensors) {
  RingShape r;
  r.vpt = nvec <= 1024 ? 1 : nvec <= 1536 ? 2 : 4;
  r.team = (int)round_up64(ceil_div64(nvec, r.vpt), 32);
  r.rows = r.team > 512 ? 1 : 512 / r.team < 8 ? 512 / r.team : 8;
  r.ctas = r.vpt == 1 && r.team * r.rows <= 512 ? 2 : 1;
  r.tensors = tensors;
  const int fit = kRingRoom / r.ctas / (tensors * r.rows * nvec * 16);
  r.stages = fit < kRingStages ? fit : kRingStages;
  return r;
}
// CTAs: by the shape with three tensors, so that the partial rows do not depend on dh
inline int64_t ring_grid(int64_t T, int64_t H) {
  const RingShape r = ring_shape((int)(H / 8), 3);
  const int64_t groups = ceil_div64(T, r.rows);
  return groups < 152 * r.ctas ? groups : 152 * r.ctas;
}

struct Ring {
  const uint4* src[3];
  int64_t T, groups;
  int nvec, slab;  // vectors of a row, of a tensor's part of a stage
  int test_stall;  // each CTA's first group is never loaded
  RingShape r;
  FP8_DEVI void load(uint4* ring, uint64_t* full, int64_t g, int s) const {
    if (g >= groups) return;
    const int64_t row = g * r.rows;
    const uint32_t bytes = (uint32_t)min((int64_t)r.rows, T - row) * (uint32_t)nvec * 16;
    mbar_arrive_expect_tx(&full[s], bytes * r.tensors);
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (i < r.tensors) bulk_load(ring + (s * r.tensors + i) * slab, src[i] + row * nvec, bytes, &full[s]);
  }
  FP8_DEVI void start(uint4* ring, uint64_t* full) const {
    if (threadIdx.x == 0) {
      for (int s = 0; s < r.stages; ++s) mbar_init(&full[s], 1);
      fence_mbar_init();
      pdl_wait();
      for (int s = test_stall ? 1 : 0; s < r.stages; ++s) load(ring, full, blockIdx.x + (int64_t)s * gridDim.x, s);
    }
    pdl_wait();
    __syncthreads();
  }
  // The loads in flight land, where group stages - 1 behind g is the last that was asked for.
  FP8_DEVI void drain(uint64_t* full, int64_t g) const {
    int64_t use = (g - blockIdx.x) / gridDim.x;
    for (int i = 0; i < r.stages && g < groups; ++i, ++use, g += gridDim.x)
      if (use > 0 || !test_stall) mbar_wait(&full[use % r.stages], (uint32_t)(use / r.stages) & 1, nullptr, kDrainNs);
  }
};
inline Ring make_ring(const void* a, const void* b, const void* c, int64_t T, int64_t H, int test_stall) {
  Ring q = {};
  int n = 0;
  for (const void* t : {a, b, c})
    if (t) q.src[n++] = static_cast<const uint4*>(t);
  q.nvec = (int)(H / 8);
  q.r = ring_shape(q.nvec, n);
  q.T = T;
  q.groups = ceil_div64(T, q.r.rows);
  q.slab = q.r.rows * q.nvec;
  q.test_stall = test_stall;
  return q;
}
inline size_t ring_bytes(const Ring& q) { return (size_t)q.r.stages * q.r.tensors * q.slab * 16; }

// Once for each device: the ring's shared memory.
template <typename K>
int allow_ring(K kern, std::atomic<uint64_t>& done, const Ctx& c) {
  const uint64_t bit = 1ull << (c.device & 63);
  if (done.load(std::memory_order_acquire) & bit) return FP8_OK;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingRoom) != cudaSuccess)
    return FP8_ERR_CUDA;
  done.fetch_or(bit, std::memory_order_release);
  return FP8_OK;
}

struct NormBwdArgs {
  const void* w;
  const float* rstd;
  uint4* dx;        // may be null
  float* part;      // [grid][H], null without dw
  float inv_H;
  uint64_t wait_ns;
};

template <int VPT, bool WF32, bool HAS_DH>
__global__ void __launch_bounds__(VPT == 1 ? 1024 : VPT == 2 ? 768 : 512, 1) rmsnorm_bwd_kernel(const NormBwdArgs p, const Ring q) {
  extern __shared__ uint4 ring[];  // [stages][dy, h, dh][rows][nvec]
  __shared__ uint64_t full[kRingStages];
  __shared__ __align__(16) float red[2][8][32];
  const int nvec = q.nvec;
  const int team = threadIdx.x / q.r.team, t = threadIdx.x % q.r.team;
  constexpr int kTensors = HAS_DH ? 3 : 2;
  __shared__ volatile int lost;       // a wait ran out
  __shared__ volatile int64_t lost_g;  // the group behind which there were no more loads
  if (threadIdx.x == 0) lost = 0, lost_g = -1;
  q.start(ring, full);
  float2 dw[VPT][4];
  uint4 wv[VPT];  // bf16 weights stay in registers; fp32 ones, twice as many, come from L1
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = t + i * q.r.team;
    wv[i] = !WF32 && c < nvec ? ld_stream(static_cast<const uint4*>(p.w) + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[i][j] = both(0.f);
  }
  int st = 0, par = 0;
  uint32_t phase = 0;
  auto row_rstd = [&](int64_t g) {
    const int64_t row = g * q.r.rows + team;
    return row < q.T ? p.rstd[row] : 0.f;
  };
  float rstd_next = row_rstd(blockIdx.x);
  for (int64_t g = blockIdx.x; g < q.groups; g += gridDim.x, par ^= 1) {
    const int64_t row = g * q.r.rows + team;
    const bool active = row < q.T;
    const float rstd = rstd_next;
    rstd_next = row_rstd(g + gridDim.x);
    if (!mbar_wait(&full[st], phase, &lost, p.wait_ns)) lost = 1;
    const uint4* in = ring + st * kTensors * q.slab + team * nvec;
    uint4 vdy[VPT], vh[VPT], vdh[VPT];
    float2 sum2 = both(0.f);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = t + i * q.r.team;
      if (!active || c >= nvec) continue;
      vdy[i] = in[c];
      vh[i] = in[q.slab + c];
      vdh[i] = HAS_DH ? in[2 * q.slab + c] : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 dyh = fmul2_rn(unpack2(word(vdy[i], j)), unpack2(word(vh[i], j)));
        dw[i][j] = ffma2_rn(dyh, both(rstd), dw[i][j]);
        sum2 = ffma2_rn(dyh, WF32 ? static_cast<const float2*>(p.w)[4 * c + j] : unpack2(word(wv[i], j)), sum2);
      }
    }
    float sum = sum2.x + sum2.y;  // of dy * w * h: rstd comes in below
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    team_put(red[par][team], t, q.r.team / 32, sum);  // two buffers: a group's are read while the next one's are written
    __syncthreads();
    if (threadIdx.x == 0) {
      if (!lost)
        q.load(ring, full, g + (int64_t)q.r.stages * gridDim.x, st);
      else if (lost_g < 0)
        lost_g = g;
    }
    if (++st == q.r.stages) st = 0, phase ^= 1;
    if (!p.dx || !active) continue;
    const float c1 = rstd * rstd * (rstd * team_sum<VPT == 1>(red[par][team], q.r.team / 32) * p.inv_H);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = t + i * q.r.team;
      if (c >= nvec) continue;
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 g2 = ffma2_rn(unpack2(word(vh[i], j)), both(-c1), unpack2(word(vdh[i], j)));
        o[j] = pack_bf16(ffma2_rn(fmul2_rn(unpack2(word(vdy[i], j)), WF32 ? static_cast<const float2*>(p.w)[4 * c + j] : unpack2(word(wv[i], j))), both(rstd), g2));
      }
      p.dx[row * nvec + c] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
  // A wait that ran out ended all other waits and the loads; what was computed from there on means nothing. NaN in all
  // of the CTA's rows and of dw. (Ending the loop there instead took 69.3 us without dh, not 67.9.)
  if (lost) {
    if (threadIdx.x == 0) q.drain(full, lost_g);
    __syncthreads();
    for (int64_t row = (int64_t)blockIdx.x * q.r.rows + team; p.dx && row < q.T; row += (int64_t)gridDim.x * q.r.rows)
      for (int c = t; c < nvec; c += q.r.team) p.dx[row * nvec + c] = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) dw[i][j] = both(__uint_as_float(0x7FC00000u));
  }
  if (p.part) {
    float4* mine = reinterpret_cast<float4*>(p.part) + (int64_t)blockIdx.x * nvec * 2;
    float4* sh = reinterpret_cast<float4*>(ring);  // [rows][2 nvec]: every load has landed and been read
    if (q.r.rows > 1) __syncthreads();
    float4* out = q.r.rows > 1 ? sh + team * nvec * 2 : mine;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = t + i * q.r.team;
      if (c >= nvec) continue;
      out[2 * c] = make_float4(dw[i][0].x, dw[i][0].y, dw[i][1].x, dw[i][1].y);
      out[2 * c + 1] = make_float4(dw[i][2].x, dw[i][2].y, dw[i][3].x, dw[i][3].y);
    }
    if (q.r.rows > 1) {
      __syncthreads();
      for (int c = threadIdx.x; c < 2 * nvec; c += blockDim.x) {
        float4 a = sh[c];
        for (int r = 1; r < q.r.rows; ++r) {
          const float4 v = sh[r * 2 * nvec + c];
          a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
        }
        mine[c] = a;
      }
    }
  }
  pdl_trigger();
}

// dw[c] = sum of `parts` partial rows: 32 float4 columns a CTA, the rows split over 16 thread rows
// that are then added in order.
__global__ void __launch_bounds__(512) dw_sum_kernel(const float4* part, int parts, int n4, void* dw, int dw_bf16) {
  __shared__ float4 sh[16][32];
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x * 32 + threadIdx.x;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < n4) {
#pragma unroll 8
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
    static_cast<uint2*>(dw)[c] = make_uint2(pack_bf16(make_float2(a.x, a.y)), pack_bf16(make_float2(a.z, a.w)));
  else
    static_cast<float4*>(dw)[c] = a;
}

template <int VPT, bool WF32, bool HAS_DH>
int run_norm_bwd(const NormBwdArgs& a, const Ring& q, int grid, const Ctx& c) {
  static std::atomic<uint64_t> done{0};
  const auto kern = rmsnorm_bwd_kernel<VPT, WF32, HAS_DH>;
  const int rc = allow_ring(kern, done, c);
  if (rc != FP8_OK) return rc;
  return launch_dependent(kern, dim3(grid), dim3(q.r.team * q.r.rows), ring_bytes(q), c.stream, a, q);
}

template <int VPT>
int norm_bwd_dispatch(const NormBwdArgs& a, const Ring& q, int w_f32, int grid, const Ctx& c) {
  if (q.r.tensors == 3) return w_f32 ? run_norm_bwd<VPT, true, true>(a, q, grid, c) : run_norm_bwd<VPT, false, true>(a, q, grid, c);
  return w_f32 ? run_norm_bwd<VPT, true, false>(a, q, grid, c) : run_norm_bwd<VPT, false, false>(a, q, grid, c);
}

}  // namespace

int64_t rmsnorm_bwd_ws_bytes(int64_t T, int64_t H) { return ring_grid(T, H) * H * 4; }

int launch_rmsnorm_bwd(const void* dy, const void* h, const void* w, int w_f32, const float* rstd, const void* dh,
                       int64_t T, int64_t H, void* dx, void* dw, int dw_bf16, float* ws, const Ctx& c) {
  const Ring q = make_ring(dy, h, dh, T, H, c.test_stall);
  const int64_t grid = ring_grid(T, H);
  if (grid > 0) {
    NormBwdArgs a;
    a.w = w;
    a.rstd = rstd;
    a.dx = static_cast<uint4*>(dx);
    a.part = dw ? ws : nullptr;
    a.inv_H = 1.0f / (float)H;
    a.wait_ns = c.wait_ns;
    const int rc = q.r.vpt == 1   ? norm_bwd_dispatch<1>(a, q, w_f32, (int)grid, c)
                   : q.r.vpt == 2 ? norm_bwd_dispatch<2>(a, q, w_f32, (int)grid, c)
                                  : norm_bwd_dispatch<4>(a, q, w_f32, (int)grid, c);
    if (rc != FP8_OK) return rc;
  }
  if (!dw) return FP8_OK;
  if (grid == 0)  // no rows: an empty sum
    return cudaMemsetAsync(dw, 0, (size_t)H * (dw_bf16 ? 2 : 4), c.stream) == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
  const int n4 = (int)(H / 4);
  return launch_dependent(dw_sum_kernel, dim3((unsigned)ceil_div64(n4, 32)), dim3(32, 16), 0, c.stream,
                          static_cast<const float4*>(static_cast<const void*>(ws)), (int)grid, n4, dw, dw_bf16);
}

}  // namespace fp8lin
