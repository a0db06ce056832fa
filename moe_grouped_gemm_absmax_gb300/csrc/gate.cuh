// The gated feed-forward's elementwise part, as the GEMM's epilogues apply it to their accumulators (sm_103a).
//
//   act(g) = g s(w),  s the logistic function:  SiLU w = g;  GELU (tanh form) w = 2 c (g + a g^3), c = sqrt(2 / pi),
//   a = 0.044715, because (1 + tanh z) / 2 = s(2 z), which keeps its relative precision where 1 + tanh z cancels.
//   act'(g) = s + g s (1 - s) w'.
//   h = act(g) u;  given dh:  dg = dh u act'(g),  du = dh act(g).
// All in fp32 from the fp32 accumulators, each output rounded once. The exponential and the quotient are the fast
// ones (2 units in the last place each, and |w| 2^-24 from the argument's rounding): 2^-17 of a value at |w| = 80,
// below which s underflows; a bf16 result's half step is 2^-9.
#pragma once

#include "common.cuh"

namespace fp8lin {

FP8_DEVI float logistic(float w) { return __fdividef(1.0f, 1.0f + __expf(-w)); }

constexpr float kGelu2C = 1.5957691216057308f, kGeluA = 0.044715f;  // 2 sqrt(2 / pi), a

FP8_DEVI float act_fwd(float g, int act) {
  const float w = act == FP8_ACT_GELU ? kGelu2C * fmaf(kGeluA * g * g, g, g) : g;
  return g * logistic(w);
}
// act(g), and its derivative in *d
FP8_DEVI float act_bwd(float g, int act, float* d) {
  float w = g, dw = 1.0f;
  if (act == FP8_ACT_GELU) {
    const float g2 = kGeluA * g * g;
    w = kGelu2C * fmaf(g2, g, g);
    dw = fmaf(3.0f * kGelu2C, g2, kGelu2C);
  }
  const float s = logistic(w), a = g * s;
  *d = fmaf(a * (1.0f - s), dw, s);
  return a;
}

FP8_DEVI uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
FP8_DEVI uint4 pack_bf16x8(const float* f) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}
FP8_DEVI void unpack_bf16x8(uint4 v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(w[i] << 16), f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
}

// max(a, b) that keeps a NaN, for a block's largest magnitude
FP8_DEVI float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// N values of a row in bf16 at o, those in front of column `left` (a multiple of 8, as is every row's width: a group of
// 8 is written whole or not at all)
template <int N>
FP8_DEVI void store_row(__nv_bfloat16* o, const float* f, int64_t left) {
#pragma unroll
  for (int j = 0; j < N; j += 8)
    if (j < left) *reinterpret_cast<uint4*>(o + j) = pack_bf16x8(f + j);
}

// Codes of N values of a row, 16 bytes at a time.
template <int FMT, int N>
FP8_DEVI void store_codes(uint8_t* o, const float* f, float scale) {
#pragma unroll
  for (int j = 0; j < N; j += 16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float* v = f + j + 4 * i;
      w[i] = cvt_fp8x2<FMT>(v[0] * scale, v[1] * scale) | (cvt_fp8x2<FMT>(v[2] * scale, v[3] * scale) << 16);
    }
    *reinterpret_cast<uint4*>(o + j) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

struct GateArgs {
  int act;
  const __nv_bfloat16* gu_in;  // backward: the projections [M, 2 I]
  __nv_bfloat16* gu;           // their values [M, 2 I] (forward, may be null), or their gradients (backward)
  __nv_bfloat16* h;            // [M, I], may be null
  uint8_t* q;                  // h in 8 bits [M, I] with inverse scales [M, I / 128] of its 1 x 128 blocks, may be null
  float* inv;
  int q_fmt;
};

// Backward, N columns from n of row m: dh (fp32) with the projections' values to their gradients, and h again. gu may be
// gu_in's own buffer: every value is read by the thread that writes its place, before it does.
template <int N>
FP8_DEVI void gate_bwd_row(const GateArgs& p, const float* dh, int64_t m, int64_t n, int64_t I) {
  const __nv_bfloat16* gi = p.gu_in + m * 2 * I + n;
  __nv_bfloat16* go = p.gu + m * 2 * I + n;
#pragma unroll
  for (int j = 0; j < N; j += 8) {
    if (n + j >= I) break;
    float g[8], u[8], h[8];
    unpack_bf16x8(*reinterpret_cast<const uint4*>(gi + j), g);
    unpack_bf16x8(*reinterpret_cast<const uint4*>(gi + I + j), u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float d;
      const float a = act_bwd(g[i], p.act, &d);
      h[i] = a * u[i];
      g[i] = dh[j + i] * u[i] * d;
      u[i] = dh[j + i] * a;
    }
    *reinterpret_cast<uint4*>(go + j) = pack_bf16x8(g);
    *reinterpret_cast<uint4*>(go + I + j) = pack_bf16x8(u);
    if (p.h) *reinterpret_cast<uint4*>(p.h + m * I + n + j) = pack_bf16x8(h);
  }
}

}  // namespace fp8lin
