// The gated feed-forward's elementwise part, as the GEMM's epilogues apply it to their accumulators (sm_103a).
//
//   act(g) = g s(w),  s the logistic function:  SiLU w = g;  GELU (tanh form) w = 2 c (g + a g^3), c = sqrt(2 / pi),
//   a = 0.044715, because (1 + tanh z) / 2 = s(2 z), which keeps its relative precision where 1 + tanh z cancels.
//   act'(g) = s + g s (1 - s) w'.
//   h = act(g) u;  given dh:  dg = dh u act'(g),  du = dh act(g).
// All in fp32 from the fp32 accumulators, each output rounded once. The exponential and the reciprocal are the approximate
// instructions (2 units in the last place, and |w| 2^-24 from the argument's rounding): below 2^-17 of a value down to
// w = -87.3, where 1 + e^-w passes 2^126, its reciprocal leaves the normal range and s is 0 (e^-87.3 is 1.2e-38); a bf16
// result's half step is 2^-9 to 2^-8 of it.
#pragma once

#include "common.cuh"

namespace fp8lin {

FP8_DEVI float logistic(float w) {
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(w * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
  return s;
}

constexpr float kGelu2C = 1.5957691216057308f, kGeluA = 0.044715f;  // 2 sqrt(2 / pi), a

template <int ACT>
FP8_DEVI float act_fwd(float g) {
  const float w = ACT == FP8_ACT_GELU ? kGelu2C * fmaf(kGeluA * g * g, g, g) : g;
  return g * logistic(w);
}
// act(g), and its derivative in *d
template <int ACT>
FP8_DEVI float act_bwd(float g, float* d) {
  float w = g, dw = 1.0f;
  if (ACT == FP8_ACT_GELU) {
    const float g2 = kGeluA * g * g;
    w = kGelu2C * fmaf(g2, g, g);
    dw = fmaf(3.0f * kGelu2C, g2, kGelu2C);
  }
  const float s = logistic(w), a = g * s, t = a * (1.0f - s);
  // a saturated gate's derivative is s alone: GELU's w' overflows from |g| = 4e19 on, where t is 0
  *d = ACT == FP8_ACT_GELU ? (t == 0.0f ? s : fmaf(t, dw, s)) : fmaf(a, 1.0f - s, s);
  return a;
}
// h[0 .. N - 1] = act(g) * u: one branch on the activation for all of them, which leaves their latencies free to overlap
template <int N>
FP8_DEVI void gate_fwd(int act, const float* g, const float* u, float* h) {
  if (act == FP8_ACT_GELU) {
#pragma unroll
    for (int j = 0; j < N; ++j) h[j] = act_fwd<FP8_ACT_GELU>(g[j]) * u[j];
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) h[j] = act_fwd<FP8_ACT_SILU>(g[j]) * u[j];
  }
}

FP8_DEVI uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// max(a, b) that keeps a NaN, for a block's largest magnitude
FP8_DEVI float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 32 values of a row, packed in 16 words, at o: those in front of column `left`, a multiple of 8 as is
// every row's width, so that a group of 8 is written whole or not at all. wide: rows are 32-byte aligned.
FP8_DEVI void store_row32(__nv_bfloat16* o, const uint32_t* w, int64_t left, int wide) {
  if (wide && left >= 32) {
    st_v8(o, w);
    st_v8(o + 16, w + 8);
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (8 * j < left) *reinterpret_cast<uint4*>(o + 8 * j) = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
}
FP8_DEVI void pack_row32(const float* f, uint32_t* w) {
#pragma unroll
  for (int j = 0; j < 16; ++j) w[j] = pack_bf16(f[2 * j], f[2 * j + 1]);
}
// Codes of N values of a row.
template <int FMT, int N>
FP8_DEVI void store_codes(uint8_t* o, const float* f, float scale, int wide) {
  uint32_t w[N / 4];
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const float* v = f + 4 * i;
    w[i] = cvt_fp8x2<FMT>(v[0] * scale, v[1] * scale) | (cvt_fp8x2<FMT>(v[2] * scale, v[3] * scale) << 16);
  }
#pragma unroll
  for (int j = 0; j < N / 4; j += 8) {
    if (wide) {
      st_v8(o + 4 * j, w + j);
    } else {
      *reinterpret_cast<uint4*>(o + 4 * j) = make_uint4(w[j], w[j + 1], w[j + 2], w[j + 3]);
      *reinterpret_cast<uint4*>(o + 4 * j + 16) = make_uint4(w[j + 4], w[j + 5], w[j + 6], w[j + 7]);
    }
  }
}

struct GateArgs {
  int act;
  __nv_bfloat16* gu;           // the projections [M, 2 I] (forward, may be null), or their gradients (backward)
  __nv_bfloat16* h;            // [M, I], may be null
  uint8_t* q;                  // h in 8 bits [M, I] with inverse scales [M, I / 128] of its 1 x 128 blocks, may be null
  float* inv;
  int q_fmt;
  int wide;                    // every row of gu, h and q in use starts on 32 bytes
};

// Backward, 32 columns of a row: in c their projections, replaced by the projections' gradients from dh (fp32); h: the
// hidden layer again.
struct GuChunk {
  uint32_t g[16], u[16];
};
template <int ACT>
FP8_DEVI void gate_bwd(GuChunk& c, const float* dh, uint32_t* h) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float a[2], d[2];
    const float g[2] = {__uint_as_float(c.g[i] << 16), __uint_as_float(c.g[i] & 0xFFFF0000u)};
    const float u[2] = {__uint_as_float(c.u[i] << 16), __uint_as_float(c.u[i] & 0xFFFF0000u)};
#pragma unroll
    for (int k = 0; k < 2; ++k) a[k] = act_bwd<ACT>(g[k], &d[k]);
    // dh act' first: act' is 0 where a gate is saturated, and up to 1.13, which times the largest u would be past fp32's range
    c.g[i] = pack_bf16(dh[2 * i] * d[0] * u[0], dh[2 * i + 1] * d[1] * u[1]);
    c.u[i] = pack_bf16(dh[2 * i] * a[0], dh[2 * i + 1] * a[1]);
    h[i] = pack_bf16(a[0] * u[0], a[1] * u[1]);
  }
}

}  // namespace fp8lin
