// The experts of a few tokens (sm_103a):
//   out[t] = sum_j weight[t, j] * W2[e] (silu(W1[e] x[t]) * (W3[e] x[t])),  e = ids[t, j],
// on FP8 weights with one inverse scale per row: w13 [E, 2 I, H] holds W1 (gate) and below it W3
// (up), w2 [E, H, I].
#include "common.cuh"
#include "internal.h"

namespace fp8lin {

namespace {

struct MoeArgs {
  const uint16_t* x;  // bf16 [T, H]
  const int32_t* ids;
  const float* weights;
  const uint8_t* w13;
  const float* s13;
  const uint8_t* w2;
  const float* s2;
  uint16_t* out;
  float* act;  // workspace [T k][I]
  int T, k, E;
  int64_t H, I;
  int32_t* status;
};

FP8_DEVI float2 e4m3x2_to_f32(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  float2 r;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(h));
  return r;
}
FP8_DEVI float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
FP8_DEVI int slot_expert(const MoeArgs& p, int slot) {
  const int e = p.ids[slot];
  if (e < -1 || e >= p.E) {
    set_status(p.status, FP8_DEV_BAD_IDS);
    return -1;
  }
  return e;
}

// A warp per (slot, row of the hidden layer).
__global__ void __launch_bounds__(256) moe_up_kernel(const MoeArgs p) {
  const int lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int slot = blockIdx.y;
  const int e = slot_expert(p, slot);
  if (e < 0 || i >= p.I) return;
  const uint16_t* x = p.x + (int64_t)(slot / p.k) * p.H;
  const int64_t r1 = (int64_t)e * 2 * p.I + i, r3 = r1 + p.I;
  float g = 0.f, u = 0.f;
  for (int64_t c = lane * 2; c < p.H; c += 64) {
    const float x0 = __uint_as_float((uint32_t)x[c] << 16), x1 = __uint_as_float((uint32_t)x[c + 1] << 16);
    const float2 a = e4m3x2_to_f32(*reinterpret_cast<const uint16_t*>(p.w13 + r1 * p.H + c));
    const float2 b = e4m3x2_to_f32(*reinterpret_cast<const uint16_t*>(p.w13 + r3 * p.H + c));
    g = fmaf(a.x, x0, fmaf(a.y, x1, g));
    u = fmaf(b.x, x0, fmaf(b.y, x1, u));
  }
  g = warp_sum(g) * p.s13[r1];
  u = warp_sum(u) * p.s13[r3];
  if (lane == 0) p.act[slot * p.I + i] = g / (1.0f + expf(-g)) * u;
}

// A warp per (token, output column), its experts in slot order.
__global__ void __launch_bounds__(256) moe_down_kernel(const MoeArgs p) {
  const int lane = threadIdx.x & 31;
  const int64_t n = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int t = blockIdx.y;
  if (n >= p.H) return;
  float y = 0.f;
  for (int j = 0; j < p.k; ++j) {
    const int slot = t * p.k + j;
    const int e = slot_expert(p, slot);
    if (e < 0) continue;
    const int64_t r = (int64_t)e * p.H + n;
    const float* a = p.act + slot * p.I;
    float d = 0.f;
    for (int64_t c = lane * 2; c < p.I; c += 64) {
      const float2 w = e4m3x2_to_f32(*reinterpret_cast<const uint16_t*>(p.w2 + r * p.I + c));
      d = fmaf(w.x, a[c], fmaf(w.y, a[c + 1], d));
    }
    y += p.weights[slot] * (warp_sum(d) * p.s2[r]);
  }
  if (lane == 0) reinterpret_cast<__nv_bfloat16*>(p.out)[t * p.H + n] = __float2bfloat16_rn(y);
}

}  // namespace

int64_t moe_tokens_ws_bytes(int64_t T, int64_t k, int64_t H, int64_t I) { return round_up64(T * k * I * 4, 16); }

int launch_moe_tokens(const void* x, const int32_t* ids, const float* weights, const void* w13, const float* s13,
                      const void* w2, const float* s2, int64_t T, int64_t k, int64_t E, int64_t H, int64_t I, void* out,
                      void* ws, const Ctx& c) {
  if (T == 0 || H == 0) return FP8_OK;
  const MoeArgs a = {static_cast<const uint16_t*>(x),
                     ids,
                     weights,
                     static_cast<const uint8_t*>(w13),
                     s13,
                     static_cast<const uint8_t*>(w2),
                     s2,
                     static_cast<uint16_t*>(out),
                     static_cast<float*>(ws),
                     (int)T,
                     (int)k,
                     (int)E,
                     H,
                     I,
                     c.status};
  if (I > 0) moe_up_kernel<<<dim3((unsigned)ceil_div64(I, 8), (unsigned)(T * k)), 256, 0, c.stream>>>(a);
  moe_down_kernel<<<dim3((unsigned)ceil_div64(H, 8), (unsigned)T), 256, 0, c.stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
}

}  // namespace fp8lin
