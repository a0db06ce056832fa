// The router of a mixture-of-experts layer (sm_103a): top-k experts of each token, their weights,
// the table of the (token, expert) slots sorted by expert that the grouped GEMM's offsets need,
// and the gradient of the logits.
//
//   sel[e] = logit[e] + bias[e] decides the k experts (ties: the lowest index; -inf and NaN are
//   never taken); v[e] = softmax(logits)[e] or sigmoid(logit[e]); w_j = scale * v[e_j], or with
//   renormalization scale * v[e_j] / sum_i v[e_i].
#include "common.cuh"
#include "internal.h"

namespace fp8lin {

namespace {

constexpr int kRouteWarps = 8;

FP8_DEVI float load_logit(const void* p, int bf16, int64_t i) {
  return bf16 ? __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(p) + i) << 16)
              : __ldg(static_cast<const float*>(p) + i);
}
FP8_DEVI void store_logit(void* p, int bf16, int64_t i, float v) {
  if (bf16)
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(p)[i] = v;
}
FP8_DEVI float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
FP8_DEVI float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Unsigned keys in the order of the values: -inf is kKeyMasked, a NaN counts as -inf, 0 is below
// every value (an expert already taken).
constexpr uint32_t kKeyMasked = 0x007FFFFFu;
FP8_DEVI uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v);
  const uint32_t k = b & 0x80000000u ? ~b : b | 0x80000000u;
  return v != v ? kKeyMasked : (v == 0.0f ? 0x80000000u : k);  // -0 and +0 are level
}

struct RouteArgs {
  const void* logits;
  int bf16;
  const float* bias;  // may be null
  int64_t T;
  int E, k;
  int softmax, renorm;
  float scale;
  int32_t* ids;
  float* weights;
  int32_t* order;  // the table's outputs: all or none
  int32_t* pos;
  int32_t* ends;
  int32_t* hist;       // workspace [chunks][E]: slots of each chunk of tokens by expert, then their places
  int64_t per_chunk;   // tokens of a chunk (one CTA's)
  int chunks;
};

// A warp per token: lane l holds experts l + 32 i.
template <int VPL>
FP8_DEVI void route_token(const RouteArgs& p, int64_t t, int lane, int32_t* hist) {
  float v[VPL];
  uint32_t key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 32 * i;
    v[i] = e < p.E ? load_logit(p.logits, p.bf16, t * p.E + e) : 0.f;
    key[i] = e < p.E ? order_key(p.bias ? v[i] + __ldg(p.bias + e) : v[i]) : 0u;
  }
  int my_id = -1;
  float my_v = 0.f;  // lane j: the j-th expert taken and its logit
  for (int j = 0; j < p.k; ++j) {
    uint32_t best = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (key[i] > best) best = key[i], at = i;
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    if (top <= kKeyMasked) break;  // nothing left that may be taken
    const uint32_t e = __reduce_min_sync(0xffffffffu, best == top ? (uint32_t)(lane + 32 * at) : 0xffffffffu);
    float val = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if ((int)e == lane + 32 * i) {
        key[i] = 0;
        val = v[i];
      }
    val = __shfl_sync(0xffffffffu, val, e & 31);
    if (lane == j) my_id = (int)e, my_v = val;
  }
  float w = 0.f;
  if (p.softmax) {
    if (p.renorm) {  // softmax over the experts taken
      const float m = warp_max(my_id >= 0 ? my_v : -INFINITY);
      w = my_id >= 0 ? expf(my_v - m) : 0.f;
      w = w / warp_sum(w);
    } else {
      float m = -INFINITY, z = 0.f;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (lane + 32 * i < p.E) m = fmaxf(m, v[i]);
      m = warp_max(m);
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (lane + 32 * i < p.E) z += expf(v[i] - m);
      w = expf(my_v - m) / warp_sum(z);
    }
  } else {
    w = my_id >= 0 ? 1.0f / (1.0f + expf(-my_v)) : 0.f;
    if (p.renorm) w = w / (warp_sum(w) + 1e-20f);
  }
  if (lane < p.k) {
    p.ids[t * p.k + lane] = my_id;
    p.weights[t * p.k + lane] = my_id >= 0 ? w * p.scale : 0.f;
    if (hist && my_id >= 0) atomicAdd(hist + my_id, 1);
  }
}

template <int VPL>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const RouteArgs p) {
  extern __shared__ int32_t hist[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (p.order)
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  const int64_t t0 = blockIdx.x * p.per_chunk;
  const int64_t t1 = t0 + p.per_chunk < p.T ? t0 + p.per_chunk : p.T;
  for (int64_t t = t0 + warp; t < t1; t += kRouteWarps) route_token<VPL>(p, t, lane, p.order ? hist : nullptr);
  if (!p.order) return;
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) p.hist[(int64_t)blockIdx.x * p.E + e] = hist[e];
}

// The places where each chunk's slots of each expert begin, and the experts' ends. One CTA, a
// thread per expert.
__global__ void __launch_bounds__(1024) route_scan_kernel(const RouteArgs p) {
  __shared__ int32_t wsum[32];
  const int e = threadIdx.x, lane = e & 31, warp = e >> 5;
  int n = 0;
  if (e < p.E)
    for (int c = 0; c < p.chunks; ++c) n += p.hist[(int64_t)c * p.E + e];
  int x = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) wsum[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int s = lane < (int)blockDim.x / 32 ? wsum[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    wsum[lane] = s;
  }
  __syncthreads();
  const int end = x + (warp ? wsum[warp - 1] : 0);
  if (e >= p.E) return;
  p.ends[e] = end;
  int at = end - n;
  for (int c = 0; c < p.chunks; ++c) {
    int32_t* h = p.hist + (int64_t)c * p.E + e;
    const int m = *h;
    *h = at;
    at += m;
  }
}

// Each slot's place: its chunk's place of its expert plus the slots of that expert before it in the
// chunk, counted by one warp in slot order.
__global__ void __launch_bounds__(32 * kRouteWarps) route_place_kernel(const RouteArgs p) {
  extern __shared__ int32_t at[];
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) at[e] = p.hist[(int64_t)blockIdx.x * p.E + e];
  __syncthreads();
  const int64_t n = p.T * p.k;
  const int64_t valid = p.ends[p.E - 1];
  for (int64_t i = valid + (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x)
    p.order[i] = -1;
  if (threadIdx.x >= 32) return;
  const int lane = threadIdx.x;
  const int64_t s0 = blockIdx.x * p.per_chunk * p.k;
  const int64_t s1 = s0 + p.per_chunk * p.k < n ? s0 + p.per_chunk * p.k : n;
  for (int64_t b = s0; b < s1; b += 32) {
    const int64_t s = b + lane;
    const int id = s < s1 ? p.ids[s] : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, id);
    const int before = __popc(same & ((1u << lane) - 1));
    int32_t place = -1;
    if (id >= 0) place = at[id] + before;
    __syncwarp();
    if (id >= 0 && before == 0) at[id] += __popc(same);
    __syncwarp();
    if (s < s1) {
      p.pos[s] = place;
      if (id >= 0) p.order[place] = (int32_t)s;
    }
  }
}

// Gradient of the logits, a warp per token. With g_j = scale * dweights_j:
//   softmax            d[e] = v[e] (g[e] - sum_j g_j v_j), every expert
//   softmax, renorm    d[e_j] = u_j (g_j - sum_i g_i u_i), u the softmax over the experts taken
//   sigmoid            d[e_j] = g_j v_j (1 - v_j)
//   sigmoid, renorm    g_j is first (g_j - sum_i g_i v_i / z) / z, z = sum_i v_i + 1e-20
struct RouteBwdArgs {
  const void* logits;
  int bf16;
  const int32_t* ids;
  const float* dw;
  void* dlogits;
  int64_t T;
  int E, k;
  int softmax, renorm;
  float scale;
  int32_t* status;
};

template <int VPL>
__global__ void __launch_bounds__(32 * kRouteWarps) route_bwd_kernel(const RouteBwdArgs p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
  if (t >= p.T) return;
  int id = lane < p.k ? p.ids[t * p.k + lane] : -1;
  float g = lane < p.k ? p.dw[t * p.k + lane] * p.scale : 0.f;
  if (id < -1 || id >= p.E) {
    set_status(p.status, FP8_DEV_BAD_IDS);
    id = -1;
  }
  if (id < 0) g = 0.f;
  const float l = id >= 0 ? load_logit(p.logits, p.bf16, t * p.E + id) : 0.f;
  float d = 0.f;
  float v[VPL];
  float base = 0.f;
  if (p.softmax && !p.renorm) {
    float m = -INFINITY, z = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 32 * i;
      v[i] = e < p.E ? load_logit(p.logits, p.bf16, t * p.E + e) : -INFINITY;
      m = fmaxf(m, v[i]);
    }
    m = warp_max(m);
    const bool none = m == -INFINITY;  // a row of masked logits: no probabilities, no gradient
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      v[i] = none || lane + 32 * i >= p.E ? 0.f : expf(v[i] - m);
      z += v[i];
    }
    z = warp_sum(z);
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = none ? 0.f : v[i] / z;
    d = id >= 0 && !none ? g * (expf(l - m) / z) : 0.f;
    base = -warp_sum(d);
  } else if (p.softmax) {
    const float m = warp_max(id >= 0 ? l : -INFINITY);
    float u = id >= 0 && m > -INFINITY ? expf(l - m) : 0.f;
    const float z = warp_sum(u);
    u = z > 0.f ? u / z : 0.f;
    d = u * (g - warp_sum(g * u));
  } else {
    const float s = id >= 0 ? 1.0f / (1.0f + expf(-l)) : 0.f;
    if (p.renorm) {
      const float z = warp_sum(s) + 1e-20f;
      g = (g - warp_sum(g * s) / z) / z;
    }
    d = g * s * (1.0f - s);
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 32 * i;
    if (e < p.E) store_logit(p.dlogits, p.bf16, t * p.E + e, p.softmax && !p.renorm ? base * v[i] : 0.f);
  }
  // an expert named twice gets the sum of its slots
  float all = 0.f;
  for (int j = 0; j < p.k; ++j) {
    const int idj = __shfl_sync(0xffffffffu, id, j);
    const float dj = __shfl_sync(0xffffffffu, d, j);
    if (idj == id) all += dj;
  }
  if (p.softmax && !p.renorm) {
    float pe = 0.f;
    for (int j = 0; j < p.k; ++j) {  // the expert's probability, from the lane that holds it
      const int idj = __shfl_sync(0xffffffffu, id, j);
      float mine = 0.f;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (idj == lane + 32 * i) mine = v[i];
      const float got = __shfl_sync(0xffffffffu, mine, idj & 31);
      if (lane == j) pe = got;
    }
    all += base * pe;
  }
  __syncwarp();  // the row's stores above come first
  if (id >= 0) store_logit(p.dlogits, p.bf16, t * p.E + id, all);
}

constexpr int64_t kRouteChunks = 304;
int64_t chunk_tokens(int64_t T) {
  const int64_t n = ceil_div64(T, kRouteChunks);
  return round_up64(n < 1 ? 1 : n, kRouteWarps);
}

#define FP8_BY_EXPERTS(E, CALL)      \
  do {                               \
    if ((E) <= 32) { CALL(1); }      \
    else if ((E) <= 64) { CALL(2); } \
    else if ((E) <= 128) { CALL(4); } \
    else if ((E) <= 256) { CALL(8); } \
    else if ((E) <= 512) { CALL(16); } \
    else { CALL(32); }               \
  } while (0)

}  // namespace

int64_t route_ws_bytes(int64_t T, int64_t E) { return ceil_div64(T, chunk_tokens(T)) * E * 4; }

int launch_route(const void* logits, int bf16, const float* bias, int64_t T, int64_t E, int64_t k, int softmax,
                 int renorm, float scale, int32_t* ids, float* weights, int32_t* order, int32_t* pos, int32_t* ends,
                 void* ws, const Ctx& c) {
  if (T == 0) {
    if (ends && cudaMemsetAsync(ends, 0, (size_t)E * 4, c.stream) != cudaSuccess) return FP8_ERR_CUDA;
    return FP8_OK;
  }
  RouteArgs a = {logits, bf16, bias, T,    (int)E, (int)k, softmax, renorm, scale, ids, weights,
                 order,  pos,  ends, static_cast<int32_t*>(ws), chunk_tokens(T), 0};
  a.chunks = (int)ceil_div64(T, a.per_chunk);
  const size_t smem = (size_t)E * 4;
#define FP8_ROUTE(V) route_kernel<V><<<(unsigned)a.chunks, 32 * kRouteWarps, smem, c.stream>>>(a)
  FP8_BY_EXPERTS(E, FP8_ROUTE);
#undef FP8_ROUTE
  if (order) {
    route_scan_kernel<<<1, (unsigned)round_up64(E, 32), 0, c.stream>>>(a);
    route_place_kernel<<<(unsigned)a.chunks, 32 * kRouteWarps, smem, c.stream>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
}

int launch_route_bwd(const void* logits, int bf16, const int32_t* ids, const float* dw, int64_t T, int64_t E,
                     int64_t k, int softmax, int renorm, float scale, void* dlogits, const Ctx& c) {
  if (T == 0) return FP8_OK;
  const RouteBwdArgs a = {logits, bf16, ids, dw, dlogits, T, (int)E, (int)k, softmax, renorm, scale, c.status};
  const unsigned grid = (unsigned)ceil_div64(T, kRouteWarps);
#define FP8_ROUTE(V) route_bwd_kernel<V><<<grid, 32 * kRouteWarps, 0, c.stream>>>(a)
  FP8_BY_EXPERTS(E, FP8_ROUTE);
#undef FP8_ROUTE
  return cudaGetLastError() == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
}

}  // namespace fp8lin
