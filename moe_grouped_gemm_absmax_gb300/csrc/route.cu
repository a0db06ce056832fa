// The router of a mixture-of-experts layer (sm_103a): top-k experts of each token, their weights,
// the table of the (token, expert) slots sorted by expert that the grouped GEMM's offsets need,
// and the gradient of the logits.
//
//   sel[e] = logit[e] + bias[e] decides the k experts (ties: the lowest index; -inf and NaN are
//   never taken); v[e] = softmax(logits)[e] or sigmoid(logit[e]); w_j = scale * v[e_j], or with
//   renormalization scale * v[e_j] / sum_i v[e_i].
//
// Up to 64 tokens one CTA chooses, counts and places; more take two launches, the second started while
// the first runs (programmatic dependent launch).
#include "common.cuh"
#include "internal.h"

namespace fp8lin {

namespace {

constexpr int kBwdWarps = 8;

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
  uint16_t* hist;      // workspace [chunks][E2]: slots of each chunk of tokens by expert
  int E2;              // E rounded up to even
  int64_t per_chunk;   // tokens of a chunk (one CTA's)
  int chunks;
};

// A warp per token: lane l holds experts l + 32 i. Each step takes the largest key left: the lanes'
// maxima meet in one warp reduction, a second one settles ties by the lowest expert, and the lane that
// holds it drops it.
template <int VPL>
FP8_DEVI void route_token(const RouteArgs& p, int64_t t, int lane, int32_t* hist) {
  float v[VPL];
  uint32_t key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 32 * i;
    v[i] = e < p.E ? load_logit(p.logits, p.bf16, t * p.E + e) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 32 * i;
    key[i] = e < p.E ? order_key(p.bias ? v[i] + __ldg(p.bias + e) : v[i]) : 0u;
  }
  int my_id = -1;  // lane j: the j-th expert taken
  for (int j = 0; j < p.k; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) best = max(best, key[i]);
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    if (top <= kKeyMasked) break;  // nothing left that may be taken
    uint32_t mine = 0xffffffffu;
#pragma unroll
    for (int i = VPL - 1; i >= 0; --i)
      if (key[i] == top) mine = (uint32_t)(lane + 32 * i);
    const uint32_t e = __reduce_min_sync(0xffffffffu, mine);
    if (e == mine) {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if ((int)e == lane + 32 * i) key[i] = 0;
    }
    if (lane == j) my_id = (int)e;
  }
  const float my_v = my_id >= 0 ? load_logit(p.logits, p.bf16, t * p.E + my_id) : 0.f;
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

// Exclusive sums over the CTA's threads (blockDim.x of them, a multiple of 32).
FP8_DEVI int block_scan(int x, int32_t* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  if (warp == 0) {
    int w = lane < (int)blockDim.x / 32 ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  return s - x + (warp ? warp_sums[warp - 1] : 0);
}

// Each slot's place: `at` holds the chunk's first place of each expert; the slots are counted in slot
// order by one warp.
FP8_DEVI void place_chunk(const RouteArgs& p, int64_t chunk, int32_t* at) {
  const int lane = threadIdx.x;
  const int64_t n = p.T * p.k, len = p.per_chunk * p.k;
  const int64_t s0 = chunk * len, s1 = s0 + len < n ? s0 + len : n;
  int next = s0 + lane < s1 ? p.ids[s0 + lane] : -1;
  for (int64_t b = s0; b < s1; b += 32) {
    const int64_t s = b + lane;
    const int id = next;
    next = s + 32 < s1 ? p.ids[s + 32] : -1;
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
// Unused slots leave the end of `order` without a slot.
FP8_DEVI void fill_order(const RouteArgs& p, int64_t valid) {
  for (int64_t i = valid + (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < p.T * p.k;
       i += (int64_t)gridDim.x * blockDim.x)
    p.order[i] = -1;
}

// The choice for a chunk of tokens, and the chunk's slots of each expert; with one chunk the table too.
template <int VPL, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) route_kernel(const RouteArgs p) {
  extern __shared__ int32_t hist[];
  __shared__ int32_t warp_sums[32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (p.order) {
    for (int e = threadIdx.x; e < p.E2; e += blockDim.x) hist[e] = 0;
    __syncthreads();
  }
  const int64_t t0 = blockIdx.x * p.per_chunk;
  const int64_t t1 = t0 + p.per_chunk < p.T ? t0 + p.per_chunk : p.T;
  for (int64_t t = t0 + warp; t < t1; t += WARPS) route_token<VPL>(p, t, lane, p.order ? hist : nullptr);
  if (!p.order) return;
  __syncthreads();
  if (p.chunks > 1) {
    for (int e = threadIdx.x; e < p.E2; e += blockDim.x) p.hist[(int64_t)blockIdx.x * p.E2 + e] = (uint16_t)hist[e];
    return;
  }
  int before = 0;
  for (int b = 0; b < p.E; b += blockDim.x) {
    const int e = b + threadIdx.x;
    const int n = e < p.E ? hist[e] : 0;
    const int start = before + block_scan(n, warp_sums);
    before += warp_sums[blockDim.x / 32 - 1];
    if (e < p.E) {
      p.ends[e] = start + n;
      hist[e] = start;
    }
    __syncthreads();
  }
  fill_order(p, before);
  if (warp == 0) place_chunk(p, 0, hist);
}

// The table from the chunks' counts. Each CTA sums the whole matrix of counts (16 bits each, 78 KB for 152
// chunks and 256 experts, from L2) into its own first places, so that no launch is spent on a scan.
constexpr int kPlaceThreads = 1024;
__global__ void __launch_bounds__(kPlaceThreads) route_place_kernel(const RouteArgs p) {
  extern __shared__ int32_t sh[];  // [E2] slots, [E2] slots in the chunks before this one
  __shared__ int32_t warp_sums[32];
  int32_t* total = sh;
  int32_t* prior = sh + p.E2;
  for (int e = threadIdx.x; e < 2 * p.E2; e += kPlaceThreads) sh[e] = 0;
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int pairs = p.E2 / 2;
  const int lanes = pairs < kPlaceThreads ? pairs : kPlaceThreads;  // threads on a row of counts
  const int split = kPlaceThreads / lanes;
  const int grp = threadIdx.x / lanes;
  if (grp < split) {
    const uint32_t* h = reinterpret_cast<const uint32_t*>(p.hist);
    const int x = threadIdx.x % lanes;
    int a0 = 0, a1 = 0, b0 = 0, b1 = 0;
#pragma unroll 8
    for (int c = grp; c < p.chunks; c += split) {
      const uint32_t v = __ldcg(h + (int64_t)c * pairs + x);
      const int lo = v & 0xFFFF, hi = v >> 16;
      a0 += lo, a1 += hi;
      if (c < (int)blockIdx.x) b0 += lo, b1 += hi;
    }
    atomicAdd(total + 2 * x, a0), atomicAdd(total + 2 * x + 1, a1);
    atomicAdd(prior + 2 * x, b0), atomicAdd(prior + 2 * x + 1, b1);
  }
  __syncthreads();
  // E <= kPlaceThreads: an expert a thread
  const int e = threadIdx.x;
  const int n = e < p.E ? total[e] : 0;
  const int start = block_scan(n, warp_sums);
  if (e < p.E) {
    if (blockIdx.x == 0) p.ends[e] = start + n;
    prior[e] += start;
  }
  const int64_t valid = warp_sums[31];
  __syncthreads();
  fill_order(p, valid);
  if (threadIdx.x < 32) place_chunk(p, blockIdx.x, prior);
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
__global__ void __launch_bounds__(32 * kBwdWarps) route_bwd_kernel(const RouteBwdArgs p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * kBwdWarps + warp;
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
  float base = 0.f, pe = 0.f;
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
    pe = id >= 0 && !none ? expf(l - m) / z : 0.f;
    d = g * pe;
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
  all += base * pe;
  __syncwarp();  // the row's stores above come first
  if (id >= 0) store_logit(p.dlogits, p.bf16, t * p.E + id, all);
}

// Chunks of tokens: one CTA does it all for as many tokens as its warps have twice over; else a chunk
// for each of 152 SMs, and not above what 16-bit counts hold.
int64_t chunk_tokens(int64_t T) {
  if (T <= 64) return T < 1 ? 1 : T;
  const int64_t n = round_up64(ceil_div64(T, 152), 8);
  return n < 65528 ? n : 65528;
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

int64_t route_ws_bytes(int64_t T, int64_t E) { return round_up64(ceil_div64(T, chunk_tokens(T)) * round_up64(E, 2) * 2, 16); }

int launch_route(const void* logits, int bf16, const float* bias, int64_t T, int64_t E, int64_t k, int softmax,
                 int renorm, float scale, int32_t* ids, float* weights, int32_t* order, int32_t* pos, int32_t* ends,
                 void* ws, const Ctx& c) {
  if (T == 0) {
    if (ends && cudaMemsetAsync(ends, 0, (size_t)E * 4, c.stream) != cudaSuccess) return FP8_ERR_CUDA;
    return FP8_OK;
  }
  RouteArgs a = {logits, bf16, bias, T,    (int)E, (int)k, softmax, renorm, scale, ids, weights,
                 order,  pos,  ends, static_cast<uint16_t*>(ws), (int)round_up64(E, 2), chunk_tokens(T), 0};
  a.chunks = (int)ceil_div64(T, a.per_chunk);
  // 32 warps a CTA where a lane holds up to 8 experts, 16 where it needs more registers
#define FP8_ROUTE(V) \
  route_kernel<V, (V <= 8 ? 32 : 16)><<<(unsigned)a.chunks, V <= 8 ? 1024 : 512, (size_t)a.E2 * 4, c.stream>>>(a)
  FP8_BY_EXPERTS(E, FP8_ROUTE);
#undef FP8_ROUTE
  if (cudaGetLastError() != cudaSuccess) return FP8_ERR_CUDA;
  if (!order || a.chunks == 1) return FP8_OK;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)a.chunks);
  cfg.blockDim = dim3(kPlaceThreads);
  cfg.dynamicSmemBytes = (size_t)a.E2 * 8;
  cfg.stream = c.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, route_place_kernel, a) == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
}

int launch_route_bwd(const void* logits, int bf16, const int32_t* ids, const float* dw, int64_t T, int64_t E,
                     int64_t k, int softmax, int renorm, float scale, void* dlogits, const Ctx& c) {
  if (T == 0) return FP8_OK;
  const RouteBwdArgs a = {logits, bf16, ids, dw, dlogits, T, (int)E, (int)k, softmax, renorm, scale, c.status};
  const unsigned grid = (unsigned)ceil_div64(T, kBwdWarps);
#define FP8_ROUTE(V) route_bwd_kernel<V><<<grid, 32 * kBwdWarps, 0, c.stream>>>(a)
  FP8_BY_EXPERTS(E, FP8_ROUTE);
#undef FP8_ROUTE
  return cudaGetLastError() == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
}

}  // namespace fp8lin
