// The router of a mixture-of-experts layer (sm_103a): top-k experts of each token, their weights,
// the table of the (token, expert) slots sorted by expert that the grouped GEMM's offsets need,
// and the gradient of the logits.
//
//   v[e] = softmax(logits)[e] or sigmoid(logit[e]); sel[e] = logit[e] + bias[e] or (BIASED) v[e] + bias[e]
//   decides the k experts (ties: the lowest index; a logit or sum of -inf or NaN is never taken);
//   w_j = scale * v[e_j], or with renormalization scale * v[e_j] / sum_i v[e_i].
//
// Few tokens: one CTA chooses, counts and places. More take two launches, the second started while the first
// runs (programmatic dependent launch). 16384 tokens of 256 experts, k = 8: 16.1 us, of which the choice 10; the
// bytes are 2.8 us. It is bound by the choice's ~500 instructions a token and their latency at 32 warps an SM. Candidates
// gathered by each lane's next one in turn, with their logits loaded again, are fewer instructions but took 1.2 us more.
#include "common.cuh"
#include "internal.h"

namespace fp8lin {

namespace {

constexpr int kBwdWarps = 8;

FP8_DEVI float load_logit(const void* p, int bf16, int64_t i) {
  return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16)
              : static_cast<const float*>(p)[i];
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

// Which experts a lane holds: VEC, where E % 4 == 0, four neighbours at a time (16- or 8-byte loads),
// else one of each 32.
template <bool VEC>
FP8_DEVI int expert_of(int lane, int i) {
  return VEC ? (i >> 2) * 128 + lane * 4 + (i & 3) : lane + 32 * i;
}
// A row's logits (or a row of fp32 values); experts past E get `none`.
template <int VPL, bool VEC>
FP8_DEVI void load_row(const void* p, int bf16, int64_t row, int E, int lane, float none, float* v) {
  if (VEC) {
#pragma unroll
    for (int i = 0; i < VPL; i += 4) {
      const int e = expert_of<true>(lane, i);
      float4 q = make_float4(none, none, none, none);
      if (e < E) {
        if (bf16) {
          const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + row * E + e);
          q = make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                          __uint_as_float(w.y & 0xFFFF0000u));
        } else {
          q = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + row * E + e);
        }
      }
      v[i] = q.x;
      if (VPL > 1) v[(i + 1) % VPL] = q.y, v[(i + 2) % VPL] = q.z, v[(i + 3) % VPL] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = lane + 32 * i < E ? load_logit(p, bf16, row * E + lane + 32 * i) : none;
  }
}
template <int VPL, bool VEC>
FP8_DEVI void store_row(void* p, int bf16, int64_t row, int E, int lane, const float* v) {
  if (VEC) {
#pragma unroll
    for (int i = 0; i < VPL; i += 4) {
      const int e = expert_of<true>(lane, i);
      if (e >= E) continue;
      const float4 q = make_float4(v[i], v[(i + 1) % VPL], v[(i + 2) % VPL], v[(i + 3) % VPL]);
      if (bf16) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(q.x, q.y), hi = __floats2bfloat162_rn(q.z, q.w);
        __nv_bfloat162* o = reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p) + row * E + e);
        o[0] = lo;
        o[1] = hi;
      } else {
        *reinterpret_cast<float4*>(static_cast<float*>(p) + row * E + e) = q;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane + 32 * i < E) store_logit(p, bf16, row * E + lane + 32 * i, v[i]);
  }
}

// The largest value of the warp's lanes; none is a NaN.
FP8_DEVI float redux_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
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
  int warps, groups, per;  // place_slots: warps that take slots, groups of them, warps of a group
};

// A warp per token. The k-th largest of the lanes' maxima is a bound that at least k experts reach, and
// few more do (9 of 256 on average for k = 8): those are gathered, one a lane, and each counts the ones
// before it. Where more than 32 reach it (level values, rows with most experts masked), k steps each take
// the largest one left. All rows by such steps took 950 instructions a token of 256 experts and k = 8, with
// each lane's best two kept 780.
struct __align__(16) Cand {
  float sel;
  int e;
  float logit;
};
template <int VPL, bool VEC, bool SOFTMAX, bool BIASED>
FP8_DEVI void route_token(const RouteArgs& p, int64_t t, int lane, const float* v, const float* bias, Cand* cand,
                          int32_t* hist) {
  float sel[VPL];
  float best = -INFINITY;
  if (BIASED) {  // the score to 4 units in the last place
    float m = 0.f, z = 0.f;
    if (SOFTMAX) {
      m = -INFINITY;
#pragma unroll
      for (int i = 0; i < VPL; ++i) m = fmaxf(m, v[i]);
      m = warp_max(m);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      sel[i] = SOFTMAX ? expf(v[i] - m) : __fdividef(1.0f, 1.0f + expf(-v[i]));
      z += fmaxf(sel[i], 0.f);  // without NaN
    }
    if (SOFTMAX) z = 1.0f / warp_sum(z);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      sel[i] = v[i] > -INFINITY ? fmaxf((SOFTMAX ? sel[i] * z : sel[i]) + bias[i], -INFINITY) : -INFINITY;
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) sel[i] = fmaxf(v[i] + bias[i], -INFINITY);  // a NaN becomes -inf; experts past E are -inf
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) best = fmaxf(best, sel[i]);
  float bound = -INFINITY;
  for (int j = 0; j < p.k; ++j) {
    bound = redux_max(best);
    if (best == bound) best = -INFINITY;
  }
  int n = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const bool in = sel[i] >= bound && sel[i] > -INFINITY;
    const uint32_t m = __ballot_sync(0xffffffffu, in);
    const int at = n + __popc(m & ((1u << lane) - 1));
    if (in && at < 32) cand[at] = {sel[i], expert_of<VEC>(lane, i), v[i]};
    n += __popc(m);
  }
  __syncwarp();
  int id = -1, rank = lane;  // this lane's expert and its place among the k
  float l = 0.f;             // its logit
  if (n <= 32) {
    if (lane < n) {
      const Cand mine = cand[lane];
      rank = 0;
#pragma unroll 4
      for (int j = 0; j < n; ++j) {
        const float2 c = *reinterpret_cast<const float2*>(&cand[j]);
        rank += c.x > mine.sel || (c.x == mine.sel && __float_as_int(c.y) < mine.e);
      }
      if (rank < p.k) id = mine.e, l = mine.logit;
    }
  } else {
    uint32_t taken = 0;
    for (int j = 0; j < p.k; ++j) {
      float b = -INFINITY;
      int bi = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (!(taken >> i & 1u) && sel[i] > b) b = sel[i], bi = i;
      const float top = redux_max(b);
      if (top == -INFINITY) break;  // nothing left that may be taken
      const uint32_t mine = b == top ? (uint32_t)expert_of<VEC>(lane, bi) : 0xffffffffu;
      const uint32_t e = __reduce_min_sync(0xffffffffu, mine);
      if (mine == e) taken |= 1u << bi;
      if (lane == j) id = (int)e;
    }
    if (id >= 0) l = load_logit(p.logits, p.bf16, t * p.E + id);
  }
  __syncwarp();  // the candidates are read before the next token's are written
  float w = 0.f;
  if (SOFTMAX) {
    if (p.renorm) {  // softmax over the experts taken
      const float m = warp_max(id >= 0 ? l : -INFINITY);
      w = id >= 0 ? expf(l - m) : 0.f;
      w = w / warp_sum(w);
    } else {
      float m = -INFINITY, z = 0.f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) m = fmaxf(m, v[i]);
      m = warp_max(m);
#pragma unroll
      for (int i = 0; i < VPL; ++i) z += expert_of<VEC>(lane, i) < p.E ? expf(v[i] - m) : 0.f;
      w = expf(l - m) / warp_sum(z);
    }
  } else {
    w = id >= 0 ? 1.0f / (1.0f + expf(-l)) : 0.f;
    if (p.renorm) w = w / (warp_sum(w) + 1e-20f);
  }
  if (id >= 0) {
    const int slot = (int)t * p.k + rank;  // T k < 2^31
    p.ids[slot] = id;
    p.weights[slot] = w * p.scale;
    if (hist) atomicAdd(hist + id, 1);
  } else if (n < p.k && lane >= n && lane < p.k) {  // fewer than k: the last slots are unused
    p.ids[t * p.k + lane] = -1;
    p.weights[t * p.k + lane] = 0.f;
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

// Each slot's place: `at` holds the chunk's first place of each expert. Warps take 32 slots each; a slot's
// place is its expert's, plus the slots of that expert in the warps before and in the lanes before. The
// warps' counts (`count`, a row of E2 a warp) are summed by two experts a thread, the warps split over up to
// 8 groups of threads whose totals (`total`, a row of E2 a group) the slots then add up.
constexpr int rank_warps(int threads, int E2) { return E2 > 512 && threads > 512 ? 16 : threads / 32; }
__host__ __device__ constexpr int most_groups(int E2) { return E2 <= 512 ? 8 : 2; }
int rank_groups(int threads, int E2) {
  int g = most_groups(E2);
  while (g > 1 && g * (E2 / 2) > threads) g >>= 1;
  return g;
}
// A batch's slots in their warps' counts (which are zero before); returns the slots of the same expert before this one
// in its warp.
FP8_DEVI int count_slot(int id, int E2, uint16_t* count) {
  const uint32_t same = __match_any_sync(0xffffffffu, id);
  const int before = __popc(same & ((1u << (threadIdx.x & 31)) - 1));
  if (id >= 0 && before == 0) count[(threadIdx.x >> 5) * E2 + id] = (uint16_t)__popc(same);
  return before;
}
FP8_DEVI void sum_counts(const RouteArgs& p, uint16_t* total, uint16_t* count) {
  const int pairs = p.E2 / 2;
  uint32_t* count2 = reinterpret_cast<uint32_t*>(count);
  for (int i = threadIdx.x; i < p.groups * pairs; i += blockDim.x) {
    const int g = i / pairs, x = i - g * pairs;
    uint32_t* c = count2 + g * p.per * pairs + x;
    uint32_t sum = 0;  // two 16-bit sums: at most 1024 slots in all
#pragma unroll 4
    for (int w = 0; w < p.per; ++w, c += pairs) {
      const uint32_t v = *c;
      *c = sum;
      sum += v;
    }
    reinterpret_cast<uint32_t*>(total)[i] = sum;
  }
}
FP8_DEVI void put_slot(const RouteArgs& p, int64_t s, int id, int before, const int32_t* at, const uint16_t* total,
                       const uint16_t* count) {
  const int warp = threadIdx.x >> 5;
  int32_t place = -1;
  if (id >= 0) {
    place = at[id] + count[warp * p.E2 + id] + before;
    for (int w = warp; w >= p.per; w -= p.per, total += p.E2) place += total[id];
    p.order[place] = (int32_t)s;
  }
  p.pos[s] = place;
}
// The slots from b to s1; `placed`: the batch before b has been placed, its totals are not yet in `at`.
FP8_DEVI void place_slots(const RouteArgs& p, int64_t b, int64_t s1, bool placed, int32_t* at, uint16_t* total,
                          uint16_t* count) {
  const int warp = threadIdx.x >> 5;
  for (; b < s1; b += 32 * p.warps, placed = true) {
    const int64_t s = b + threadIdx.x;
    const int id = warp < p.warps && s < s1 ? p.ids[s] : -1;
    if (placed) {
      __syncthreads();
      for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
        int sum = 0;
        for (int g = 0; g < p.groups; ++g) sum += total[g * p.E2 + e];
        at[e] += sum;
      }
    }
    for (int i = threadIdx.x; i < p.warps * (p.E2 / 2); i += blockDim.x) reinterpret_cast<uint32_t*>(count)[i] = 0;
    __syncthreads();
    int before = 0;
    if (warp < p.warps) before = count_slot(id, p.E2, count);
    __syncthreads();
    sum_counts(p, total, count);
    __syncthreads();
    if (warp < p.warps && s < s1) put_slot(p, s, id, before, at, total, count);
  }
}
// Unused slots leave the end of `order` without a slot.
FP8_DEVI void fill_order(const RouteArgs& p, int64_t valid) {
  for (int64_t i = valid + (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < p.T * p.k;
       i += (int64_t)gridDim.x * blockDim.x)
    p.order[i] = -1;
}

// The choice for a chunk of tokens, and the chunk's slots of each expert; with one chunk the table too.
template <int VPL, bool VEC, int WARPS, bool BF16, bool SOFTMAX, bool BIASED>
__global__ void __launch_bounds__(32 * WARPS) route_kernel(const RouteArgs p) {
  extern __shared__ __align__(16) int32_t hist[];  // [E2], then the warps' candidates, or place_slots' arrays
  __shared__ int32_t warp_sums[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Cand* cand = reinterpret_cast<Cand*>(hist + (p.E2 + 3) / 4 * 4) + warp * 32;
  if (p.order) {
    for (int e = threadIdx.x; e < p.E2; e += blockDim.x) hist[e] = 0;
    __syncthreads();
  }
  pdl_wait();
  pdl_trigger();
  const int64_t t0 = blockIdx.x * p.per_chunk;
  const int64_t t1 = t0 + p.per_chunk < p.T ? t0 + p.per_chunk : p.T;
  float bias[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) bias[i] = 0.f;
  if (p.bias) load_row<VPL, VEC>(p.bias, 0, 0, p.E, lane, 0.f, bias);
  // a warp's next row is asked for before it works on this one, where there are registers for it
  constexpr bool kAhead = VPL <= 8;
  float v[VPL], next[VPL];
  if (kAhead && t0 + warp < t1) load_row<VPL, VEC>(p.logits, BF16, t0 + warp, p.E, lane, -INFINITY, next);
  for (int64_t t = t0 + warp; t < t1; t += WARPS) {
    if (kAhead) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) v[i] = next[i];
      if (t + WARPS < t1) load_row<VPL, VEC>(p.logits, BF16, t + WARPS, p.E, lane, -INFINITY, next);
    } else {
      load_row<VPL, VEC>(p.logits, BF16, t, p.E, lane, -INFINITY, v);
    }
    route_token<VPL, VEC, SOFTMAX, BIASED>(p, t, lane, v, bias, cand, p.order ? hist : nullptr);
  }
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
  uint16_t* sums = reinterpret_cast<uint16_t*>(hist + p.E2);
  place_slots(p, 0, p.T * p.k, false, hist, sums, sums + most_groups(p.E2) * p.E2);
}

// The table from the chunks' counts. Each CTA sums the whole matrix of counts (16 bits each, 78 KB for 152
// chunks and 256 experts, from L2) into its own first places, so that no launch is spent on a scan. What it takes is a
// chain of latencies: its slots are read together with the matrix, and counted while that is summed.
constexpr int kPlaceThreads = 1024;
// ROWS: loads of the matrix in flight; 20 are all of a thread's for 152 chunks. REGS: with up to 40 a CTA fits an SM
// beside one of route_kernel for few experts (24 to 46 registers and 32 warps, too), so that it has started when the
// choice ends.
template <int ROWS, int REGS>
__global__ void __maxnreg__(REGS) route_place_kernel(const RouteArgs p) {
  extern __shared__ int32_t sh[];  // [E2] slots in the chunks before this one, [E2] slots, then place_slots' arrays
  __shared__ int32_t warp_sums[32];
  int32_t* prior = sh;
  int32_t* all = sh + p.E2;
  uint16_t* total = reinterpret_cast<uint16_t*>(sh + 2 * p.E2);
  uint16_t* count = total + most_groups(p.E2) * p.E2;
  const int warp = threadIdx.x >> 5, warps = p.warps;
  const int pairs = p.E2 / 2;  // at most kPlaceThreads / 2
  for (int e = threadIdx.x; e < 2 * p.E2; e += kPlaceThreads) sh[e] = 0;
  for (int i = threadIdx.x; i < warps * pairs; i += kPlaceThreads) reinterpret_cast<uint32_t*>(count)[i] = 0;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const int64_t n_slots = p.T * p.k, len = p.per_chunk * p.k;
  const int64_t s0 = blockIdx.x * len, s1 = s0 + len < n_slots ? s0 + len : n_slots, s = s0 + threadIdx.x;
  const int id = warp < warps && s < s1 ? p.ids[s] : -1;
  const int split = min(kPlaceThreads / pairs, 8);  // threads that share a pair of experts
  const int grp = threadIdx.x / pairs;
  if (grp < split) {
    const uint32_t* h = reinterpret_cast<const uint32_t*>(p.hist);
    const int x = threadIdx.x - grp * pairs;
    int a0 = 0, a1 = 0, b0 = 0, b1 = 0;
    const int step = split * pairs;
    for (int c0 = grp; c0 < p.chunks; c0 += ROWS * split) {
      const uint32_t* row = h + (int64_t)c0 * pairs + x;
      uint32_t v[ROWS];
#pragma unroll
      for (int i = 0; i < ROWS; ++i) v[i] = c0 + i * split < p.chunks ? row[i * step] : 0u;
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {  // both halves in one addition measured slower (1024 tokens 8.3 us, not 7.8)
        const int lo = v[i] & 0xFFFF, hi = v[i] >> 16;
        a0 += lo, a1 += hi;
        if (c0 + i * split < (int)blockIdx.x) b0 += lo, b1 += hi;
      }
    }
    atomicAdd(all + 2 * x, a0), atomicAdd(all + 2 * x + 1, a1);
    atomicAdd(prior + 2 * x, b0), atomicAdd(prior + 2 * x + 1, b1);
  }
  int before = 0;
  if (warp < warps) before = count_slot(id, p.E2, count);
  __syncthreads();
  sum_counts(p, total, count);
  // E <= kPlaceThreads: an expert a thread
  const int e = threadIdx.x;
  const int n = e < p.E ? all[e] : 0;
  const int start = block_scan(n, warp_sums);
  if (e < p.E) {
    if (blockIdx.x == 0) p.ends[e] = start + n;
    prior[e] += start;
  }
  const int64_t valid = warp_sums[31];
  __syncthreads();
  fill_order(p, valid);
  if (warp < warps && s < s1) put_slot(p, s, id, before, prior, total, count);
  place_slots(p, s0 + 32 * warps, s1, true, prior, total, count);
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

// ALL: softmax without renormalization, which every expert's logit has a gradient of.
template <int VPL, bool VEC, bool BF16, bool ALL>
__global__ void __launch_bounds__(32 * kBwdWarps) route_bwd_kernel(const RouteBwdArgs p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * kBwdWarps + warp;
  pdl_wait();
  pdl_trigger();
  if (t >= p.T) return;
  int id = lane < p.k ? p.ids[t * p.k + lane] : -1;
  float g = lane < p.k ? p.dw[t * p.k + lane] * p.scale : 0.f;
  if (id < -1 || id >= p.E) {
    set_status(p.status, FP8_DEV_BAD_IDS);
    id = -1;
  }
  if (id < 0) g = 0.f;
  const float l = id >= 0 ? load_logit(p.logits, BF16, t * p.E + id) : 0.f;
  float d = 0.f;
  float v[VPL];
  float base = 0.f, pe = 0.f;
  if (ALL) {
    float m = -INFINITY, z = 0.f;
    load_row<VPL, VEC>(p.logits, BF16, t, p.E, lane, -INFINITY, v);
#pragma unroll
    for (int i = 0; i < VPL; ++i) m = fmaxf(m, v[i]);
    m = warp_max(m);
    const bool none = m == -INFINITY;  // a row of masked logits: no probabilities, no gradient
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      v[i] = none ? 0.f : expf(v[i] - m);
      z += v[i];
    }
    z = none ? 0.f : 1.0f / warp_sum(z);
    pe = id >= 0 && !none ? expf(l - m) * z : 0.f;
    d = g * pe;
    base = -warp_sum(d);
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] *= base * z;
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
  if (!ALL) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = 0.f;
  }
  store_row<VPL, VEC>(p.dlogits, BF16, t, p.E, lane, v);
  // an expert named twice gets the sum of its slots
  float all = 0.f;
  for (int j = 0; j < p.k; ++j) {
    const int idj = __shfl_sync(0xffffffffu, id, j);
    const float dj = __shfl_sync(0xffffffffu, d, j);
    if (idj == id) all += dj;
  }
  all += base * pe;
  __syncwarp();  // the row's stores above come first
  if (id >= 0) store_logit(p.dlogits, BF16, t * p.E + id, all);
}

// Chunks of tokens: one CTA does it all for a token a warp (32 tokens of 256 experts 5.7 us, in chunks 6.0; 64 tokens 8.9
// and 6.1, of 512 experts 14.3 and 6.6, of 16 experts 5.4 and 4.9); else a chunk for each of 152 SMs, and not
// above what 16-bit counts hold.
int64_t chunk_tokens(int64_t T, int64_t E) {
  if (T <= (E <= 256 ? 32 : 16)) return T < 1 ? 1 : T;
  const int64_t n = round_up64(ceil_div64(T, 152), 8);
  return n < 65528 ? n : 65528;
}

// CALL(vectors a lane, VEC) by the number of experts
#define FP8_BY_EXPERTS(E, CALL)                                                        \
  do {                                                                                 \
    if ((E) <= 32) { CALL(1, false); }                                                 \
    else if ((E) <= 64) { CALL(2, false); }                                            \
    else if ((E) <= 128) { if ((E) % 4 == 0) { CALL(4, true); } else { CALL(4, false); } }   \
    else if ((E) <= 256) { if ((E) % 4 == 0) { CALL(8, true); } else { CALL(8, false); } }   \
    else if ((E) <= 512) { if ((E) % 4 == 0) { CALL(16, true); } else { CALL(16, false); } } \
    else { if ((E) % 4 == 0) { CALL(32, true); } else { CALL(32, false); } }                 \
  } while (0)

// Shared memory of place_slots: first places, group totals, a row of counts a warp.
size_t place_bytes(int E2) { return (size_t)E2 * (4 + 2 * most_groups(E2) + 2 * (E2 <= 512 ? 32 : 16)); }

// 32 warps a CTA where a lane holds up to 8 experts, 16 where it needs more registers. Kernels by the logits' type and
// the score: with both decided in the kernel 16384 tokens of 256 experts took 17.1 us instead of 16.5. And by where the
// bias goes: on the score, 256 sigmoids or exponentials a token more, they take 17.6.
template <int VPL, bool VEC, bool BIASED>
int run_route_on(const RouteArgs& a, size_t smem, const Ctx& c) {
  constexpr int W = VPL <= 8 ? 32 : 16;
  const auto kern = a.bf16 ? (a.softmax ? route_kernel<VPL, VEC, W, true, true, BIASED> : route_kernel<VPL, VEC, W, true, false, BIASED>)
                           : (a.softmax ? route_kernel<VPL, VEC, W, false, true, BIASED> : route_kernel<VPL, VEC, W, false, false, BIASED>);
  return launch_dependent(kern, dim3((unsigned)a.chunks), dim3(32 * W), smem, c.stream, a);
}

template <int VPL, bool VEC>
int run_route(const RouteArgs& a, bool biased, size_t smem, const Ctx& c) {
  return biased ? run_route_on<VPL, VEC, true>(a, smem, c) : run_route_on<VPL, VEC, false>(a, smem, c);
}

template <int VPL, bool VEC>
int run_route_bwd(const RouteBwdArgs& a, const Ctx& c) {
  const bool all = a.softmax && !a.renorm;
  const auto kern = a.bf16 ? (all ? route_bwd_kernel<VPL, VEC, true, true> : route_bwd_kernel<VPL, VEC, true, false>)
                           : (all ? route_bwd_kernel<VPL, VEC, false, true> : route_bwd_kernel<VPL, VEC, false, false>);
  return launch_dependent(kern, dim3((unsigned)ceil_div64(a.T, kBwdWarps)), dim3(32 * kBwdWarps), 0, c.stream, a);
}

}  // namespace

// A row of counts a chunk; 152 rows at least, so that a workspace for many tokens serves fewer too.
int64_t route_ws_bytes(int64_t T, int64_t E) {
  const int64_t chunks = ceil_div64(T, chunk_tokens(T, E));
  return round_up64((chunks < 152 ? 152 : chunks) * round_up64(E, 2) * 2, 16);
}

int launch_route(const void* logits, int bf16, const float* bias, int64_t T, int64_t E, int64_t k, int softmax,
                 int biased, int renorm, float scale, int32_t* ids, float* weights, int32_t* order, int32_t* pos, int32_t* ends,
                 void* ws, const Ctx& c) {
  if (T == 0) {
    if (ends && cudaMemsetAsync(ends, 0, (size_t)E * 4, c.stream) != cudaSuccess) return FP8_ERR_CUDA;
    return FP8_OK;
  }
  RouteArgs a = {logits, bf16, bias, T,    (int)E, (int)k, softmax, renorm, scale, ids, weights,
                 order,  pos,  ends, static_cast<uint16_t*>(ws), (int)round_up64(E, 2), chunk_tokens(T, E), 0, 0, 0, 0};
  a.chunks = (int)ceil_div64(T, a.per_chunk);
  const int threads = a.chunks > 1 ? kPlaceThreads : E <= 256 ? 1024 : 512;
  a.warps = rank_warps(threads, a.E2);
  a.groups = rank_groups(threads, a.E2);
  a.per = a.warps / a.groups;
  // up to 48 KB, which needs no attribute: place_slots' 40 to 43 KB and the candidates' 8 to 16 KB share it
  const size_t choose = (size_t)(a.E2 + 3) / 4 * 16 + (E <= 256 ? 32 : 16) * 32 * sizeof(Cand);
  const size_t smem = a.chunks == 1 && place_bytes(a.E2) > choose ? place_bytes(a.E2) : choose;
#define FP8_ROUTE(V, X) rc = run_route<V, X>(a, biased && bias, smem, c)
  int rc;
  FP8_BY_EXPERTS(E, FP8_ROUTE);
#undef FP8_ROUTE
  if (rc != FP8_OK || !order || a.chunks == 1) return rc;
  // Up to 40 chunks a thread has at most 5 rows (100 tokens of 256 experts 6.7 us, with 20 loads 7.5); few registers for
  // few experts (1024 tokens of 8 experts 5.3 us instead of 6.2, but of 256 8.3 instead of 7.9).
  const auto place = a.chunks <= 40 ? route_place_kernel<5, 40> : E <= 64 ? route_place_kernel<20, 40> : route_place_kernel<20, 64>;
  return launch_dependent(place, dim3((unsigned)a.chunks), dim3(kPlaceThreads),
                          place_bytes(a.E2) + (size_t)a.E2 * 4, c.stream, a);
}

int launch_route_bwd(const void* logits, int bf16, const int32_t* ids, const float* dw, int64_t T, int64_t E,
                     int64_t k, int softmax, int renorm, float scale, void* dlogits, const Ctx& c) {
  if (T == 0) return FP8_OK;
  const RouteBwdArgs a = {logits, bf16, ids, dw, dlogits, T, (int)E, (int)k, softmax, renorm, scale, c.status};
#define FP8_ROUTE(V, X) rc = run_route_bwd<V, X>(a, c)
  int rc;
  FP8_BY_EXPERTS(E, FP8_ROUTE);
#undef FP8_ROUTE
  return rc;
}

}  // namespace fp8lin
