// The experts of a few tokens (sm_103a):
//   out[t] = sum_j weight[t, j] * W2[e] (silu(W1[e] x[t]) * (W3[e] x[t])),  e = ids[t, j],
// on FP8 weights with one inverse scale per row: w13 [E, 2 I, H] holds W1 (gate) and below it W3
// (up), w2 [E, H, I].
//
// With a few tokens the work is reading the named experts' weights once; everything here serves to
// keep that stream going. One persistent cooperative launch, one CTA per SM:
//  - The weights are the MMA's A operand (tcgen05.mma kind::f8f6f4, M = 128 weight rows), so they go
//    from HBM by TMA into a shared-memory ring and from there into the tensor cores without
//    passing through registers. The tokens are its N.
//  - The activations keep their precision although the MMA takes 8-bit operands: a value v, scaled
//    by a power of two so that its row's largest lies in [128, 256), is split into e4m3 parts
//    v = p0 + p1 / 16 + p2 / 256, each part the rounding of 16 times what the ones before left. e4m3
//    has 4 significant bits, so two parts hold a bf16 value's 8 bits exactly (to 2^-21 of the row's
//    largest for the smallest values) and three hold the hidden layer to 2^-13 or better. The parts
//    are neighbouring columns of N; the epilogue adds the columns up. That costs columns of N,
//    which an MMA this narrow has to spare.
//  - Both products are cut into units of 128 rows x 128 K bytes (16 KB), in a fixed order, and each
//    CTA takes an equal contiguous run of them, whatever tile it ends in (the tail is at most one
//    unit). A tile that several CTAs share leaves fp32 partial sums in the workspace; the last to
//    arrive adds them in CTA order, so the result does not depend on who was last.
//  - Between the two products all CTAs meet at a grid barrier (the hidden layer is complete); the
//    weight ring is filled for the second product meanwhile.
//
// Warps: 0 the weights' TMA producer; 1 the MMA issuer; 2-9 build the activation operand, every
// eighth unit each, into the weights' ring stages; 10-13 the epilogue, a thread per row of
// the tile. The MMA issuer's loop runs warp-uniform (elect.sync picks the issuing lane), with one
// commit a unit: with a lane's own control flow and a ring of its own for the activations a unit took
// 980 cycles, above the 700 that its 16 KB take to arrive.
// Every wait is bounded; on a timeout the kernel raises FP8_DEV_TIMEOUT, drains its loads and MMAs,
// frees its tensor memory and returns.
#include "common.cuh"
#include "internal.h"

namespace fp8lin {

namespace {

constexpr int kRows = 128;             // weight rows of a tile (64 gate + 64 up rows in the first product)
constexpr int kUnitBytes = kRows * 128;
constexpr int kMaxStages = 12;
constexpr int kBuilders = 8;           // warps 2 .. 9
constexpr int kEpi0 = 2 + kBuilders;   // first epilogue warp
constexpr int kThreads = 32 * (kEpi0 + 4);
constexpr int kMaxEntry = 40;          // slots of an entry at most: 128 columns of N in three parts
constexpr int kSmemMax = 232448;       // 227 KB
constexpr uint64_t kDrainNs = 2000000000ull;
// columns of N: groups of 16 hold 8 tokens in two parts, or 5 in three
constexpr int kPerGroup1 = 8, kPerGroup2 = 5;

struct MoeArgs {
  const int32_t* ids;
  const float* weights;
  const float* s13;
  const float* s2;
  __nv_bfloat16* out;
  int T, k, E, H, I;
  int cap;                // slots of an entry at most
  int stages, b_bytes;    // ring stages; bytes of a stage's activations, after its weights
  int tiles1, nk1, tiles2, nk2;
  // workspace
  uint32_t* counters;     // [0] the grid barrier, [1 + ph * grid + c] arrivals at the tile that CTA c starts and leaves
  const uint8_t* xq;      // the tokens' parts [T][2][128 nk1], zeros past H
  const float* xinv;      // [T]: their powers of two
  float* act;             // hidden layer [slots sorted by expert][I]
  uint32_t* amax;         // |hidden| maxima as bit patterns [slots][2 tiles1]
  float* part;            // partial sums [CTA][2][T][128]
  int32_t* status;
  uint64_t wait_ns;
  int test_stall;
};

struct Shared {
  uint64_t full[kMaxStages], built[kMaxStages], empty[kMaxStages];  // weights landed; activations written; both read
  uint64_t tfull[2], tempty[2];
  uint64_t drain, never, scales;
  uint32_t tmem_base;
  int abort;
  int n_act;
  int last;
};

// Shared memory after the rings: offsets in bytes (n = T k slots).
struct Layout {
  int acc, xch, shared, wt, inv1, mult2, inv2, hist, ids, ent, slot, total;
};
__host__ __device__ inline Layout layout(int T, int k, int E) {
  const int n = T * k;
  Layout L;
  int o = 0;
  L.acc = o, o += T * kRows * 4;
  L.xch = o, o += kPerGroup1 * 64 * 4;
  L.shared = o, o += (int)sizeof(Shared);
  L.wt = o, o += n * 4;
  L.inv1 = o, o += n * 4;
  L.mult2 = o, o += n * 4;
  L.inv2 = o, o += n * 4;
  L.hist = o, o += E * 4;
  L.ids = o, o += n * 4;
  L.ent = o, o += n * 4;   // per entry: expert, first slot
  L.slot = o, o += n * 4;  // per entry: slots; per sorted slot: token
  L.total = o;
  return L;
}

FP8_DEVI float2 e4m3x2_to_f32(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  float2 r;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(h));
  return r;
}
FP8_DEVI void tma_load_3d_hint(void* dst, const CUtensorMap* m, uint64_t* bar, int32_t x, int32_t y, int32_t z,
                               uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "l"(pol)
      : "memory");
}
FP8_DEVI bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
FP8_DEVI uint32_t atom_add_acq_rel(uint32_t* p, uint32_t v) {
  uint32_t r;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(r) : "l"(p), "r"(v) : "memory");
  return r;
}

// The power of two that brings a row's largest magnitude (bit pattern of an fp32) into [128, 256), and
// its inverse. A row with an infinity or a NaN gets NaN, which makes all of its values NaN.
FP8_DEVI void row_scale(uint32_t amax_bits, float* mult, float* inv) {
  const int ef = (int)(amax_bits >> 23);
  const int s = min(134 - ef, 126);
  *mult = ef == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float((uint32_t)(127 + s) << 23);
  *inv = ef == 255 ? 1.0f : __uint_as_float((uint32_t)(127 - s) << 23);
}

// Four values, already scaled, into PARTS words of e4m3 codes.
template <int PARTS>
FP8_DEVI void split4(float4 v, uint32_t* out) {
#pragma unroll
  for (int p = 0; p < PARTS; ++p) {
    const uint32_t lo = cvt_fp8x2<FP8_DT_E4M3>(v.x, v.y), hi = cvt_fp8x2<FP8_DT_E4M3>(v.z, v.w);
    out[p] = lo | (hi << 16);
    if (p + 1 < PARTS) {
      const float2 a = e4m3x2_to_f32(lo), b = e4m3x2_to_f32(hi);
      v = make_float4((v.x - a.x) * 16.f, (v.y - a.y) * 16.f, (v.z - b.x) * 16.f, (v.w - b.y) * 16.f);
    }
  }
}

// One product's share of a CTA: units [it0, it1) of `total`, tile after tile of nk units each.
struct Run {
  int total, nk, it0, it1, grid;  // grid: CTAs with a share
  FP8_DEVI int owner(int64_t it) const { return (int)(((it + 1) * grid - 1) / total); }
  FP8_DEVI int first(int c) const { return (int)((int64_t)c * total / grid); }
};
FP8_DEVI Run make_run(int tiles, int nk, int cta, int grid) {
  Run r;
  r.total = tiles * nk;
  r.nk = nk;
  r.grid = min(grid, r.total);
  r.it0 = cta < r.grid ? r.first(cta) : 0;
  r.it1 = cta < r.grid ? r.first(cta + 1) : 0;
  return r;
}

// A place in a CTA's share, stepped without divisions: unit kk of the nk of a (tile, entry).
struct Walk {
  int kk, nk, tile, a;
  FP8_DEVI void step1(int by, int tiles1) {  // first product: tiles of an entry are consecutive
    for (kk += by; kk >= nk; kk -= nk)
      if (++tile == tiles1) tile = 0, ++a;
  }
  FP8_DEVI void step2(int by, int n_act) {  // second: entries of a tile are consecutive
    for (kk += by; kk >= nk; kk -= nk)
      if (++a == n_act) a = 0, ++tile;
  }
};
FP8_DEVI Walk walk1(int it, int nk, int tiles1) {
  const int X = it / nk;
  return {it - X * nk, nk, X % tiles1, X / tiles1};
}
FP8_DEVI Walk walk2(int it, int nk, int n_act) {
  const int X = it / nk;
  return {it - X * nk, nk, X / n_act, X % n_act};
}

// The tokens' parts, a CTA per token, and the counters' zeros. The product kernel is launched while
// this one runs (programmatic dependent launch) and waits for it where it first needs the parts: by
// then it has sorted the slots and filled its ring with weights.
constexpr int kSplitThreads = 512;
__global__ void __launch_bounds__(kSplitThreads) moe_split_kernel(const uint16_t* __restrict__ x, int H, int Hp,
                                                                  uint8_t* __restrict__ xq, float* __restrict__ xinv,
                                                                  uint32_t* __restrict__ counters, int n_counters) {
  __shared__ uint32_t red[kSplitThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int t = blockIdx.x, tid = threadIdx.x;
  if (t == 0)
    for (int i = tid; i < n_counters; i += kSplitThreads) counters[i] = 0;
  const uint4* row = reinterpret_cast<const uint4*>(x + (int64_t)t * H);
  uint32_t m = 0;
  for (int c = tid; c < H / 8; c += kSplitThreads) m = absmax_vec8(m, row[c]);
  m = __reduce_max_sync(0xffffffffu, absmax_fold(m));
  if ((tid & 31) == 0) red[tid >> 5] = m;
  __syncthreads();
  m = 0;
#pragma unroll
  for (int w = 0; w < kSplitThreads / 32; ++w) m = max(m, red[w]);
  float mult, inv;
  row_scale(m << 16, &mult, &inv);
  if (tid == 0) xinv[t] = inv;
  for (int c = tid; c < Hp / 8; c += kSplitThreads) {
    const uint4 v = c < H / 8 ? row[c] : make_uint4(0, 0, 0, 0);
    uint32_t a[2] = {0, 0}, b[2] = {0, 0};
    if (c < H / 8) {
      split4<2>(make_float4(__uint_as_float(v.x << 16) * mult, __uint_as_float(v.x & 0xFFFF0000u) * mult,
                            __uint_as_float(v.y << 16) * mult, __uint_as_float(v.y & 0xFFFF0000u) * mult), a);
      split4<2>(make_float4(__uint_as_float(v.z << 16) * mult, __uint_as_float(v.z & 0xFFFF0000u) * mult,
                            __uint_as_float(v.w << 16) * mult, __uint_as_float(v.w & 0xFFFF0000u) * mult), b);
    }
    uint2* o = reinterpret_cast<uint2*>(xq + (int64_t)t * 2 * Hp) + c;
    o[0] = make_uint2(a[0], b[0]);
    o[Hp / 8] = make_uint2(a[1], b[1]);
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    moe_tokens_kernel(const __grid_constant__ CUtensorMap tm13, const __grid_constant__ CUtensorMap tm2, const MoeArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const Layout L = layout(p.T, p.k, p.E);
  const int stage_bytes = kUnitBytes + p.b_bytes;
  uint8_t* rest = smem + p.stages * stage_bytes;
  float* acc = reinterpret_cast<float*>(rest + L.acc);
  float* xch = reinterpret_cast<float*>(rest + L.xch);
  Shared& S = *reinterpret_cast<Shared*>(rest + L.shared);
  float* wt = reinterpret_cast<float*>(rest + L.wt);
  float* inv1 = reinterpret_cast<float*>(rest + L.inv1);
  float* mult2 = reinterpret_cast<float*>(rest + L.mult2);
  float* inv2 = reinterpret_cast<float*>(rest + L.inv2);
  int* hist = reinterpret_cast<int*>(rest + L.hist);
  int* ids = reinterpret_cast<int*>(rest + L.ids);
  uint16_t* ent_e = reinterpret_cast<uint16_t*>(rest + L.ent);
  const int n = p.T * p.k;
  uint16_t* ent_start = ent_e + n;
  uint16_t* ent_cnt = reinterpret_cast<uint16_t*>(rest + L.slot);
  uint16_t* tok = ent_cnt + n;
  int* slot_tmp = reinterpret_cast<int*>(wt);  // a sorted slot's index, until its weight takes the place
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, grid = gridDim.x;
  volatile int* abort_flag = &S.abort;
  auto fail = [&]() {
    if (!*abort_flag) {
      *abort_flag = 1;
      set_status(p.status, FP8_DEV_TIMEOUT);
    }
  };

  // ---- slots by expert: each entry is an expert with up to `cap` of its slots ----
  for (int e = tid; e < p.E; e += kThreads) hist[e] = 0;
  if (tid == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&S.full[s], 1);
      mbar_init(&S.built[s], 1);
      mbar_init(&S.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&S.tfull[b], 1);
      mbar_init(&S.tempty[b], 4);
    }
    mbar_init(&S.drain, 1);
    mbar_init(&S.never, 1);
    mbar_init(&S.scales, kBuilders);
    S.abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm13);
    tma_prefetch_desc(&tm2);
  }
  if (warp == 1) {
    tmem_alloc(&S.tmem_base, 512);
    tmem_relinquish();
  }
  __syncthreads();
  for (int s = tid; s < n; s += kThreads) {
    int id = p.ids[s];
    if (id < -1 || id >= p.E) {
      if (cta == 0) set_status(p.status, FP8_DEV_BAD_IDS);
      id = -1;
    }
    ids[s] = id;
    if (id >= 0) atomicAdd(hist + id, 1);
  }
  __syncthreads();
  if (warp == 0) {
    int slots = 0, ents = 0;
    for (int b = 0; b < p.E; b += 32) {
      const int e = b + lane;
      const int cnt = e < p.E ? hist[e] : 0;
      const int ne = (cnt + p.cap - 1) / p.cap;
      int xs = cnt, xe = ne;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int ys = __shfl_up_sync(0xffffffffu, xs, o), ye = __shfl_up_sync(0xffffffffu, xe, o);
        if (lane >= o) xs += ys, xe += ye;
      }
      const int s0 = slots + xs - cnt, a0 = ents + xe - ne;
      if (e < p.E) hist[e] = s0;
      for (int q = 0; q < ne; ++q) {
        ent_e[a0 + q] = (uint16_t)e;
        ent_start[a0 + q] = (uint16_t)(s0 + q * p.cap);
        ent_cnt[a0 + q] = (uint16_t)min(p.cap, cnt - q * p.cap);
      }
      slots += __shfl_sync(0xffffffffu, xs, 31);
      ents += __shfl_sync(0xffffffffu, xe, 31);
    }
    if (lane == 0) S.n_act = ents;
    __syncwarp();
    for (int b = 0; b < n; b += 32) {  // in slot order, so that every CTA has the same order
      const int s = b + lane;
      const int id = s < n ? ids[s] : -1;
      const uint32_t same = __match_any_sync(0xffffffffu, id);
      const int before = __popc(same & ((1u << lane) - 1));
      const int at = id >= 0 ? hist[id] + before : 0;
      __syncwarp();
      if (id >= 0) {
        slot_tmp[at] = s;
        tok[at] = (uint16_t)(s / p.k);
        if (before == 0) hist[id] += __popc(same);
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = S.tmem_base;
  const int n_act = S.n_act;

  if (n_act == 0) {  // nothing to read: zeros
    asm volatile("griddepcontrol.wait;" ::: "memory");  // not done before the kernel before it is
    for (int64_t i = (int64_t)cta * kThreads + tid; i < (int64_t)p.T * p.H; i += (int64_t)grid * kThreads)
      p.out[i] = __float2bfloat16_rn(0.f);
    if (warp == 1) tmem_dealloc(tmem_base, 512);
    return;
  }
  // first product: tiles by entry, then rows; second: tiles by rows, each over all entries
  const Run R1 = make_run(n_act * p.tiles1, p.nk1, cta, grid);
  const Run R2 = make_run(p.tiles2 * n_act, p.nk2, cta, grid);
  const int units1 = R1.it1 - R1.it0, units = units1 + R2.it1 - R2.it0;

  if (warp == 0) {
    // ============================== weights: TMA producer ==============================
    if (lane == 0) {
      const uint64_t pol = l2_evict_first();
      int li = 0, s = 0;
      uint32_t phase = 0;
      Walk w1 = walk1(R1.it0, p.nk1, p.tiles1), w2 = walk2(R2.it0, p.nk2, n_act);
      for (; li < units; ++li) {
        if (!mbar_wait(&S.empty[s], phase ^ 1, abort_flag, p.wait_ns)) {
          fail();
          break;
        }
        uint8_t* dst = smem + s * stage_bytes;
        mbar_arrive_expect_tx(&S.full[s], kUnitBytes);
        if (li < units1) {
          tma_load_3d_hint(dst, &tm13, &S.full[s], w1.kk * 128, w1.tile * 64, 2 * ent_e[w1.a], pol);
          w1.step1(1, p.tiles1);
        } else {
          tma_load_3d_hint(dst, &tm2, &S.full[s], w2.kk * 128, w2.tile * kRows, ent_e[w2.a], pol);
          w2.step2(1, n_act);
        }
        if (++s == p.stages) s = 0, phase ^= 1;
      }
      for (int i = li > p.stages ? li - p.stages : 0; i < li; ++i)  // loads in flight land before exit
        mbar_wait(&S.full[i % p.stages], (uint32_t)((i / p.stages) & 1), nullptr, kDrainNs);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ================================== MMA issuer ==================================
    const bool leader = elect_one();
    const uint32_t idesc0 = make_idesc(kFmtE4M3, kFmtE4M3, 0, 0, kRows, 0);
    const uint64_t desc0 = smem_desc(smem_u32(smem), 16, 1024);
    const uint32_t stage16 = (uint32_t)stage_bytes >> 4;
    bool ok = true;
    if (p.test_stall && !mbar_wait(&S.never, 0, abort_flag, p.wait_ns)) {
      fail();
      ok = false;
    }
    int li = 0, seg = 0, s = 0;
    uint32_t phase = 0;
    Walk w = walk1(R1.it0, p.nk1, p.tiles1);
    if (units1 == 0) w = walk2(R2.it0, p.nk2, n_act);
    while (li < units && ok) {
      const bool one = li < units1;
      const int left = min(w.nk - w.kk, (one ? units1 : units) - li);
      const int cnt = ent_cnt[w.a];
      const int groups = one ? (cnt + kPerGroup1 - 1) / kPerGroup1 : (cnt + kPerGroup2 - 1) / kPerGroup2;
      const uint32_t idesc = idesc0 | ((uint32_t)(2 * groups) << 17);
      const int buf = seg & 1;
      if (!mbar_wait(&S.tempty[buf], (uint32_t)(((seg >> 1) & 1) ^ 1), abort_flag, p.wait_ns)) {
        fail();
        break;
      }
      tc_fence_after();
      const uint32_t d = tmem_base + (uint32_t)(buf * 256);
      for (int i = 0; i < left; ++i) {
        if (!mbar_wait(&S.full[s], phase, abort_flag, p.wait_ns) || !mbar_wait(&S.built[s], phase, abort_flag, p.wait_ns)) {
          fail();
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t ad = desc0 + (uint64_t)((uint32_t)s * stage16);
        const uint64_t bd = ad + (kUnitBytes >> 4);
        if (leader) {
          umma_f8f6f4(d, ad, bd, idesc, i > 0 ? 1u : 0u);
          umma_f8f6f4(d, ad + 2, bd + 2, idesc, 1u);
          umma_f8f6f4(d, ad + 4, bd + 4, idesc, 1u);
          umma_f8f6f4(d, ad + 6, bd + 6, idesc, 1u);
          umma_commit(&S.empty[s]);
          if (i + 1 == left) umma_commit(&S.tfull[buf]);
        }
        __syncwarp();
        if (++s == p.stages) s = 0, phase ^= 1;
      }
      li += left;
      ++seg;
      if (one) {
        w.step1(left, p.tiles1);
        if (li == units1) w = walk2(R2.it0, p.nk2, n_act);
      } else {
        w.step2(left, n_act);
      }
    }
    if (leader) umma_commit(&S.drain);
    __syncwarp();
  } else {
    // ---- each slot's weight and its token's power of two: builders and epilogue warps together ----
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the tokens' parts and the counters are there
    const int used = ent_start[n_act - 1] + ent_cnt[n_act - 1];
    for (int i = tid - 64; i < used; i += 32 * (kBuilders + 4)) {
      wt[i] = __ldg(p.weights + slot_tmp[i]);
      inv1[i] = __ldcg(p.xinv + tok[i]);
    }
    named_bar_sync(1, 32 * (kBuilders + 4));
    if (warp < kEpi0) {
      // ============================ activations: B operand ============================
      const int w = warp - 2;
      bool ok = true;
      const uint32_t col = 4u * (uint32_t)lane;  // this lane's 4 of the unit's 128 K values
      // A builder waits for the use of its stage before its own. It must not get two uses ahead (their
      // parities are the same), so no more builders work than there are stages.
      const int builders = min(kBuilders, p.stages);
      int li = w < builders ? w : units, s = w;
      uint32_t phase = 0;
      uint8_t* stage = nullptr;
      auto enter = [&]() {
        const bool got = mbar_wait(&S.empty[s], phase ^ 1, abort_flag, p.wait_ns);
        if (!got) fail();
        stage = smem + s * stage_bytes + kUnitBytes;
        return __all_sync(0xffffffffu, got) != 0;
      };
      auto put = [&](int row, uint32_t word) {  // 128-byte swizzled row
        *reinterpret_cast<uint32_t*>(stage + row * 128 + (col ^ ((uint32_t)(row & 7) << 4))) = word;
      };
      auto leave = [&]() {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.built[s]);
        for (s += builders; s >= p.stages; s -= p.stages) phase ^= 1;
        li += builders;
      };
      // Rows are loaded four at a time, the first ones before the wait for the stage.
      constexpr int kBatch = 4;
      {
        Walk at = walk1(R1.it0, p.nk1, p.tiles1);
        at.step1(w, p.tiles1);
        while (li < units1) {
          // the entry's 2 cnt rows of 128 codes: 8 lanes a row, 4 rows a step
          const int rows = 2 * ent_cnt[at.a], start = ent_start[at.a];
          const uint8_t* src = p.xq + at.kk * 128 + (lane & 7) * 16;
          uint4 v[kBatch];
          auto fetch = [&](int r0) {
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
              const int row = r0 + 4 * b + (lane >> 3);
              if (row < rows) v[b] = __ldcg(reinterpret_cast<const uint4*>(src + (int64_t)(2 * tok[start + (row >> 1)] + (row & 1)) * (p.nk1 * 128)));
            }
          };
          fetch(0);
          if (!enter()) {
            ok = false;
            break;
          }
          for (int r0 = 0; r0 < rows; r0 += 4 * kBatch) {
            if (r0) fetch(r0);
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
              const int row = r0 + 4 * b + (lane >> 3);
              if (row < rows) *reinterpret_cast<uint4*>(stage + row * 128 + (((lane & 7) ^ (row & 7)) << 4)) = v[b];
            }
          }
          leave();
          at.step1(builders, p.tiles1);
        }
      }
      // ---- the hidden layer is complete once every CTA has arrived ----
      if (ok) {
        bool there = true;
        if (lane == 0) there = wait_count_geq(p.counters, (uint32_t)grid, p.wait_ns);
        ok = __shfl_sync(0xffffffffu, (int)there, 0);
        if (!ok && lane == 0) fail();
      }
      if (ok) {
        for (int pos = w; pos < used; pos += kBuilders) {
          uint32_t m = 0;
          for (int i = lane; i < 2 * p.tiles1; i += 32) m = max(m, __ldcg(p.amax + (int64_t)pos * 2 * p.tiles1 + i));
          m = __reduce_max_sync(0xffffffffu, m);
          if (lane == 0) row_scale(m, mult2 + pos, inv2 + pos);
        }
      }
      named_bar_sync(3, 32 * kBuilders);
      if (ok && lane == 0) mbar_arrive(&S.scales);
      if (ok && li < units) {
        Walk at = walk2(R2.it0, p.nk2, n_act);
        at.step2(li - units1, n_act);
        while (li < units) {
          const int k0 = at.kk * 128 + (int)col;
          const int cnt = ent_cnt[at.a], start = ent_start[at.a];
          float4 v[kBatch];
          auto fetch = [&](int j0) {
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
              v[b] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (j0 + b < cnt && k0 < p.I)
                v[b] = __ldcg(reinterpret_cast<const float4*>(p.act + (int64_t)(start + j0 + b) * p.I + k0));
            }
          };
          fetch(0);
          if (!enter()) break;
          for (int j0 = 0; j0 < cnt; j0 += kBatch) {
            if (j0) fetch(j0);
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
              const int j = j0 + b;
              if (j >= cnt) break;
              const float mult = mult2[start + j];
              uint32_t o[3];
              split4<3>(make_float4(v[b].x * mult, v[b].y * mult, v[b].z * mult, v[b].w * mult), o);
              const int row = 16 * (j / kPerGroup2) + 3 * (j % kPerGroup2);
              put(row, o[0]);
              put(row + 1, o[1]);
              put(row + 2, o[2]);
            }
          }
          leave();
          at.step2(builders, n_act);
        }
      }
    } else {
      // ================================== epilogue ==================================
      const int q = warp & 3, r = q * 32 + lane;  // tensor-memory lane quarter, row of the tile
      const uint32_t lanes = tmem_base + ((uint32_t)(q * 32) << 16);
      bool ok = true;
      int seg = 0;
      float* my_part = p.part + (int64_t)cta * 2 * p.T * kRows;
      auto part_of = [&](int c, int which) { return p.part + ((int64_t)c * 2 + which) * p.T * kRows; };
      // the four warps go on or stop together: they meet at named barriers further down
      auto wait_all = [&](uint64_t* bar, uint32_t parity) {
        const bool got = mbar_wait(bar, parity, abort_flag, p.wait_ns);
        if (!got) fail();
        return named_bar_and(2, 128, got);
      };
      auto wait_tile = [&](int buf) {
        if (!wait_all(&S.tfull[buf], (uint32_t)((seg >> 1) & 1))) return false;
        tc_fence_after();
        return true;
      };
      auto release_tile = [&](int buf) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed(&S.tempty[buf]);
        ++seg;
      };
      // this CTA's partial sums of a shared tile are written: true for the CTA that came last
      auto came_last = [&](int ph, int c_first, int c_last) {
        named_bar_sync(2, 128);
        if (tid == 32 * kEpi0) S.last = atom_add_acq_rel(p.counters + 1 + ph * grid + c_first, 1u) == (uint32_t)(c_last - c_first);
        named_bar_sync(2, 128);
        return S.last != 0;
      };

      // ---- first product: hidden = silu(gate) * up ----
      for (int it = R1.it0; it < R1.it1;) {
        const int X = it / p.nk1, first = X * p.nk1, len = min(first + p.nk1, R1.it1) - it;
        const int a = X / p.tiles1, tile = X - a * p.tiles1;
        const int cnt = ent_cnt[a], start = ent_start[a];
        const int i = tile * 64 + (r & 63);
        const float s = i < p.I ? __ldg(p.s13 + ((int64_t)ent_e[a] * 2 + (r >> 6)) * p.I + i) : 0.f;
        const bool whole = len == p.nk1;
        // gate and up of 8 tokens' row r -> the hidden layer and its maxima
        auto finish = [&](int g, const float* v) {
          if (r >= 64) {
#pragma unroll
            for (int j = 0; j < kPerGroup1; ++j) xch[j * 64 + r - 64] = v[j] * s;
          }
          named_bar_sync(2, 128);
          if (r < 64) {
#pragma unroll
            for (int j = 0; j < kPerGroup1; ++j) {
              if (g * kPerGroup1 + j >= cnt) break;
              const int64_t pos = start + g * kPerGroup1 + j;
              const float gate = v[j] * s;
              const float h = gate / (1.0f + expf(-gate)) * xch[j * 64 + r];
              if (i < p.I) p.act[pos * p.I + i] = h;
              const uint32_t m = __reduce_max_sync(0xffffffffu, i < p.I ? __float_as_uint(h) & 0x7FFFFFFFu : 0u);
              if (lane == 0) p.amax[pos * 2 * p.tiles1 + 2 * tile + q] = m;
            }
          }
          named_bar_sync(2, 128);
        };
        const int buf = seg & 1;
        if (!wait_tile(buf)) {
          ok = false;
          break;
        }
        float* mine = my_part + (it == R1.it0 ? 0 : p.T * kRows);
        for (int g = 0; g * kPerGroup1 < cnt; ++g) {
          uint32_t d[16];
          tmem_ld16(lanes + (uint32_t)(buf * 256 + 16 * g), d);
          tmem_ld_wait_regs16(d);
          float v[kPerGroup1];
#pragma unroll
          for (int j = 0; j < kPerGroup1; ++j) {
            const int idx = g * kPerGroup1 + j;
            v[j] = (__uint_as_float(d[2 * j]) + __uint_as_float(d[2 * j + 1]) * 0.0625f) * (idx < cnt ? inv1[start + idx] : 0.f);
            if (!whole && idx < cnt) mine[idx * kRows + r] = v[j];
          }
          if (whole) finish(g, v);
        }
        release_tile(buf);
        if (!whole) {
          const int c0 = R1.owner(first), c1 = R1.owner(first + p.nk1 - 1);
          if (came_last(0, c0, c1)) {
            for (int g = 0; g * kPerGroup1 < cnt; ++g) {
              float v[kPerGroup1];
#pragma unroll
              for (int j = 0; j < kPerGroup1; ++j) v[j] = 0.f;
              for (int c = c0; c <= c1; ++c) {
                const float* o = part_of(c, R1.first(c) >= first ? 0 : 1) + r;
#pragma unroll
                for (int j = 0; j < kPerGroup1; ++j)
                  if (g * kPerGroup1 + j < cnt) v[j] += __ldcg(o + (g * kPerGroup1 + j) * kRows);
              }
              finish(g, v);
            }
          }
        }
        it += len;
      }
      named_bar_sync(2, 128);
      if (ok && tid == 32 * kEpi0) red_add_release_gpu(p.counters, 1u);

      // ---- second product: the weighted sum over a token's experts, in entry order ----
      if (ok) ok = wait_all(&S.scales, 0);
      const int per = n_act * p.nk2;  // units of a tile of the output
      for (int it = R2.it0; it < R2.it1 && ok;) {
        const int tile = it / per, first = tile * per, end = min(first + per, R2.it1);
        const int nrow = tile * kRows + r;
        const bool whole = it == first && end == first + per;
        float* mine = my_part + (it == R2.it0 ? 0 : p.T * kRows);
        for (int t = 0; t < p.T; ++t) acc[t * kRows + r] = 0.f;
        while (it < end) {
          const int X = it / p.nk2, len = min((X + 1) * p.nk2, end) - it;
          const int a = X - tile * n_act, cnt = ent_cnt[a], start = ent_start[a];
          const float s = nrow < p.H ? __ldg(p.s2 + (int64_t)ent_e[a] * p.H + nrow) : 0.f;
          const int buf = seg & 1;
          if (!wait_tile(buf)) {
            ok = false;
            break;
          }
          for (int g = 0; g * kPerGroup2 < cnt; ++g) {
            uint32_t d[16];
            tmem_ld16(lanes + (uint32_t)(buf * 256 + 16 * g), d);
            tmem_ld_wait_regs16(d);
#pragma unroll
            for (int j = 0; j < kPerGroup2; ++j) {
              if (g * kPerGroup2 + j >= cnt) break;
              const int pos = start + g * kPerGroup2 + j;
              const float v = __uint_as_float(d[3 * j]) + __uint_as_float(d[3 * j + 1]) * 0.0625f +
                              __uint_as_float(d[3 * j + 2]) * 0.00390625f;
              acc[tok[pos] * kRows + r] += wt[pos] * (v * inv2[pos] * s);
            }
          }
          release_tile(buf);
          it += len;
        }
        if (!ok) break;
        if (whole) {
          if (nrow < p.H)
            for (int t = 0; t < p.T; ++t) p.out[(int64_t)t * p.H + nrow] = __float2bfloat16_rn(acc[t * kRows + r]);
          continue;
        }
        for (int t = 0; t < p.T; ++t) mine[t * kRows + r] = acc[t * kRows + r];
        const int c0 = R2.owner(first), c1 = R2.owner(first + per - 1);
        if (came_last(1, c0, c1)) {
          for (int t = 0; t < p.T; ++t) {
            float v = 0.f;
            for (int c = c0; c <= c1; ++c) v += __ldcg(part_of(c, R2.first(c) >= first ? 0 : 1) + t * kRows + r);
            if (nrow < p.H) p.out[(int64_t)t * p.H + nrow] = __float2bfloat16_rn(v);
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    if (lane == 0) mbar_wait(&S.drain, 0, nullptr, kDrainNs);  // the MMAs that write tensor memory
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// The workspace: counters (cleared by each call), the tokens' parts, hidden layer, its maxima, partial
// sums.
struct WsLayout {
  int64_t xq, xinv, act, amax, part, total;
};
constexpr int64_t kMaxGrid = 160;  // CTAs that the workspace holds partial sums for
WsLayout ws_layout(int64_t T, int64_t k, int64_t H, int64_t I) {
  WsLayout L;
  const int64_t n = T * k, tiles1 = ceil_div64(I, 64);
  int64_t o = round_up64((1 + 2 * kMaxGrid) * 4, 256);
  L.xq = o, o += T * 2 * round_up64(H, 128);
  L.xinv = o, o += round_up64(T * 4, 256);
  L.act = o, o += round_up64(n * I * 4, 256);
  L.amax = o, o += round_up64(n * 2 * tiles1 * 4, 256);
  L.part = o, o += kMaxGrid * 2 * T * kRows * 4;
  L.total = o;
  return L;
}

}  // namespace

int64_t moe_tokens_ws_bytes(int64_t T, int64_t k, int64_t H, int64_t I) {
  return ws_layout(T, k, H, I).total;
}

int launch_moe_tokens(const void* x, const int32_t* ids, const float* weights, const void* w13, const float* s13,
                      const void* w2, const float* s2, int64_t T, int64_t k, int64_t E, int64_t H, int64_t I, void* out,
                      void* ws, const Ctx& c) {
  if (T == 0) return FP8_OK;
  const WsLayout W = ws_layout(T, k, H, I);
  uint8_t* base = static_cast<uint8_t*>(ws);
  MoeArgs a;
  a.xq = base + W.xq;
  a.xinv = reinterpret_cast<const float*>(base + W.xinv);
  a.ids = ids;
  a.weights = weights;
  a.s13 = s13;
  a.s2 = s2;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.T = (int)T, a.k = (int)k, a.E = (int)E, a.H = (int)H, a.I = (int)I;
  a.tiles1 = (int)ceil_div64(I, 64);
  a.nk1 = (int)ceil_div64(H, 128);
  a.tiles2 = (int)ceil_div64(H, kRows);
  a.nk2 = (int)ceil_div64(I, 128);
  a.counters = reinterpret_cast<uint32_t*>(base);
  a.act = reinterpret_cast<float*>(base + W.act);
  a.amax = reinterpret_cast<uint32_t*>(base + W.amax);
  a.part = reinterpret_cast<float*>(base + W.part);
  a.status = c.status;
  a.wait_ns = c.wait_ns;
  a.test_stall = c.test_stall;
  a.cap = (int)(T < kMaxEntry ? T : kMaxEntry);
  // columns of N for an entry, in the layout that needs more of them (5 slots to a group of 16)
  a.b_bytes = (int)ceil_div64(a.cap, kPerGroup2) * 16 * 128;
  const Layout L = layout((int)T, (int)k, (int)E);
  const int stage_bytes = kUnitBytes + a.b_bytes;
  const int fit = (kSmemMax - 1024 - L.total) / stage_bytes;  // at least 4: T, k and E are bounded
  a.stages = fit < kMaxStages ? fit : kMaxStages;
  const int grid = (int)(c.sm_count < kMaxGrid ? c.sm_count : kMaxGrid);
  const size_t smem = 1024 + (size_t)a.stages * stage_bytes + L.total;

  CUtensorMap t13, t2;
  {
    // [2 E][I][H]: a box of 64 rows of the gate and the same 64 rows of the up projection
    const uint64_t dims[3] = {(uint64_t)H, (uint64_t)I, (uint64_t)(2 * E)};
    const uint64_t strides[2] = {(uint64_t)H, (uint64_t)(H * I)};
    const uint32_t box[3] = {128, 64, 2};
    const int rc = make_tmap(&t13, w13, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc != FP8_OK) return rc;
  }
  {
    const uint64_t dims[3] = {(uint64_t)I, (uint64_t)H, (uint64_t)E};
    const uint64_t strides[2] = {(uint64_t)I, (uint64_t)(H * I)};
    const uint32_t box[3] = {128, kRows, 1};
    const int rc = make_tmap(&t2, w2, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc != FP8_OK) return rc;
  }
  if (cudaFuncSetAttribute(moe_tokens_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return FP8_ERR_CUDA;
  moe_split_kernel<<<(unsigned)T, kSplitThreads, 0, c.stream>>>(
      static_cast<const uint16_t*>(x), a.H, a.nk1 * 128, base + W.xq, reinterpret_cast<float*>(base + W.xinv), a.counters,
      1 + 2 * grid);
  if (cudaGetLastError() != cudaSuccess) return FP8_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeCooperative;  // all CTAs resident: they meet at the grid barrier
  attr[0].val.cooperative = 1;
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = c.stream;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, moe_tokens_kernel, t13, t2, a) == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
}

}  // namespace fp8lin
