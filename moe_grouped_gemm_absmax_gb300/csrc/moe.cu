// The experts of a few tokens (sm_103a):
//   out[t] = sum_j weight[t, j] * W2[e] (silu(W1[e] x[t]) * (W3[e] x[t])),  e = ids[t, j],
// on FP8 weights with one inverse scale per row: w13 [E, 2 I, H] holds W1 (gate) and below it W3
// (up), w2 [E, H, I].
//
// With a few tokens the work is reading the named experts' weights once (once for each 40 slots of an expert,
// kMaxEntry); everything here serves to keep that stream going. Persistent CTAs, one for each SM:
//  - The weights are the MMA's A operand (tcgen05.mma kind::f8f6f4, M = 128 weight rows), so they go
//    from HBM by TMA into a shared-memory ring and from there into the tensor cores without
//    passing through registers. The tokens are its N.
//  - The activations keep their precision although the MMA takes 8-bit operands: a value v, scaled
//    by a power of two so that the largest around it lies in [128, 256), is split into e4m3 parts
//    v = p0 + p1 / 16 + p2 / 256, each part the rounding of 16 times what the ones before left. e4m3
//    has 4 significant bits, so two parts hold a bf16 value's 8 bits exactly (to 2^-21 of the row's
//    largest for the smallest values) and three hold the hidden layer to 2^-13 or better. The parts
//    are neighbouring columns of N; the epilogue adds the columns up. That costs columns of N,
//    which an MMA this narrow has to spare. A token is scaled as a row. The hidden layer is scaled in
//    blocks of 32, whose scales the block-scaled MMA applies (kind::mxf8f6f4, E8M0; the weights' are one):
//    a row's scale would need its whole row, another pass over it and another wait.
//  - Each product is cut into units of 128 rows x 128 K bytes (16 KB), in a fixed order, and each CTA
//    takes a contiguous run of them, equal or in whole tiles (make_run). A tile that several CTAs share
//    leaves fp32 partial sums in the workspace; the last to arrive adds them in CTA order, so the
//    result does not depend on who was last.
//
// Three launches, each started while the one before it runs (programmatic dependent launch) and
// waiting for it only where it needs its results:
//   moe_split_kernel   the tokens' parts, and the zeros that the others count from;
//   moe_kernel<1>      the hidden layer: it sorts the slots and fills its ring with weights meanwhile;
//   moe_kernel<2>      the output: with few tokens both kernels fit an SM side by side, so its ring is
//                      full when the hidden layer is complete.
// No CTA waits for another of its own launch, so nothing has to be resident together. One cooperative
// launch with a grid barrier between the products, built and measured early on, started 3 us later and
// took 74 us instead of 65 for one token (8 of 256 experts, 7168 x 2048).
//
// Warps: 0 the weights' TMA producer; 1 the MMA issuer; then the builders of the activation operand, one
// unit after the other in turn, into the weights' ring stages; the last four are the epilogue, a thread
// per row of the tile. The MMA issuer's loop runs warp-uniform (elect.sync picks the issuing lane),
// with one commit a unit: with a lane's own control flow and a ring of its own for the activations a
// unit took 980 cycles, above the 700 that its 16 KB take to arrive.
// Bound by memory: the weights stream at 7.1-7.5 TB/s once they flow (one token 64-66 us, 5.4 TB/s overall; 32
// tokens of the same layer on 137 experts 900-920 us, 6.9 TB/s, where a copy reaches 6.8). What a call adds is 5
// us to start, 4 us between the products and 3 us at the end: of a small layer (1040 x 528) nothing else is left.
// Every wait is bounded; on a timeout the kernel raises FP8_DEV_TIMEOUT, drains its loads and MMAs,
// frees its tensor memory and returns.
#include <atomic>

#include "common.cuh"
#include "internal.h"

namespace fp8lin {

namespace {

constexpr int kRows = 128;             // weight rows of a tile (64 gate + 64 up rows in the first product)
constexpr int kUnitBytes = kRows * 128;
constexpr int kMaxStages = 12;
constexpr int kFewTokens = 8;          // two CTAs an SM up to here; an entry's slots are at most as many
constexpr int kMaxEntry = 40;          // slots of an entry at most: 128 columns of N in three parts
// Tensor-memory columns: an accumulator's (two of them), then the weights' scales (all one) and those of each
// stage's activations, 4 columns each; a power of two in all.
constexpr int buf_cols(int NB) { return NB <= 4 ? 32 : 128; }
constexpr int tmem_cols(int ph, int NB) {
  const int need = 2 * buf_cols(NB) + (ph == 2 ? 4 + 4 * 12 : 0);
  return need <= 64 ? 64 : need <= 128 ? 128 : need <= 256 ? 256 : 512;
}
constexpr int kScaleBytes = 512;       // a stage's activation scales, in the MX scale layout's block of 128 rows
constexpr int kSmemMax = 232448;       // 227 KB a CTA
constexpr int kSmemPair = 115712;      // two CTAs an SM: half of 228 KB less the 1 KB reserved for each
// columns of N: groups of 16 hold 8 slots in two parts (columns 2 j, 2 j + 1), or 5 in three
constexpr int kPerGroup1 = 8, kPerGroup2 = 5;
constexpr int kPrefetchUnits = 8;      // units a CTA brings into L2 for the second product

struct MoeArgs {
  const int32_t* ids;
  const float* weights;
  const float* scales;    // s13 / s2
  __nv_bfloat16* out;
  int T, k, E, H, I;
  int cap;                // slots of an entry at most
  int stages, b_bytes;    // ring stages; bytes of a stage's activations, after its weights
  int tiles1, nk1, tiles2, nk2;
  // workspace; the first two start at zero
  uint32_t* arrived1;     // [CTA c] arrivals at the tile that c starts and does not finish
  uint32_t* arrived2;
  const uint8_t* xq;      // the tokens' parts [T][2][128 nk1], zeros past H
  const float* xinv;      // [T]: their powers of two
  uint8_t* hq;            // the hidden layer's parts [sorted slot][3][128 nk2]
  uint8_t* hs;            // and E8M0 codes of its blocks of 32 [sorted slot][4 nk2]
  float* part;            // partial sums [CTA][2][T][128]
  int32_t* status;
  uint64_t wait_ns;
  int test_stall;
};

struct Shared {
  uint64_t full[kMaxStages], built[kMaxStages], empty[kMaxStages];  // weights landed; activations written; both read
  uint64_t tfull[2], tempty[2];
  uint64_t drain, never, ready;  // ready: the slots' factors are in shared memory
  uint32_t tmem_base;
  int abort;
  int n_act, used;  // entries, sorted slots
  int last;
};

// Shared memory after the ring: offsets in bytes (n = T k slots).
struct Layout {
  int acc, shared, wt, inv, hist, ids, ent, slot, total;
};
__host__ __device__ inline Layout layout(int ph, int T, int k, int E) {
  const int n = T * k;
  Layout L;
  int o = 0;
  L.acc = o, o += ph == 1 ? 2 * kPerGroup1 * 64 * 4 : T * kRows * 4;  // gate and up on their way; output sums
  L.shared = o, o += (int)sizeof(Shared);
  L.wt = o, o += n * 4;    // per sorted slot: its index, then its weight
  L.inv = o, o += n * 4;   // its token's power of two; in the second product, per token, what its sum starts from
  L.hist = o, o += n > 32 ? E * 4 : 0;
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
FP8_DEVI void tma_prefetch_3d(const CUtensorMap* m, int32_t x, int32_t y, int32_t z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(x), "r"(y), "r"(z)
               : "memory");
}
// 16 bytes global -> shared without passing through registers; zeros where `valid` is false.
FP8_DEVI void cp_async16(void* dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(valid ? 16 : 0)
               : "memory");
}
FP8_DEVI uint32_t atom_add_acq_rel(uint32_t* p, uint32_t v) {
  uint32_t r;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(r) : "l"(p), "r"(v) : "memory");
  return r;
}

// The power of two that brings a row's largest magnitude (bit pattern of an fp32) into [128, 256), and
// its inverse. A row with an infinity or a NaN gets NaN for both, which makes all of its values NaN, and its
// output even where no expert takes it.
FP8_DEVI void row_scale(uint32_t amax_bits, float* mult, float* inv) {
  const int ef = (int)(amax_bits >> 23);
  const int s = min(134 - ef, 126);
  *mult = ef == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float((uint32_t)(127 + s) << 23);
  *inv = ef == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float((uint32_t)(127 - s) << 23);
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

// One product's share of a CTA: units [it0, it1) of `total`, tile after tile of `per` units each. Shares are
// contiguous and equal, to a unit or (whole) to a tile.
struct Run {
  int total, it0, it1, grid;  // grid: CTAs with a share
  int quantum, quanta;        // 1, or the units of a tile; how many of them
  FP8_DEVI int owner(int64_t it) const { return (int)(((it + 1) * grid - 1) / total); }  // for quantum 1
  FP8_DEVI int first(int c) const { return (int)((int64_t)c * quanta / grid) * quantum; }
};
// How to share, by the time it takes. All units take kUsAll each at the memory's rate; a CTA's own take at
// least kUsOne each, by the latency of its ring. Whole tiles may leave CTAs unequal, which costs nothing while
// the memory is the limit. A tile that P CTAs share is joined: kUsJoin for the stores, an atomic and loads one
// after the other, and kUsColumn for each of its `cols` slots from each of the P. (A 1040 x 528
// layer, one token: 14.6 us with whole tiles, 16.4 shared equally; 9 tokens on 13 experts of 1024 x 256 16 and
// 20 us.)
constexpr float kUsAll = 0.0023f, kUsOne = 0.35f, kUsJoin = 3.f, kUsColumn = 0.025f;
FP8_DEVI Run make_run(int tiles, int per, int cols, int cta, int grid) {
  Run r;
  r.total = tiles * per;
  const float all = r.total * kUsAll;
  auto cost = [&](float most, float P) { return fmaxf(all, most * kUsOne) + kUsJoin + P * cols * kUsColumn; };
  const int g = min(grid, r.total);
  const float whole = fmaxf(all, (float)((tiles + grid - 1) / grid * per) * kUsOne);
  const float equal = cost((float)r.total / g, fmaxf((float)g / tiles, 1.f) + 1.f);
  r.grid = g;
  r.quantum = 1, r.quanta = r.total;
  float best = equal;
  if (tiles <= grid) {
    const int P = max(1, min((int)(sqrtf(per * kUsOne / (cols * kUsColumn)) + 0.5f), grid / tiles));
    const float some = cost((float)per / P, (float)P);
    if (some < best && tiles * P <= r.total) best = some, r.grid = tiles * P;
  }
  if (whole <= best) r.grid = min(grid, tiles), r.quantum = per, r.quanta = tiles;
  r.it0 = cta < r.grid ? r.first(cta) : 0;
  r.it1 = cta < r.grid ? r.first(cta + 1) : 0;
  return r;
}

// A place in a CTA's share, stepped without divisions: unit kk of the nk of a (tile, entry). In the first
// product the tiles of an entry are consecutive, in the second the entries of a tile.
template <int PH>
struct Walk {
  int kk, nk, tile, a, lim;  // lim: tiles of an entry / entries of a tile
  FP8_DEVI Walk(int it, const MoeArgs& p, int n_act) {
    nk = PH == 1 ? p.nk1 : p.nk2;
    lim = PH == 1 ? p.tiles1 : n_act;
    const int X = it / nk;
    kk = it - X * nk;
    tile = PH == 1 ? X % lim : X / lim;
    a = PH == 1 ? X / lim : X % lim;
  }
  FP8_DEVI void step(int by) {
    for (kk += by; kk >= nk; kk -= nk) {
      if (PH == 1) {
        if (++tile == lim) tile = 0, ++a;
      } else {
        if (++a == lim) a = 0, ++tile;
      }
    }
  }
};

// The tokens' parts, a CTA per token, and the counters' zeros. The first product is launched while
// this one runs.
constexpr int kSplitThreads = 512;
__global__ void __launch_bounds__(kSplitThreads) moe_split_kernel(const uint16_t* x, int H, int Hp,
                                                                  uint8_t* xq, float* xinv,
                                                                  uint32_t* counters, int n_counters) {
  __shared__ uint32_t red[kSplitThreads / 32];
  pdl_wait();
  pdl_trigger();  // after the wait: the next kernel reads ids ahead of its own
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

// Slots by expert: entries of an expert with up to `cap` of its slots, and the slots in that order. The
// order depends on the ids only, so that every CTA has the same one.
FP8_DEVI void put_entries(const MoeArgs& p, int e, int cnt, int s0, int a0, uint16_t* ent_e, uint16_t* ent_start,
                          uint16_t* ent_cnt) {
  for (int q = 0; q * p.cap < cnt; ++q) {
    ent_e[a0 + q] = (uint16_t)e;
    ent_start[a0 + q] = (uint16_t)(s0 + q * p.cap);
    ent_cnt[a0 + q] = (uint16_t)min(p.cap, cnt - q * p.cap);
  }
}
// Exclusive sums over the lanes, and the totals.
FP8_DEVI void scan2(int x, int y, int lane, int* ex, int* ey, int* tx, int* ty) {
  int a = x, b = y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int c = __shfl_up_sync(0xffffffffu, a, o), d = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) a += c, b += d;
  }
  *ex = a - x, *ey = b - y;
  *tx = __shfl_sync(0xffffffffu, a, 31);
  *ty = __shfl_sync(0xffffffffu, b, 31);
}
FP8_DEVI int valid_id(const MoeArgs& p, int s) {
  const int id = ld_l2(p.ids + s);  // ahead of this kernel's own wait, see moe_split_kernel
  if (id >= -1 && id < p.E) return id;
  if (blockIdx.x == 0) set_status(p.status, FP8_DEV_BAD_IDS);
  return -1;
}

template <int N>
struct Width {
  static constexpr int value = N;
};

// PH: 1 the hidden layer, 2 the output. NB: builder warps.
template <int PH, int NB>
__global__ void __launch_bounds__(32 * (6 + NB), NB <= 4 ? 2 : 1)
    moe_kernel(const __grid_constant__ CUtensorMap tm, const __grid_constant__ CUtensorMap tm_next, const MoeArgs p) {
  constexpr int kThreads = 32 * (6 + NB);
  constexpr int kEpi0 = 2 + NB;  // first epilogue warp
  constexpr int kPer = PH == 1 ? kPerGroup1 : kPerGroup2;
  constexpr int kBufCols = buf_cols(NB), kTmem = tmem_cols(PH, NB);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const Layout L = layout(PH, p.T, p.k, p.E);
  const int stage_bytes = kUnitBytes + p.b_bytes + (PH == 2 ? 1024 : 0);  // scales: 512 bytes, stages on 1 KB
  uint8_t* rest = smem + p.stages * stage_bytes;
  float* acc = reinterpret_cast<float*>(rest + L.acc);
  Shared& S = *reinterpret_cast<Shared*>(rest + L.shared);
  float* wt = reinterpret_cast<float*>(rest + L.wt);
  int* slot_tmp = reinterpret_cast<int*>(wt);
  float* inv = reinterpret_cast<float*>(rest + L.inv);
  int* hist = reinterpret_cast<int*>(rest + L.hist);
  int* ids = reinterpret_cast<int*>(rest + L.ids);
  const int n = p.T * p.k;
  uint16_t* ent_e = reinterpret_cast<uint16_t*>(rest + L.ent);
  uint16_t* ent_start = ent_e + n;
  uint16_t* ent_cnt = reinterpret_cast<uint16_t*>(rest + L.slot);
  uint16_t* tok = ent_cnt + n;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, grid = gridDim.x;
  volatile int* abort_flag = &S.abort;
  auto fail = [&]() {
    if (!*abort_flag) {
      *abort_flag = 1;
      set_status(p.status, FP8_DEV_TIMEOUT);
    }
  };
  pdl_trigger();

  if (tid == 32) {
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
    mbar_init(&S.ready, NB);
    S.abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm);
  }
  if (PH == 2) {  // the weights' scales, all one (E8M0 127), for the MMA issuer
    uint32_t* one = reinterpret_cast<uint32_t*>(smem + kUnitBytes + p.b_bytes + kScaleBytes);
    for (int i = tid; i < kScaleBytes / 4; i += kThreads) one[i] = 0x7F7F7F7Fu;
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc(&S.tmem_base, kTmem);
    tmem_relinquish();
  }
  if (n <= 32) {  // one warp, a slot a lane: experts in the order of their first slots
    if (warp == 0) {
      const int id = lane < n ? valid_id(p, lane) : -1;
      const uint32_t same = __match_any_sync(0xffffffffu, id);
      const int lead = __ffs(same) - 1;
      const int cnt = id >= 0 && lane == lead ? __popc(same) : 0;
      int s0, a0, slots, ents;
      scan2(cnt, (cnt + p.cap - 1) / p.cap, lane, &s0, &a0, &slots, &ents);
      put_entries(p, id, cnt, s0, a0, ent_e, ent_start, ent_cnt);
      const int at = __shfl_sync(0xffffffffu, s0, lead) + __popc(same & ((1u << lane) - 1));
      if (id >= 0) {
        slot_tmp[at] = lane;
        tok[at] = (uint16_t)(lane / p.k);
      }
      if (lane == 0) S.n_act = ents, S.used = slots;
    }
  } else {
    // Each 32 slots count theirs by expert; the counts of the 32s before (in the ring, which is still empty) and
    // of the experts before are a slot's place.
    uint16_t* count = reinterpret_cast<uint16_t*>(smem + stage_bytes);  // [groups][E]
    const int groups = (n + 31) / 32, chunks = (p.E + 31) / 32;
    int* chunk_sum = reinterpret_cast<int*>(smem + stage_bytes + (groups * p.E * 2 + 15) / 16 * 16);  // [chunks][2]
    for (int i = tid; i < groups * p.E; i += kThreads) count[i] = 0;
    __syncthreads();
    for (int g = warp; g < groups; g += kThreads / 32) {
      const int s = g * 32 + lane;
      const int id = s < n ? valid_id(p, s) : -1;
      const uint32_t same = __match_any_sync(0xffffffffu, id);
      const int before = __popc(same & ((1u << lane) - 1));
      if (id >= 0 && before == 0) count[g * p.E + id] = (uint16_t)__popc(same);
      if (s < n) ids[s] = id < 0 ? -1 : id | before << 16;
    }
    __syncthreads();
    for (int c = warp; c < chunks; c += kThreads / 32) {
      const int e = c * 32 + lane;
      int cnt = 0;
      if (e < p.E)
        for (int g = 0; g < groups; ++g) {
          const int x = count[g * p.E + e];
          count[g * p.E + e] = (uint16_t)cnt;
          cnt += x;
        }
      if (e < p.E) hist[e] = cnt;
      const int ts = __reduce_add_sync(0xffffffffu, cnt), te = __reduce_add_sync(0xffffffffu, (cnt + p.cap - 1) / p.cap);
      if (lane == 0) chunk_sum[2 * c] = ts, chunk_sum[2 * c + 1] = te;
    }
    __syncthreads();
    for (int c = warp; c < chunks; c += kThreads / 32) {
      const int e = c * 32 + lane;
      const int cnt = e < p.E ? hist[e] : 0;
      int s0, a0, ts, te;
      scan2(cnt, (cnt + p.cap - 1) / p.cap, lane, &s0, &a0, &ts, &te);
      const int bs = __reduce_add_sync(0xffffffffu, lane < c ? chunk_sum[2 * lane] : 0);  // E <= 1024: a chunk a lane
      const int ba = __reduce_add_sync(0xffffffffu, lane < c ? chunk_sum[2 * lane + 1] : 0);
      if (e < p.E) hist[e] = bs + s0;
      put_entries(p, e, cnt, bs + s0, ba + a0, ent_e, ent_start, ent_cnt);
      if (c == chunks - 1 && lane == 0) S.n_act = ba + te, S.used = bs + ts;
    }
    __syncthreads();
    for (int s = tid; s < n; s += kThreads) {
      const int v = ids[s];
      if (v < 0) continue;
      const int id = v & 0xFFFF, at = hist[id] + count[(s >> 5) * p.E + id] + (v >> 16);
      slot_tmp[at] = s;
      tok[at] = (uint16_t)(s / p.k);
    }
    fence_proxy_async_smem();  // the ring's first loads come after these accesses
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = S.tmem_base;
  const int n_act = S.n_act, used = S.used;

  if (n_act == 0) {  // nothing to read: zeros, NaN for a token that holds one
    pdl_wait();  // not done before the kernel before it is
    if (PH == 2)
      for (int64_t i = (int64_t)cta * kThreads + tid; i < (int64_t)p.T * p.H; i += (int64_t)grid * kThreads)
        p.out[i] = __float2bfloat16_rn(0.f * ld_l2(p.xinv + i / p.H));
    if (warp == 1) tmem_dealloc(tmem_base, kTmem);
    return;
  }
  const int nk = PH == 1 ? p.nk1 : p.nk2;
  const Run R = PH == 1 ? make_run(n_act * p.tiles1, nk, (used + n_act - 1) / n_act, cta, grid)
                        : make_run(p.tiles2, n_act * nk, p.T, cta, grid);
  const int units = R.it1 - R.it0;

  if (warp == 0) {
    // ============================== weights: TMA producer ==============================
    if (lane == 0) {
      const uint64_t pol = l2_evict_first();
      int li = 0, s = 0;
      uint32_t phase = 0;
      Walk<PH> at(R.it0, p, n_act);
      for (; li < units; ++li, at.step(1)) {
        if (!mbar_wait(&S.empty[s], phase ^ 1, abort_flag, p.wait_ns)) {
          fail();
          break;
        }
        mbar_arrive_expect_tx(&S.full[s], kUnitBytes);
        tma_load_3d_hint(smem + s * stage_bytes, &tm, &S.full[s], at.kk * 128, at.tile * (PH == 1 ? 64 : kRows),
                         (PH == 1 ? 2 : 1) * ent_e[at.a], pol);
        if (++s == p.stages) s = 0, phase ^= 1;
      }
      for (int i = li > p.stages ? li - p.stages : 0; i < li; ++i)  // loads in flight land before exit
        mbar_wait(&S.full[i % p.stages], (uint32_t)((i / p.stages) & 1), nullptr, kDrainNs);
      // While the last tiles' sums are joined and the second product starts up, memory would idle: where that
      // product is short, the first units of its weights go to L2 meanwhile (63.9 us against 65.5 for one token
      // of the 7168 x 2048 layer; for 32 tokens 908 against 899). Asking for them before the last loads have
      // landed delays those.
      if (PH == 1 && !*abort_flag) {
        const Run R2 = make_run(p.tiles2, n_act * p.nk2, p.T, cta, grid);
        if (R2.it1 - R2.it0 <= 16 * kPrefetchUnits) {
          Walk<2> at2(R2.it0, p, n_act);
          for (int i = R2.it0; i < min(R2.it1, R2.it0 + kPrefetchUnits); ++i, at2.step(1))
            tma_prefetch_3d(&tm_next, at2.kk * 128, at2.tile * kRows, ent_e[at2.a]);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ================================== MMA issuer ==================================
    const bool leader = elect_one();
    const uint32_t idesc0 =
        PH == 1 ? make_idesc(kFmtE4M3, kFmtE4M3, 0, 0, kRows, 0) : make_idesc_mx(kFmtE4M3, kFmtE4M3, kRows, 0);
    // the weights' scales, all one, from a block of shared memory that the stages' own scales do not reach
    const uint32_t sfa = tmem_base + 2 * kBufCols, sfb0 = sfa + 4;
    const uint64_t sf_desc0 = smem_desc_plain(smem_u32(smem) + kUnitBytes + p.b_bytes, 128);
    if (PH == 2) {
      if (leader) tmem_cp_sf(sfa, sf_desc0 + (kScaleBytes >> 4));
      __syncwarp();
    }
    const uint64_t desc0 = smem_desc(smem_u32(smem), 16, 1024);
    const uint32_t stage16 = (uint32_t)stage_bytes >> 4;
    bool ok = true;
    if (p.test_stall && !mbar_wait(&S.never, 0, abort_flag, p.wait_ns)) {
      fail();
      ok = false;
    }
    int li = 0, seg = 0, s = 0;
    uint32_t phase = 0;
    Walk<PH> at(R.it0, p, n_act);
    while (li < units && ok) {
      const int left = min(nk - at.kk, units - li);
      const int groups = (ent_cnt[at.a] + kPer - 1) / kPer;
      const uint32_t idesc = idesc0 | ((uint32_t)(2 * groups) << 17);
      const int buf = seg & 1;
      if (!mbar_wait(&S.tempty[buf], (uint32_t)(((seg >> 1) & 1) ^ 1), abort_flag, p.wait_ns)) {
        fail();
        break;
      }
      tc_fence_after();
      const uint32_t d = tmem_base + (uint32_t)(buf * kBufCols);
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
          if (PH == 1) {
            umma_f8f6f4(d, ad, bd, idesc, i > 0 ? 1u : 0u);
            umma_f8f6f4(d, ad + 2, bd + 2, idesc, 1u);
            umma_f8f6f4(d, ad + 4, bd + 4, idesc, 1u);
            umma_f8f6f4(d, ad + 6, bd + 6, idesc, 1u);
          } else {
            const uint32_t sfb = sfb0 + 4 * s;
            tmem_cp_sf(sfb, sf_desc0 + (uint64_t)((uint32_t)s * stage16));
            umma_mx(d, ad, bd, idesc_sf_ids(idesc, 0, 0), sfa, sfb, i > 0 ? 1u : 0u);
            umma_mx(d, ad + 2, bd + 2, idesc_sf_ids(idesc, 1, 1), sfa, sfb, 1u);
            umma_mx(d, ad + 4, bd + 4, idesc_sf_ids(idesc, 2, 2), sfa, sfb, 1u);
            umma_mx(d, ad + 6, bd + 6, idesc_sf_ids(idesc, 3, 3), sfa, sfb, 1u);
          }
          umma_commit(&S.empty[s]);
          if (i + 1 == left) umma_commit(&S.tfull[buf]);
        }
        __syncwarp();
        if (++s == p.stages) s = 0, phase ^= 1;
      }
      li += left;
      ++seg;
      at.step(left);
    }
    if (leader) umma_commit(&S.drain);
    __syncwarp();
  } else if (warp < kEpi0) {
    // ============================ activations: B operand ============================
    const int w = warp - 2;
    // A builder waits for the use of its stage before its own. It must not get two uses ahead (their
    // parities are the same), so no more builders work than there are stages.
    const int builders = min(NB, p.stages);
    int li = w < builders ? w : units, s = w;
    uint32_t phase = 0;
    uint8_t* stage = nullptr;
    Walk<PH> at(R.it0 + w, p, n_act);
    auto enter = [&]() {
      const bool got = mbar_wait(&S.empty[s], phase ^ 1, abort_flag, p.wait_ns);
      if (!got) fail();
      stage = smem + s * stage_bytes + kUnitBytes;
      return __all_sync(0xffffffffu, got) != 0;
    };
    auto leave = [&]() {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.built[s]);
      for (s += builders; s >= p.stages; s -= p.stages) phase ^= 1;
      li += builders;
      at.step(builders);
    };
    // 8 lanes copy a row of 128 codes. An entry of few slots (NB 4) has its rows in flight, in registers, before the
    // wait for the unit's stage: that is worth 2 us of one token's 65. Entries of more are copied
    // asynchronously, all rows at once, one memory latency a unit whatever its rows (through registers, 16 at a
    // time, 32 tokens on 11 experts of 1392 x 1024 took 52 us instead of 39).
    const int chunk = lane & 7;
    constexpr bool kAhead = NB <= 4;
    constexpr int kBatch = kAhead ? (PH + 1) * kFewTokens / 4 : 1;  // loads a lane for an entry's rows
    pdl_wait();  // the tokens' parts / the hidden layer are there
    if (PH == 2) {
      for (int i = tid - 64; i < used; i += 32 * NB) wt[i] = p.weights[slot_tmp[i]];
      if (used < n)  // a token without experts: its sum starts from 0, or from NaN
        for (int i = tid - 64; i < p.T; i += 32 * NB) inv[i] = 0.f * ld_l2(p.xinv + i);
      named_bar_sync(1, 32 * NB);
      if (lane == 0) mbar_arrive(&S.ready);
    }
    while (li < units) {
      const int cnt = ent_cnt[at.a], start = ent_start[at.a];
      const int k0 = at.kk * 128 + chunk * 16;
      // the codes of four blocks of slot `lane`'s hidden layer; blocks past I have none
      auto codes = [&](int j) {
        const uint32_t w = ld_l2(reinterpret_cast<const uint32_t*>(p.hs) + (int64_t)(start + j) * p.nk2 + at.kk);
        const int blocks = (p.I - at.kk * 128 + 31) / 32;
        return blocks >= 4 ? w : w & ((1u << (8 * blocks)) - 1);
      };
      uint32_t code = PH == 2 && lane < cnt ? codes(lane) : 0u;
      // row `row` of the entry's: 2 a slot (its token's parts), or 3 a slot, 15 to a group of 16 columns, zeros past I
      const int rows = (PH + 1) * cnt;
      const bool in = PH == 1 || k0 < p.I;
      auto from = [&](int row) {
        return PH == 1 ? p.xq + (int64_t)(2 * tok[start + (row >> 1)] + (row & 1)) * (p.nk1 * 128) + k0
                       : p.hq + ((int64_t)start * 3 + row) * (p.nk2 * 128) + k0;
      };
      auto to = [&](int row) {
        const int t = PH == 1 ? row : row + row / 15;
        return stage + t * 128 + ((chunk ^ (t & 7)) << 4);
      };
      uint4 v[kBatch];
      if (kAhead) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const int row = 4 * b + (lane >> 3);
          v[b] = row < rows && in ? ld_l2(reinterpret_cast<const uint4*>(from(row))) : make_uint4(0, 0, 0, 0);
        }
      }
      if (!enter()) break;
      if (kAhead) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const int row = 4 * b + (lane >> 3);
          if (row < rows) *reinterpret_cast<uint4*>(to(row)) = v[b];
        }
      } else {
        for (int row = lane >> 3; row < rows; row += 4) cp_async16(to(row), from(row), in);
      }
      if (PH == 2) {
        uint8_t* scales = stage + p.b_bytes;
        for (int j = lane; j < cnt; j += 32) {
          if (j >= 32) code = codes(j);
          const int row = 3 * j + j / kPerGroup2;
#pragma unroll
          for (int q = 0; q < 3; ++q) {  // part q is worth 16^-q: 4 q less in the exponent
            const uint32_t c = __vsubus4(code, 0x04040404u * q);
            *reinterpret_cast<uint32_t*>(scales + ((row + q) & 31) * 16 + ((row + q) >> 5) * 4) = c;
          }
        }
      }
      if (!kAhead) {
        cp_async_commit();
        cp_async_wait<0>();
      }
      leave();
    }
  } else {
    // ================================== epilogue ==================================
    const int q = warp & 3, r = q * 32 + lane;  // tensor-memory lane quarter, row of the tile
    const uint32_t lanes = tmem_base + ((uint32_t)(q * 32) << 16);
    int seg = 0;
    uint32_t* arrived = PH == 1 ? p.arrived1 : p.arrived2;
    float* my_part = p.part + (int64_t)cta * 2 * p.T * kRows;
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
    auto came_last = [&](int c0, int c1) {
      named_bar_sync(2, 128);
      if (tid == 32 * kEpi0) S.last = atom_add_acq_rel(arrived + c0, 1u) == (uint32_t)(c1 - c0);
      named_bar_sync(2, 128);
      return S.last != 0;
    };
    // W of a tile's columns (slots or tokens), from `col0` on: the sums of row r over the partial sums of CTAs
    // c0 .. c1, in that order. All but c0 begin inside the tile, so theirs are their first.
    auto add_parts = [&](auto width, int c0, int c1, int first, int col0, int cols, float* v) {
      constexpr int W = decltype(width)::value;
      const int64_t step = (int64_t)2 * p.T * kRows;
      const float* o = p.part + c0 * step + (R.first(c0) >= first ? 0 : p.T * kRows) + col0 * kRows + r;
#pragma unroll
      for (int j = 0; j < W; ++j) v[j] = col0 + j < cols ? ld_l2(o + j * kRows) : 0.f;
      o = p.part + (c0 + 1) * step + col0 * kRows + r;
#pragma unroll 2
      for (int c = c0 + 1; c <= c1; ++c, o += step) {
        float u[W];
#pragma unroll
        for (int j = 0; j < W; ++j) u[j] = col0 + j < cols ? ld_l2(o + j * kRows) : 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] += u[j];
      }
    };

    if (PH == 1) {
      // ---- hidden = silu(gate) * up ----
      int xbuf = 0;
      pdl_wait();
      for (int i = tid - 32 * kEpi0; i < used; i += 128) inv[i] = ld_l2(p.xinv + tok[i]);
      named_bar_sync(2, 128);
      for (int it = R.it0; it < R.it1;) {
        const int X = it / nk, first = X * nk, len = min(first + nk, R.it1) - it;
        const int a = X / p.tiles1, tile = X - a * p.tiles1;
        const int cnt = ent_cnt[a], start = ent_start[a];
        const int i = tile * 64 + (r & 63);
        const float s = i < p.I ? p.scales[((int64_t)ent_e[a] * 2 + (r >> 6)) * p.I + i] : 0.f;
        const bool whole = len == nk;
        // Gate or up of 8 slots' row r -> the hidden layer, its parts and scales. The gate rows' threads take the
        // first four slots, the up rows' the others; each gives the other side what it lacks.
        auto finish = [&](int g, const float* v) {
          float* xch = acc + xbuf * (kPer * 64);
          xbuf ^= 1;  // two buffers: one is read while the next group's is written
          const bool gate_row = r < 64;
          const int row = r & 63;
#pragma unroll
          for (int j = 0; j < 4; ++j) xch[(gate_row ? j + 4 : j) * 64 + row] = (gate_row ? v[j + 4] : v[j]) * s;
          named_bar_sync(2, 128);
          const int j0 = gate_row ? 0 : 4;
          float h[4];
          uint32_t m[4];
          // with few slots (NB 4) only those there are, else all four side by side
          const int live = NB <= 4 ? cnt - g * kPer - j0 : 4;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (j >= live) break;
            const float other = xch[(j0 + j) * 64 + row];
            const float own = (gate_row ? v[j] : v[j + 4]) * s;
            const float gate = gate_row ? own : other, up = gate_row ? other : own;
            h[j] = i < p.I ? gate / (1.0f + expf(-gate)) * up : 0.f;
          }
          // this warp's 32 rows are a block of the hidden layer: its largest in [128, 256) times 2^(code - 127)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (j >= live) break;
            m[j] = __reduce_max_sync(0xffffffffu, __float_as_uint(h[j]) & 0x7FFFFFFFu);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (j >= live) break;
            const int idx = g * kPer + j0 + j;
            const int ef = (int)(m[j] >> 23);
            const uint32_t code = ef == 255 ? 0xFFu : (uint32_t)max(ef - 7, 8);  // 8: the third part's is 0
            float u = h[j] * mx_inv(code);
            const int64_t pos = start + idx;
            uint8_t* o = p.hq + pos * 3 * (p.nk2 * 128) + i;
            const bool put = idx < cnt && i < p.I;
#pragma unroll
            for (int part = 0; part < 3; ++part) {
              const uint32_t e = cvt_fp8x2<FP8_DT_E4M3>(u, 0.f);
              if (put) o[part * (p.nk2 * 128)] = (uint8_t)e;
              u = (u - e4m3x2_to_f32(e).x) * 16.f;
            }
            if (lane == 0 && put) p.hs[pos * (4 * p.nk2) + i / 32] = (uint8_t)code;
          }
        };
        const int buf = seg & 1;
        if (!wait_tile(buf)) break;
        float* mine = my_part + (it == R.it0 ? 0 : p.T * kRows);
        for (int g = 0; g * kPer < cnt; ++g) {
          uint32_t d[16];
          tmem_ld16(lanes + (uint32_t)(buf * kBufCols + 16 * g), d);
          tmem_ld_wait_regs16(d);
          float v[kPer];
#pragma unroll
          for (int j = 0; j < kPer; ++j) {
            const int idx = g * kPer + j;
            v[j] = (__uint_as_float(d[2 * j]) + __uint_as_float(d[2 * j + 1]) * 0.0625f) * (idx < cnt ? inv[start + idx] : 0.f);
            if (!whole && idx < cnt) mine[idx * kRows + r] = v[j];
          }
          if (whole) finish(g, v);
        }
        release_tile(buf);
        if (!whole) {
          const int c0 = R.owner(first), c1 = R.owner(first + nk - 1);
          if (came_last(c0, c1)) {
            for (int g = 0; g * kPer < cnt; ++g) {
              float v[kPer];
              add_parts(Width<kPer>{}, c0, c1, first, g * kPer, cnt, v);
              finish(g, v);
            }
          }
        }
        it += len;
      }
    } else {
      // ---- the weighted sum over a token's experts, in entry order ----
      bool ok = units == 0 || wait_all(&S.ready, 0);
      const int per = n_act * nk;  // units of a tile of the output
      for (int it = R.it0; it < R.it1 && ok;) {
        const int tile = it / per, first = tile * per, end = min(first + per, R.it1);
        const int nrow = tile * kRows + r;
        const bool whole = it == first && end == first + per;
        float* mine = my_part + (it == R.it0 ? 0 : p.T * kRows);
        for (int t = 0; t < p.T; ++t) acc[t * kRows + r] = used < n ? inv[t] : 0.f;
        while (it < end) {
          const int X = it / nk, len = min((X + 1) * nk, end) - it;
          const int a = X - tile * n_act, cnt = ent_cnt[a], start = ent_start[a];
          const float s = nrow < p.H ? p.scales[(int64_t)ent_e[a] * p.H + nrow] : 0.f;
          const int buf = seg & 1;
          if (!wait_tile(buf)) {
            ok = false;
            break;
          }
          for (int g = 0; g * kPer < cnt; ++g) {
            uint32_t d[16];
            tmem_ld16(lanes + (uint32_t)(buf * kBufCols + 16 * g), d);
            tmem_ld_wait_regs16(d);
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
              if (g * kPer + j >= cnt) break;
              const int pos = start + g * kPer + j;
              const float v = __uint_as_float(d[3 * j]) + __uint_as_float(d[3 * j + 1]) + __uint_as_float(d[3 * j + 2]);
              acc[tok[pos] * kRows + r] += wt[pos] * (v * s);
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
        const int c0 = R.owner(first), c1 = R.owner(first + per - 1);
        if (came_last(c0, c1)) {
          constexpr int W = NB <= 4 ? kFewTokens : 16;
          for (int t0 = 0; t0 < p.T; t0 += W) {
            float v[W];
            add_parts(Width<W>{}, c0, c1, first, t0, p.T, v);
#pragma unroll
            for (int j = 0; j < W; ++j)
              if (t0 + j < p.T && nrow < p.H) p.out[(int64_t)(t0 + j) * p.H + nrow] = __float2bfloat16_rn(v[j]);
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
    tmem_dealloc(tmem_base, kTmem);
  }
}

// The workspace: counts (cleared by each call), the tokens' parts, the hidden layer's, partial sums.
struct WsLayout {
  int64_t arrived2, zeros, xq, xinv, hq, hs, part, total;
};
constexpr int64_t kMaxGrid = 160;  // CTAs that the workspace holds partial sums for
WsLayout ws_layout(int64_t T, int64_t k, int64_t H, int64_t I) {
  WsLayout L;
  const int64_t n = T * k;
  int64_t o = kMaxGrid * 4;
  L.arrived2 = o, o += kMaxGrid * 4;
  L.zeros = o / 4;
  o = round_up64(o, 256);
  L.xq = o, o += T * 2 * round_up64(H, 128);
  L.xinv = o, o += round_up64(T * 4, 256);
  L.hq = o, o += n * 3 * round_up64(I, 128);
  L.hs = o, o += round_up64(n * 4 * ceil_div64(I, 128), 256);
  L.part = o, o += kMaxGrid * 2 * T * kRows * 4;
  L.total = o;
  return L;
}

// The ring of a product in `room` bytes of shared memory; returns what its CTA takes.
int ring(int ph, MoeArgs* a, int room) {
  const int per = ph == 1 ? kPerGroup1 : kPerGroup2;
  a->b_bytes = (a->cap + per - 1) / per * 16 * 128;  // columns of N for an entry
  const int stage_bytes = kUnitBytes + a->b_bytes + (ph == 2 ? 1024 : 0);
  const int rest = 1024 + layout(ph, a->T, a->k, a->E).total;
  const int fit = (room - rest) / stage_bytes;  // at least 4: T, k and E are bounded
  a->stages = fit < kMaxStages ? fit : kMaxStages;
  return rest + a->stages * stage_bytes;
}
template <int PH, int NB>
int run_moe(const CUtensorMap& tm, const CUtensorMap& tm_next, MoeArgs a, int room, int grid, const Ctx& c) {
  const int smem = ring(PH, &a, room);
  auto kern = moe_kernel<PH, NB>;
  // Once for each device: all of an SM's memory as shared memory, so that the two products' CTAs fit
  // together.
  static std::atomic<uint64_t> done{0};
  const uint64_t bit = 1ull << (c.device & 63);
  if (!(done.load(std::memory_order_acquire) & bit)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax) != cudaSuccess ||
        cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) !=
            cudaSuccess)
      return FP8_ERR_CUDA;
    done.fetch_or(bit, std::memory_order_release);
  }
  return launch_dependent(kern, dim3((unsigned)grid), dim3(32 * (6 + NB)), smem, c.stream, tm, tm_next, a);
}

}  // namespace

int64_t moe_tokens_ws_bytes(int64_t T, int64_t k, int64_t H, int64_t I) { return ws_layout(T, k, H, I).total; }

int launch_moe_tokens(const void* x, const int32_t* ids, const float* weights, const void* w13, const float* s13,
                      const void* w2, const float* s2, int64_t T, int64_t k, int64_t E, int64_t H, int64_t I, void* out,
                      void* ws, const Ctx& c) {
  if (T == 0) return FP8_OK;
  const WsLayout W = ws_layout(T, k, H, I);
  uint8_t* base = static_cast<uint8_t*>(ws);
  MoeArgs a;
  a.ids = ids;
  a.weights = weights;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.T = (int)T, a.k = (int)k, a.E = (int)E, a.H = (int)H, a.I = (int)I;
  a.tiles1 = (int)ceil_div64(I, 64);
  a.nk1 = (int)ceil_div64(H, 128);
  a.tiles2 = (int)ceil_div64(H, kRows);
  a.nk2 = (int)ceil_div64(I, 128);
  a.arrived1 = reinterpret_cast<uint32_t*>(base);
  a.arrived2 = reinterpret_cast<uint32_t*>(base + W.arrived2);
  a.xq = base + W.xq;
  a.xinv = reinterpret_cast<const float*>(base + W.xinv);
  a.hq = base + W.hq;
  a.hs = base + W.hs;
  a.part = reinterpret_cast<float*>(base + W.part);
  a.status = c.status;
  a.wait_ns = c.wait_ns;
  a.test_stall = c.test_stall;
  a.cap = (int)(T < kMaxEntry ? T : kMaxEntry);
  const int grid = (int)(c.sm_count < kMaxGrid ? c.sm_count : kMaxGrid);

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
  int rc = launch_dependent(moe_split_kernel, dim3((unsigned)T), dim3(kSplitThreads), 0, c.stream,
                            static_cast<const uint16_t*>(x), a.H, a.nk1 * 128, base + W.xq,
                            reinterpret_cast<float*>(base + W.xinv), reinterpret_cast<uint32_t*>(base), (int)W.zeros);
  if (rc != FP8_OK) return rc;
  // With few tokens a stage is hardly more than its weights, and half an SM's shared memory holds
  // enough of them in flight: the two products run side by side. More tokens need longer stages and
  // more builders, and the second product then follows on each SM as the first leaves it.
  if (T <= kFewTokens) {
    a.scales = s13;
    // twice as many bytes pass through the first product: it gets what the second one's whole stages leave
    MoeArgs second = a;
    rc = run_moe<1, 4>(t13, t2, a, 2 * kSmemPair - ring(2, &second, kSmemPair), grid, c);
    if (rc != FP8_OK) return rc;
    a.scales = s2;
    return run_moe<2, 4>(t2, t2, a, kSmemPair, grid, c);
  }
  a.scales = s13;
  rc = run_moe<1, 8>(t13, t2, a, kSmemMax, grid, c);
  if (rc != FP8_OK) return rc;
  a.scales = s2;
  return run_moe<2, 8>(t2, t2, a, kSmemMax, grid, c);
}

}  // namespace fp8lin
