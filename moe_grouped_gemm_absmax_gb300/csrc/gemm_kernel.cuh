// Scaled FP8 (and BF16) GEMMs on the 5th-generation tensor cores (sm_103a): dense, and the MoE
// grouped GEMM with rows or contraction jagged by expert.
//
//   D[m, n] = sA[m] * sB[n] * sum_k A[m, k] * B[n, k]       (dequant contract: "FP8 Training:
//   Quantization, Autograd, Torchao", section 2; operand layouts: section 4)
//   grouped: per-row sA, per-expert-column sB, rows routed by cumulative offsets ("FP8 training
//   on AMD GPUs with TorchTitan and TorchAO", "Scaling FP8 to MoE Architectures", Figure 3).
//
// Design (persistent; 320 threads per CTA, 384 with block scales, 608 with MX; CG = 1 or 2 CTAs per MMA):
//   CG = 1: one CTA per SM computes 128 x 256 tiles (block scales by expert and the gated kernels: or 128 or 64
//           columns, NT, where that takes shorter rounds);
//   CG = 2: a cluster of two CTAs (a CTA pair on two SMs) computes 256 x 256 tiles with
//           tcgen05.mma.cta_group::2: each CTA stages its own 128 rows of A and 128 of the 256
//           rows of B, the even CTA issues the MMAs for both, and each CTA's tensor memory
//           holds the accumulator of its own 128 rows. Per CTA a stage is 32 KB instead of
//           48 KB, so the ring is deeper (5 or 6 stages, not 4) and B is read from L2 once per pair.
//   warp 0      TMA producer (128-byte swizzle; K blocks of 128 bytes) into the stage ring,
//               guarded by full/empty mbarriers (the pair's full barrier lives in the even CTA
//               and counts both CTAs' bytes);
//   warp 1      allocates 512 TMEM columns; in the issuing CTA its loop runs warp-uniform (waits and descriptors
//               in all lanes, an elected lane's MMAs: 8192 x 14336 x 4096 took 270 us with lane 0
//               in the loop alone, 259 so). MMAs (M=128 or 256, N=256; K=32 for FP8, K=16 for BF16) go into one of two fp32
//               accumulators and commits each stage back to the producers and each finished
//               tile to the epilogues (multicast to both CTAs of a pair);
//   warps 2..9  epilogue: each warp owns 32 TMEM lanes (tile rows) and one half (128 columns)
//               of its CTA's tile; the tile's column scales are staged once in shared memory;
//               tcgen05.ld 32 columns at a time, sA[m] * sB[n] applied once, one rounding to
//               bf16/fp32, masked stores. The second accumulator lets the next tile's MMAs
//               overlap this epilogue.
// Grouped with rows jagged by expert (FP8, pairs): an expert's last tile, when it has fewer than
// 256 rows, is computed transposed: its 256 weight rows are the MMA's M and its rows, rounded up
// to 16, the MMA's N, loaded with a row box of 32, 64 or 128 per CTA. These GEMMs are bound by
// operand traffic from L2, so a short tail costs the bytes and MMAs of its own rows.
// Block scales (kBLK; single CTAs): below, at the promotion.
// The gated feed-forward (EPI kGate, kGateBwd; formulas: gate.cuh) has the same main loop and epilogues of its own.
// Every wait is bounded; on a timeout the kernel raises FP8_DEV_TIMEOUT, drains in-flight TMA
// and MMA work, frees its tensor memory and returns.
#pragma once

#include <string.h>

#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "gate.cuh"
#include "internal.h"

namespace fp8lin {

namespace {

constexpr int BM = 128, BN = 256, BKB = 128;  // rows per CTA, tile columns (FP8 / BF16), K bytes per stage
constexpr int kTmemCols = 512;
constexpr int kMaxExperts = 2048;
constexpr int64_t kGroupBytes = 32ll << 20;  // rasterization: the A panels of a group of M-blocks, in L2
constexpr int kStageOut = 4096;  // per epilogue warp: output staging for TMA stores (pairs)
constexpr int kMaxStages = 6;    // ring stages the barrier arrays hold
constexpr int kSharedBytes = 2304;
constexpr int kSmemMax = 232448;  // 227 KB a CTA
constexpr int kGateBox = 2048;   // a box of 32 rows x 32 bf16 columns
// kDenseAmax: the dense schedule whose epilogue also folds max |out| into the side outputs;
// kDenseQuant: the dense schedule whose epilogue writes the next quantization of the (bf16) result:
// FP8 codes and 1 x 128 or MX scales along the rows
enum { kDense = 0, kJagM = 1, kJagK = 2, kDenseAmax = 3, kDenseQuant = 4 };
constexpr bool is_dense(int sched) { return sched == kDense || sched == kDenseAmax || sched == kDenseQuant; }
// kBLK: FP8 operands with blockwise scales (A: 1 x 128 tiles, B: 128 x 128 tiles); the MMAs of
// each 128-deep K block go to a fresh tensor-memory partial, which the epilogue warps scale by
// sA[m, kb] * sB[n / 128, kb] and add into register accumulators ("promotion")
enum { kFP8 = 0, kBF16 = 1, kMX = 2, kBLK = 3 };

// What becomes of a finished tile. kStore: its values, scaled. kGate: columns 0 .. 127 are the gate's projection and
// 128 .. 255 the up projection's of the same 128 columns of the hidden layer, which is formed and stored (gate.cuh);
// kGateBwd: the values are the hidden layer's gradient, from which the projections' gradients are formed and stored.
enum { kStore = 0, kGate = 1, kGateBwd = 2 };

// MX (block-scaled) tiles are 256 columns wide like the FP8 ones (an MMA's cost is set per
// instruction, so narrower tiles run the tensor cores below their rate), but they keep ONE
// accumulator: its 256 tensor-memory columns plus one 16-column scale-factor slot per ring stage
// fit in the 512 columns, two accumulators would not. Sixteen epilogue warps (four per lane
// quarter, 64 columns each) move the accumulator into registers right after the tile's MMAs and
// release it at once, so the next tile's MMAs wait only for those loads, not for the stores.
template <int KIND, int CG, int SCHED = 0, int EPI = kStore, int NT = BN>
struct Cfg {
  // kBLK: two K-block partials, so the MMAs run one K block ahead of the promotion.
  static constexpr int TBN = NT;                          // tile columns (less than 256 on single CTAs: tile_width)
  static constexpr int NBUF = KIND == kMX ? 1 : 2;        // accumulators / K-block partials
  static constexpr int EPI_WARPS = KIND == kMX ? 16 : 8;
  static constexpr int EPI_THREADS = 32 * EPI_WARPS;
  static constexpr int EPI0 = KIND == kBLK ? 4 : 2;      // first epilogue warp (kBLK: warpgroups share registers)
  static constexpr int SF_WARP = 2 + EPI_WARPS;          // MX: the warp that copies scales to tensor memory
  static constexpr int THREADS = 32 * EPI0 + EPI_THREADS + (KIND == kMX ? 32 : 0);
  static constexpr int WCOLS = TBN * 4 / EPI_WARPS;      // columns per epilogue warp: 128 or 64
  static constexpr int A_BYTES = BM * BKB;               // this CTA's 128 rows of A
  static constexpr int B_ROWS = TBN / CG;                // this CTA's rows of B
  static constexpr int B_BYTES = B_ROWS * BKB;
  static constexpr int SF_BYTES = KIND == kMX ? 3 * 512 : 0;  // one A scale block, two B scale blocks
  static constexpr int TX_BYTES = A_BYTES + B_BYTES + SF_BYTES;  // bytes the loads of a stage deliver
  static constexpr int STAGE_BYTES = (TX_BYTES + 1023) / 1024 * 1024;
  // MX with the contraction jagged: short K loops make the epilogue's stores the critical path,
  // so those tiles store through shared memory with TMA (64 KB of staging for 16 warps), which
  // leaves room for 4 stages; the other MX schedules store from registers and keep 5
  static constexpr bool MX_TMA_OUT = KIND == kMX && CG == 2 && SCHED == 2;
  // The gated epilogues' stores, and the backward's loads of the projections, pass through shared memory too: boxes of
  // 32 rows x 32 columns, two a warp, or two of either projection's.
  static constexpr bool GATE_BOXES = EPI == kGateBwd || (EPI == kGate && KIND != kBLK);
  static constexpr int OUT_BYTES = GATE_BOXES ? EPI_WARPS * (EPI == kGate ? 2 : 4) * kGateBox
                                   : (CG == 2 && ((KIND != kMX && KIND != kBLK) || MX_TMA_OUT)) ? EPI_WARPS * kStageOut : 0;
  // Gated and blockwise: as many stages as fit beside that, the barriers and the experts' offsets (the dense backward on
  // pairs with 4 stages: 437 us at 8192 x 14336 x 4096, with 5 400)
  static constexpr int FIT = (kSmemMax - kSharedBytes - OUT_BYTES - (EPI == kGate ? 2048 : EPI == kGateBwd ? 128 : 0) -
                              (SCHED == 0 ? 0 : EPI == kStore ? 8 * (kMaxExperts + 1) : 8 * ((int)kMaxGatedExperts + 1))) /
                             STAGE_BYTES;
  static constexpr int STAGES = EPI != kStore || KIND == kBLK ? (FIT < kMaxStages ? FIT : kMaxStages)
                                : (CG == 2 && !MX_TMA_OUT ? 5 : 4);
  static constexpr int RING_BYTES = STAGES * STAGE_BYTES;
  static constexpr int TILE_M = BM * CG;
  static constexpr int SF_COL0 = NBUF * TBN;             // first scale-factor slot (16 columns each)
};
static_assert(Cfg<kMX, 2>::SF_COL0 + 16 * Cfg<kMX, 2>::STAGES <= kTmemCols, "MX tensor-memory budget");
static_assert(Cfg<kMX, 2, 2>::STAGES <= Cfg<kMX, 2>::STAGES, "MX jagged-K ring");

struct GemmParams {
  int64_t M, N, K;     // tile space: rows of D, columns of D, contraction length (elements)
  int64_t num_m, num_n;
  int64_t nkb;         // K blocks per tile (dense, jagged M)
  int64_t group_m;     // dense: tiles walk group_m M-blocks per N-block (group_n == 0), or
  int64_t group_n;     //        group_n N-blocks per M-block
  const float* sA;
  const float* sB;
  int sa_scalar, sb_scalar;
  int sc_vec;          // kBLK: four K blocks' scales start on 16 bytes (nkb % 4 == 0)
  void* out;
  int out_f32;
  int vec_ok;          // 16-byte aligned output rows
  int wide;            // 32-byte aligned output rows (kBLK)
  int64_t ldo;         // output row stride (elements)
  const int32_t* ends;
  int E;
  int64_t total_rows;  // jagged M: last valid offset
  int tma_out;         // CTA pairs with 16-byte aligned output rows: TMA bulk-tensor stores
  int test_stall;      // wait first on a barrier nothing signals (failure-detection tests)
  uint32_t* row_amax;  // side outputs (bf16 out): max |out| per row / column as fp32 words
  uint32_t* col_amax;
  int amax_whole;      // col_amax is a single word: the maximum over the whole output
  uint32_t idesc;
  int32_t* status;
  uint64_t wait_ns;
  // kDenseQuant: the result's quantization (codes [M, N] row-major in q_fmt; scales: fp32 [M, N / 128]
  // for 1 x 128 blocks, or E8M0 bytes in the MX scale layout for rows M, contraction N)
  uint8_t* q_out;
  void* q_scales;
  int q_mx;
  int q_fmt;
  ScaleTab q_tab;
  // FP8 jagged M on CTA pairs: an expert's last tile, when it holds fewer than 256 rows, is
  // computed transposed (weight rows on the MMA's M side, the tile's rows as its N)
  int tail_t;
  uint32_t idesc_t;    // the transposed tile's instruction descriptor, N field zero
  GateArgs gate;       // kGate, kGateBwd (N: the hidden layer's columns)
};

struct Tile {
  int32_t m0, n0;   // first row / column of the (pair's) tile of D
  int32_t row_end;  // rows >= row_end are masked (segment end, or M)
  int32_t k0;       // first contraction coordinate
  int32_t nkb;      // K blocks
  int e;            // expert (jagged)
  int tt;           // jagged M, transposed tail tile: its rows (1..255); 0 for an ordinary tile
  int64_t pm0;      // m0 in the segment-padded row space of the MX A scales (jagged M), else m0
};

struct Shared {
  float sb[2][BN];  // per-tile column scales, alternating between consecutive tiles
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t tfull[4];   // accumulators / K-block partials ready (NBUF of them in use)
  uint64_t tempty[4];
  uint64_t drain;
  uint64_t never;   // signalled by no one: the failure-detection test hook waits on it
  uint64_t sff[kMaxStages];  // MX: a stage's scales are in tensor memory
  uint64_t sf_drain;
  uint32_t tmem_base;
  int abort;
};
// kBLK: K blocks whose scales a promoting lane loads together, one group ahead
constexpr int kScGroup = 4;
// kBLK: registers a thread of the four warps that issue and of the eight that promote: 128 x 40 + 256 x 232 = 384 x 168,
// what the block is launched with
constexpr int kIssueRegs = 40, kPromoteRegs = 232;
static_assert(sizeof(Shared) <= kSharedBytes, "shared block");
// kGate with codes: the largest magnitudes of a row's columns that the warps of a lane quarter hold, alternating between
// consecutive tiles
struct AmaxShare {
  float a[2][2][128];
};
// kGateBwd: a warp's boxes of the projections have landed
struct BoxBars {
  uint64_t full[8][2];
};

FP8_DEVI int find_expert(const int32_t* tpre, int E, int64_t t) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tpre[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Tile t of the persistent schedule. Tile indices, tile counts and block coordinates fit in 32
// bits (the launcher checks), so the divisions here are 32-bit: they sit on the MMA issuer's and
// the epilogue's per-tile path.
template <int SCHED, int TILE_M, int TBN>
FP8_DEVI Tile get_tile(const GemmParams& p, int64_t t64, const int32_t* tpre, const int32_t* aux,
                       const int32_t* pst) {
  Tile T;
  const uint32_t t = (uint32_t)t64, num_n = (uint32_t)p.num_n;
  if (is_dense(SCHED)) {
    uint32_t mb, nb;
    if (p.group_n == 0) {
      const uint32_t gm = (uint32_t)p.group_m;
      const uint32_t per_group = gm * num_n;
      const uint32_t g = t / per_group, r = t - g * per_group;
      const uint32_t first_m = g * gm;
      const uint32_t left = (uint32_t)p.num_m - first_m;
      const uint32_t gsz = left < gm ? left : gm;
      nb = r / gsz;
      mb = first_m + (r - nb * gsz);
    } else {
      const uint32_t gn = (uint32_t)p.group_n;
      const uint32_t per_group = gn * (uint32_t)p.num_m;
      const uint32_t g = t / per_group, r = t - g * per_group;
      const uint32_t first_n = g * gn;
      const uint32_t left = num_n - first_n;
      const uint32_t gsz = left < gn ? left : gn;
      mb = r / gsz;
      nb = first_n + (r - mb * gsz);
    }
    T.m0 = (int32_t)(mb * TILE_M);
    T.pm0 = T.m0;
    T.n0 = (int32_t)(nb * TBN);
    T.row_end = (int32_t)p.M;
    T.k0 = 0;
    T.nkb = (int32_t)p.nkb;
    T.e = 0;
    T.tt = 0;
  } else if (SCHED == kJagM) {
    const int e = find_expert(tpre, p.E, t64);
    const uint32_t local = t - (uint32_t)tpre[e];
    // as dense tiles: a group of the expert's M-blocks per N-block, so that its weights pass once for each group
    const uint32_t gm = (uint32_t)p.group_m, per_group = gm * num_n;
    const uint32_t first_m = local / per_group * gm, r = local - first_m * num_n;
    const uint32_t left = ((uint32_t)tpre[e + 1] - (uint32_t)tpre[e]) / num_n - first_m;
    const uint32_t gsz = left < gm ? left : gm;
    const uint32_t nb = r / gsz, mb = first_m + (r - nb * gsz);
    T.m0 = aux[e] + (int32_t)(mb * TILE_M);  // aux[e] = segment start row
    T.pm0 = pst ? pst[e] + (int64_t)mb * TILE_M : T.m0;
    T.n0 = (int32_t)(nb * TBN);
    T.row_end = aux[e + 1];
    T.k0 = 0;
    T.nkb = (int32_t)p.nkb;
    T.e = e;
    T.tt = (p.tail_t && T.row_end - T.m0 < TILE_M) ? T.row_end - T.m0 : 0;
  } else {
    const uint32_t per = (uint32_t)p.num_m * num_n;
    const uint32_t e = t / per;
    const uint32_t local = t - e * per;
    const uint32_t mb = local / num_n, nb = local - mb * num_n;
    T.m0 = (int32_t)(mb * TILE_M);
    T.pm0 = T.m0;
    T.n0 = (int32_t)(nb * TBN);
    T.row_end = (int32_t)p.M;
    T.k0 = aux[e];                             // aux[e] = padded start of segment e
    T.nkb = (aux[e + 1] - aux[e]) / BKB;       // padded length / 128
    T.e = (int)e;
    T.tt = 0;
  }
  return T;
}

// K blocks of tile t (all the MMA issuer needs to know about a tile).
template <int SCHED>
FP8_DEVI int64_t tile_nkb(const GemmParams& p, int64_t t, const int32_t* aux) {
  if (SCHED != kJagK) return p.nkb;
  const uint32_t e = (uint32_t)t / ((uint32_t)p.num_m * (uint32_t)p.num_n);
  return (aux[e + 1] - aux[e]) / BKB;
}

template <int KIND, int SCHED, int A_MN, int B_MN, int CG, int EPI, int NT>
__global__ void __launch_bounds__(Cfg<KIND, CG, SCHED, EPI, NT>::THREADS, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const __grid_constant__ CUtensorMap tmO, const __grid_constant__ CUtensorMap tmSA,
                const __grid_constant__ CUtensorMap tmSB, const GemmParams p) {
  using C = Cfg<KIND, CG, SCHED, EPI, NT>;
  static_assert(KIND != kBLK || CG == 1, "blockwise scaling runs on single CTAs");
  static_assert(C::STAGES <= kMaxStages && C::NBUF <= 4, "ring and accumulator barriers fit the shared block");
  constexpr int STAGES = C::STAGES;
  constexpr int kThreads = C::THREADS;
  constexpr int kEpiThreads = C::EPI_THREADS;
  constexpr int TBN = C::TBN;
  constexpr int TN = EPI == kGate ? TBN / 2 : TBN;  // columns of D (kGate: of the hidden layer) of a tile
  constexpr bool kPadRows = KIND == kMX && SCHED == kJagM;  // A scales in the segment-padded row space
  // FP8 jagged M on pairs: transposed tail tiles, whose row boxes of 32 and 64 rows come in the
  // tmSA and tmSB slots (unused by FP8 operands); 128-row boxes are tmA's own
  constexpr bool kTail = KIND == kFP8 && SCHED == kJagM && CG == 2 && EPI == kStore;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* out_stage = smem + C::RING_BYTES;  // [8 warps][kStageOut], pairs only
  Shared& S = *reinterpret_cast<Shared*>(smem + C::RING_BYTES + C::OUT_BYTES);
  uint8_t* rest = smem + C::RING_BYTES + C::OUT_BYTES + kSharedBytes;
  AmaxShare& AS = *reinterpret_cast<AmaxShare*>(rest);  // kGate
  if (EPI == kGate) rest += sizeof(AmaxShare);
  BoxBars& BB = *reinterpret_cast<BoxBars*>(rest);  // kGateBwd
  if (EPI == kGateBwd) rest += sizeof(BoxBars);
  int32_t* tpre = reinterpret_cast<int32_t*>(rest);
  int32_t* aux = tpre + (p.E + 1);
  int32_t* pst = kPadRows ? aux + (p.E + 1) : nullptr;  // padded segment starts
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &S.abort;
  const uint32_t rank = CG == 2 ? cluster_ctarank() : 0;  // 0 issues the pair's MMAs
  const bool issuer = rank == 0;
  const int64_t unit = blockIdx.x / CG, n_units = gridDim.x / CG;

  // ---- jagged schedules: validate offsets, per-expert tile prefix and row / K starts ----
  int64_t total;
  if (is_dense(SCHED)) {
    total = p.num_m * p.num_n;
  } else {
    int bad = 0;
    for (int e = tid; e < p.E; e += kThreads) {
      const int32_t cur = p.ends[e], prev = e ? p.ends[e - 1] : 0;
      if (cur < prev || (SCHED != kJagK && e == p.E - 1 && cur != p.total_rows)) bad = 1;
      const int64_t cnt = cur > prev ? cur - prev : 0;
      if (SCHED == kJagM) {
        tpre[e + 1] = (int32_t)(((cnt + C::TILE_M - 1) / C::TILE_M) * p.num_n);
        aux[e + 1] = cur;
        if (kPadRows) pst[e + 1] = (int32_t)((cnt + 127) / 128 * 128);
      } else {
        tpre[e + 1] = (int32_t)(p.num_m * p.num_n);
        aux[e + 1] = (int32_t)(((cnt + BKB - 1) / BKB) * BKB);
      }
    }
    if (tid == 0) {
      tpre[0] = 0;
      aux[0] = 0;
      if (kPadRows) pst[0] = 0;
    }
    bad = __syncthreads_or(bad);
    if (bad) {  // both CTAs of a pair see the same offsets and leave together
      if (blockIdx.x == 0 && tid == 0) set_status(p.status, FP8_DEV_BAD_OFFSETS);
      return;
    }
    if (warp == 0) {  // inclusive scans (tile prefix always; padded prefix for jagged K / MX rows)
      constexpr bool kScan2 = SCHED == kJagK || kPadRows;
      int32_t* w_arr = SCHED == kJagK ? aux : pst;
      int carry = 0, carry2 = 0;
      for (int base = 0; base < p.E; base += 32) {
        const int i = base + lane;
        int v = i < p.E ? tpre[i + 1] : 0;
        int w = (kScan2 && i < p.E) ? w_arr[i + 1] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, v, o);
          const int z = __shfl_up_sync(0xffffffffu, w, o);
          if (lane >= o) {
            v += y;
            w += z;
          }
        }
        if (i < p.E) {
          tpre[i + 1] = v + carry;
          if (kScan2) w_arr[i + 1] = w + carry2;
        }
        carry += __shfl_sync(0xffffffffu, v, 31);
        carry2 += __shfl_sync(0xffffffffu, w, 31);
      }
    }
    __syncthreads();
    total = tpre[p.E];
    if (SCHED == kJagK && aux[p.E] > p.K) {  // segments do not fit the padded operand
      if (blockIdx.x == 0 && tid == 0) set_status(p.status, FP8_DEV_BAD_OFFSETS);
      return;
    }
  }

  // ---- barriers and tensor memory ----
  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&S.full[s], 1);
      mbar_init(&S.empty[s], 1);
    }
    for (int b = 0; b < C::NBUF; ++b) {
      mbar_init(&S.tfull[b], 1);
      mbar_init(&S.tempty[b], CG * kEpiThreads / 32);
    }
    mbar_init(&S.drain, 1);
    for (int s2 = 0; s2 < STAGES; ++s2) mbar_init(&S.sff[s2], 1);
    mbar_init(&S.sf_drain, 1);
    mbar_init(&S.never, 1);
    if (EPI == kGateBwd)
      for (int i = 0; i < 16; ++i) mbar_init(&BB.full[i >> 1][i & 1], 1);
    S.abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    if (EPI != kStore || CG == 2) tma_prefetch_desc(&tmO);
    if (KIND == kMX || (kTail && p.tail_t)) {
      tma_prefetch_desc(&tmSA);
      tma_prefetch_desc(&tmSB);
    }
  }
  if (warp == 1) {
    if (CG == 2) {
      tmem_alloc_pair(&S.tmem_base, kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&S.tmem_base, kTmemCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_barrier();  // the peer's barriers are initialised before any remote use
  tc_fence_after();
  const uint32_t tmem_base = S.tmem_base;

  auto fail = [&]() {
    *abort_flag = 1;
    set_status(p.status, FP8_DEV_TIMEOUT);
  };

  if (KIND == kBLK) {
    if (warp < C::EPI0)
      setmaxnreg_dec<kIssueRegs>();
    else
      setmaxnreg_inc<kPromoteRegs>();
  }
  if (warp == 0) {
    // ================================ TMA producer ================================
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int64_t issued = 0;
      bool ok = true;
      for (int64_t t = unit; t < total && ok; t += n_units) {
        const Tile T = get_tile<SCHED, C::TILE_M, TN>(p, t, tpre, aux, pst);
        const int32_t am = T.m0 + (int32_t)rank * BM;        // this CTA's A rows
        // this CTA's B rows; kGate on a pair: the gate's 128 in the even CTA, the up projection's in the other
        const int32_t bn = (int32_t)(T.n0 + (int64_t)rank * (EPI == kGate ? p.N : C::B_ROWS));
        // MX scale blocks: this CTA's 128 A rows; the two 128-row B blocks holding the tile's
        // columns (each CTA of a pair loads them in full: its accumulator spans all columns)
        const int32_t sfa_rb = (int32_t)((T.pm0 + (int64_t)rank * BM) / 128);
        const int32_t sfb_rb = (int32_t)(T.n0 / 128);
        // transposed tail tile: each CTA holds N' / 2 of its rows (N' = rows rounded up to 16),
        // loaded with the smallest row box that covers them; the weight rows take the A side
        int tail_half = 0, tail_box = 0;
        if (kTail && T.tt) {
          tail_half = (T.tt + 15) / 16 * 8;
          tail_box = tail_half <= 32 ? 32 : (tail_half <= 64 ? 64 : 128);
        }
        const uint32_t tx = tail_box ? (uint32_t)(C::A_BYTES + tail_box * BKB) : (uint32_t)C::TX_BYTES;
        for (int32_t kb = 0; kb < T.nkb; ++kb) {
          if (!mbar_wait(&S.empty[stage], phase ^ 1, abort_flag, p.wait_ns)) {
            if (!*abort_flag) fail();
            ok = false;
            break;
          }
          uint8_t* sa = smem + stage * C::STAGE_BYTES;
          uint8_t* sb = sa + C::A_BYTES;
          uint8_t* ssf = sa + C::A_BYTES + C::B_BYTES;
          if (CG == 1) {
            uint64_t* fb = &S.full[stage];
            mbar_arrive_expect_tx(fb, C::TX_BYTES);
            if (KIND == kMX) {
              const int32_t kx = (int32_t)(T.k0 + kb * BKB);
              tma_load_2d(sa, &tmA, fb, kx, am);
              if (SCHED == kJagM) {
                tma_load_3d(sb, &tmB, fb, kx, bn, T.e);
                tma_load_4d(ssf + 512, &tmSB, fb, 0, kx / 128, sfb_rb, T.e);
              } else {
                tma_load_2d(sb, &tmB, fb, kx, bn);
                tma_load_3d(ssf + 512, &tmSB, fb, 0, kx / 128, sfb_rb);
              }
              tma_load_3d(ssf, &tmSA, fb, 0, kx / 128, sfa_rb);
            } else if (KIND == kFP8 || KIND == kBLK) {
              const int32_t kx = (int32_t)(T.k0 + kb * BKB);
              tma_load_2d(sa, &tmA, fb, kx, am);
              // kGate: the up projection's rows after the gate's (kBLK: either half of them)
              constexpr int kBoxes = EPI == kGate ? (KIND == kBLK ? 4 : 2) : 1;
#pragma unroll
              for (int h = 0; h < kBoxes; ++h) {
                const int32_t r = bn + (h & 1) * (int32_t)p.N + h / 2 * (TBN / 4);
                if (SCHED == kJagM)
                  tma_load_3d(sb + h * (C::B_BYTES / kBoxes), &tmB, fb, kx, r, T.e);
                else
                  tma_load_2d(sb + h * (C::B_BYTES / kBoxes), &tmB, fb, kx, r);
              }
            } else {
              const int32_t kx = (int32_t)(kb * (BKB / 2));  // 64 bf16 per block
              if (A_MN) {
                tma_load_2d(sa, &tmA, fb, am, kx);
                tma_load_2d(sa + 8192, &tmA, fb, am + 64, kx);
              } else {
                tma_load_2d(sa, &tmA, fb, kx, am);
              }
              if (B_MN) {
#pragma unroll
                for (int h = 0; h < C::B_ROWS / 64; ++h) tma_load_2d(sb + h * 8192, &tmB, fb, bn + 64 * h, kx);
              } else {
                tma_load_2d(sb, &tmB, fb, kx, bn);
                if (EPI == kGate) tma_load_2d(sb + C::B_BYTES / 2, &tmB, fb, kx, bn + (int32_t)p.N);
              }
            }
          } else {
            // both CTAs' bytes are counted on the issuing CTA's full barrier
            const uint32_t fb = mapa_shared(smem_u32(&S.full[stage]), 0);
            if (issuer) mbar_arrive_expect_tx(&S.full[stage], 2 * tx);
            if (KIND == kMX) {
              const int32_t kx = (int32_t)(T.k0 + kb * BKB);
              tma_load_2d_pair(sa, &tmA, fb, kx, am);
              if (SCHED == kJagM) {
                tma_load_3d_pair(sb, &tmB, fb, kx, bn, T.e);
                tma_load_4d_pair(ssf + 512, &tmSB, fb, 0, kx / 128, sfb_rb, T.e);
              } else {
                tma_load_2d_pair(sb, &tmB, fb, kx, bn);
                tma_load_3d_pair(ssf + 512, &tmSB, fb, 0, kx / 128, sfb_rb);
              }
              tma_load_3d_pair(ssf, &tmSA, fb, 0, kx / 128, sfa_rb);
            } else if (KIND == kFP8) {
              const int32_t kx = (int32_t)(T.k0 + kb * BKB);
              if (kTail && tail_box) {
                tma_load_3d_pair(sa, &tmB, fb, kx, bn, T.e);  // this CTA's 128 weight rows
                const CUtensorMap* tm = tail_box == 32 ? &tmSA : (tail_box == 64 ? &tmSB : &tmA);
                tma_load_2d_pair(sb, tm, fb, kx, (int32_t)(T.m0 + (int64_t)rank * tail_half));
              } else {
                tma_load_2d_pair(sa, &tmA, fb, kx, am);
                if (SCHED == kJagM)
                  tma_load_3d_pair(sb, &tmB, fb, kx, bn, T.e);
                else
                  tma_load_2d_pair(sb, &tmB, fb, kx, bn);
              }
            } else {
              const int32_t kx = (int32_t)(kb * (BKB / 2));
              if (A_MN) {
                tma_load_2d_pair(sa, &tmA, fb, am, kx);
                tma_load_2d_pair(sa + 8192, &tmA, fb, am + 64, kx);
              } else {
                tma_load_2d_pair(sa, &tmA, fb, kx, am);
              }
              if (B_MN) {
#pragma unroll
                for (int h = 0; h < C::B_ROWS / 64; ++h) tma_load_2d_pair(sb + h * 8192, &tmB, fb, bn + 64 * h, kx);
              } else {
                tma_load_2d_pair(sb, &tmB, fb, kx, bn);
              }
            }
          }
          ++issued;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      // Drain: the last (up to STAGES) loads must land before the CTA (pair) may exit. For a
      // pair, the issuing CTA's full barriers count both CTAs' loads; after an abort the other
      // CTA cannot observe them and lets its own last loads settle for 100 us instead.
      if (issuer) {
        const int64_t first = issued > STAGES ? issued - STAGES : 0;
        for (int64_t i = first; i < issued; ++i)
          mbar_wait(&S.full[i % STAGES], (uint32_t)((i / STAGES) & 1), nullptr, kDrainNs);
      } else if (!ok) {
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 100000ull) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ================================ MMA issuer ================================
    // The loop runs warp-uniform: elect.sync picks the lane that issues, all lanes wait. Descriptors are offsets of
    // per-kernel bases (address field in 16-byte units). Control flow of one lane alone, and descriptors built for
    // every MMA, cost the blockwise loop a third of its time. A K block costs the warp 98 cycles a wait, 200 for the MMAs,
    // 160 for the first commit and 100 for the second, ready or not.
    if (issuer) {
      const bool leader = elect_one();
      int stage = 0;
      uint32_t phase = 0;
      int buf = 0;
      uint32_t aphase = 0;
      bool ok = true;
      const uint64_t a_desc0 = smem_desc(smem_u32(smem), A_MN ? 8192 : 16, 1024);
      const uint64_t b_desc0 = smem_desc(smem_u32(smem) + C::A_BYTES, B_MN ? 8192 : 16, 1024);
      constexpr uint64_t kStepA = (A_MN ? 2048 : 32) >> 4, kStepB = (B_MN ? 2048 : 32) >> 4;
      uint32_t mx_id[4];  // MX: the four scale-factor ids
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) mx_id[kk] = idesc_sf_ids(p.idesc, (uint32_t)kk, (uint32_t)kk);
      if (p.test_stall && !mbar_wait(&S.never, 0, abort_flag, p.wait_ns)) {
        fail();
        ok = false;
      }
      for (int64_t t = unit; t < total && ok; t += n_units) {
        const int nkb = (int)tile_nkb<SCHED>(p, t, aux);
        if (nkb == 0) continue;
        uint32_t idesc = p.idesc;
        if (kTail && p.tail_t) {  // transposed tail tile: swapped formats, N = N'
          const int tt = get_tile<SCHED, C::TILE_M, TN>(p, t, tpre, aux, pst).tt;
          if (tt) idesc = p.idesc_t | ((uint32_t)((tt + 15) / 16 * 2) << 17);
        }
        if (KIND != kBLK) {
          if (!mbar_wait(&S.tempty[buf], aphase ^ 1, abort_flag, p.wait_ns)) {
            if (!*abort_flag) fail();
            break;
          }
          tc_fence_after();
        }
        for (int kb = 0; kb < nkb; ++kb) {
          // kBLK: each K block into the next free partial. MX: the scale warp's commit on sff[stage] follows the
          // stage's full barrier
          if (!(KIND == kBLK ? mbar_wait_both(&S.tempty[buf], aphase ^ 1, &S.full[stage], phase, abort_flag, p.wait_ns)
                             : mbar_wait(KIND == kMX ? &S.sff[stage] : &S.full[stage], phase, abort_flag, p.wait_ns))) {
            if (!*abort_flag) fail();
            ok = false;
            break;
          }
          tc_fence_after();
          const bool done = KIND == kBLK || kb + 1 == nkb;  // the accumulator is complete with these MMAs
          if (leader) {
            const uint32_t d_tmem = tmem_base + (uint32_t)(buf * TBN);
            const uint64_t soff = (uint64_t)((uint32_t)(stage * C::STAGE_BYTES) >> 4);
            const uint64_t ad0 = a_desc0 + soff, bd0 = b_desc0 + soff;
            // MX: the stage's scales are in its tensor-memory slot (copied by the scale warp)
            const uint32_t sf_t = tmem_base + (uint32_t)(C::SF_COL0 + 16 * stage);
            const uint32_t sfb_t = sf_t + 4;  // 256-column tiles start on a 128-row scale block
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint64_t ad = ad0 + kk * kStepA, bd = bd0 + kk * kStepB;
              const uint32_t acc = ((KIND != kBLK && kb > 0) || kk > 0) ? 1u : 0u;
              if (KIND == kMX) {
                if (CG == 2)
                  umma_mx_pair(d_tmem, ad, bd, mx_id[kk], sf_t, sfb_t, acc);
                else
                  umma_mx(d_tmem, ad, bd, mx_id[kk], sf_t, sfb_t, acc);
              } else if (KIND == kBF16) {
                if (CG == 2)
                  umma_f16_pair(d_tmem, ad, bd, p.idesc, acc);
                else
                  umma_f16(d_tmem, ad, bd, p.idesc, acc);
              } else {
                if (CG == 2)
                  umma_f8f6f4_pair(d_tmem, ad, bd, idesc, acc);
                else
                  umma_f8f6f4(d_tmem, ad, bd, p.idesc, acc);
              }
            }
            // frees the stage (in both CTAs of a pair) once these MMAs have read it
            if (CG == 2)
              umma_commit_pair(&S.empty[stage], 0x3);
            else
              umma_commit(&S.empty[stage]);
            if (done) {
              if (CG == 2)
                umma_commit_pair(&S.tfull[buf], 0x3);
              else
                umma_commit(&S.tfull[buf]);
            }
          }
          __syncwarp();
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
          if (done && ++buf == C::NBUF) {
            buf = 0;
            aphase ^= 1;
          }
        }
      }
      // Drain every MMA issued before the tensor memory is released.
      if (leader) {
        if (CG == 2)
          umma_commit_pair(&S.drain, 0x3);
        else
          umma_commit(&S.drain);
      }
    }
    __syncwarp();
  } else if (KIND == kBLK && warp < C::EPI0) {
    // no role: these warps complete the warpgroup
  } else if (KIND == kMX && warp == C::SF_WARP) {
    // ============================ MX scale copies ============================
    // For every stage the MMA thread will consume: wait for its loads, copy its three scale
    // blocks into the stage's tensor-memory slot (shared memory -> tensor memory), and commit
    // them to sff[stage]. Issued apart from the MMAs so that a copy never waits behind them;
    // the slot is free because the stage was refilled only after its previous MMAs completed.
    if (lane == 0 && issuer) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      const uint64_t cp_desc0 = smem_desc_plain(smem_u32(smem) + C::A_BYTES + C::B_BYTES, 128);
      for (int64_t t = unit; t < total && ok; t += n_units) {
        const int64_t nkb = tile_nkb<SCHED>(p, t, aux);
        for (int64_t kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(&S.full[stage], phase, abort_flag, p.wait_ns)) {
            if (!*abort_flag) fail();
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sf_t = tmem_base + (uint32_t)(C::SF_COL0 + 16 * stage);
          const uint64_t cd = cp_desc0 + (uint64_t)((stage * C::STAGE_BYTES) >> 4);
#pragma unroll
          for (int j = 0; j < 3; ++j) {
            if (CG == 2)
              tmem_cp_sf_pair(sf_t + 4 * j, cd + 32 * j);
            else
              tmem_cp_sf(sf_t + 4 * j, cd + 32 * j);
          }
          if (CG == 2)
            umma_commit_pair(&S.sff[stage], 0x1);
          else
            umma_commit(&S.sff[stage]);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      // every copy into either CTA's tensor memory completes before it is released
      if (CG == 2)
        umma_commit_pair(&S.sf_drain, 0x3);
      else
        umma_commit(&S.sf_drain);
    }
    __syncwarp();
  } else {
    // ================================ epilogue ================================
    const int q = warp & 3;              // TMEM lane quarter this warp may access
    const int c0 = ((warp - C::EPI0) >> 2) * C::WCOLS;  // first tile column of this warp's share
    const int etid = tid - 32 * C::EPI0;  // 0..255 across the epilogue warps
    const int row = (int)rank * BM + q * 32 + lane;  // row within the pair's tile
    const bool stage_sb = KIND == kFP8 && !p.sb_scalar;
    int buf = 0, sbi = 0;
    uint32_t oseq = 0;  // TMA stores issued by this warp
    uint32_t aphase = 0;
    // The next tile and the scales it needs (this thread's row scale; its column scale, or the
    // scalar one) are fetched one tile ahead, so the memory latency hides behind this tile.
    Tile Tn;
    float sa_nx = 1.0f, sb_nx = 1.0f;
    auto fetch = [&](int64_t tt) {
      Tn = get_tile<SCHED, C::TILE_M, TN>(p, tt, tpre, aux, pst);
      if (KIND != kFP8) return;
      if (kTail && Tn.tt) {  // this thread's weight-row scale; the staged scales are the rows'
        const int64_t n = Tn.n0 + row;
        sa_nx = n < p.N ? __ldg(p.sB + (int64_t)Tn.e * p.N + n) : 0.0f;
        sb_nx = etid < Tn.tt ? (p.sa_scalar ? __ldg(p.sA) : __ldg(p.sA + Tn.m0 + etid)) : 0.0f;
        return;
      }
      const int64_t m = (int64_t)Tn.m0 + row;
      const float* sbp = p.sB;
      if (!is_dense(SCHED)) sbp += (int64_t)Tn.e * (EPI == kGate ? 2 * p.N : p.N);
      sa_nx = 1.0f;
      if (m < Tn.row_end) {
        if (SCHED == kJagK)
          sa_nx = __ldg(p.sA + (int64_t)Tn.e * p.M + m);
        else
          sa_nx = p.sa_scalar ? __ldg(p.sA) : __ldg(p.sA + m);
      }
      if (stage_sb) {
        const int part = EPI == kGate ? etid / TN : 0;  // kGate: the gate's columns, then the up projection's
        const int64_t n = Tn.n0 + etid - part * TN;
        sb_nx = n < p.N && part < 2 ? __ldg(sbp + n + part * p.N) : 0.0f;
      } else {
        sb_nx = __ldg(sbp);
      }
    };
    // kGate: the codes of the hidden layer's columns n .. n + W - 1 of row m. A row's 128-column block lies in the warps of
    // one lane quarter, 64 columns each: they share its largest magnitude through shared memory.
    int amax_buf = 0;
    auto gate_codes = [&](const float* hv, auto width, int64_t m, int64_t n, bool row_ok) {
      constexpr int W = decltype(width)::value;
      if (W < 64 || !p.gate.q) return;  // codes: tiles of whole blocks
      float a = 0.0f;
#pragma unroll
      for (int j = 0; j < W; ++j) a = max_nan(a, fabsf(hv[j]));
      const int at = q * 32 + lane, part = (warp - C::EPI0) >> 2;
      AS.a[amax_buf][part][at] = a;
      named_bar_sync(3 + q, 128 / W * 32);
#pragma unroll
      for (int i = 0; i < 128 / W; ++i) a = max_nan(a, AS.a[amax_buf][i][at]);
      amax_buf ^= 1;
      a = max_nan(a, (float)kEps);
      if (!row_ok || n >= p.N) return;  // N % 128 == 0: the block is all in range or all out
      const bool e4 = p.gate.q_fmt == FP8_DT_E4M3;
      if (part == 0) p.gate.inv[m * (p.N / 128) + n / 128] = a * (e4 ? 1.0f / kE4M3Max : 1.0f / kE5M2Max);
      uint8_t* o = p.gate.q + m * p.N + n;
      if (e4)
        store_codes<FP8_DT_E4M3, W>(o, hv, __fdiv_rn(kE4M3Max, a), p.gate.wide);
      else
        store_codes<FP8_DT_E5M2, W>(o, hv, __fdiv_rn(kE5M2Max, a), p.gate.wide);
    };
    // Boxes of 32 rows x 32 columns in shared memory, 64 bytes a row, swizzled (16-byte chunk ^ row / 2 % 4): lane `lane`
    // reads and writes its own row.
    uint8_t* box0 = out_stage + (warp - C::EPI0) * ((EPI == kGate ? 2 : 4) * kGateBox);
    auto box_at = [&](uint8_t* box, int c) {
      return reinterpret_cast<uint4*>(box + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4));
    };
    auto box_put = [&](uint8_t* box, const uint32_t* w) {
#pragma unroll
      for (int c = 0; c < 4; ++c) *box_at(box, c) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
    };
    auto box_get = [&](uint8_t* box, uint32_t* w) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint4 v = *box_at(box, c);
        w[4 * c] = v.x, w[4 * c + 1] = v.y, w[4 * c + 2] = v.z, w[4 * c + 3] = v.w;
      }
    };
    // kGate: 32 columns from n of the warp's rows: the hidden layer (half < 0) or a projection. Past a segment's end rows
    // belong to others: such a warp's rows are stored by the lanes that hold them.
    uint32_t box_seq = 0;
    auto put32 = [&](const float* f, int half, int64_t m, int64_t n, const Tile& T, bool row_ok) {
      uint32_t w[16];
      pack_row32(f, w);
      const int64_t wrow0 = m - lane;
      if (C::GATE_BOXES && (SCHED != kJagM || wrow0 + 32 <= T.row_end)) {
        if (n >= p.N) return;
        uint8_t* box = box0 + (box_seq++ & 1) * kGateBox;
        if (lane == 0) bulk_wait_read_1();  // the store before the last one has read this box
        __syncwarp();
        box_put(box, w);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (half < 0)
            tma_store_2d(&tmO, box, (int32_t)n, (int32_t)wrow0);
          else
            tma_store_3d(&tmSA, box, (int32_t)n, half, (int32_t)wrow0);
          bulk_commit();
        }
      } else if (row_ok) {
        store_row32(half < 0 ? p.gate.h + m * p.N + n : p.gate.gu + m * 2 * p.N + half * p.N + n, w, p.N - n, p.gate.wide);
      }
    };
    // kGateBwd: the warp's chunks (32 rows x 32 columns of a tile that hold any element of D) in the order of its tiles; the
    // projections' boxes of two of them are in shared memory or on their way. `ahead` is the next one to ask for.
    struct Ahead {
      int64_t t;
      int32_t m0, n0, row_end;
      int ch;
    } ahead = {unit, 0, 0, 0, 0};
    uint32_t asked = 0, done = 0;
    bool dead = false;  // a wait ran out: the warp goes on to the next vote
    auto chunk_live = [&](int32_t m0, int32_t n0, int32_t row_end, int ch) {
      return m0 + (int32_t)rank * BM + q * 32 < row_end && n0 + c0 + 32 * ch < p.N;
    };
    auto seek = [&]() {  // to the next live chunk, from ahead.ch of tile ahead.t on
      while (ahead.t < total) {
        if (ahead.ch == 0) {
          const Tile A = get_tile<SCHED, C::TILE_M, TN>(p, ahead.t, tpre, aux, pst);
          ahead.m0 = A.m0, ahead.n0 = A.n0, ahead.row_end = A.row_end;
        }
        if (ahead.ch < C::WCOLS / 32 && chunk_live(ahead.m0, ahead.n0, ahead.row_end, ahead.ch)) return;
        ahead.t += n_units, ahead.ch = 0;  // the chunks behind a dead one are dead
      }
    };
    auto ask = [&]() {  // loads of the next chunk into the boxes that chunk asked - 2 had
      if (ahead.t >= total) return;
      if (lane == 0) {
        uint8_t* box = box0 + (asked & 1) * (2 * kGateBox);
        uint64_t* bar = &BB.full[warp - C::EPI0][asked & 1];
        mbar_arrive_expect_tx(bar, 2 * kGateBox);
        const int32_t x = ahead.n0 + c0 + 32 * ahead.ch, y = ahead.m0 + (int32_t)rank * BM + q * 32;
        tma_load_3d(box, &tmSA, bar, x, 0, y);
        tma_load_3d(box + kGateBox, &tmSA, bar, x, 1, y);
      }
      ++asked;
      ++ahead.ch;
      seek();
    };
    auto bwd_chunk = [&](const float* dh, const Tile& T, int ch, int64_t m, bool row_ok) {
      if (!chunk_live(T.m0, T.n0, T.row_end, ch)) return;
      if (done > 0) {  // the chunk before this one: its boxes have been read by its stores
        if (lane == 0) bulk_wait_read_all();
        __syncwarp();
        ask();
      }
      uint8_t* box = box0 + (done & 1) * (2 * kGateBox);
      if (!mbar_wait(&BB.full[warp - C::EPI0][done & 1], (done >> 1) & 1, abort_flag, p.wait_ns)) {
        if (!*abort_flag) fail();
        dead = true;
        mbar_wait(&BB.full[warp - C::EPI0][done & 1], (done >> 1) & 1, nullptr, kDrainNs);  // it may still land
      }
      ++done;
      GuChunk c;
      box_get(box, c.g);
      box_get(box + kGateBox, c.u);
      fence_proxy_async_smem();  // these reads come before the next loads' writes to the boxes, which are another proxy's
      const int64_t n = T.n0 + c0 + 32 * ch, wrow0 = m - lane;
      const bool boxes = SCHED != kJagM || wrow0 + 32 <= T.row_end;
      uint32_t h[16];
      if (p.gate.act == FP8_ACT_GELU)
        gate_bwd<FP8_ACT_GELU>(c, dh, h);
      else
        gate_bwd<FP8_ACT_SILU>(c, dh, h);
      if (boxes) {
        box_put(box, c.g);
        box_put(box + kGateBox, c.u);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_3d(&tmO, box, (int32_t)n, 0, (int32_t)wrow0);
          tma_store_3d(&tmO, box + kGateBox, (int32_t)n, 1, (int32_t)wrow0);
          bulk_commit();
        }
      } else if (row_ok) {
        __nv_bfloat16* go = p.gate.gu + m * 2 * p.N + n;
        store_row32(go, c.g, p.N - n, p.gate.wide);
        store_row32(go + p.N, c.u, p.N - n, p.gate.wide);
      }
      if (p.gate.h && row_ok) store_row32(p.gate.h + m * p.N + n, h, p.N - n, p.gate.wide);
      __syncwarp();
    };
    if (EPI == kGateBwd) {
      seek();
      ask();
      ask();
    }
    // kBLK: the scales of kScGroup K blocks from kb0 on: this lane's row of A, and the 128-column block of B that the
    // warp's columns lie in (kGate: the gate's and the up projection's). Loaded a group ahead, so that no promotion
    // waits for memory.
    float ra[kScGroup], rb[kScGroup], rc[kScGroup];
    const float *pa = p.sA, *pb = p.sB, *pc = p.sB;  // sc_vec: the tile's (rows and columns past the end: any scales)
    auto load_scales = [&](const Tile& T, int32_t kb0) {
      const int64_t KB = p.nkb, r = (int64_t)T.m0 + row;
      const int64_t blocks = (EPI == kGate ? 2 * p.N : p.N + 127) / 128;
      const int64_t nb = (T.n0 + (EPI == kGate ? 0 : c0)) / 128;
      const float* a = p.sA + r * KB;
      const float* b = p.sB + ((int64_t)T.e * blocks + nb) * KB;
      if (p.sc_vec) {  // one load for a group: its 32 rows' lines pass the L1 once, not four times
        if (kb0 == 0) pa = r < p.M ? a : p.sA, pb = nb < blocks ? b : p.sB, pc = b + (p.N / 128) * KB;
        if (kb0 >= KB) return;
        const float4 va = __ldg(reinterpret_cast<const float4*>(pa + kb0));
        const float4 vb = __ldg(reinterpret_cast<const float4*>(pb + kb0));
        ra[0] = va.x, ra[1] = va.y, ra[2] = va.z, ra[3] = va.w;
        rb[0] = vb.x, rb[1] = vb.y, rb[2] = vb.z, rb[3] = vb.w;
        if (EPI == kGate) {
          const float4 vc = __ldg(reinterpret_cast<const float4*>(pc + kb0));
          rc[0] = vc.x, rc[1] = vc.y, rc[2] = vc.z, rc[3] = vc.w;
        }
        return;
      }
#pragma unroll
      for (int j = 0; j < kScGroup; ++j) {
        const bool live = kb0 + j < KB;
        ra[j] = live && r < p.M ? __ldg(a + kb0 + j) : 0.0f;
        rb[j] = live && nb < blocks ? __ldg(b + kb0 + j) : 0.0f;
        if (EPI == kGate) rc[j] = live ? __ldg(b + (p.N / 128) * KB + kb0 + j) : 0.0f;
      }
    };
    if (unit < total) fetch(unit);
    if (KIND == kBLK && unit < total) load_scales(Tn, 0);
    for (int64_t t = unit; t < total; t += n_units) {
      const Tile T = Tn;
      const float sa = sa_nx, sb_mine = sb_nx;
      if (KIND != kBLK && t + n_units < total) fetch(t + n_units);
      const int64_t m = (int64_t)T.m0 + row;
      const bool row_ok = m < T.row_end;
      const int64_t orow = SCHED == kJagK ? (int64_t)T.e * p.M + m : m;
      if (stage_sb || (kTail && T.tt)) {  // one column scale per epilogue thread; reused by all 128 rows
        S.sb[sbi][etid] = sb_mine;
        named_bar_sync(1, kEpiThreads);
      }
      const float* sbs = S.sb[sbi];
      sbi ^= 1;
      if (T.nkb == 0) {  // empty segment (jagged K): the result is zero
        if (row_ok) {
          for (int64_t n = T.n0 + c0; n < T.n0 + c0 + C::WCOLS && n < p.N; ++n) {
            if (p.out_f32)
              static_cast<float*>(p.out)[orow * p.ldo + n] = 0.0f;
            else
              static_cast<uint16_t*>(p.out)[orow * p.ldo + n] = 0;
          }
        }
        continue;
      }
      if constexpr (KIND == kBLK) {
        // promotion: for every K block, this warp's half of the partial into registers, the partial back to the MMAs,
        // acc += partial * sA[m, kb] * sB[n / 128, kb]. The next 16 columns are on their way while these are added.
        // What bounds it: the chain of each promoting warp. Two warps a scheduler read 16 columns, 50 cycles after they
        // asked, and add them: 400 cycles to the partial's release, 620 to the last addition, 200 to the next partial (a test
        // of a barrier alone takes 98), and the first K block of a group of scales 350 more. 870 cycles a K block, 512 of
        // them MMAs: 355 us at 8192 x 14336 x 4096 (2710 TFLOP/s). Sixteen warps with 64 accumulators a thread 394, loads of
        // 32 columns 406, the row's scales by TMA 381, a second warp issuing every other K block 3345; CTA pairs, before
        // these steps, 523 for 452.
        constexpr int WC = C::WCOLS;
        static_assert(WC % 32 == 0 && WC <= 128, "a warp's columns, in one block of B's scales");
        float acc[WC];
#pragma unroll
        for (int j = 0; j < WC; ++j) acc[j] = 0.0f;
        auto add16 = [](float* a, const uint32_t* v, float sc) {
#pragma unroll
          for (int j = 0; j < 16; ++j) a[j] = fmaf(__uint_as_float(v[j]), sc, a[j]);
        };
        bool live = true;
        for (int32_t kb0 = 0; kb0 < T.nkb && live; kb0 += kScGroup) {
          float sk[kScGroup], su[kScGroup];
#pragma unroll
          for (int j = 0; j < kScGroup; ++j) {
            sk[j] = ra[j] * rb[j];
            su[j] = EPI == kGate ? ra[j] * rc[j] : sk[j];
          }
          load_scales(T, kb0 + kScGroup);
#pragma unroll 1  // (unrolled, the same time and four times the code)
          for (int j = 0; j < kScGroup && kb0 + j < T.nkb; ++j) {
            const float skj = sk[0], suj = su[0];
#pragma unroll
            for (int i = 0; i + 1 < kScGroup; ++i) sk[i] = sk[i + 1], su[i] = su[i + 1];
            if (!mbar_wait(&S.tfull[buf], aphase, abort_flag, p.wait_ns)) {
              if (!*abort_flag) fail();
              live = false;
              break;
            }
            tc_fence_after();
            const uint32_t taddr = tmem_base + (uint32_t)(buf * TBN + c0) + ((uint32_t)(q * 32) << 16);
            uint32_t va[16], vb[16];
            tmem_ld16(taddr, va);
            tmem_ld_wait_regs16(va);
#pragma unroll
            for (int c = 0; c < WC; c += 32) {
              tmem_ld16(taddr + c + 16, vb);
              add16(acc + c, va, c < WC / 2 ? skj : suj);
              tmem_ld_wait_regs16(vb);
              if (c + 32 == WC) break;
              tmem_ld16(taddr + c + 32, va);
              add16(acc + c + 16, vb, c < WC / 2 ? skj : suj);
              tmem_ld_wait_regs16(va);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if (CG == 2)
                mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&S.tempty[buf]), 0));
              else
                mbar_arrive_relaxed(&S.tempty[buf]);
            }
            if (++buf == 2) {
              buf = 0;
              aphase ^= 1;
            }
            add16(acc + WC - 16, vb, suj);
          }
        }
        if (t + n_units < total) {  // the next tile, not held in registers before
          fetch(t + n_units);
          load_scales(Tn, 0);
        }
        // the decision is uniform where warps meet at a barrier below
        if (EPI == kGate && p.gate.q) live = named_bar_and(2, kEpiThreads, live);
        if (!live) break;
        if constexpr (EPI == kGate) {
          const int64_t n = T.n0 + c0 / 2;
#pragma unroll
          for (int j = 0; j < WC / 2; j += 32) {
            if (p.gate.gu) {
              put32(acc + j, 0, m, n + j, T, row_ok);
              put32(acc + WC / 2 + j, 1, m, n + j, T, row_ok);
            }
            gate_fwd<32>(p.gate.act, acc + j, acc + WC / 2 + j, acc + j);
            if (p.gate.h) put32(acc + j, -1, m, n + j, T, row_ok);
          }
          gate_codes(acc, std::integral_constant<int, WC / 2>(), m, n, row_ok);
          continue;
        }
        if constexpr (EPI == kGateBwd) {
#pragma unroll
          for (int ch = 0; ch < WC / 32; ++ch) bwd_chunk(acc + 32 * ch, T, ch, m, row_ok);
          if (dead) break;
          continue;
        }
        if (row_ok) {
#pragma unroll
          for (int h = 0; h < WC / 32; ++h) {
            const int64_t n = T.n0 + c0 + 32 * h;
            if (n >= p.N) break;
            const float* a = acc + 32 * h;
            const bool full = p.vec_ok && n + 32 <= p.N;
            if (p.out_f32) {
              float* o = static_cast<float*>(p.out) + orow * p.ldo + n;
              if (full && p.wide) {
#pragma unroll
                for (int j = 0; j < 32; j += 8) st_v8(o + j, reinterpret_cast<const uint32_t*>(a + j));
              } else if (full) {
#pragma unroll
                for (int j = 0; j < 32; j += 4) *reinterpret_cast<float4*>(o + j) = make_float4(a[j], a[j + 1], a[j + 2], a[j + 3]);
              } else {
                for (int j = 0; j < 32 && n + j < p.N; ++j) o[j] = a[j];
              }
            } else {
              __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + orow * p.ldo + n;
              uint32_t wd[16];
              pack_row32(a, wd);
              if (p.vec_ok) {
                store_row32(o, wd, p.N - n, p.wide);
              } else {
                for (int j = 0; j < 32 && n + j < p.N; ++j)
                  reinterpret_cast<uint16_t*>(o)[j] = (uint16_t)(wd[j >> 1] >> (16 * (j & 1)));
              }
            }
          }
        }
        continue;
      }
      const bool got = !dead && mbar_wait(&S.tfull[buf], aphase, abort_flag, p.wait_ns);
      if (!named_bar_and(2, kEpiThreads, got)) {  // uniform decision across the epilogue warps
        if (!got && !*abort_flag) fail();
        break;
      }
      tc_fence_after();
      if (KIND == kMX) {
        // this warp's 64 columns into registers, the accumulator back to the MMAs, then stores
        const uint32_t taddr = tmem_base + (uint32_t)c0 + ((uint32_t)(q * 32) << 16);
        uint32_t va[32], vb[32];
        tmem_ld32(taddr, va);
        tmem_ld32(taddr + 32, vb);
        tmem_ld_wait_regs(va);
        tmem_ld_wait_regs(vb);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (CG == 2)
            mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&S.tempty[0]), 0));
          else
            mbar_arrive_relaxed(&S.tempty[0]);
        }
        aphase ^= 1;
        if (C::MX_TMA_OUT && p.tma_out && !p.out_f32 && T.n0 + c0 < p.N) {
          // jagged K: bf16 through a 128-byte-swizzled [32 rows][128 B] box and one TMA store
          // per warp and tile (columns past N are clipped by the copy)
          const int64_t wrow0 = T.m0 + (int64_t)rank * BM + q * 32;
          uint8_t* st = out_stage + (warp - 2) * kStageOut;
          uint32_t w[32];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const __nv_bfloat162 h0 = __floats2bfloat162_rn(__uint_as_float(va[2 * j]), __uint_as_float(va[2 * j + 1]));
            const __nv_bfloat162 h1 = __floats2bfloat162_rn(__uint_as_float(vb[2 * j]), __uint_as_float(vb[2 * j + 1]));
            w[j] = *reinterpret_cast<const uint32_t*>(&h0);
            w[16 + j] = *reinterpret_cast<const uint32_t*>(&h1);
          }
          if (lane == 0) bulk_wait_read_all();  // the previous tile's store has read the buffer
          __syncwarp();
#pragma unroll
          for (int c8 = 0; c8 < 8; ++c8)
            *reinterpret_cast<uint4*>(st + lane * 128 + ((c8 ^ (lane & 7)) << 4)) =
                make_uint4(w[4 * c8], w[4 * c8 + 1], w[4 * c8 + 2], w[4 * c8 + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&tmO, st, (int32_t)(T.n0 + c0), (int32_t)wrow0, T.e);
            bulk_commit();
          }
          continue;
        }
        if (row_ok) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t* v = h ? vb : va;
            const int64_t n = T.n0 + c0 + 32 * h;
            if (n >= p.N) break;
            const bool full = p.vec_ok && n + 32 <= p.N;
            if (p.out_f32) {
              float* o = static_cast<float*>(p.out) + orow * p.ldo + n;
              if (full) {
#pragma unroll
                for (int j = 0; j < 32; j += 4)
                  *reinterpret_cast<uint4*>(o + j) = make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
              } else {
                for (int j = 0; j < 32 && n + j < p.N; ++j) o[j] = __uint_as_float(v[j]);
              }
            } else {
              uint16_t* o = static_cast<uint16_t*>(p.out) + orow * p.ldo + n;
              uint32_t wd[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const __nv_bfloat162 hb = __floats2bfloat162_rn(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
                wd[j] = *reinterpret_cast<const uint32_t*>(&hb);
              }
              if (full) {
#pragma unroll
                for (int j = 0; j < 16; j += 4)
                  *reinterpret_cast<uint4*>(o + 2 * j) = make_uint4(wd[j], wd[j + 1], wd[j + 2], wd[j + 3]);
              } else {
                for (int j = 0; j < 32 && n + j < p.N; ++j) o[j] = (uint16_t)(wd[j >> 1] >> (16 * (j & 1)));
              }
            }
          }
        }
        continue;
      }
      const float sb_all = (KIND == kFP8 && p.sb_scalar) ? sb_mine : 1.0f;
      const uint32_t taddr = tmem_base + (uint32_t)(buf * TBN + c0) + ((uint32_t)(q * 32) << 16);
      if (kTail && T.tt) {
        // transposed tail tile: lane = weight row n (an output column), tensor-memory column j =
        // the tile's row m0 + j. Rounded as the ordinary tiles round, (acc * sA[m]) * sB[n]. For
        // each row the warp's lanes hold 32 consecutive output columns: every store instruction
        // writes 64 (bf16) or 128 (fp32) contiguous bytes; rows past the tile's end are skipped.
        const int64_t n = T.n0 + row;
        const bool n_ok = n < p.N;
        const float2 sn2 = make_float2(sa, sa);
        uint32_t v[32];
        for (int ch = 0; ch < C::WCOLS / 32; ++ch) {
          const int cl = c0 + ch * 32;
          if (cl >= T.tt) break;  // uniform across the warp
          tmem_ld32(taddr + ch * 32, v);
          tmem_ld_wait_regs(v);
          const int nr = T.tt - cl < 32 ? T.tt - cl : 32;
          const int64_t o0 = (T.m0 + cl) * p.ldo + n;
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float2 x = fmul2_rn(fmul2_rn(make_float2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])),
                                               *reinterpret_cast<const float2*>(sbs + cl + j)),
                                      sn2);
            if (n_ok && j < nr) {
              if (p.out_f32) {
                float* o = static_cast<float*>(p.out) + o0 + j * p.ldo;
                o[0] = x.x;
                if (j + 1 < nr) o[p.ldo] = x.y;
              } else {
                __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + o0 + j * p.ldo;
                o[0] = __float2bfloat16_rn(x.x);
                if (j + 1 < nr) o[p.ldo] = __float2bfloat16_rn(x.y);
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&S.tempty[buf]), 0));
        if (++buf == 2) {
          buf = 0;
          aphase ^= 1;
        }
        continue;
      }
      if constexpr (EPI != kStore) {
        // kGate: the warp's columns of the hidden layer, 32 at a time, from either half of the accumulator. kGateBwd: its
        // columns of the hidden layer's gradient.
        const float2 sa2 = make_float2(sa, sa);
        auto load32 = [&](int col, float* f) {  // 32 tile columns, scaled
          uint32_t v[32];
          __syncwarp();
          tmem_ld32(tmem_base + (uint32_t)(buf * TBN + col) + ((uint32_t)(q * 32) << 16), v);
          tmem_ld_wait_regs(v);
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            float2 x = make_float2(__uint_as_float(v[j]), __uint_as_float(v[j + 1]));
            if (KIND == kFP8)
              x = fmul2_rn(fmul2_rn(x, sa2), stage_sb ? *reinterpret_cast<const float2*>(sbs + col + j) : make_float2(sb_all, sb_all));
            f[j] = x.x;
            f[j + 1] = x.y;
          }
        };
        auto release = [&]() {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (CG == 2)
              mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&S.tempty[buf]), 0));
            else
              mbar_arrive_relaxed(&S.tempty[buf]);
          }
          if (++buf == 2) {
            buf = 0;
            aphase ^= 1;
          }
        };
        if constexpr (EPI == kGate) {
          const int hc = c0 / 2;  // the warp's first column of the hidden layer's
          const int64_t n = T.n0 + hc;
          constexpr int W = C::WCOLS / 2;
          float hv[W];
#pragma unroll
          for (int ch = 0; ch < W / 32; ++ch) {
            float u[32];
            load32(hc + 32 * ch, hv + 32 * ch);
            load32(TN + hc + 32 * ch, u);
            if (ch + 1 == W / 32) release();
            if (p.gate.gu) {
              put32(hv + 32 * ch, 0, m, n + 32 * ch, T, row_ok);
              put32(u, 1, m, n + 32 * ch, T, row_ok);
            }
            gate_fwd<32>(p.gate.act, hv + 32 * ch, u, hv + 32 * ch);
            if (p.gate.h) put32(hv + 32 * ch, -1, m, n + 32 * ch, T, row_ok);
          }
          gate_codes(hv, std::integral_constant<int, W>(), m, n, row_ok);
        } else {
#pragma unroll
          for (int ch = 0; ch < C::WCOLS / 32; ++ch) {
            float dh[32];
            load32(c0 + 32 * ch, dh);
            if (ch + 1 == C::WCOLS / 32) release();
            bwd_chunk(dh, T, ch, m, row_ok);
          }
        }
        continue;
      }
      if constexpr (SCHED == kDenseQuant) {
        // The next quantization from the epilogue ("Triton Kernel Optimization", Level 1): this
        // lane holds row m's tile columns c0 .. c0 + 127. They are scaled and rounded once to bf16
        // (the result as fp8_scaled_mm stores it), the accumulator goes back to the MMAs, and the
        // bf16 values are quantized along the row: one 1 x 128 block (scale by the recipe's table)
        // or four MX blocks of 32 (E8M0 scales). Codes leave as the row's 128 bytes; the scales
        // beside them.
        static_assert(C::WCOLS == 128, "one 128-column row segment per lane");
        uint32_t h[64];
        const float2 sa2 = make_float2(sa, sa);
        uint32_t v[32];
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          tmem_ld32(taddr + ch * 32, v);
          tmem_ld_wait_regs(v);
          const int cl = c0 + ch * 32;
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float2 sb2 = stage_sb ? *reinterpret_cast<const float2*>(sbs + cl + j) : make_float2(sb_all, sb_all);
            const float2 x = fmul2_rn(fmul2_rn(make_float2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), sa2), sb2);
            const __nv_bfloat162 hb = __floats2bfloat162_rn(x.x, x.y);
            h[ch * 16 + j / 2] = *reinterpret_cast<const uint32_t*>(&hb);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (CG == 2)
            mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&S.tempty[buf]), 0));
          else
            mbar_arrive_relaxed(&S.tempty[buf]);
        }
        if (++buf == 2) {
          buf = 0;
          aphase ^= 1;
        }
        const int64_t n0 = T.n0 + c0;
        if (!row_ok || n0 >= p.N) continue;  // N % 128 == 0: the segment is all in range or all out
        const bool e4 = p.q_fmt == FP8_DT_E4M3;
        uint32_t qw[32];
        if (p.q_mx) {
          uint32_t codes = 0;
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            uint32_t am = 0;
#pragma unroll
            for (int j = 0; j < 16; ++j) am = absmax2(am, h[16 * b + j]);
            const uint32_t code = e4 ? mx_code<FP8_DT_E4M3>(absmax_fold(am)) : mx_code<FP8_DT_E5M2>(absmax_fold(am));
            const float inv = mx_inv(code);
            codes |= code << (8 * b);
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              const uint32_t lo = e4 ? mx_cast2<FP8_DT_E4M3>(h[16 * b + j], inv) : mx_cast2<FP8_DT_E5M2>(h[16 * b + j], inv);
              const uint32_t hi = e4 ? mx_cast2<FP8_DT_E4M3>(h[16 * b + j + 1], inv) : mx_cast2<FP8_DT_E5M2>(h[16 * b + j + 1], inv);
              qw[8 * b + j / 2] = lo | (hi << 16);
            }
          }
          // row m's four block codes: one aligned word of the MX scale layout (rows M, contraction N)
          const int64_t off = ((m / 128) * (p.N / 128) + n0 / 128) * 512 + (m % 32) * 16 + ((m / 32) % 4) * 4;
          *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.q_scales) + off) = codes;
        } else {
          uint32_t am = 0;
#pragma unroll
          for (int j = 0; j < 64; ++j) am = absmax2(am, h[j]);
          const Scale sc = tab_scale(p.q_tab, absmax_fold(am));
          const float2 s2 = make_float2(sc.s32, sc.s32);
#pragma unroll
          for (int j = 0; j < 64; j += 2) {
            const float2 a = fmul2_rn(make_float2(__uint_as_float(h[j] << 16), __uint_as_float(h[j] & 0xFFFF0000u)), s2);
            const float2 b = fmul2_rn(make_float2(__uint_as_float(h[j + 1] << 16), __uint_as_float(h[j + 1] & 0xFFFF0000u)), s2);
            const uint32_t lo = e4 ? cvt_fp8x2<FP8_DT_E4M3>(a.x, a.y) : cvt_fp8x2<FP8_DT_E5M2>(a.x, a.y);
            const uint32_t hi = e4 ? cvt_fp8x2<FP8_DT_E4M3>(b.x, b.y) : cvt_fp8x2<FP8_DT_E5M2>(b.x, b.y);
            qw[j / 2] = lo | (hi << 16);
          }
          static_cast<float*>(p.q_scales)[m * (p.N / 128) + n0 / 128] = sc.inv32;
        }
        uint4* dst = reinterpret_cast<uint4*>(p.q_out + m * p.N + n0);
#pragma unroll
        for (int i = 0; i < 8; ++i) dst[i] = make_uint4(qw[4 * i], qw[4 * i + 1], qw[4 * i + 2], qw[4 * i + 3]);
        continue;
      }
      // Pairs write through shared memory with TMA bulk-tensor stores of 32 rows x 128 bytes
      // (64 bf16 columns, or 32 fp32), unless this warp's 32 rows run past the end of an
      // expert's segment.
      const int64_t wrow0 = T.m0 + (int64_t)rank * BM + q * 32;
      const bool via_tma = CG == 2 && p.tma_out && (SCHED != kJagM || wrow0 + 32 <= T.row_end);
      uint8_t* st = out_stage + (warp - 2) * kStageOut;
      // Two register sets: the load of the next 32 columns is in flight while the current ones
      // are scaled and stored (tcgen05.wait::ld names the set it completes, so the compiler
      // keeps that set in place until then).
      uint32_t va[32], vb[32];
      uint32_t w[32];  // bf16 pairs of two consecutive 32-column chunks (one 128-byte row)
      // Side outputs (dense schedule with amax): the maxima of |out| as stored (bf16), per row over
      // this warp's columns (one relaxed atomic max per row and tile) and per column over this
      // warp's 32 rows. Magnitudes of non-negative values order like their bit patterns, so all
      // maxima are integer maxima on packed pairs (vmax2). The column maxima of a 32 x 32 chunk
      // come from a butterfly across the lanes: each step keeps half of the words and folds in
      // the partner lane's other half (16 shuffles per chunk); the lanes then hold one column
      // pair each. Rows past the tile's end and columns past N count as zero.
      uint32_t racc = 0;
      auto amax_chunk = [&](const uint32_t* wv, int64_t n) {
        const int64_t left = p.N - n;
        const int valid = left >= 32 ? 32 : (left > 0 ? (int)left : 0);
        uint32_t m[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          uint32_t v = wv[i] & 0x7FFF7FFFu;
          if (!row_ok || 2 * i >= valid) v = 0;
          else if (2 * i + 1 >= valid) v &= 0xFFFFu;
          m[i] = v;
          racc = __vmaxu2(racc, v);
        }
        if (!p.col_amax) return;
        // step with distance d (16, 8, 4, 2): the lanes with bit d clear keep words [0, h), the
        // others [h, 2h), each folding in the partner's copy of its kept half
#pragma unroll
        for (int h = 8; h >= 1; h >>= 1) {
          const int d = 2 * h;
          const bool upper = (lane & d) != 0;
#pragma unroll
          for (int i = 0; i < h; ++i) {
            const uint32_t keep = upper ? m[i + h] : m[i];
            const uint32_t give = upper ? m[i] : m[i + h];
            m[i] = __vmaxu2(keep, __shfl_xor_sync(0xffffffffu, give, d));
          }
        }
        m[0] = __vmaxu2(m[0], __shfl_xor_sync(0xffffffffu, m[0], 1));
        // the step of distance 2^k kept word bit (k - 1) from lane bit k, so lane l now holds the
        // column pair of word l >> 1; the even lane reports its low column, the odd one its high
        const int col = 2 * (lane >> 1) + (lane & 1);
        const uint32_t mc = (lane & 1) ? (m[0] >> 16) : (m[0] & 0xFFFFu);
        if (p.amax_whole) {
          const uint32_t mw = __reduce_max_sync(0xffffffffu, mc);
          if (lane == 0 && mw) red_max_relaxed(p.col_amax, mw << 16);
        } else if (col < valid && mc) {
          red_max_relaxed(p.col_amax + n + col, mc << 16);
        }
      };
      tmem_ld32(taddr, va);
      constexpr int NCH = C::WCOLS / 32;
#pragma unroll
      for (int ch = 0; ch < NCH; ++ch) {
        uint32_t* v = (ch & 1) ? vb : va;
        tmem_ld_wait_regs(v);
        if (ch + 1 < NCH) tmem_ld32(taddr + (ch + 1) * 32, (ch & 1) ? va : vb);
        const int cl = c0 + ch * 32;  // tile column of v[0]
        const int64_t n = T.n0 + cl;
        // bf16 through TMA: the pair (ch - 1, ch) is stored once ch is done, unless the pair
        // starts at or past N (uniform across the warp); columns past N are clipped by the copy
        const bool pair_live = T.n0 + c0 + (ch & ~1) * 32 < p.N;
        if (n >= p.N && !(via_tma && !p.out_f32 && pair_live)) continue;
        float f[32];
        if (KIND == kMX) {  // the block scales were applied inside the MMA
#pragma unroll
          for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(v[j]);
        } else {
          const float2 sa2 = make_float2(sa, sa);
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float2 sb2 = stage_sb ? *reinterpret_cast<const float2*>(sbs + cl + j) : make_float2(sb_all, sb_all);
            const float2 x = fmul2_rn(fmul2_rn(make_float2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), sa2), sb2);
            f[j] = x.x;
            f[j + 1] = x.y;
          }
        }
        if (via_tma) {
          if (!p.out_f32) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
              w[(ch & 1) * 16 + j] = *reinterpret_cast<const uint32_t*>(&h);
            }
            if (SCHED == kDenseAmax) amax_chunk(w + (ch & 1) * 16, n);
            if ((ch & 1) == 0) continue;
            if (lane == 0 && oseq >= 1) bulk_wait_read_all();  // the previous store has read the buffer
            __syncwarp();
            // row `lane` of a [32][128 B] box, 128-byte swizzle (16-byte chunk ^ row % 8)
#pragma unroll
            for (int c8 = 0; c8 < 8; ++c8)
              *reinterpret_cast<uint4*>(st + lane * 128 + ((c8 ^ (lane & 7)) << 4)) =
                  make_uint4(w[4 * c8], w[4 * c8 + 1], w[4 * c8 + 2], w[4 * c8 + 3]);
          } else {
            if (lane == 0 && oseq >= 1) bulk_wait_read_all();
            __syncwarp();
#pragma unroll
            for (int c8 = 0; c8 < 8; ++c8)
              *reinterpret_cast<float4*>(st + lane * 128 + ((c8 ^ (lane & 7)) << 4)) =
                  make_float4(f[4 * c8], f[4 * c8 + 1], f[4 * c8 + 2], f[4 * c8 + 3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            const int32_t n_st = (int32_t)(p.out_f32 ? n : n - 32);
            if (SCHED == kJagK)
              tma_store_3d(&tmO, st, n_st, (int32_t)wrow0, T.e);
            else
              tma_store_2d(&tmO, st, n_st, (int32_t)wrow0);
            bulk_commit();
          }
          ++oseq;
          continue;
        }
        uint32_t wd[16];
        if (!p.out_f32) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
            wd[j] = *reinterpret_cast<const uint32_t*>(&h);
          }
          if (SCHED == kDenseAmax) amax_chunk(wd, n);
        }
        if (row_ok) {
          const bool full = p.vec_ok && n + 32 <= p.N;
          if (p.out_f32) {
            float* o = static_cast<float*>(p.out) + orow * p.ldo + n;
            if (full) {
#pragma unroll
              for (int j = 0; j < 32; j += 4) *reinterpret_cast<float4*>(o + j) = make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
            } else {
              for (int j = 0; j < 32 && n + j < p.N; ++j) o[j] = f[j];
            }
          } else {
            uint16_t* o = static_cast<uint16_t*>(p.out) + orow * p.ldo + n;
            if (full) {
#pragma unroll
              for (int j = 0; j < 16; j += 4) *reinterpret_cast<uint4*>(o + 2 * j) = make_uint4(wd[j], wd[j + 1], wd[j + 2], wd[j + 3]);
            } else {
              for (int j = 0; j < 32 && n + j < p.N; ++j) o[j] = (uint16_t)(wd[j >> 1] >> (16 * (j & 1)));
            }
          }
        }
      }
      if (SCHED == kDenseAmax && p.row_amax && row_ok) {
        const uint32_t r = (racc & 0xFFFFu) > (racc >> 16) ? (racc & 0xFFFFu) : (racc >> 16);
        if (r) red_max_relaxed(p.row_amax + orow, r << 16);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {  // the issuing CTA's barrier counts the epilogue warps of both CTAs
        if (CG == 2)
          mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&S.tempty[buf]), 0));
        else
          mbar_arrive_relaxed(&S.tempty[buf]);
      }
      if (++buf == 2) {
        buf = 0;
        aphase ^= 1;
      }
    }
    if (EPI == kGateBwd)  // loads asked for and not used land before the CTA may exit
      for (; done < asked; ++done) mbar_wait(&BB.full[warp - C::EPI0][done & 1], (done >> 1) & 1, nullptr, kDrainNs);
  }

  if ((CG == 2 || C::GATE_BOXES) && warp >= C::EPI0 && warp < C::EPI0 + C::EPI_WARPS && lane == 0)
    bulk_wait_all();  // this warp's stores are done
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_barrier();  // no remote arrive or load into a CTA that has left
  if (warp == 1) {
    if (lane == 0) {
      mbar_wait(&S.drain, 0, nullptr, kDrainNs);  // the MMAs writing this CTA's TMEM
      if (KIND == kMX) mbar_wait(&S.sf_drain, 0, nullptr, kDrainNs);  // and the scale copies
    }
    __syncwarp();
    tc_fence_after();
    if (CG == 2)
      tmem_dealloc_pair(tmem_base, kTmemCols);
    else
      tmem_dealloc(tmem_base, kTmemCols);
  }
}

// Dense tiles walk a group of M-blocks before the next N-block (or a group of N-blocks before
// the next M-block): the group's panels (tile rows x K) are re-read by every block of the other
// dimension, from L2 while the group fits in ~32 MB, and every group reads all of the other
// operand once. The orientation with fewer bytes read by that count is taken. Measured on the
// Llama3 MLP shapes (DRAM bytes read): the forward (1 MB panels) 152 MB with 16 M-blocks per
// group, 115 MB with all 32; the grad-input and bf16 weight-gradient GEMMs (~4 MB panels)
// 573 / 1179 MB with 16 M-blocks, 483 / 1048 MB with 8. pa, pb: panel bytes of A and B.
void set_walk(GemmParams& p, int64_t pa, int64_t pb) {
  auto group = [](int64_t panel, int64_t blocks) {
    int64_t gsz = panel > 0 ? kGroupBytes / panel : blocks;
    if (gsz > blocks) gsz = blocks;
    return gsz < 1 ? (int64_t)1 : gsz;  // never zero: it divides the tile index
  };
  const int64_t gm = group(pa, p.num_m), gn = group(pb, p.num_n);
  const int64_t by_m = p.num_m * pa + (p.num_m + gm - 1) / gm * p.num_n * pb;  // A once, B per group
  const int64_t by_n = p.num_n * pb + (p.num_n + gn - 1) / gn * p.num_m * pa;  // B once, A per group
  p.group_m = gm;
  p.group_n = by_n < by_m ? gn : 0;
}

// Columns of a tile on single CTAs: 256, or 128 or 64 (least) of them where that takes fewer or shorter rounds of CTAs.
// A narrower tile's K blocks and its epilogue take less time, not in proportion: kCost (100 rows, K 4096, 2048 columns of
// the hidden layer in bf16: the backward in 28.7, 22.6 and 19.5 us at 256, 128 and 64 columns, the forward in 24.4 and
// 20.6; but where 256 take one round and 128 two, 37.9 and 53.4). tiles(width): their number.
template <typename F>
int tile_width(int least, int sm_count, F tiles) {
  constexpr int kWidth[3] = {256, 128, 64};
  constexpr float kCost[3] = {1.0f, 0.78f, 0.62f};
  int best = 256;
  float cost = 0.0f;
  for (int i = 0; i < 3 && kWidth[i] >= least; ++i) {
    const float c = (float)((tiles(kWidth[i]) + sm_count - 1) / sm_count) * kCost[i];
    if (i == 0 || c < cost) best = kWidth[i], cost = c;
  }
  return best;
}

template <int KIND, int SCHED, int A_MN, int B_MN, int CG, int EPI = kStore, int NT = BN>
int run(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& o, const CUtensorMap& sfa,
        const CUtensorMap& sfb, GemmParams p, int64_t total_tiles_hint, const Ctx& c) {
  auto kern = gemm_kernel<KIND, SCHED, A_MN, B_MN, CG, EPI, NT>;
  using C = Cfg<KIND, CG, SCHED, EPI, NT>;
  constexpr int kThreads = C::THREADS, kEpiThreads = C::EPI_THREADS;
  const int n_arrays = is_dense(SCHED) ? 0 : (KIND == kMX && SCHED == kJagM) ? 3 : 2;
  const size_t smem = C::RING_BYTES + C::OUT_BYTES + kSharedBytes + (size_t)n_arrays * 4 * (p.E + 1) +
                     (EPI == kGate ? sizeof(AmaxShare) : EPI == kGateBwd ? sizeof(BoxBars) : 0);
  // Once for each device, and all that a CTA may have: the limit is the process's, and the experts' offsets make `smem`
  // another for each E, so a limit set by one thread's call could be below what another's is about to launch with.
  static std::atomic<uint64_t> done{0};
  const uint64_t bit = 1ull << (c.device & 63);
  if (!(done.load(std::memory_order_acquire) & bit)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax) != cudaSuccess)
      return FP8_ERR_CUDA;
    if (KIND == kBLK) {  // the promoting warps would wait without end for registers that a build did not give the block
      cudaFuncAttributes fa;
      if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess ||
          fa.numRegs * kThreads < 32 * C::EPI0 * kIssueRegs + kEpiThreads * kPromoteRegs)
        return FP8_ERR_CUDA;
    }
    done.fetch_or(bit, std::memory_order_release);
  }
  if (KIND == kBLK)
    p.sc_vec = p.nkb % kScGroup == 0 && ((reinterpret_cast<uintptr_t>(p.sA) | reinterpret_cast<uintptr_t>(p.sB)) & 15) == 0;
  int64_t units = c.sm_count / CG;
  if (total_tiles_hint > 0 && total_tiles_hint < units) units = total_tiles_hint;
  if (units < 1) units = 1;
  if (CG == 1) {
    kern<<<(unsigned)units, kThreads, smem, c.stream>>>(a, b, o, sfa, sfb, p);
    return cudaGetLastError() == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CG;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(units * CG));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = c.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, a, b, o, sfa, sfb, p) != cudaSuccess) return FP8_ERR_CUDA;
  return FP8_OK;
}

}  // namespace

}  // namespace fp8lin
