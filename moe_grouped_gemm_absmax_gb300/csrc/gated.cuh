// The gated feed-forward's GEMMs (sm_103a): both projections of a row with the activation and the product, and its
// backward pass, as epilogues of the scaled GEMM (gemm_kernel.cuh; formulas: gate.cuh).
//
//   h = act(x W1^T) * (x W3^T)          a tile of 128 columns of h takes the MMA's 256 columns: 128 rows of W1 and the
//                                       same 128 of W3, so both values of an element meet in one thread
//   dh = dY W2, du = dh act(g), dg = dh u act'(g)     dh stays in the accumulator
#pragma once

#include "args.h"
#include "gemm_kernel.cuh"

namespace fp8lin {

namespace {

// Operands; out: the hidden layer (forward) or the projections' gradients; gu: the projections
struct Maps {
  CUtensorMap a, b, out, gu;
};

template <int KIND, int SCHED, int B_MN, int EPI>
int run_width(int width, const Maps& m, const GemmParams& p, const Ctx& c) {
  const int64_t tiles = SCHED == kDense ? p.num_m * p.num_n : 0;
  if constexpr (EPI == kGateBwd)
    if (width == 64) return run<KIND, SCHED, 0, B_MN, 1, EPI, 64>(m.a, m.b, m.out, m.gu, m.gu, p, tiles, c);
  if (width == 128) return run<KIND, SCHED, 0, B_MN, 1, EPI, 128>(m.a, m.b, m.out, m.gu, m.gu, p, tiles, c);
  return run<KIND, SCHED, 0, B_MN, 1, EPI>(m.a, m.b, m.out, m.gu, m.gu, p, tiles, c);
}

template <int KIND, int SCHED, int B_MN, int EPI>
int run_kind(bool pair, int width, const Maps& m, const GemmParams& p, const Ctx& c) {
  if constexpr (KIND != kBLK)
    if (pair) return run<KIND, SCHED, 0, B_MN, 2, EPI>(m.a, m.b, m.out, m.gu, m.gu, p, SCHED == kDense ? p.num_m * p.num_n : 0, c);
  return run_width<KIND, SCHED, B_MN, EPI>(width, m, p, c);
}

template <int EPI>
int launch_gated_epi(const GatedArgs& g, const Ctx& c) {
  constexpr bool kForward = EPI == kGate;
  const bool fp8 = g.a_dtype != FP8_DT_BF16, grouped = g.ends != nullptr;
  const int esz = fp8 ? 1 : 2;
  GemmParams p = {};
  p.M = g.M;
  p.N = g.I;
  p.K = g.K;
  p.sA = g.sA;
  p.sB = g.sB;
  p.sa_scalar = g.sa_scalar;
  p.sb_scalar = g.sb_scalar;
  p.ends = g.ends;
  p.E = (int)g.E;
  p.total_rows = g.M;
  p.status = c.status;
  p.wait_ns = c.wait_ns;
  p.test_stall = c.test_stall;
  p.gate.act = g.act;
  p.gate.gu = static_cast<__nv_bfloat16*>(g.gu);
  p.gate.h = static_cast<__nv_bfloat16*>(g.h);
  p.gate.q = static_cast<uint8_t*>(g.q);
  p.gate.inv = g.inv;
  p.gate.q_fmt = g.q_fmt;
  p.gate.wide = ((reinterpret_cast<uintptr_t>(g.gu) | reinterpret_cast<uintptr_t>(g.h) |
                  reinterpret_cast<uintptr_t>(g.q)) & 31) == 0 && g.I % 16 == 0;
  if (grouped && (g.E < 1 || g.E > kMaxGatedExperts)) return FP8_ERR_UNSUPPORTED;
  p.nkb = (g.K * esz + BKB - 1) / BKB;
  // CTA pairs, whose tiles have 256 rows, where they fill the GPU; by experts, where these have rows for such tiles (no
  // transposed tails here; 4096 x 2048, forward: 16 experts of 256 rows 67 us on pairs, 81 on single CTAs; 32 of 128 rows
  // 109 and 101; 64 of 64 rows 197 and 181).
  const int64_t per = kForward ? 2 : 1;  // tile columns for each column of the hidden layer
  auto num_n = [&](int w) { return (g.I * per + w - 1) / w; };
  const bool pair = !g.blockwise && (grouped ? g.M >= 2048 && g.M >= 192 * g.E : ((g.M + 255) / 256) * num_n(BN) * 2 >= c.sm_count);
  const int tile_m = pair ? 2 * BM : BM;
  p.num_m = (g.M + tile_m - 1) / tile_m;
  int width = BN;
  if (!pair && !g.q) {  // (codes: a tile has whole blocks)
    const int64_t mb = p.num_m + (grouped ? (g.E < g.M ? g.E : g.M) / 2 : 0);  // half of the last tiles' rows are empty
    width = tile_width(kForward ? 128 : 64, c.sm_count, [&](int w) { return mb * num_n(w); });
  }
  p.num_n = num_n(width);
  set_walk(p, (int64_t)tile_m * g.K * esz, (int64_t)width * g.K * esz);
  if ((p.num_m + (grouped ? g.E : 0)) * p.num_n >= (int64_t)1 << 31) return FP8_ERR_UNSUPPORTED;

  // operand maps: 128-byte rows of K. The forward's B boxes have rows of one projection, the backward's all of a CTA's.
  const CUtensorMapDataType dt = fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const uint32_t kbox = (uint32_t)(BKB / esz),
                 b_rows = (uint32_t)width / (kForward ? (g.blockwise ? 4 : 2) : pair ? 2 : 1);
  const uint64_t rows = (uint64_t)(kForward ? 2 * g.I : g.I);
  Maps m;
  memset(&m, 0, sizeof(m));
  {
    const uint64_t d[2] = {(uint64_t)g.K, (uint64_t)g.M}, st[1] = {(uint64_t)(g.K * esz)};
    const uint32_t box[2] = {kbox, BM};
    FP8_TRY(make_tmap(&m.a, g.A, dt, 2, d, st, box, CU_TENSOR_MAP_SWIZZLE_128B));
  }
  if (grouped) {
    const uint64_t d[3] = {(uint64_t)g.K, rows, (uint64_t)g.E}, st[2] = {(uint64_t)g.K, rows * (uint64_t)g.K};
    const uint32_t box[3] = {kbox, b_rows, 1};
    FP8_TRY(make_tmap(&m.b, g.B, dt, 3, d, st, box, CU_TENSOR_MAP_SWIZZLE_128B));
  } else if (g.b_mn) {
    const uint64_t d[2] = {rows, (uint64_t)g.K}, st[1] = {rows * 2};
    const uint32_t box[2] = {64, 64};
    FP8_TRY(make_tmap(&m.b, g.B, dt, 2, d, st, box, CU_TENSOR_MAP_SWIZZLE_128B));
  } else {
    const uint64_t d[2] = {(uint64_t)g.K, rows}, st[1] = {(uint64_t)(g.K * esz)};
    const uint32_t box[2] = {kbox, b_rows};
    FP8_TRY(make_tmap(&m.b, g.B, dt, 2, d, st, box, CU_TENSOR_MAP_SWIZZLE_128B));
  }
  m.out = m.gu = m.a;  // maps without a use are valid ones all the same
  // boxes of 32 rows x 32 columns of the hidden layer [M, I] and of the projections [M][2][I]
  const uint64_t I = (uint64_t)g.I;
  auto gu_map = [&](CUtensorMap* t, const void* base) {
    const uint64_t d[3] = {I, 2, (uint64_t)g.M}, st[2] = {2 * I, 4 * I};
    const uint32_t box[3] = {32, 1, 32};
    return make_tmap(t, base, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, d, st, box, CU_TENSOR_MAP_SWIZZLE_64B);
  };
  if (!kForward) {
    FP8_TRY(gu_map(&m.gu, g.gu_in));
    FP8_TRY(gu_map(&m.out, g.gu));
  } else {
    if (g.gu) FP8_TRY(gu_map(&m.gu, g.gu));
    if (g.h) {
      const uint64_t d[2] = {I, (uint64_t)g.M}, st[1] = {2 * I};
      const uint32_t box[2] = {32, 32};
      FP8_TRY(make_tmap(&m.out, g.h, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, d, st, box, CU_TENSOR_MAP_SWIZZLE_64B));
    }
  }
  if (!fp8) {
    p.idesc = make_idesc(kFmtBF16, kFmtBF16, 0, (uint32_t)g.b_mn, tile_m, width);
    if constexpr (!kForward)
      if (g.b_mn) return run_kind<kBF16, kDense, 1, EPI>(pair, width, m, p, c);
    return run_kind<kBF16, kDense, 0, EPI>(pair, width, m, p, c);
  }
  p.idesc = make_idesc(g.a_dtype == FP8_DT_E4M3 ? kFmtE4M3 : kFmtE5M2, g.b_dtype == FP8_DT_E4M3 ? kFmtE4M3 : kFmtE5M2,
                       0, 0, tile_m, width);
  if (grouped)
    return g.blockwise ? run_kind<kBLK, kJagM, 0, EPI>(false, width, m, p, c)
                       : run_kind<kFP8, kJagM, 0, EPI>(pair, width, m, p, c);
  return g.blockwise ? run_kind<kBLK, kDense, 0, EPI>(false, width, m, p, c)
                     : run_kind<kFP8, kDense, 0, EPI>(pair, width, m, p, c);
}

}  // namespace

}  // namespace fp8lin
