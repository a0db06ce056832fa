// Launch of the scaled FP8 (and BF16) GEMMs: operand tensor maps, tile shapes and schedules (the kernel:
// gemm_kernel.cuh).
#include "gemm_kernel.cuh"

namespace fp8lin {

namespace {

// MX operands: the FP8 codes load as on the FP8 path; the E8M0 scales, stored as
// [row blocks][K / 128][512 bytes], load through tensor maps over 128-word rows: a 3-D map
// [row block][K group][128 words] (4-D with the expert for the grouped weights). Box: one A
// block, two consecutive B blocks (a 192-column tile spans parts of at most two).
int launch_mx(const GemmArgs& g, GemmParams& p, const CUtensorMap& to, bool pair, int tile_m, const Ctx& c) {
  if (g.K % 128 || !g.sfa || !g.sfb) return FP8_ERR_UNSUPPORTED;
  const uint32_t af = g.a_dtype == FP8_DT_E4M3 ? kFmtE4M3 : kFmtE5M2;
  const uint32_t bf = g.b_dtype == FP8_DT_E4M3 ? kFmtE4M3 : kFmtE5M2;
  constexpr int TBN = Cfg<kMX, 1>::TBN;
  p.idesc = make_idesc_mx(af, bf, (uint32_t)tile_m, TBN);
  const uint32_t b_rows = pair ? TBN / 2 : TBN;
  const uint64_t kbg = (uint64_t)(g.K / 128);
  const uint64_t rba = (uint64_t)((g.sfa_rows + 127) / 128);
  const uint64_t rbb = (uint64_t)((g.N + 127) / 128);
  CUtensorMap ta, tb, tsa, tsb;
  const uint64_t dA[2] = {(uint64_t)g.K, (uint64_t)g.M};
  const uint64_t strideK[1] = {(uint64_t)g.K};
  const uint32_t boxA[2] = {BKB, BM};
  int rc = make_tmap(&ta, g.A, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, dA, strideK, boxA, CU_TENSOR_MAP_SWIZZLE_128B);
  if (rc) return rc;
  {
    const uint64_t d[3] = {128, kbg, rba};
    const uint64_t st[2] = {512, 512 * kbg};
    const uint32_t box[3] = {128, 1, 1};
    rc = make_tmap(&tsa, g.sfa, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, d, st, box, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (rc) return rc;
  }
  if (g.mode == FP8_GROUPED_JAGGED_M) {
    const uint64_t dB[3] = {(uint64_t)g.K, (uint64_t)g.N, (uint64_t)g.E};
    const uint64_t sB_[2] = {(uint64_t)g.K, (uint64_t)(g.N * g.K)};
    const uint32_t boxB[3] = {BKB, b_rows, 1};
    rc = make_tmap(&tb, g.B, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, dB, sB_, boxB, CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
    const uint64_t d[4] = {128, kbg, rbb, (uint64_t)g.E};
    const uint64_t st[3] = {512, 512 * kbg, 512 * kbg * rbb};
    const uint32_t box[4] = {128, 1, 2, 1};
    rc = make_tmap(&tsb, g.sfb, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, d, st, box, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (rc) return rc;
    p.total_rows = g.M;
    return pair ? run<kMX, kJagM, 0, 0, 2>(ta, tb, to, tsa, tsb, p, 0, c)
                : run<kMX, kJagM, 0, 0, 1>(ta, tb, to, tsa, tsb, p, 0, c);
  }
  const uint64_t dB[2] = {(uint64_t)g.K, (uint64_t)g.N};
  const uint32_t boxB[2] = {BKB, b_rows};
  rc = make_tmap(&tb, g.B, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, dB, strideK, boxB, CU_TENSOR_MAP_SWIZZLE_128B);
  if (rc) return rc;
  {
    const uint64_t d[3] = {128, kbg, rbb};
    const uint64_t st[2] = {512, 512 * kbg};
    const uint32_t box[3] = {128, 1, 2};
    rc = make_tmap(&tsb, g.sfb, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, d, st, box, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (rc) return rc;
  }
  if (g.mode == -1) {
    const int64_t tiles = p.num_m * p.num_n;
    return pair ? run<kMX, kDense, 0, 0, 2>(ta, tb, to, tsa, tsb, p, tiles, c)
                : run<kMX, kDense, 0, 0, 1>(ta, tb, to, tsa, tsb, p, tiles, c);
  }
  p.total_rows = -1;
  const int64_t tiles = (int64_t)g.E * p.num_m * p.num_n;
  return pair ? run<kMX, kJagK, 0, 0, 2>(ta, tb, to, tsa, tsb, p, tiles, c)
              : run<kMX, kJagK, 0, 0, 1>(ta, tb, to, tsa, tsb, p, tiles, c);
}

}  // namespace

// Pairs (CG = 2) serve problems with enough 256-row tiles to fill the GPU; small ones run on
// single CTAs (CG = 1).
int launch_gemm(const GemmArgs& g, const Ctx& c) {
  const bool fp8 = g.a_dtype != FP8_DT_BF16;
  GemmParams p = {};
  p.M = g.M;
  p.N = g.N;
  p.K = g.K;
  p.sA = g.sA;
  p.sB = g.sB;
  p.out = g.out;
  p.out_f32 = g.out_dtype == FP8_DT_F32;
  p.status = c.status;
  p.wait_ns = c.wait_ns;
  p.test_stall = c.test_stall;
  p.row_amax = g.row_amax;
  p.col_amax = g.col_amax;
  p.amax_whole = g.amax_whole;
  p.ends = g.ends;
  p.E = (int)g.E;
  const bool mx = g.mx != 0;
  if (g.mode != -1 && (g.E < 1 || g.E > kMaxExperts)) return FP8_ERR_UNSUPPORTED;
  int blk_cols = BN;  // jagged M with block scales: columns of a tile
  if (g.blockwise && g.mode == FP8_GROUPED_JAGGED_M) {
    if (g.M <= kFewRows) return launch_few_blockwise(g, c);
    const int64_t mb = (g.M + BM - 1) / BM + (g.E < g.M ? g.E : g.M) / 2;  // half of the last tiles' rows are empty
    blk_cols = tile_width(128, c.sm_count, [&](int w) { return mb * ((g.N + w - 1) / w); });
  }
  p.num_n = (g.N + blk_cols - 1) / blk_cols;
  const int esz = fp8 ? 1 : 2;
  p.nkb = (g.K * esz + BKB - 1) / BKB;
  p.ldo = g.N;
  p.vec_ok = p.out_f32 ? (p.ldo % 4 == 0) : (p.ldo % 8 == 0);
  p.wide = ((reinterpret_cast<uintptr_t>(g.out) | (uintptr_t)(p.ldo * (p.out_f32 ? 4 : 2))) & 31) == 0;
  // pair tiles when there are at least ~one per SM pair. Blockwise scaling runs on single CTAs: each K block's
  // partial goes from the MMAs to the promoting warps and back, and across a pair that takes longer than
  // the pair saves in operand traffic (8192 x 14336 x 4096: 523 us on pairs when single CTAs took 452; since then their
  // promotion, for a single CTA's registers, has come to 353).
  const int64_t pair_tiles = ((g.M + 255) / 256) * p.num_n * (g.mode == FP8_GROUPED_JAGGED_K ? g.E : 1);
  const bool pair = !g.blockwise && (g.mode == FP8_GROUPED_JAGGED_M ? g.M >= 2048 : pair_tiles * 2 >= c.sm_count);
  const int tile_m = pair ? 256 : 128;
  p.num_m = (g.M + tile_m - 1) / tile_m;
  set_walk(p, (int64_t)tile_m * g.K * esz, (int64_t)BN * g.K * esz);
  // the kernels index tiles with 32-bit arithmetic
  const int64_t max_tiles = g.mode == FP8_GROUPED_JAGGED_K ? g.E * p.num_m * p.num_n
                            : g.mode == FP8_GROUPED_JAGGED_M ? (p.num_m + g.E) * p.num_n
                                                             : p.num_m * p.num_n;
  if (max_tiles >= (int64_t)1 << 31) return FP8_ERR_UNSUPPORTED;
  // output tensor map for the pairs' TMA stores: boxes of 32 rows x 128 bytes
  CUtensorMap to, none;
  memset(&to, 0, sizeof(to));
  memset(&none, 0, sizeof(none));
  p.tma_out = 0;
  if (pair && p.vec_ok && (reinterpret_cast<uintptr_t>(g.out) & 15) == 0) {
    const CUtensorMapDataType odt = p.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const CUtensorMapSwizzle osw = CU_TENSOR_MAP_SWIZZLE_128B;
    const uint32_t bx = p.out_f32 ? 32 : 64;  // 128-byte box rows
    const uint64_t oes = p.out_f32 ? 4 : 2;
    int rc;
    if (g.mode == FP8_GROUPED_JAGGED_K) {
      const uint64_t d[3] = {(uint64_t)g.N, (uint64_t)g.M, (uint64_t)g.E};
      const uint64_t st[2] = {(uint64_t)g.N * oes, (uint64_t)(g.M * g.N) * oes};
      const uint32_t box[3] = {bx, 32, 1};
      rc = make_tmap(&to, g.out, odt, 3, d, st, box, osw);
    } else {
      const uint64_t d[2] = {(uint64_t)g.N, (uint64_t)g.M};
      const uint64_t st[1] = {(uint64_t)g.N * oes};
      const uint32_t box[2] = {bx, 32};
      rc = make_tmap(&to, g.out, odt, 2, d, st, box, osw);
    }
    if (rc) return rc;
    p.tma_out = 1;
  }

  if (mx) {
    if (g.mode != FP8_GROUPED_JAGGED_K) p.tma_out = 0;  // MX stores from registers except jagged K
    return launch_mx(g, p, to, pair, tile_m, c);
  }
  if (fp8) {
    const uint32_t af = g.a_dtype == FP8_DT_E4M3 ? kFmtE4M3 : kFmtE5M2;
    const uint32_t bf = g.b_dtype == FP8_DT_E4M3 ? kFmtE4M3 : kFmtE5M2;
    p.idesc = make_idesc(af, bf, 0, 0, tile_m, BN);
    p.sa_scalar = g.sA_len == 1;
    p.sb_scalar = g.sB_len == 1;
    CUtensorMap ta, tb;
    const uint32_t boxA[2] = {BKB, BM};
    const uint64_t dA[2] = {(uint64_t)g.K, (uint64_t)g.M};
    const uint64_t strideK[1] = {(uint64_t)g.K};
    const uint32_t b_rows = pair ? BN / 2 : BN;
    int rc = make_tmap(&ta, g.A, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, dA, strideK, boxA, CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
    if (g.mode == -1 || g.mode == FP8_GROUPED_JAGGED_K) {
      const uint64_t dB[2] = {(uint64_t)g.K, (uint64_t)g.N};
      const uint32_t boxB[2] = {BKB, b_rows};
      rc = make_tmap(&tb, g.B, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, dB, strideK, boxB, CU_TENSOR_MAP_SWIZZLE_128B);
      if (rc) return rc;
      if (g.mode == -1) {
        const int64_t tiles = p.num_m * p.num_n;
        if (g.blockwise) {  // sA [M, K/128], sB [ceil(N/128), K/128]
          if (g.K % 128 || p.row_amax || p.col_amax) return FP8_ERR_UNSUPPORTED;
          return run<kBLK, kDense, 0, 0, 1>(ta, tb, to, none, none, p, tiles, c);
        }
        if (p.row_amax || p.col_amax)
          return pair ? run<kFP8, kDenseAmax, 0, 0, 2>(ta, tb, to, none, none, p, tiles, c)
                      : run<kFP8, kDenseAmax, 0, 0, 1>(ta, tb, to, none, none, p, tiles, c);
        if (g.q_out) {
          p.q_out = static_cast<uint8_t*>(g.q_out);
          p.q_scales = g.q_scales;
          p.q_mx = g.q_mx;
          p.q_fmt = g.q_fmt;
          p.q_tab = scale_tab(g.q_fmt);
          return pair ? run<kFP8, kDenseQuant, 0, 0, 2>(ta, tb, to, none, none, p, tiles, c)
                      : run<kFP8, kDenseQuant, 0, 0, 1>(ta, tb, to, none, none, p, tiles, c);
        }
        return pair ? run<kFP8, kDense, 0, 0, 2>(ta, tb, to, none, none, p, tiles, c) : run<kFP8, kDense, 0, 0, 1>(ta, tb, to, none, none, p, tiles, c);
      }
      if (g.blockwise) return FP8_ERR_UNSUPPORTED;
      // jagged K: A = G^T [N_out, P], B = X^T [Kd, P]; tile space M = N_out, N = Kd; the
      // offsets are checked for order and for fitting the padded length P.
      p.total_rows = -1;
      const int64_t tiles = (int64_t)g.E * p.num_m * p.num_n;
      return pair ? run<kFP8, kJagK, 0, 0, 2>(ta, tb, to, none, none, p, tiles, c) : run<kFP8, kJagK, 0, 0, 1>(ta, tb, to, none, none, p, tiles, c);
    }
    if (g.mode == FP8_GROUPED_JAGGED_M) {
      p.total_rows = g.M;
      const uint64_t dB[3] = {(uint64_t)g.K, (uint64_t)g.N, (uint64_t)g.E};
      const uint64_t sB_[2] = {(uint64_t)g.K, (uint64_t)(g.N * g.K)};
      const uint32_t boxB[3] = {BKB, g.blockwise ? (uint32_t)blk_cols : b_rows, 1};
      rc = make_tmap(&tb, g.B, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, dB, sB_, boxB, CU_TENSOR_MAP_SWIZZLE_128B);
      if (rc) return rc;
      if (g.blockwise) {
        p.idesc = make_idesc(af, bf, 0, 0, tile_m, blk_cols);
        return blk_cols == 256 ? run<kBLK, kJagM, 0, 0, 1>(ta, tb, to, none, none, p, 0, c)
                               : run<kBLK, kJagM, 0, 0, 1, kStore, 128>(ta, tb, to, none, none, p, 0, c);
      }
      if (!pair) return run<kFP8, kJagM, 0, 0, 1>(ta, tb, to, none, none, p, 0, c);
      // An expert's last tile with fewer than 256 rows runs transposed: the expert's 256 weight
      // rows as the MMA's M, the tile's rows rounded up to 16 as its N, and only the row boxes
      // that cover them loaded (32, 64 or 128 rows per CTA), so a short tail costs the MMAs and
      // the operand bytes of its rows, not of 256.
      CUtensorMap t32, t64;
      const uint32_t box32[2] = {BKB, 32}, box64[2] = {BKB, 64};
      rc = make_tmap(&t32, g.A, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, dA, strideK, box32, CU_TENSOR_MAP_SWIZZLE_128B);
      if (rc) return rc;
      rc = make_tmap(&t64, g.A, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, dA, strideK, box64, CU_TENSOR_MAP_SWIZZLE_128B);
      if (rc) return rc;
      p.tail_t = 1;
      p.idesc_t = make_idesc(bf, af, 0, 0, 256, 0);
      return run<kFP8, kJagM, 0, 0, 2>(ta, tb, to, t32, t64, p, 0, c);
    }
    return FP8_ERR_INVALID_ARG;
  }

  // BF16 (dense only)
  if (g.mode != -1) return FP8_ERR_UNSUPPORTED;
  p.idesc = make_idesc(kFmtBF16, kFmtBF16, (uint32_t)g.a_mn, (uint32_t)g.b_mn, tile_m, BN);
  const uint32_t b_rows = pair ? BN / 2 : BN;
  CUtensorMap ta, tb;
  int rc;
  if (g.a_mn) {
    const uint64_t d[2] = {(uint64_t)g.M, (uint64_t)g.K};
    const uint64_t s[1] = {(uint64_t)g.M * 2};
    const uint32_t box[2] = {64, 64};
    rc = make_tmap(&ta, g.A, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, d, s, box, CU_TENSOR_MAP_SWIZZLE_128B);
  } else {
    const uint64_t d[2] = {(uint64_t)g.K, (uint64_t)g.M};
    const uint64_t s[1] = {(uint64_t)g.K * 2};
    const uint32_t box[2] = {64, BM};
    rc = make_tmap(&ta, g.A, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, d, s, box, CU_TENSOR_MAP_SWIZZLE_128B);
  }
  if (rc) return rc;
  if (g.b_mn) {
    const uint64_t d[2] = {(uint64_t)g.N, (uint64_t)g.K};
    const uint64_t s[1] = {(uint64_t)g.N * 2};
    const uint32_t box[2] = {64, 64};
    rc = make_tmap(&tb, g.B, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, d, s, box, CU_TENSOR_MAP_SWIZZLE_128B);
  } else {
    const uint64_t d[2] = {(uint64_t)g.K, (uint64_t)g.N};
    const uint64_t s[1] = {(uint64_t)g.K * 2};
    const uint32_t box[2] = {64, b_rows};
    rc = make_tmap(&tb, g.B, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, d, s, box, CU_TENSOR_MAP_SWIZZLE_128B);
  }
  if (rc) return rc;
  const int64_t tiles = p.num_m * p.num_n;
  if (p.row_amax || p.col_amax) {  // side outputs: the weight-gradient layout (both MN-major) only
    if (!(g.a_mn && g.b_mn)) return FP8_ERR_UNSUPPORTED;
    return pair ? run<kBF16, kDenseAmax, 1, 1, 2>(ta, tb, to, none, none, p, tiles, c)
                : run<kBF16, kDenseAmax, 1, 1, 1>(ta, tb, to, none, none, p, tiles, c);
  }
  if (pair) {
    if (g.a_mn && g.b_mn) return run<kBF16, kDense, 1, 1, 2>(ta, tb, to, none, none, p, tiles, c);
    if (g.a_mn) return run<kBF16, kDense, 1, 0, 2>(ta, tb, to, none, none, p, tiles, c);
    if (g.b_mn) return run<kBF16, kDense, 0, 1, 2>(ta, tb, to, none, none, p, tiles, c);
    return run<kBF16, kDense, 0, 0, 2>(ta, tb, to, none, none, p, tiles, c);
  }
  if (g.a_mn && g.b_mn) return run<kBF16, kDense, 1, 1, 1>(ta, tb, to, none, none, p, tiles, c);
  if (g.a_mn) return run<kBF16, kDense, 1, 0, 1>(ta, tb, to, none, none, p, tiles, c);
  if (g.b_mn) return run<kBF16, kDense, 0, 1, 1>(ta, tb, to, none, none, p, tiles, c);
  return run<kBF16, kDense, 0, 0, 1>(ta, tb, to, none, none, p, tiles, c);
}

}  // namespace fp8lin
