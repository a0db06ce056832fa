// Host-side internals of fp8lin: launch context, tensor-map encoding and the kernel launchers
// that the C ABI (api.cu) composes.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/fp8lin.h"

namespace fp8lin {

struct Ctx {
  cudaStream_t stream;
  int32_t* status;   // device status word (may be null)
  uint64_t wait_ns;  // bound of every on-device wait
  int sm_count;
  int device;
  int test_stall;    // failure-detection test hook (see fp8_set_test_stall)
};

// Launch that may begin before the kernel before it on the stream has ended (see pdl_wait()): its launch
// and the kernel's start overlap that one's tail.
template <typename... P, typename... A>
int launch_dependent(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...) == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
}

struct ScaleTab;
// The scale table of a format (FP8_DT_E4M3 / FP8_DT_E5M2), built once on the host in fp64.
const ScaleTab& scale_tab(int fmt);

// Fills ctx for the current device; returns FP8_OK or FP8_ERR_DEVICE.
int make_ctx(Ctx* ctx, void* stream, int32_t* status);

// 2-D / 3-D tiled tensor maps (row-major tensors; dims listed innermost first).
int make_tmap(CUtensorMap* map, const void* base, CUtensorMapDataType dt, int rank, const uint64_t* dims,
              const uint64_t* strides_bytes /* rank-1 entries */, const uint32_t* box, CUtensorMapSwizzle swz);

// --- quantize launchers (quantize.cu) ---
// Rowwise: x bf16 [R, C] -> q [R, C], inv [R].
int launch_quant_rows(const void* x, int64_t R, int64_t C, int fmt, void* q, float* inv, const Ctx& c);
// Blockwise 1 x 128 by the row kernel: x bf16 [R, C] -> q [R, C], inv [R, C / 128]; 512 <= C <= 16384,
// C % 128 == 0, else FP8_ERR_UNSUPPORTED (nothing launched).
int launch_quant_rows_blk128(const void* x, int64_t R, int64_t C, int fmt, void* q, float* inv, const Ctx& c);
// Tensorwise in one cooperative launch: amax of x [R, C] into ws[0], a grid barrier on ws[1] (both
// zeroed here), then the cast into q (row-major, may be null) and/or qt ([C, R], may be null); inv [1].
int launch_quant_tensor(const void* x, int64_t R, int64_t C, int fmt, void* q, void* qt, float* inv,
                        uint32_t* amax_ws, const Ctx& c);
// The same with up to 12 tiles of 128 x 64 per SM kept in shared memory between the two reads
// (tensor.cu); for shapes where tensor_stash_ok holds (the outputs can leave by TMA).
bool tensor_stash_ok(int64_t R, int64_t C, bool has_q, bool has_qt);
int launch_quant_tensor_stash(const void* x, int64_t R, int64_t C, int fmt, void* q, void* qt, float* inv,
                              uint32_t* amax_ws, const Ctx& c);
// Columnwise with column-major output. x viewed as [rows_total, C]. Groups of rows share one
// scale per column: either n_groups consecutive groups of group_rows rows (ends == null) or the
// segments given by ends[n_groups] (segment-padded output, padded row count ld_out).
// out_t row (g, c) starts at out_t + (g * C + c) * ld_out (dense) or out_t + c * ld_out + pstart_g
// (segments). inv [n_groups, C]. scratch: col_ws_words(n_groups, C, rows_total) words of device
// memory, 16-byte aligned (unused when the maxima are given).
// Workspace words (4 bytes each) a column quantize of `groups` x C scales over rows_total rows of
// input (all groups) needs.
int64_t col_ws_words(int64_t groups, int64_t C, int64_t rows_total);
// amax_given (optional): the column maxima as fp32 words [n_groups, C] (bf16 values); pass 1 is
// skipped and scratch is not used.
int launch_quant_cols(const void* x, int64_t rows_total, int64_t C, int64_t n_groups, int64_t group_rows,
                      const int32_t* ends, int fmt, void* out_t, int64_t ld_out, float* inv, uint32_t* scratch,
                      const Ctx& c, const uint32_t* amax_given = nullptr);

// --- MX quantize (mx.cu) ---
// Bytes of the E8M0 scales of an operand with `rows` rows and contraction length k (k % 128 == 0):
// [ceil(rows / 128)][k / 128][512]; -1 for bad arguments.
int64_t mx_scale_bytes(int64_t rows, int64_t k);
// x bf16 [batches, R, C] (C % 128 == 0). q: row-major codes (blocks along C) with scales sf; qt:
// column-major codes [batches, C, ld_t] (blocks along R; R % 128 == 0 unless segmented) with
// scales sft. Either output may be null. With ends (batches == 1): segments of rows, padded row
// space of ld_t rows (ld_t % 128 == 0) for sf's rows and qt's columns; pstart_ws: E + 1 words.
int launch_mx_quant(const void* x, int64_t batches, int64_t R, int64_t C, int fmt, void* q, void* sf, void* qt,
                    int64_t ld_t, void* sft, const int32_t* ends, int64_t E, int32_t* pstart_ws, const Ctx& c);

// --- blockwise quantize (blockwise.cu) ---
// x bf16 [R, C] (C % 128 == 0). tile128 false: 1 x 128 tiles, row-major codes q, inv [R, C/128].
// tile128 true: 128 x 128 tiles; q row-major and/or qt column-major [C, R] (R % 128 == 0);
// inv [ceil(R/128), C/128] (may be null when qt is given) and inv_t [C/128, R/128] (with qt).
int launch_blk_quant(const void* x, int64_t R, int64_t C, int fmt, bool tile128, void* q, void* qt, float* inv,
                     float* inv_t, const Ctx& c);

// --- norm with the residual's addition (norm.cu) ---
// x, res (may be null), h, y bf16 [T, H]; w [H] bf16 or fp32; q FP8 [T, H] with inv in the layout of
// gran (row, 1 x 128 or MX); h, y, q and rstd [T] may be null. H % 8 == 0, H <= 16384.
int launch_add_rmsnorm(const void* x, const void* res, const void* w, int w_f32, float eps, int64_t T, int64_t H,
                       int gran, int fmt, void* h, void* y, void* q, void* inv, float* rstd, const Ctx& c);
int64_t rmsnorm_bwd_ws_bytes(int64_t T, int64_t H);
int launch_rmsnorm_bwd(const void* dy, const void* h, const void* w, int w_f32, const float* rstd, const void* dh,
                       int64_t T, int64_t H, void* dx, void* dw, int dw_bf16, float* ws, const Ctx& c);

// --- router (route.cu) ---
// logits [T, E] bf16 or fp32; order, pos and ends all given or all null. E <= 1024, k <= 16. biased: bias is added to
// the score, else to the logit.
int64_t route_ws_bytes(int64_t T, int64_t E);
int launch_route(const void* logits, int bf16, const float* bias, int64_t T, int64_t E, int64_t k, int softmax,
                 int biased, int renorm, float scale, int32_t* ids, float* weights, int32_t* order, int32_t* pos, int32_t* ends,
                 void* ws, const Ctx& c);
int launch_route_bwd(const void* logits, int bf16, const int32_t* ids, const float* dw, int64_t T, int64_t E,
                     int64_t k, int softmax, int renorm, float scale, void* dlogits, const Ctx& c);

// --- experts of a few tokens (moe.cu) ---
int64_t moe_tokens_ws_bytes(int64_t T, int64_t k, int64_t H, int64_t I);
int launch_moe_tokens(const void* x, const int32_t* ids, const float* weights, const void* w13, const float* s13,
                      const void* w2, const float* s2, int64_t T, int64_t k, int64_t E, int64_t H, int64_t I, void* out,
                      void* ws, const Ctx& c);

// --- GEMM launchers (gemm.cu) ---
struct GemmArgs {
  // operands
  const void* A;
  const void* B;
  int a_dtype, b_dtype;   // FP8_DT_*
  int a_mn, b_mn;         // BF16 only: operand stored MN-major
  const float* sA;        // [1] or [M] (dense), [M] (jagged M), [E, M-dim] (jagged K); null for BF16
  const float* sB;
  int64_t sA_len, sB_len; // dense: 1 or M / 1 or N
  void* out;
  int out_dtype;          // FP8_DT_BF16 / FP8_DT_F32
  int64_t M, N, K;        // dense problem; jagged M: M = total rows; jagged K: K = padded rows P
  // grouped
  int mode;               // -1 dense, FP8_GROUPED_JAGGED_M, FP8_GROUPED_JAGGED_K
  const int32_t* ends;
  int64_t E;
  int64_t k_dim;          // jagged K: the output's last dimension (X's columns)
  // MX (block-scaled) operands: E8M0 scales in [row blocks][K / 128][512 B] blocks
  int mx;
  const void* sfa;        // A's scales; rows: M, or the segment-padded row count (jagged M)
  const void* sfb;        // B's scales; rows: N (per expert for jagged M)
  int64_t sfa_rows;
  // side outputs (dense, bf16 out): max |out| per row / per column as fp32 words, or null
  uint32_t* row_amax;
  uint32_t* col_amax;
  int amax_whole;         // col_amax is one word: the maximum over the whole output
  int blockwise;          // FP8 operands with blockwise inverse scales: sA [M, K/128] (1 x 128 tiles),
                          // sB [ceil(N/128), K/128] (128 x 128 tiles), per expert for jagged M
  // quantized output (dense FP8, N % 128 == 0): codes [M, N] in q_fmt and scales of the result's
  // bf16 rounding, 1 x 128 blocks (q_mx 0: fp32 inverse scales [M, N/128]) or MX blocks of 32
  // (q_mx 1: E8M0 bytes in the MX scale layout for rows M, contraction N); out is then unused
  void* q_out;
  void* q_scales;
  int q_mx;
  int q_fmt;
};
int launch_gemm(const GemmArgs& g, const Ctx& c);

// --- the gated feed-forward's GEMMs (gated.cu) ---
constexpr int64_t kMaxGatedExperts = 1024;  // offsets, loads and stores share an SM's memory with the ring
struct GatedArgs {
  const void* A;          // [M, K] FP8 or bf16: the rows (forward), the output's gradient (backward)
  const void* B;          // forward [2 I, K] ([E, 2 I, K]), the gate's rows before the up projection's; backward [I, K]
  int a_dtype, b_dtype;   // ([E, I, K]), or with b_mn [K, I] (bf16 only)
  int b_mn;
  const float* sA;        // [1], [M], or [M, K / 128] (blockwise); null for bf16
  const float* sB;        // [1], one for each of B's rows, or for each 128 x 128 block
  int sa_scalar, sb_scalar;
  int blockwise;
  int64_t M, I, K;
  const int32_t* ends;    // null: dense
  int64_t E;
  int backward;
  int act;
  const void* gu_in;      // backward: the projections [M, 2 I] bf16
  void* gu;               // the projections (forward, may be null) or their gradients (backward) [M, 2 I] bf16
  void* h;                // bf16 [M, I] or null
  void* q;                // forward: FP8 [M, I] with inv fp32 [M, I / 128], or null
  float* inv;
  int q_fmt;
};
int launch_gated(const GatedArgs& g, const Ctx& c);

// --- FP8 products of a few rows (few.cu) ---
// Most rows of a call that takes it: those of its widest tile, so that no call reads its weights twice there. us on either
// kernel (few / tiles), gated, row scales and block scales:
//              16 rows                 48                      64                      65                      128
//   4096 x 14336   23 / 33, 24 / 29    23 / 31, 27 / 27        24 / 31, 28 / 27        35 / 31, 47 / 26        39 / 31, 52 / 27
//   7168 x 2048    12 / 19, 12 / 26    16 / 19, 16 / 26        17 / 20, 17 / 27        16 / 19, 17 / 27        17 / 20, 17 / 27
//   2048 x 1024     7 /  8,  8 / 10    11 /  8, 10 / 11        12 /  9, 11 / 11        12 /  9, 11 / 11        12 /  9, 11 / 11
// and 8 experts' block-scaled products of 2048 x 7168: 23 / 33, 27 / 32, 27 / 27, 27 / 27, 28 / 28. The rows alone are
// not the whole rule: with few output tiles the border lies above 128 rows, with a short contraction below 48.
constexpr int64_t kFewRows = 64;
int launch_few_gated(const GatedArgs& g, const Ctx& c);          // forward, FP8
int launch_few_blockwise(const GemmArgs& g, const Ctx& c);       // jagged M, block scales

}  // namespace fp8lin

namespace fp8lin {
// Cast phase of the tensorwise quantize alone: reads the bf16 pattern of amax at `amax_word`
// (already reduced) and writes q / qt / inv exactly as launch_quant_tensor does.
// amax_shift: 0 when amax_word holds a bf16 pattern, 16 when it holds the fp32 value.
// Test hook: out[i] = the kernels' cast (fmt) of the fp32 value with bit pattern first + i.
int launch_cast_bits(uint32_t first, int64_t n, int fmt, void* out, const Ctx& c);
int launch_quant_tensor_cast(const void* x, int64_t R, int64_t C, int fmt, void* q, void* qt, float* inv,
                             const uint32_t* amax_word, const Ctx& c, int amax_shift = 0);
}  // namespace fp8lin
