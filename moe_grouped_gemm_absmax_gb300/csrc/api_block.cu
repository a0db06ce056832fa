// C ABI of the operators around a mixture-of-experts layer: argument checking for the norm with the
// residual, the router and the experts of a few tokens. Every check comes before any device work.
#include "args.h"
#include "internal.h"

using namespace fp8lin;

static bool shape_max(const fp8_tensor* t, int64_t most) {
  for (int i = 0; i < t->ndim; ++i)
    if (t->shape[i] > most) return false;
  return true;
}
// a usable dense tensor of this dtype and shape, 16-byte aligned
static int check_tensor(const fp8_tensor* t, int dtype, int nd, int64_t a, int64_t b = -1, int64_t c = -1) {
  FP8_CHECK(valid_desc(t) && t->dtype == dtype && shape_is(t, nd, a, b, c), FP8_ERR_INVALID_ARG);
  FP8_CHECK(aligned16(t->ptr), FP8_ERR_ALIGNMENT);
  return FP8_OK;
}
static int check_workspace(const void* ws, size_t bytes, int64_t need) {
  FP8_CHECK(need == 0 || (ws && (reinterpret_cast<uintptr_t>(ws) & 15u) == 0 && bytes >= (size_t)need),
            FP8_ERR_WORKSPACE);
  return FP8_OK;
}

constexpr int64_t kMaxDim = (int64_t)1 << 31;

// ------------------------------------------------------------------------------------------
// norm

static bool norm_width(int64_t H) { return H > 0 && H <= 16384 && H % 8 == 0; }

static int check_norm_input(const fp8_tensor* x, const fp8_tensor* weight) {
  FP8_CHECK(valid_desc(x) && x->dtype == FP8_DT_BF16 && x->ndim == 2, FP8_ERR_INVALID_ARG);
  FP8_CHECK(shape_max(x, kMaxDim - 1), FP8_ERR_UNSUPPORTED);
  const int64_t H = x->shape[1];
  FP8_CHECK(H % 8 == 0, FP8_ERR_ALIGNMENT);
  FP8_CHECK(norm_width(H), FP8_ERR_UNSUPPORTED);
  FP8_CHECK(aligned16(x->ptr), FP8_ERR_ALIGNMENT);
  FP8_CHECK(valid_desc(weight) && is_out(weight->dtype) && shape_is(weight, 1, H), FP8_ERR_INVALID_ARG);
  FP8_CHECK(aligned16(weight->ptr), FP8_ERR_ALIGNMENT);
  return FP8_OK;
}

extern "C" int fp8_add_rmsnorm(const fp8_tensor* x, const fp8_tensor* residual, const fp8_tensor* weight, float eps,
                               int granularity, fp8_tensor* h, fp8_tensor* y, fp8_tensor* q, fp8_tensor* inv_scales,
                               fp8_tensor* rstd, void* stream) {
  FP8_TRY(check_norm_input(x, weight));
  FP8_CHECK(eps >= 0.0f, FP8_ERR_INVALID_ARG);
  const int64_t T = x->shape[0], H = x->shape[1];
  if (residual) FP8_TRY(check_tensor(residual, FP8_DT_BF16, 2, T, H));
  if (h) FP8_TRY(check_tensor(h, FP8_DT_BF16, 2, T, H));
  if (y) FP8_TRY(check_tensor(y, FP8_DT_BF16, 2, T, H));
  if (rstd) FP8_TRY(check_tensor(rstd, FP8_DT_F32, 1, T));
  FP8_CHECK((q != nullptr) == (inv_scales != nullptr), FP8_ERR_INVALID_ARG);
  FP8_CHECK(h || y || q || rstd, FP8_ERR_INVALID_ARG);
  if (q) {
    FP8_CHECK(valid_desc(q) && is_fp8(q->dtype), FP8_ERR_INVALID_ARG);
    FP8_TRY(check_tensor(q, q->dtype, 2, T, H));
    FP8_CHECK(valid_desc(inv_scales) && shape_max(inv_scales, (int64_t)1 << 40), FP8_ERR_INVALID_ARG);
    FP8_CHECK(aligned16(inv_scales->ptr), FP8_ERR_ALIGNMENT);
    switch (granularity) {
      case FP8_GRAN_ROW:
        FP8_CHECK(inv_scales->dtype == FP8_DT_F32 && shape_is(inv_scales, 1, T), FP8_ERR_INVALID_ARG);
        break;
      case FP8_GRAN_BLOCK_1x128:
        FP8_CHECK(H % 128 == 0, FP8_ERR_UNSUPPORTED);
        FP8_CHECK(inv_scales->dtype == FP8_DT_F32 && shape_is(inv_scales, 2, T, H / 128), FP8_ERR_INVALID_ARG);
        break;
      case FP8_GRAN_MX:
        FP8_CHECK(H % 128 == 0, FP8_ERR_UNSUPPORTED);
        FP8_CHECK(inv_scales->dtype == FP8_DT_E8M0 && shape_is(inv_scales, 1, mx_scale_bytes(T, H)),
                  FP8_ERR_INVALID_ARG);
        break;
      default:
        return FP8_ERR_UNSUPPORTED;
    }
  }
  Ctx c;
  FP8_TRY(make_ctx(&c, stream, nullptr));
  return launch_add_rmsnorm(x->ptr, residual ? residual->ptr : nullptr, weight->ptr, weight->dtype == FP8_DT_F32, eps,
                            T, H, granularity, q ? q->dtype : FP8_DT_E4M3, h ? h->ptr : nullptr, y ? y->ptr : nullptr,
                            q ? q->ptr : nullptr, q ? inv_scales->ptr : nullptr,
                            rstd ? static_cast<float*>(rstd->ptr) : nullptr, c);
}

extern "C" size_t fp8_rmsnorm_bwd_workspace_size(int64_t T, int64_t H) {
  // the widths that the call takes: the shape of its ring is defined for those only
  return T > 0 && T < kMaxDim && norm_width(H) ? (size_t)rmsnorm_bwd_ws_bytes(T, H) : 0;
}

extern "C" int fp8_add_rmsnorm_bwd(const fp8_tensor* dy, const fp8_tensor* h, const fp8_tensor* weight,
                                   const fp8_tensor* rstd, const fp8_tensor* dh, fp8_tensor* dx, fp8_tensor* dw,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  FP8_TRY(check_norm_input(dy, weight));
  const int64_t T = dy->shape[0], H = dy->shape[1];
  FP8_TRY(check_tensor(h, FP8_DT_BF16, 2, T, H));
  FP8_TRY(check_tensor(rstd, FP8_DT_F32, 1, T));
  if (dh) FP8_TRY(check_tensor(dh, FP8_DT_BF16, 2, T, H));
  if (dx) FP8_TRY(check_tensor(dx, FP8_DT_BF16, 2, T, H));
  FP8_CHECK(dx || dw, FP8_ERR_INVALID_ARG);
  if (dw) {
    FP8_CHECK(valid_desc(dw) && is_out(dw->dtype), FP8_ERR_INVALID_ARG);
    FP8_TRY(check_tensor(dw, dw->dtype, 1, H));
    FP8_TRY(check_workspace(workspace, workspace_bytes, rmsnorm_bwd_ws_bytes(T, H)));
  }
  Ctx c;
  FP8_TRY(make_ctx(&c, stream, nullptr));
  return launch_rmsnorm_bwd(dy->ptr, h->ptr, weight->ptr, weight->dtype == FP8_DT_F32,
                            static_cast<const float*>(rstd->ptr), dh ? dh->ptr : nullptr, T, H, dx ? dx->ptr : nullptr,
                            dw ? dw->ptr : nullptr, dw && dw->dtype == FP8_DT_BF16, static_cast<float*>(workspace), c);
}

// ------------------------------------------------------------------------------------------
// router

static int score_kind(int score) { return score & ~FP8_SCORE_BIASED; }

static int check_route(const fp8_tensor* logits, const fp8_tensor* ids, int score) {
  FP8_CHECK(valid_desc(logits) && is_out(logits->dtype) && logits->ndim == 2, FP8_ERR_INVALID_ARG);
  FP8_CHECK(valid_desc(ids) && ids->dtype == FP8_DT_I32 && ids->ndim == 2, FP8_ERR_INVALID_ARG);
  FP8_CHECK(score_kind(score) == FP8_SCORE_SOFTMAX || score_kind(score) == FP8_SCORE_SIGMOID, FP8_ERR_INVALID_ARG);
  const int64_t T = logits->shape[0], E = logits->shape[1], k = ids->shape[1];
  FP8_CHECK(ids->shape[0] == T && k >= 1 && k <= E, FP8_ERR_INVALID_ARG);
  FP8_CHECK(E <= 1024 && k <= 16 && T < kMaxDim && T * k < kMaxDim, FP8_ERR_UNSUPPORTED);
  FP8_CHECK(aligned16(logits->ptr) && aligned16(ids->ptr), FP8_ERR_ALIGNMENT);
  return FP8_OK;
}

extern "C" size_t fp8_moe_route_workspace_size(int64_t T, int64_t E) {
  return T > 0 && E > 0 && T < kMaxDim && E <= 1024 ? (size_t)route_ws_bytes(T, E) : 0;
}

extern "C" int fp8_moe_route(const fp8_tensor* logits, const fp8_tensor* bias, int score, int renormalize, float scale,
                             fp8_tensor* ids, fp8_tensor* weights, fp8_tensor* order, fp8_tensor* pos,
                             fp8_tensor* ends, void* workspace, size_t workspace_bytes, int32_t* d_status,
                             void* stream) {
  FP8_TRY(check_route(logits, ids, score));
  const int64_t T = logits->shape[0], E = logits->shape[1], k = ids->shape[1];
  FP8_TRY(check_tensor(weights, FP8_DT_F32, 2, T, k));
  if (bias) FP8_TRY(check_tensor(bias, FP8_DT_F32, 1, E));
  FP8_CHECK((order != nullptr) == (ends != nullptr) && (pos != nullptr) == (ends != nullptr), FP8_ERR_INVALID_ARG);
  if (ends) {
    FP8_TRY(check_tensor(order, FP8_DT_I32, 1, T * k));
    FP8_TRY(check_tensor(pos, FP8_DT_I32, 2, T, k));
    FP8_TRY(check_tensor(ends, FP8_DT_I32, 1, E));
    FP8_TRY(check_workspace(workspace, workspace_bytes, T > 0 ? route_ws_bytes(T, E) : 0));
  }
  Ctx c;
  FP8_TRY(make_ctx(&c, stream, d_status));
  return launch_route(logits->ptr, logits->dtype == FP8_DT_BF16, bias ? static_cast<const float*>(bias->ptr) : nullptr,
                      T, E, k, score_kind(score) == FP8_SCORE_SOFTMAX, (score & FP8_SCORE_BIASED) != 0, renormalize != 0,
                      scale, static_cast<int32_t*>(ids->ptr), static_cast<float*>(weights->ptr), ends ? static_cast<int32_t*>(order->ptr) : nullptr,
                      ends ? static_cast<int32_t*>(pos->ptr) : nullptr,
                      ends ? static_cast<int32_t*>(ends->ptr) : nullptr, workspace, c);
}

extern "C" int fp8_moe_route_bwd(const fp8_tensor* logits, const fp8_tensor* ids, const fp8_tensor* dweights,
                                 int score, int renormalize, float scale, fp8_tensor* dlogits, int32_t* d_status,
                                 void* stream) {
  FP8_TRY(check_route(logits, ids, score));
  const int64_t T = logits->shape[0], E = logits->shape[1], k = ids->shape[1];
  FP8_TRY(check_tensor(dweights, FP8_DT_F32, 2, T, k));
  FP8_TRY(check_tensor(dlogits, logits->dtype, 2, T, E));
  Ctx c;
  FP8_TRY(make_ctx(&c, stream, d_status));
  return launch_route_bwd(logits->ptr, logits->dtype == FP8_DT_BF16, static_cast<const int32_t*>(ids->ptr),
                          static_cast<const float*>(dweights->ptr), T, E, k, score_kind(score) == FP8_SCORE_SOFTMAX,
                          renormalize != 0, scale, dlogits->ptr, c);
}

// ------------------------------------------------------------------------------------------
// experts of a few tokens

extern "C" size_t fp8_moe_tokens_workspace_size(int64_t T, int64_t top_k, int64_t H, int64_t I) {
  if (T <= 0 || T > FP8_MOE_MAX_TOKENS || top_k <= 0 || top_k > 16 || H <= 0 || I <= 0 || H >= kMaxDim || I >= kMaxDim)
    return 0;
  return (size_t)moe_tokens_ws_bytes(T, top_k, H, I);
}

extern "C" int fp8_moe_tokens(const fp8_tensor* x, const fp8_tensor* ids, const fp8_tensor* weights,
                              const fp8_tensor* w13, const fp8_tensor* s13, const fp8_tensor* w2, const fp8_tensor* s2,
                              fp8_tensor* out, void* workspace, size_t workspace_bytes, int32_t* d_status,
                              void* stream) {
  FP8_CHECK(valid_desc(x) && x->dtype == FP8_DT_BF16 && x->ndim == 2, FP8_ERR_INVALID_ARG);
  FP8_CHECK(valid_desc(ids) && ids->dtype == FP8_DT_I32 && ids->ndim == 2, FP8_ERR_INVALID_ARG);
  FP8_CHECK(valid_desc(w13) && w13->dtype == FP8_DT_E4M3 && w13->ndim == 3, FP8_ERR_INVALID_ARG);
  const int64_t T = x->shape[0], H = x->shape[1], k = ids->shape[1], E = w13->shape[0], I = w13->shape[1] / 2;
  FP8_CHECK(w13->shape[1] % 2 == 0 && w13->shape[2] == H && ids->shape[0] == T && k >= 1 && E >= 1,
            FP8_ERR_INVALID_ARG);
  FP8_CHECK(T <= FP8_MOE_MAX_TOKENS && k <= 16 && E <= 1024 && H <= 65536 && I <= 65536, FP8_ERR_UNSUPPORTED);
  FP8_CHECK(H % 16 == 0 && I % 16 == 0, FP8_ERR_ALIGNMENT);
  FP8_CHECK(H > 0 && I > 0, FP8_ERR_UNSUPPORTED);
  FP8_CHECK(aligned16(x->ptr) && aligned16(ids->ptr) && aligned16(w13->ptr), FP8_ERR_ALIGNMENT);
  FP8_TRY(check_tensor(weights, FP8_DT_F32, 2, T, k));
  FP8_TRY(check_tensor(s13, FP8_DT_F32, 2, E, 2 * I));
  FP8_TRY(check_tensor(w2, FP8_DT_E4M3, 3, E, H, I));
  FP8_TRY(check_tensor(s2, FP8_DT_F32, 2, E, H));
  FP8_TRY(check_tensor(out, FP8_DT_BF16, 2, T, H));
  FP8_TRY(check_workspace(workspace, workspace_bytes, T > 0 ? moe_tokens_ws_bytes(T, k, H, I) : 0));
  Ctx c;
  FP8_TRY(make_ctx(&c, stream, d_status));
  return launch_moe_tokens(x->ptr, static_cast<const int32_t*>(ids->ptr), static_cast<const float*>(weights->ptr),
                           w13->ptr, static_cast<const float*>(s13->ptr), w2->ptr, static_cast<const float*>(s2->ptr),
                           T, k, E, H, I, out->ptr, workspace, c);
}

// ------------------------------------------------------------------------------------------
// gated feed-forward

// The operands of fp8_gated_mm (per = 2: B has the gate's rows and the up projection's) and of its backward pass (1).
static int check_gated(const fp8_tensor* A, const fp8_tensor* B, const fp8_tensor* offsets, const fp8_tensor* sA,
                       const fp8_tensor* sB, int act, int flags, int per, GatedArgs* g) {
  FP8_CHECK(valid_desc(A) && A->ndim == 2 && valid_desc(B), FP8_ERR_INVALID_ARG);
  FP8_CHECK(act == FP8_ACT_SILU || act == FP8_ACT_GELU, FP8_ERR_INVALID_ARG);
  FP8_CHECK(shape_max(A, kMaxDim - 1) && shape_max(B, kMaxDim - 1), FP8_ERR_UNSUPPORTED);
  const bool fp8 = is_fp8(A->dtype);
  FP8_CHECK(fp8 ? is_fp8(B->dtype) : A->dtype == FP8_DT_BF16 && B->dtype == FP8_DT_BF16, FP8_ERR_INVALID_ARG);
  FP8_CHECK(!(A->dtype == FP8_DT_E5M2 && B->dtype == FP8_DT_E5M2), FP8_ERR_UNSUPPORTED);
  const int known = FP8_MM_FAST_ACCUM | (fp8 ? FP8_MM_BLOCKWISE : per == 1 ? FP8_MM_B_MN_MAJOR : 0);
  FP8_CHECK((flags & ~known) == 0, FP8_ERR_UNSUPPORTED);
  int64_t E = 0;
  if (offsets) {
    FP8_CHECK(valid_desc(offsets) && offsets->dtype == FP8_DT_I32 && offsets->ndim == 1 && offsets->shape[0] >= 1,
              FP8_ERR_INVALID_ARG);
    E = offsets->shape[0];
    FP8_CHECK(fp8 && E <= kMaxGatedExperts, FP8_ERR_UNSUPPORTED);
    FP8_CHECK(B->ndim == 3 && B->shape[0] == E, FP8_ERR_INVALID_ARG);
    FP8_CHECK(word_aligned({offsets}), FP8_ERR_ALIGNMENT);
  } else {
    FP8_CHECK(B->ndim == 2, FP8_ERR_INVALID_ARG);
  }
  const int b_mn = (flags & FP8_MM_B_MN_MAJOR) ? 1 : 0;
  const int64_t M = A->shape[0], K = A->shape[1];
  const int64_t rows = B->shape[b_mn ? 1 : B->ndim - 2], kb = B->shape[b_mn ? 0 : B->ndim - 1], I = rows / per;
  FP8_CHECK(kb == K && rows % per == 0, FP8_ERR_INVALID_ARG);
  FP8_CHECK(K % (fp8 ? 16 : 8) == 0 && I % 8 == 0, FP8_ERR_ALIGNMENT);
  FP8_CHECK(K > 0, FP8_ERR_UNSUPPORTED);  // an empty contraction: not implemented here
  FP8_CHECK(aligned16(A->ptr) && aligned16(B->ptr), FP8_ERR_ALIGNMENT);
  const bool block = (flags & FP8_MM_BLOCKWISE) != 0;
  if (fp8) {
    FP8_CHECK(valid_desc(sA) && valid_desc(sB), FP8_ERR_INVALID_ARG);
    FP8_CHECK(sA->dtype != FP8_DT_E8M0 && sB->dtype != FP8_DT_E8M0, FP8_ERR_UNSUPPORTED);  // MX block scales
    FP8_CHECK(sA->dtype == FP8_DT_F32 && sB->dtype == FP8_DT_F32, FP8_ERR_INVALID_ARG);
    FP8_CHECK(shape_max(sA, kMaxDim - 1) && shape_max(sB, kMaxDim - 1), FP8_ERR_UNSUPPORTED);
    const int64_t la = numel(sA), lb = numel(sB), n = E ? E : 1;
    if (block) {
      FP8_CHECK(K % 128 == 0 && (per == 1 || I % 128 == 0), FP8_ERR_UNSUPPORTED);
      FP8_CHECK(la == M * (K / 128) && lb == n * ((rows + 127) / 128) * (K / 128), FP8_ERR_INVALID_ARG);
    } else {
      g->sa_scalar = !E && la == 1;
      g->sb_scalar = !E && lb == 1;
      FP8_CHECK((la == M || g->sa_scalar) && (lb == n * rows || g->sb_scalar), FP8_ERR_INVALID_ARG);
    }
    // read word by word: the scales of a transposed weight may follow those of the weight at any word
    FP8_CHECK(word_aligned({sA, sB}), FP8_ERR_ALIGNMENT);
    g->sA = static_cast<const float*>(sA->ptr);
    g->sB = static_cast<const float*>(sB->ptr);
  } else {
    FP8_CHECK(sA == nullptr && sB == nullptr, FP8_ERR_INVALID_ARG);
  }
  g->A = A->ptr;
  g->B = B->ptr;
  g->a_dtype = A->dtype;
  g->b_dtype = B->dtype;
  g->b_mn = b_mn;
  g->blockwise = block;
  g->M = M;
  g->I = I;
  g->K = K;
  g->ends = offsets ? static_cast<const int32_t*>(offsets->ptr) : nullptr;
  g->E = E;
  g->act = act;
  return FP8_OK;
}

extern "C" int fp8_gated_mm(const fp8_tensor* A, const fp8_tensor* B, const fp8_tensor* offsets, const fp8_tensor* sA,
                            const fp8_tensor* sB, int act, int flags, fp8_tensor* h, fp8_tensor* gu, fp8_tensor* q,
                            fp8_tensor* inv_scales, int32_t* d_status, void* stream) {
  GatedArgs g = {};
  FP8_TRY(check_gated(A, B, offsets, sA, sB, act, flags, 2, &g));
  FP8_CHECK((q != nullptr) == (inv_scales != nullptr), FP8_ERR_INVALID_ARG);
  FP8_CHECK(h || gu || q, FP8_ERR_INVALID_ARG);
  if (h) {
    FP8_TRY(check_tensor(h, FP8_DT_BF16, 2, g.M, g.I));
    g.h = h->ptr;
  }
  if (gu) {
    FP8_TRY(check_tensor(gu, FP8_DT_BF16, 2, g.M, 2 * g.I));
    g.gu = gu->ptr;
  }
  if (q) {
    FP8_CHECK(valid_desc(q) && is_fp8(q->dtype), FP8_ERR_INVALID_ARG);
    FP8_CHECK(g.I % 128 == 0, FP8_ERR_UNSUPPORTED);
    FP8_TRY(check_tensor(q, q->dtype, 2, g.M, g.I));
    FP8_TRY(check_tensor(inv_scales, FP8_DT_F32, 2, g.M, g.I / 128));
    g.q = q->ptr;
    g.inv = static_cast<float*>(inv_scales->ptr);
    g.q_fmt = q->dtype;
  }
  Ctx c;
  FP8_TRY(make_ctx(&c, stream, d_status));
  if (g.M == 0 || g.I == 0) return FP8_OK;
  return launch_gated(g, c);
}

extern "C" int fp8_gated_mm_bwd(const fp8_tensor* dy, const fp8_tensor* B, const fp8_tensor* offsets,
                                const fp8_tensor* sdy, const fp8_tensor* sB, int act, int flags, const fp8_tensor* gu,
                                fp8_tensor* dgu, fp8_tensor* h, int32_t* d_status, void* stream) {
  GatedArgs g = {};
  FP8_TRY(check_gated(dy, B, offsets, sdy, sB, act, flags, 1, &g));
  FP8_TRY(check_tensor(gu, FP8_DT_BF16, 2, g.M, 2 * g.I));
  FP8_TRY(check_tensor(dgu, FP8_DT_BF16, 2, g.M, 2 * g.I));
  if (h) {
    FP8_TRY(check_tensor(h, FP8_DT_BF16, 2, g.M, g.I));
    g.h = h->ptr;
  }
  g.backward = 1;
  g.gu_in = gu->ptr;
  g.gu = dgu->ptr;
  Ctx c;
  FP8_TRY(make_ctx(&c, stream, d_status));
  if (g.M == 0 || g.I == 0) return FP8_OK;
  return launch_gated(g, c);
}
