"""A thin training-code wrapper over the C ABI: a torch.autograd.Function for the FP8 Linear and a
module swap in the style of the pages' Float8Linear ("FP8 Training: Quantization, Autograd,
Torchao", sections 5-6: the Linear keeps a bf16 weight, quantizes x and W in the forward pass,
dY in the backward pass, and returns bf16).

Every step runs in the library's kernels through fp8_linear_fwd / fp8_linear_bwd; this module only
allocates the caller-owned buffers (FP8 copies, inverse scales, workspaces) with PyTorch and wires
them into autograd. No bias: the pages' hot path is the bias-free matmul, and a bias would add a
non-FP8 step."""
import torch

from . import (ACT_SILU, DT_E4M3, DT_E5M2, GRAN_BLOCK_1x128, GRAN_COL, GRAN_MX, GRAN_ROW, GRAN_TENSOR, LAYOUT_COL_MAJOR,
               MM_A_MN_MAJOR, MM_B_MN_MAJOR, MM_BLOCKWISE, MM_FAST_ACCUM, OP_LINEAR_BWD, OP_LINEAR_FWD, SCORE_BIASED,
               SCORE_SOFTMAX, WGRAD_BF16, WGRAD_FP8, add_rmsnorm_alloc, blk_quantize_alloc, fp8_add_rmsnorm_bwd,
               fp8_linear_bwd, fp8_linear_fwd, fp8_moe_route_bwd, fp8_scaled_mm, fp8_workspace_size, gated_mm_alloc,
               gated_mm_bwd_alloc, linear_saved_alloc, make_saved, moe_route_alloc, quantize_alloc, rmsnorm_bwd_workspace)


def _workspace(nbytes, device):
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


class Fp8LinearFunction(torch.autograd.Function):
    """y = x W^T in FP8 (forward with fast accumulation, as the pages' recipe does), dX and dW in
    the backward pass; x [..., K] bf16, W [N, K] bf16 -> y [..., N] bf16."""

    @staticmethod
    def forward(ctx, x, weight, granularity=GRAN_ROW, wgrad_mode=WGRAD_BF16):
        if x.dtype != torch.bfloat16 or weight.dtype != torch.bfloat16:
            raise TypeError("Fp8LinearFunction takes bf16 x and weight")
        K = x.shape[-1]
        N = weight.shape[0]
        x2 = x.reshape(-1, K).contiguous()
        w = weight.contiguous()
        M = x2.shape[0]
        dev = x.device
        saved, bufs = linear_saved_alloc(M, K, N, granularity, keep_xt=wgrad_mode == WGRAD_FP8, device=dev)
        y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        fp8_linear_fwd(x2, w, granularity, MM_FAST_ACCUM, y, saved,
                       _workspace(fp8_workspace_size(OP_LINEAR_FWD, M, K, N, granularity), dev))
        # the FP8 copies and scales for the backward pass (absent ones as empty placeholders)
        ctx.save_for_backward(x2, w, *(b if b is not None else x2.new_empty(0) for b in bufs))
        ctx.present = tuple(b is not None for b in bufs)
        ctx.granularity, ctx.wgrad_mode, ctx.x_shape = granularity, wgrad_mode, x.shape
        return y.reshape(*x.shape[:-1], N)

    @staticmethod
    def backward(ctx, dy):
        x2, w, *bufs = ctx.saved_tensors
        bufs = [b if keep else None for b, keep in zip(bufs, ctx.present)]
        saved = make_saved(*bufs)
        M, K = x2.shape
        N = w.shape[0]
        dy2 = dy.reshape(-1, N).to(torch.bfloat16).contiguous()
        dx = torch.empty((M, K), dtype=torch.bfloat16, device=dy.device) if ctx.needs_input_grad[0] else None
        dw = torch.empty((N, K), dtype=torch.bfloat16, device=dy.device) if ctx.needs_input_grad[1] else None
        ws = _workspace(fp8_workspace_size(OP_LINEAR_BWD, M, K, N, ctx.granularity, ctx.wgrad_mode), dy.device)
        fp8_linear_bwd(dy2, saved, x2, w, ctx.granularity, ctx.wgrad_mode, dx, dw, ws)
        return (dx.reshape(ctx.x_shape) if dx is not None else None), dw, None, None


class Fp8Linear(torch.nn.Module):
    """Drop-in for a bias-free torch.nn.Linear: the weight stays bf16; the matmuls run in FP8
    (granularity GRAN_TENSOR, GRAN_ROW, GRAN_MX or GRAN_BLOCK_1x128; MX and blockwise need
    dimensions that are multiples of 128, blockwise a bf16 weight gradient)."""

    def __init__(self, in_features, out_features, granularity=GRAN_ROW, wgrad_mode=WGRAD_BF16, weight=None,
                 device=None):
        super().__init__()
        if in_features % 16 or out_features % 16:
            raise ValueError("FP8 GEMM operands need in_features and out_features divisible by 16")
        self.in_features, self.out_features = in_features, out_features
        self.granularity, self.wgrad_mode = granularity, wgrad_mode
        if weight is None:
            weight = torch.nn.Parameter(torch.empty((out_features, in_features), dtype=torch.bfloat16, device=device))
            torch.nn.init.kaiming_uniform_(weight, a=5 ** 0.5)
        self.weight = weight

    def forward(self, x):
        return Fp8LinearFunction.apply(x.to(torch.bfloat16), self.weight, self.granularity, self.wgrad_mode)

    def extra_repr(self):
        g = {GRAN_ROW: "row", GRAN_TENSOR: "tensor", GRAN_MX: "mx", GRAN_BLOCK_1x128: "blockwise"}[self.granularity]
        w = {WGRAD_BF16: "bf16", WGRAD_FP8: "fp8"}[self.wgrad_mode]
        return f"in_features={self.in_features}, out_features={self.out_features}, scaling={g}, wgrad={w}"


def swap_linears(module, granularity=GRAN_ROW, wgrad_mode=WGRAD_BF16, module_filter=None):
    """Replace, in place, every bias-free bf16 torch.nn.Linear child (recursively) whose shape the
    FP8 GEMMs accept and that `module_filter(fqn, linear)` admits, by an Fp8Linear that shares
    its weight Parameter. Returns the names of the swapped modules."""
    swapped = []

    def visit(mod, prefix):
        for name, child in list(mod.named_children()):
            fqn = f"{prefix}.{name}" if prefix else name
            ok = (isinstance(child, torch.nn.Linear) and child.bias is None and child.weight.dtype == torch.bfloat16
                  and child.in_features % 16 == 0 and child.out_features % 16 == 0
                  and (module_filter is None or module_filter(fqn, child)))
            if ok:
                setattr(mod, name, Fp8Linear(child.in_features, child.out_features, granularity, wgrad_mode,
                                             weight=child.weight))
                swapped.append(fqn)
            else:
                visit(child, fqn)

    visit(module, "")
    return swapped


class _OnceFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, grad):
        return grad.view_as(grad)

    @staticmethod
    def backward(ctx, _):
        raise RuntimeError("the gradients of the fp8lin functions are not differentiable")


def _once(*grads):
    """Gradients whose own derivative is refused, not taken for zero. (once_differentiable refuses it only where the
    incoming gradient requires one; these depend on the saved inputs too.)"""
    if not torch.is_grad_enabled():
        return grads
    return tuple(g if g is None else _OnceFunction.apply(g.detach().requires_grad_(True)) for g in grads)


class AddRmsNormFunction(torch.autograd.Function):
    """(y, h) = norm(x + residual) * weight and the new residual stream; x, residual [..., H] bf16, weight [H] bf16 or
    fp32. Without a residual (None), h is x. Gradients of x, residual and weight."""

    @staticmethod
    def forward(ctx, x, residual, weight, eps=1e-6):
        if x.dtype != torch.bfloat16:
            raise TypeError("AddRmsNormFunction takes bf16 x")
        H = x.shape[-1]
        x2 = x.reshape(-1, H).contiguous()
        r2 = residual.reshape(-1, H).contiguous() if residual is not None else None
        w = weight.contiguous()
        h, y, _, _, rstd = add_rmsnorm_alloc(x2, w, eps, r2, want_rstd=True)
        ctx.save_for_backward(h, w, rstd)
        ctx.shape, ctx.has_residual = x.shape, residual is not None
        ctx.set_materialize_grads(False)  # an output that nothing uses costs no gradient of zeros
        return y.reshape(x.shape), (h.reshape(x.shape) if residual is not None else x.view_as(x))

    @staticmethod
    def backward(ctx, dy, dh):
        h, w, rstd = ctx.saved_tensors
        T, H = h.shape
        dh2 = dh.reshape(T, H).to(torch.bfloat16).contiguous() if dh is not None else None
        need_x = ctx.needs_input_grad[0] or ctx.needs_input_grad[1]
        dw = (torch.zeros_like if dy is None else torch.empty_like)(w) if ctx.needs_input_grad[2] else None
        dx = dh2  # where only h is used, its gradient passes through
        if dy is not None and (need_x or dw is not None):
            dx = torch.empty_like(h) if need_x else None
            fp8_add_rmsnorm_bwd(dy.reshape(T, H).to(torch.bfloat16).contiguous(), h, w, rstd, dx, dw, dh2,
                                rmsnorm_bwd_workspace(T, H, h.device) if dw is not None else None)
        g = dx.reshape(ctx.shape) if dx is not None else None
        return _once(g if ctx.needs_input_grad[0] else None,
                     g if ctx.has_residual and ctx.needs_input_grad[1] else None, dw, None)


class MoERouteFunction(torch.autograd.Function):
    """(weights fp32 [T, k], ids int32 [T, k]) of fp8_moe_route, with bias the balancing bias, added to the scores for the
    choice; the gradient of the weights reaches the logits, the choice and its bias get none."""

    @staticmethod
    def forward(ctx, logits, top_k, bias=None, score=SCORE_SOFTMAX, renormalize=True, scale=1.0):
        logits = logits.contiguous()
        ids, weights, _, _, _ = moe_route_alloc(logits, top_k, bias, score | SCORE_BIASED, renormalize, scale, table=False)
        ctx.save_for_backward(logits, ids)
        ctx.args = (score, renormalize, scale)
        ctx.mark_non_differentiable(ids)
        return weights, ids

    @staticmethod
    def backward(ctx, dweights, _):
        logits, ids = ctx.saved_tensors
        dlogits = torch.empty_like(logits)
        fp8_moe_route_bwd(logits, ids, dweights.float().contiguous(), dlogits, *ctx.args)
        return _once(dlogits, None, None, None, None, None)


def _mm(a, b, sa=None, sb=None, flags=0):
    """a b^T in bf16; with flags' MN-major layouts a [K, M], b [K, N]."""
    M = a.shape[1] if flags & MM_A_MN_MAJOR else a.shape[0]
    N = b.shape[1] if flags & MM_B_MN_MAJOR else b.shape[0]
    out = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    fp8_scaled_mm(a, b, sa, sb, out, flags)
    return out


class GatedMLPFunction(torch.autograd.Function):
    """y = W2 (act(W1 x) * (W3 x)) in FP8: x [..., H] bf16, w13 bf16 [2 I, H] (W1 above W3), w2 bf16 [H, I] -> y [..., H]
    bf16. Scales per row, or with GRAN_BLOCK_1x128 per 1 x 128 of the activations and 128 x 128 of the weights (H and I
    multiples of 128). The forward keeps x and both projections in bf16; the backward makes the hidden layer again, takes
    dY and the projections' gradients in e5m2, and the weight gradients in bf16. (A backward pass is captured into a CUDA
    graph only while no eager graph of the same weights lives: torch's own rule.)"""

    @staticmethod
    def forward(ctx, x, w13, w2, granularity=GRAN_ROW, act=ACT_SILU):
        if any(t.dtype != torch.bfloat16 for t in (x, w13, w2)):
            raise TypeError("GatedMLPFunction takes bf16 x, w13 and w2")
        if granularity not in (GRAN_ROW, GRAN_BLOCK_1x128):
            raise ValueError("GatedMLPFunction takes GRAN_ROW or GRAN_BLOCK_1x128")
        x2, w13, w2 = x.reshape(-1, x.shape[-1]).contiguous(), w13.contiguous(), w2.contiguous()
        ctx.granularity, ctx.act, ctx.x_shape = granularity, act, x.shape
        if x2.shape[0] == 0:  # nothing to quantize
            ctx.save_for_backward(x2, w13, w2, x2)
            return torch.empty_like(x)
        if granularity == GRAN_ROW:
            xq, _, xi = quantize_alloc(x2, GRAN_ROW, DT_E4M3)
            wq, _, wi = quantize_alloc(w13, GRAN_ROW, DT_E4M3)
            h, gu, _, _ = gated_mm_alloc(xq, wq, xi, wi, act=act, want_gu=True)
            hq, _, hi = quantize_alloc(h, GRAN_ROW, DT_E4M3)
            wq, _, wi = quantize_alloc(w2, GRAN_ROW, DT_E4M3)
            y = _mm(hq, wq, hi, wi)
        else:
            xq, _, xi, _ = blk_quantize_alloc(x2, DT_E4M3)
            wq, _, wi, _ = blk_quantize_alloc(w13, DT_E4M3, tile128=True)
            _, gu, hq, hi = gated_mm_alloc(xq, wq, xi, wi, act=act, flags=MM_BLOCKWISE, want_h=False, want_gu=True,
                                           q_dtype=DT_E4M3)
            wq, _, wi, _ = blk_quantize_alloc(w2, DT_E4M3, tile128=True)
            y = _mm(hq, wq, hi, wi, MM_BLOCKWISE)
        ctx.save_for_backward(x2, w13, w2, gu)
        return y.reshape(x.shape)

    @staticmethod
    def backward(ctx, dy):
        x2, w13, w2, gu = ctx.saved_tensors
        need_x, need_13, need_2 = ctx.needs_input_grad[:3]
        if x2.shape[0] == 0:
            return _once(torch.empty_like(dy) if need_x else None, torch.zeros_like(w13) if need_13 else None,
                         torch.zeros_like(w2) if need_2 else None, None, None)
        dy2 = dy.reshape(x2.shape).to(torch.bfloat16).contiguous()
        row = ctx.granularity == GRAN_ROW

        def left(t):  # gradients, the GEMM's left operand
            if row:
                q, _, inv = quantize_alloc(t, GRAN_ROW, DT_E5M2)
                return q, inv
            q, _, inv, _ = blk_quantize_alloc(t, DT_E5M2)
            return q, inv

        def transposed(w):  # a weight, its transpose the right operand
            if row:
                _, q, inv = quantize_alloc(w, GRAN_COL, DT_E4M3)
                return q, inv
            _, q, _, inv = blk_quantize_alloc(w, DT_E4M3, tile128=True, layout=LAYOUT_COL_MAJOR)
            return q, inv

        flags = 0 if row else MM_BLOCKWISE
        dx = dw13 = None
        outer = MM_A_MN_MAJOR | MM_B_MN_MAJOR  # sums over the rows
        dyq, sdy = left(dy2)
        wq, wi = transposed(w2)
        dgu, h = gated_mm_bwd_alloc(dyq, wq, sdy, wi, gu, act=ctx.act, flags=flags, want_h=need_2)
        dw2 = _mm(dy2, h, flags=outer) if need_2 else None
        if need_13:
            dw13 = _mm(dgu, x2, flags=outer)
        if need_x:
            dq, sd = left(dgu)
            wq, wi = transposed(w13)
            dx = _mm(dq, wq, sd, wi, flags).reshape(ctx.x_shape)
        return _once(dx, dw13, dw2, None, None)


class Fp8GatedMLP(torch.nn.Module):
    """The gated feed-forward of a transformer layer, y = W2 (act(W1 x) * (W3 x)), with bf16 weights w13 [2 I, H] and w2
    [H, I] and its products in FP8 (GatedMLPFunction)."""

    def __init__(self, hidden, inner, granularity=GRAN_ROW, act=ACT_SILU, device=None):
        super().__init__()
        if hidden % 16 or inner % 16:
            raise ValueError("FP8 GEMM operands need hidden and inner divisible by 16")
        if granularity == GRAN_BLOCK_1x128 and (hidden % 128 or inner % 128):
            raise ValueError("block scales need hidden and inner divisible by 128")
        self.granularity, self.act = granularity, act
        self.w13 = torch.nn.Parameter(torch.empty((2 * inner, hidden), dtype=torch.bfloat16, device=device))
        self.w2 = torch.nn.Parameter(torch.empty((hidden, inner), dtype=torch.bfloat16, device=device))
        for w in (self.w13, self.w2):
            torch.nn.init.kaiming_uniform_(w, a=5 ** 0.5)

    def forward(self, x):
        return GatedMLPFunction.apply(x.to(torch.bfloat16), self.w13, self.w2, self.granularity, self.act)

    def extra_repr(self):
        g = {GRAN_ROW: "row", GRAN_BLOCK_1x128: "blockwise"}[self.granularity]
        return f"hidden={self.w13.shape[1]}, inner={self.w2.shape[1]}, scaling={g}, act={'silu' if self.act == ACT_SILU else 'gelu'}"
