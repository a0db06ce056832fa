"""The mixture-of-experts block of a transformer on FP8 weights, for serving: the norm with the residual, the
router and the experts, through the library's entry points.

Up to MOE_MAX_TOKENS tokens (decode) take fp8_moe_tokens, which reads the named experts' weights once (for each 40
slots of an expert) and holds the activations to bf16's precision; more take the grouped GEMM on rows sorted by
expert, with the norm's 8-bit output as its operand and the hidden layer in 8 bits too (a scale per row): the results
of the two differ by the rounding to e4m3.

With block scales (GRAN_BLOCK_1x128) any number of tokens takes one path: fp8_gated_mm on the sorted rows of the norm's
codes, whose hidden layer leaves as codes with 1 x 128 scales, and the block-scaled grouped GEMM."""
import torch

from . import (DT_E4M3, GRAN_BLOCK_1x128, GRAN_ROW, GROUPED_JAGGED_M, MM_BLOCKWISE, MOE_MAX_TOKENS, SCORE_BIASED,
               SCORE_SOFTMAX, add_rmsnorm_alloc, blk_quantize_alloc, fp8_grouped_mm, fp8_scaled_mm, gated_mm_alloc,
               moe_route_alloc, moe_tokens_alloc, quantize_alloc)


class Fp8MoEBlock:
    """norm_weight [H]; router_weight bf16 [E, H]; w1 (gate), w3 (up) bf16 [E, I, H]; w2 bf16 [E, H, I]; bias fp32
    [E] or None, the balancing bias: added to the router's scores for the choice. The experts' weights are quantized
    once, e4m3 with a scale per row, or with granularity GRAN_BLOCK_1x128 per 128 x 128 block (H and I multiples of 128;
    the activations per 1 x 128)."""

    def __init__(self, norm_weight, router_weight, w1, w3, w2, top_k, eps=1e-6, bias=None, score=SCORE_SOFTMAX,
                 renormalize=True, scale=1.0, granularity=GRAN_ROW):
        E, I, H = w1.shape
        if granularity not in (GRAN_ROW, GRAN_BLOCK_1x128):
            raise ValueError("Fp8MoEBlock takes GRAN_ROW or GRAN_BLOCK_1x128")
        self.block = granularity == GRAN_BLOCK_1x128
        if self.block and (H % 128 or I % 128):
            raise ValueError("block scales need H and I divisible by 128")
        self.norm_weight, self.router_weight, self.bias = norm_weight.contiguous(), router_weight.contiguous(), bias
        self.top_k, self.eps, self.score, self.renormalize, self.scale = top_k, eps, score | SCORE_BIASED, renormalize, scale

        def rows(w):
            n = w.shape[1]
            if self.block:
                q, _, inv, _ = blk_quantize_alloc(w.reshape(E * n, -1).contiguous(), DT_E4M3, tile128=True)
                return q.view(w.shape), inv.view(E, n // 128, -1)
            q, _, inv = quantize_alloc(w.reshape(E * n, -1).contiguous(), GRAN_ROW, DT_E4M3)
            return q.view(w.shape), inv.view(E, n)

        self.w13, self.s13 = rows(torch.cat([w1, w3], 1))
        self.w2, self.s2 = rows(w2)

    def __call__(self, x, residual=None, status=None):
        """x (and residual) bf16 [T, H] -> (the experts' weighted sum bf16 [T, H], the new residual stream bf16 [T, H]).
        A token with fewer than top_k experts that can be chosen (see fp8_moe_route) gets the sum over those there are,
        one with none zeros. A NaN or an infinity in a token gives NaN in its row of both."""
        T, H = x.shape
        few = T <= MOE_MAX_TOKENS and not self.block
        h, y, q, inv, _ = add_rmsnorm_alloc(x, self.norm_weight, self.eps, residual,
                                            None if few else GRAN_BLOCK_1x128 if self.block else GRAN_ROW, want_y=True)
        logits = torch.empty((T, self.router_weight.shape[0]), dtype=torch.float32, device=x.device)
        if T:
            fp8_scaled_mm(y, self.router_weight, None, None, logits, status=status)
        ids, weights, order, pos, ends = moe_route_alloc(logits, self.top_k, self.bias, self.score, self.renormalize,
                                                         self.scale, table=not few, status=status)
        if few:
            return moe_tokens_alloc(y, ids, weights, self.w13, self.s13, self.w2, self.s2, status=status), h
        # rows by expert: codes and scales of the slots' tokens. Unused slots leave rows at the end; they go to the last
        # expert with any token's codes (the offsets cover all rows, without a look at the device's counts), and
        # `pos` -1 takes the last row, of zeros, behind the product's.
        ends[-1:].fill_(T * self.top_k)
        token = order.div(self.top_k, rounding_mode="floor").clamp_(min=0).long()
        a = q.view(torch.uint8)[token].view(q.dtype)
        if self.block:
            _, _, aq, ainv = gated_mm_alloc(a, self.w13, inv[token], self.s13, ends, flags=MM_BLOCKWISE, want_h=False,
                                            q_dtype=DT_E4M3, status=status)
            inv = inv.sum(1)
        else:
            gate_up = self._grouped(a, inv[token], self.w13, self.s13, ends, status).float()
            gate, up = gate_up.chunk(2, 1)
            act = (torch.nn.functional.silu(gate) * up).to(torch.bfloat16)
            aq, _, ainv = quantize_alloc(act, GRAN_ROW, DT_E4M3)
        out = self._grouped(aq, ainv, self.w2, self.s2, ends, status, spare=1)
        out[-1:].zero_()
        out = out[pos.view(-1).long()].float()
        # A NaN or an infinity makes all logits of its token NaN: no expert takes it, and none would show it. The row's
        # scale is NaN too.
        weights = weights + inv[:, None] * 0
        return (out.view(T, self.top_k, H) * weights[..., None]).sum(1).to(torch.bfloat16), h

    def _grouped(self, a, inv, w, s, ends, status, spare=0):
        """The product's rows, and `spare` more that it does not write."""
        out = torch.empty((a.shape[0] + spare, w.shape[1]), dtype=torch.bfloat16, device=a.device)
        fp8_grouped_mm(a, w, ends, inv, s, out[:a.shape[0]], GROUPED_JAGGED_M, MM_BLOCKWISE if self.block else 0, status)
        return out
