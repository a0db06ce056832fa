"""The gated feed-forward's backward pass where the up projection is as large as bf16 goes and the activation's derivative
is above 1: u act'(g) is past fp32's range there, dh u act'(g) is not."""
import pytest
import torch

from tests.gated_util import E5, HALF_BF16, act64, check, ends, gen, operand, product, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("kind,M,counts", [("bf16", 5, None), ("row", 70, None), ("block", 130, [100, 0, 30]), ("row", 2304, [2300, 4])])
def test_largest_up_projection(kind, M, counts, act):
    import moe_grouped_gemm_absmax_gb300 as f
    K, I = 128, 128
    g = gen(M)
    D, sD, d = operand(g, (M, K), kind, E5, size=1e-4)
    W, sW, w = operand(g, ((len(counts), I, K) if counts else (I, K)), kind, rows=128, size=0.25)
    gate = (2.4 if act == "silu" else 1.4) + 0.25 * randn(g, M, I)  # the derivative's maximum is near: 1.10, 1.13
    big = torch.finfo(torch.bfloat16).max
    u = torch.where(torch.rand(M, I, generator=g, device="cuda") < 0.5, -big, big)
    gu = torch.cat([gate, u], 1).to(torch.bfloat16)
    dgu, _ = f.gated_mm_bwd_alloc(D, W, sD, sW, gu, ends(counts) if counts else None, act=f.ACT_SILU if act == "silu" else f.ACT_GELU,
                                  flags=f.MM_BLOCKWISE if kind == "block" else 0)
    dh, err = product(d, w, counts)
    g64, u64 = gu.double().split(I, 1)
    _, d64, _, ed = act64(g64, act)
    assert (u64 * d64).abs().max() > torch.finfo(torch.float32).max
    dg = dh * u64 * d64
    assert dg.abs().max() < 0.5 * big
    bound = err * (u64 * d64).abs() + (dh.abs() + err) * u64.abs() * ed + 2.0 ** -22 * dg.abs()
    check(dgu[:, :I], dg, bound + HALF_BF16 * (dg.abs() + bound))
