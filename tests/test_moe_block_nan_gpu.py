"""A token whose hidden state holds a NaN or an infinity has no experts (its logits are NaN); the serving block shows
that as NaN in the token's row, for few and for many tokens, and in no other row."""
import pytest
import torch

from tests.test_moe_block_gpu import _weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 5, 64, 65, 300])
@pytest.mark.parametrize("residual", [True, False])
def test_nan_reaches_the_output(T, residual):
    from moe_grouped_gemm_absmax_gb300.moe import Fp8MoEBlock
    E, H, I, k = 8, 512, 256, 2
    norm, router, w1, w3, w2, g = _weights(E, H, I, T)
    block = Fp8MoEBlock(norm, router, w1, w3, w2, k)
    x, r = (torch.randn(T, H, generator=g, device="cuda").bfloat16() for _ in range(2))
    bad = {0: float("nan")} if T == 1 else {0: float("nan"), 3: float("inf"), T - 1: float("-inf")}
    for t, v in bad.items():
        x[t, 17] = v
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, _ = block(x, r if residual else None, st)
    assert int(st) == 0
    assert out.isnan().all(1).tolist() == [t in bad for t in range(T)]
    assert torch.isfinite(out[[t for t in range(T) if t not in bad]].float()).all()


@pytest.mark.parametrize("T", [1, 6, 40])
def test_experts_of_a_nan_token(T):
    """fp8_moe_tokens itself: NaN in x reaches the token's row whether experts take it or not, and only that row."""
    import moe_grouped_gemm_absmax_gb300 as fp8
    from tests.test_moe_tokens_gpu import _layer, _tokens
    layer, g = _layer(4, 272, 144, T)
    x, ids, wt = _tokens(g, T, 272, 4, 2)
    x[T - 1, 271] = float("nan")
    x[T // 2, 3] = float("inf")
    bad = sorted({T - 1, T // 2})
    for unused in ([], [T - 1], list(range(T))):
        ids2 = ids.clone()
        ids2[unused] = -1
        out = fp8.moe_tokens_alloc(x, ids2, wt, *layer)
        assert out.isnan().all(1).tolist() == [t in bad for t in range(T)]
        good = [t for t in range(T) if t not in bad]
        assert torch.isfinite(out[good].float()).all()
        if len(unused) == T:
            assert not out[good].any()
