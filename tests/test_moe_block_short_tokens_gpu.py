"""The serving block with tokens that have fewer selectable experts than top_k, on both sides of MOE_MAX_TOKENS: such a
token concerns itself only. A row of the grouped products depends on its own operands alone, so above
MOE_MAX_TOKENS the other tokens keep their bits; below, the experts' sums may be split over the SMs otherwise, and
the other tokens are held to the bounds of the block's own test (2^-7 and 2^-4 of the 2-norm)."""
import pytest
import torch

from tests.test_moe_block_gpu import _reference, _weights

pytestmark = pytest.mark.gpu
E, H, I, K = 8, 512, 256, 3
MASKED, PARTLY = 1, 4  # tokens; the last token is masked too


@pytest.fixture(scope="module")
def fp8():
    import moe_grouped_gemm_absmax_gb300 as m
    return m


def _block(fp8, T):
    """A block whose router masks by the hidden state: column 0 takes every expert from a token (logit -inf), column 1 all
    but expert 5; both columns are zero in the other tokens."""
    from moe_grouped_gemm_absmax_gb300.moe import Fp8MoEBlock
    norm, router, w1, w3, w2, g = _weights(E, H, I, 7 * T)
    router[:, 0] = -3e38
    router[:, 1] = -3e38
    router[5, 1] = 0
    block = Fp8MoEBlock(norm, router, w1, w3, w2, K)
    x, r = (torch.randn(T, H, generator=g, device="cuda").bfloat16() for _ in range(2))
    x[:, :2] = 0
    r[:, :2] = 0
    return block, x, r


def _logits_ids(fp8, block, x, r):
    _, y, _, _, _ = fp8.add_rmsnorm_alloc(x, block.norm_weight, block.eps, r, want_y=True)
    logits = torch.empty(x.shape[0], E, device="cuda")
    fp8.fp8_scaled_mm(y, block.router_weight, None, None, logits)
    return (logits, *fp8.moe_route_alloc(logits, K, table=False)[:2])


@pytest.mark.parametrize("T", [6, 64, 65, 300])
def test_masked_tokens(fp8, T):
    block, x, r = _block(fp8, T)
    clean, _ = block(x, r)
    for t, column in ((MASKED, 0), (PARTLY, 1), (T - 1, 0)):
        x[t, column] = 30.0
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, h = block(x, r, st)
    assert int(st) == 0 and torch.equal(h, (x.float() + r.float()).bfloat16())
    logits, ids, weights = _logits_ids(fp8, block, x, r)
    assert (logits[MASKED] == -torch.inf).all() and (ids[MASKED] == -1).all()
    assert ids[PARTLY].tolist() == [5, -1, -1] and float(weights[PARTLY, 0]) == 1.0
    assert not out[MASKED].any() and not out[T - 1].any()
    _, ref = _reference(block, x, r, ids, weights)
    bound = 2.0 ** -7 if T <= fp8.MOE_MAX_TOKENS else 2.0 ** -4
    assert float((out[PARTLY].double() - ref[PARTLY]).norm() / ref[PARTLY].norm()) <= bound
    others = torch.ones(T, dtype=torch.bool, device="cuda")
    others[[MASKED, PARTLY, T - 1]] = False
    assert float((out[others].double() - ref[others]).norm() / ref[others].norm()) <= bound
    if T > fp8.MOE_MAX_TOKENS:
        assert torch.equal(out[others], clean[others])


@pytest.mark.parametrize("T", [65, 300])
def test_every_token_masked(fp8, T):
    block, x, r = _block(fp8, T)
    x[:, 0] = 30.0
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, _ = block(x, r, st)
    assert int(st) == 0 and not out.any()


@pytest.mark.parametrize("T", [65, 300])
def test_a_nan_token_leaves_the_others(fp8, T):
    block, x, r = _block(fp8, T)
    clean, _ = block(x, r)
    for t, v in ((0, float("nan")), (MASKED, float("inf")), (T - 1, float("nan"))):
        x[t, 9] = v
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, h = block(x, r, st)
    assert int(st) == 0 and h[0].isnan().any()
    others = torch.ones(T, dtype=torch.bool, device="cuda")
    others[[0, MASKED, T - 1]] = False
    assert torch.equal(out[others], clean[others])
