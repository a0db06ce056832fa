"""The router with its bias on the score (SCORE_BIASED): auxiliary-loss-free load balancing chooses the top k of
score + bias and weighs with the score alone. The reference is that definition in 64 bits, from the logits.

Bounds: u = 2^-24. A sigmoid in fp32 takes an exponential (4 u), a sum (u) and a quotient (4 u): 12 u of its value; a
softmax 64 u (test_route_gpu.py); the sum with the bias u more. Values that move by at most d keep each order statistic
within d, so the j-th expert taken has a sum within 2 d of the j-th largest."""
import numpy as np
import pytest
import torch

from tests.test_route_gpu import _check_table, _weights

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def fp8():
    import moe_grouped_gemm_absmax_gb300 as m
    return m


def _score(logits, softmax):
    l64 = logits.double()
    return torch.softmax(l64, 1) if softmax else 1 / (1 + torch.exp(-l64))


def _run(fp8, logits, k, bias, softmax, renorm=True, scale=1.0):
    kind = (fp8.SCORE_SOFTMAX if softmax else fp8.SCORE_SIGMOID) | fp8.SCORE_BIASED
    ids, w, order, pos, ends = fp8.moe_route_alloc(logits, k, bias, kind, renorm, scale)
    _check_table(ids, order, pos, ends, logits.shape[1])
    return ids, w


def _check_choice(ids, logits, bias, softmax):
    v = _score(logits, softmax)
    sel = v + bias.double()
    d = (64 if softmax else 12) * U * v.amax(1, keepdim=True) + U * sel.abs().amax(1, keepdim=True)
    assert (ids >= 0).all()
    assert all(len(set(r)) == len(r) for r in ids.tolist())
    best = sel.sort(1, descending=True).values[:, :ids.shape[1]]
    got = sel.gather(1, ids.long())
    assert ((got - best).abs() <= 2 * d).all()


@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (5, 7, 7), (8, 256, 8), (33, 100, 6), (64, 64, 6), (129, 130, 16), (1000, 256, 8),
                                   (5003, 256, 8), (37, 1000, 10), (300, 500, 4), (20000, 17, 2)])
@pytest.mark.parametrize("softmax,renorm", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_choice_and_weights(fp8, T, E, k, softmax, renorm, dtype):
    g = torch.Generator(device="cuda").manual_seed(T + E)
    logits = (2 * torch.randn(T, E, generator=g, device="cuda")).to(dtype)
    bias = 0.1 * torch.randn(E, generator=g, device="cuda")
    ids, w = _run(fp8, logits, k, bias, softmax, renorm, 2.5)
    _check_choice(ids, logits, bias, softmax)
    ref = _weights(logits.double(), ids, softmax, renorm, 2.5)
    assert ((w.double() - ref).abs() <= 64 * U * ref).all()
    # without a bias the flag changes nothing
    plain = fp8.moe_route_alloc(logits, k, None, fp8.SCORE_SOFTMAX if softmax else fp8.SCORE_SIGMOID, renorm, 2.5)
    flag = _run(fp8, logits, k, None, softmax, renorm, 2.5)
    assert torch.equal(plain[0], flag[0]) and torch.equal(plain[1], flag[1])


def test_by_hand(fp8):
    """sigmoid(2, 1, 0, -1) = .881, .731, .5, .269; with the bias .881, .781, .9, .869: experts 2 and 0. (On the logits
    the same bias would choose 0 and 1.)"""
    logits = torch.tensor([[2.0, 1.0, 0.0, -1.0]], device="cuda")
    bias = torch.tensor([0.0, 0.05, 0.4, 0.6], device="cuda")
    ids, w = _run(fp8, logits, 2, bias, False)
    assert ids.tolist() == [[2, 0]]
    assert w.tolist()[0] == pytest.approx([0.5 / (0.5 + 0.880797), 0.880797 / (0.5 + 0.880797)], rel=1e-6)
    assert fp8.moe_route_alloc(logits, 2, bias, fp8.SCORE_SIGMOID)[0].tolist() == [[0, 1]]


def test_flat_part_of_the_sigmoid(fp8):
    """Logits of 18 to 40: every score is one to 2^-25, so the bias alone decides, whatever the logits. Logits of -40 to
    -18: every score is nought to 2^-25."""
    T, E, k = 500, 256, 8
    g = torch.Generator(device="cuda").manual_seed(5)
    bias = 1e-3 * torch.randperm(E, generator=g, device="cuda").float()
    want = bias.argsort(descending=True)[:k].tolist()
    logits = 18 + 22 * torch.rand(T, E, generator=g, device="cuda")
    for lg in (logits, -logits):
        ids, _ = _run(fp8, lg, k, bias, False)
        assert ids.tolist() == [want] * T
    # level sums: the lowest index
    ids, _ = _run(fp8, logits, k, torch.full((E,), 0.25, device="cuda"), False)
    assert ids.tolist() == [list(range(k))] * T
    ids, _ = _run(fp8, torch.full((9, 1000), -3.0, device="cuda"), 16, torch.zeros(1000, device="cuda"), True)
    assert ids.tolist() == [list(range(16))] * 9


@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("E", [40, 256, 1000])
def test_masks(fp8, softmax, E):
    """A logit of -inf or NaN is not taken however large its bias; a bias of -inf or NaN takes an expert out."""
    T, k = 41, 4
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.randn(T, E, generator=g, device="cuda")
    bias = 0.1 * torch.randn(E, generator=g, device="cuda")
    bias[0] = 100.0
    bias[10:20] = -torch.inf
    bias[20] = float("nan")
    logits[1] = -torch.inf
    logits[2, 3:] = -torch.inf
    logits[3, 0] = -torch.inf
    logits[4, 0] = float("nan")
    logits[5] = float("nan")
    ids, w = _run(fp8, logits, k, bias, softmax)
    got = ids.cpu()
    assert not torch.isin(got, torch.arange(10, 21)).any()
    assert (got[1] == -1).all() and (got[5] == -1).all() and not w[1].any() and not w[5].any()
    assert sorted(got[2].tolist()) == [-1, 0, 1, 2]
    assert not (got[3] == 0).any() and not (got[4] == 0).any() and (got[4] >= 0).all()
    assert torch.isfinite(w).all()
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[1:6] = False
    assert (got[rest.cpu()][:, 0] == 0).all()
    allowed = torch.where(bias.isnan(), -torch.inf, bias)
    keep = allowed > -torch.inf
    index = torch.arange(E, device="cuda")[keep]
    back = torch.full((E,), -1, dtype=torch.int32, device="cuda")
    back[index] = torch.arange(len(index), dtype=torch.int32, device="cuda")
    if not softmax:  # the experts that are left, renumbered
        _check_choice(back[ids[rest].long()], logits[rest][:, keep], bias[keep], False)


def test_training_function_and_block(fp8):
    """MoERouteFunction and Fp8MoEBlock take the balancing bias as published."""
    from moe_grouped_gemm_absmax_gb300.autograd import MoERouteFunction
    from moe_grouped_gemm_absmax_gb300.moe import Fp8MoEBlock
    from tests.test_moe_block_gpu import _reference, _weights as block_weights
    T, E, H, I, k = 50, 32, 256, 128, 4
    g = torch.Generator(device="cuda").manual_seed(8)
    logits = (1.5 * torch.randn(T, E, generator=g, device="cuda")).requires_grad_(True)
    bias = 0.3 * torch.randn(E, generator=g, device="cuda")
    for softmax in (False, True):
        kind = fp8.SCORE_SOFTMAX if softmax else fp8.SCORE_SIGMOID
        w, ids = MoERouteFunction.apply(logits, k, bias, kind, True, 2.5)
        _check_choice(ids, logits.detach(), bias, softmax)
        c = torch.randn(T, k, generator=g, device="cuda")
        grad, = torch.autograd.grad((w * c).sum(), logits)
        l64 = logits.detach().double().requires_grad_(True)
        want, = torch.autograd.grad((_weights(l64, ids, softmax, True, 2.5) * c.double()).sum(), l64)
        assert float((grad.double() - want).norm() / want.norm()) <= 2.0 ** -18
    norm, router, w1, w3, w2, _ = block_weights(E, H, I, 3)
    for tokens in (6, 200):
        block = Fp8MoEBlock(norm, router, w1, w3, w2, k, bias=bias, score=fp8.SCORE_SIGMOID, scale=2.5)
        x, r = (torch.randn(tokens, H, generator=g, device="cuda").bfloat16() for _ in range(2))
        out, _ = block(x, r)
        _, y, _, _, _ = fp8.add_rmsnorm_alloc(x, norm, block.eps, r, want_y=True)
        lg = torch.empty(tokens, E, device="cuda")
        fp8.fp8_scaled_mm(y, router, None, None, lg)
        ids = (_score(lg, False) + bias.double()).sort(dim=1, descending=True, stable=True).indices[:, :k]
        weights = _weights(lg.double(), ids, False, True, 2.5)
        ref = _reference(block, x, r, ids, weights)[1]
        # a token whose k-th and next sums are level to fp32 may take either: none here
        top = (_score(lg, False) + bias.double()).sort(1, descending=True).values
        assert (top[:, k - 1] - top[:, k] > 32 * U).all()
        rel = float((out.double() - ref).norm() / ref.norm())
        assert rel <= (2.0 ** -7 if tokens <= fp8.MOE_MAX_TOKENS else 2.0 ** -4), rel
