"""The norm, the router and the experts together: the serving block on few and on many tokens, and the training
functions. The block's own roundings (the norm's output and the hidden layer in bf16, with many tokens both in e4m3
with a scale per row, 2^-4 relative a value) bound how far it may be from the same chain in 64 bits: they
are independent from value to value, so the result's relative error in the 2-norm stays below them."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8():
    import moe_grouped_gemm_absmax_gb300 as m
    return m


def _weights(E, H, I, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return (1 + 0.1 * r(H)).bfloat16(), (0.05 * r(E, H)).bfloat16(), (0.05 * r(E, I, H)).bfloat16(), \
        (0.05 * r(E, I, H)).bfloat16(), (0.05 * r(E, H, I)).bfloat16(), g


def _reference(block, x, residual, ids, weights):
    """The block in 64 bits, with its choice of experts and its quantized weights."""
    s = x.double() + residual.double()
    y = s / (s.square().mean(1, keepdim=True) + block.eps).sqrt() * block.norm_weight.double()
    out = torch.zeros_like(y)
    I = block.w2.shape[2]
    for e in range(block.w2.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        gu = y[t] @ (block.w13[e].double() * block.s13[e].double()[:, None]).T
        act = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
        out.index_add_(0, t, weights[t, j].double()[:, None] *
                       (act @ (block.w2[e].double() * block.s2[e].double()[:, None]).T))
    return y, out


@pytest.mark.parametrize("T,E,H,I,k", [(1, 8, 256, 128, 2), (7, 16, 1040, 528, 3), (64, 8, 512, 256, 2), (65, 8, 512, 256, 2),
                                       (300, 16, 1024, 512, 4)])
def test_serving_block(fp8, T, E, H, I, k):
    from moe_grouped_gemm_absmax_gb300.moe import Fp8MoEBlock
    norm, router, w1, w3, w2, g = _weights(E, H, I, T)
    block = Fp8MoEBlock(norm, router, w1, w3, w2, k, renormalize=True)
    x, r = (torch.randn(T, H, generator=g, device="cuda").bfloat16() for _ in range(2))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, h = block(x, r, st)
    assert int(st) == 0 and torch.equal(h, (x.float() + r.float()).bfloat16())
    # the block's own choice: the same calls on the same inputs
    _, y, _, _, _ = fp8.add_rmsnorm_alloc(x, norm, block.eps, r, want_y=True)
    logits = torch.empty(T, E, device="cuda")
    fp8.fp8_scaled_mm(y, router, None, None, logits)
    ids, weights, _, _, _ = fp8.moe_route_alloc(logits, k, table=False)
    y64, ref = _reference(block, x, r, ids, weights)
    l64 = y64 @ router.double().T
    assert ((logits.double() - l64).abs() <= 2.0 ** -7 * (y64.abs() @ router.double().abs().T)).all()
    rel = float((out.double() - ref).norm() / ref.norm())
    assert rel <= (2.0 ** -7 if T <= fp8.MOE_MAX_TOKENS else 2.0 ** -4), rel


def test_training_functions(fp8):
    """Gradients of a loss through the norm and the router against autograd in 64 bits on the same bf16 inputs."""
    from moe_grouped_gemm_absmax_gb300.autograd import AddRmsNormFunction, MoERouteFunction
    T, H, E, k = 37, 520, 24, 3
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, res = (r(T, H).bfloat16().requires_grad_(True) for _ in range(2))
    w = (1 + 0.1 * r(H)).requires_grad_(True)
    cy, ch, cw = r(T, H), r(T, H), r(T, k)
    y, h = AddRmsNormFunction.apply(x.view(1, T, H), res.view(1, T, H), w)
    assert y.shape == (1, T, H)
    ((y.float() * cy).sum() + (h.float() * ch).sum()).backward()
    a, b, c = (t.detach().double().requires_grad_(True) for t in (x, res, w))
    s = a + b
    ((s / (s.square().mean(1, keepdim=True) + 1e-6).sqrt() * c * cy.double()).sum() + (s * ch.double()).sum()).backward()
    # incoming gradients and h are rounded to bf16 on the way (2^-8 each), dx once more
    for got, want in ((x.grad, a.grad), (res.grad, b.grad), (w.grad, c.grad)):
        assert float((got.double() - want).norm() / want.norm()) <= 2.0 ** -7
    assert torch.equal(x.grad, res.grad)
    y0, h0 = AddRmsNormFunction.apply(x, None, w)
    assert torch.equal(h0, x)

    logits = r(T, E).requires_grad_(True)
    weights, ids = MoERouteFunction.apply(logits, k, None, fp8.SCORE_SIGMOID, True, 2.5)
    (weights * cw).sum().backward()
    l64 = logits.detach().double().requires_grad_(True)
    v = torch.sigmoid(l64).gather(1, ids.long())
    (2.5 * v / v.sum(1, keepdim=True) * cw.double()).sum().backward()
    assert float((logits.grad.double() - l64.grad).norm() / l64.grad.norm()) <= 2.0 ** -18
