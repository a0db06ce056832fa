"""The training functions of the norm and the router where a gradient is absent, and where a second derivative is asked
for."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ag():
    import moe_grouped_gemm_absmax_gb300.autograd as m
    return m


def _inputs(T=37, H=520):
    g = torch.Generator(device="cuda").manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, res = (r(T, H).bfloat16().requires_grad_(True) for _ in range(2))
    return x, res, (1 + 0.1 * r(H)).requires_grad_(True), r(T, H), r


def test_a_stream_without_gradient_is_not_read(ag, monkeypatch):
    """Only y is used: the backward pass gets no dh, and the gradients are those of a dh of zeros."""
    seen = []
    real = ag.fp8_add_rmsnorm_bwd

    def spy(dy, h, w, rstd, dx=None, dw=None, dh=None, workspace=None, stream=None):
        seen.append(dh)
        return real(dy, h, w, rstd, dx, dw, dh, workspace, stream)

    monkeypatch.setattr(ag, "fp8_add_rmsnorm_bwd", spy)
    x, res, w, c, _ = _inputs()
    y, _ = ag.AddRmsNormFunction.apply(x, res, w)
    (y.float() * c).sum().backward()
    assert seen == [None]
    got = [t.grad.clone() for t in (x, res, w)]
    for t in (x, res, w):
        t.grad = None
    y, h = ag.AddRmsNormFunction.apply(x, res, w)
    ((y.float() * c).sum() + (h * 0).float().sum()).backward()
    assert seen[1] is not None
    assert all(torch.equal(a, t.grad) for a, t in zip(got, (x, res, w)))


@pytest.mark.parametrize("residual", [True, False])
def test_only_the_stream_has_a_gradient(ag, residual):
    """Only h is used: its gradient passes through unchanged, the weight's is zero."""
    x, res, w, c, _ = _inputs()
    _, h = ag.AddRmsNormFunction.apply(x, res if residual else None, w)
    (h.float() * c).sum().backward()
    assert torch.equal(x.grad, c.bfloat16())
    if residual:
        assert torch.equal(res.grad, c.bfloat16())
    assert w.grad is not None and not w.grad.any()


def test_a_second_derivative_is_refused(ag):
    """A gradient penalty would lose its terms through these functions without a word; it raises instead."""
    x, res, w, c, r = _inputs()
    y, _ = ag.AddRmsNormFunction.apply(x, res, w)
    gx, = torch.autograd.grad((y.float() * c).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        (gx.float().sum() + x.float().sum()).backward()
    logits = r(12, 16).requires_grad_(True)
    weights, _ = ag.MoERouteFunction.apply(logits, 3)
    gl, = torch.autograd.grad((weights * r(12, 3)).sum(), logits, create_graph=True)
    with pytest.raises(RuntimeError):
        (gl.sum() + logits.sum()).backward()
