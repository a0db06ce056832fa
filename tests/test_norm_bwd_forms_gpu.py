"""The norm's backward pass in the forms between which its kernels differ: fp32 weights at every width class with dx
written, with and without dh, and dx over each of the buffers that it may share. Bounds as in test_norm_gpu.py."""
import pytest
import torch

from tests.test_norm_gpu import EPS, U, _bwd_reference, _inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8():
    import moe_grouped_gemm_absmax_gb300 as m
    return m


@pytest.mark.parametrize("T,H", [(1, 8), (77, 520), (610, 2056), (500, 7168), (160, 8200), (157, 12288), (155, 12296),
                                 (310, 16384)])
@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("over", ["new", "dy", "h", "dh"])
def test_forms(fp8, T, H, f32, over):
    x, r, w = _inputs(T, H, 5 * T + H)
    if f32:
        w = w.float() * 1.000123  # values that bf16 does not hold
    h, _, _, _, rstd = fp8.add_rmsnorm_alloc(x, w, EPS, r, want_rstd=True)
    g = torch.Generator(device="cuda").manual_seed(T)
    dy, dh = (torch.randn(T, H, generator=g, device="cuda").bfloat16() for _ in range(2))
    for stream in ([dh] if over == "dh" else [dh, None]):
        rx, rw = _bwd_reference(dy, h, w, rstd, stream)
        xhat = h.double().abs() * rstd.double()[:, None]
        gabs = dy.double().abs() * w.double().abs()
        terms = rstd.double()[:, None] * (gabs + xhat * (gabs * xhat).mean(1, keepdim=True))
        a, b, c = dy.clone(), h.clone(), stream.clone() if stream is not None else None
        dx = {"new": torch.empty_like(h), "dy": a, "h": b, "dh": c}[over]
        dw = torch.empty(H, device="cuda")
        fp8.fp8_add_rmsnorm_bwd(a, b, w, rstd, dx, dw, dh=c, workspace=fp8.rmsnorm_bwd_workspace(T, H, "cuda"))
        assert ((dx.double() - rx).abs() <= 2.0 ** -8 * rx.abs() + 64 * U * terms + 1e-30).all()
        bound = (T / 152 + 60) * U * (dy.double().abs() * xhat).sum(0) + 1e-30
        assert ((dw.double() - rw).abs() <= bound).all()
