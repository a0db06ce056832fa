"""Codes and scales of the norm's 8-bit output where the largest |y| nears fp32's own: a scale is fp8_max over that
maximum whatever its size. Bounds as in test_norm_gpu.py."""
import pytest
import torch

from tests.test_norm_gpu import EPS, FMAX, U, _check_codes, _reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8():
    import moe_grouped_gemm_absmax_gb300 as m
    return m


@pytest.mark.parametrize("gran", ["row", "block"])
@pytest.mark.parametrize("dt", [3, 4])
@pytest.mark.parametrize("size", [1e-6, 1e30, 5e36, 2.5e37, 5e37])
@pytest.mark.parametrize("w_type", [torch.bfloat16, torch.float32])
def test_large_and_small_weights(fp8, gran, dt, size, w_type):
    """Weights of `size`: block maxima of about 2 to 4 times that, past 2^126 (8.5e37) for the largest."""
    T, H = 37, 2176
    g = torch.Generator(device="cuda").manual_seed(dt)
    x = torch.randn(T, H, generator=g, device="cuda").clamp_(-4, 4).bfloat16()
    w = (size * (0.5 + torch.rand(H, generator=g, device="cuda"))).to(w_type)
    gr = fp8.GRAN_ROW if gran == "row" else fp8.GRAN_BLOCK_1x128
    _, _, q, inv, _ = fp8.add_rmsnorm_alloc(x, w, EPS, None, gr, dt)
    yr = _reference(x, None, w)[2].view(T, -1, H if gran == "row" else 128)
    assert yr.abs().max() < 3.4e38
    want = yr.abs().amax(2).clamp_min(1e-12) / FMAX[dt]
    inv = inv.double().view_as(want)
    assert ((inv - want).abs() <= 80 * U * want).all()
    _check_codes(q.double().view_as(yr) * inv[..., None], yr, inv[..., None], dt)
