"""The norm's backward pass when a wait for its rows runs out: each CTA's first rows are never loaded (the test hook), the
wait ends after 2 ms, the copies behind it are drained, and everything that the call gives is NaN: all rows, since
every CTA lost one of its own, and all of dw. The next call on the same buffers is right, bit for bit."""
import pytest
import torch

from tests.test_norm_gpu import EPS, _inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8():
    import moe_grouped_gemm_absmax_gb300 as m
    return m


# one row; several rows a CTA (one, two or four vectors a thread), the last group short; several groups a CTA
@pytest.mark.parametrize("T,H", [(1, 264), (13, 520), (2003, 1024), (700, 7168), (400, 12288), (310, 16384)])
@pytest.mark.parametrize("stream_grad", [True, False])
def test_wait_limit_expiry_gives_nan_and_context_survives(fp8, T, H, stream_grad):
    x, r, w = _inputs(T, H, T + H)
    h, _, _, _, rstd = fp8.add_rmsnorm_alloc(x, w, EPS, r, want_rstd=True)
    g = torch.Generator(device="cuda").manual_seed(T)
    dy = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    dh = torch.randn(T, H, generator=g, device="cuda").bfloat16() if stream_grad else None
    ws = fp8.rmsnorm_bwd_workspace(T, H, "cuda")

    def run():
        dx, dw = torch.zeros_like(h), torch.zeros(H, device="cuda")
        fp8.fp8_add_rmsnorm_bwd(dy, h, w, rstd, dx, dw, dh=dh, workspace=ws)
        torch.cuda.synchronize()
        return dx, dw

    want = run()
    old = fp8.fp8_set_wait_limit_ns(2_000_000)  # 2 ms
    fp8.fp8_set_test_stall(True)
    try:
        dx, dw = run()
    finally:
        fp8.fp8_set_test_stall(False)
        fp8.fp8_set_wait_limit_ns(old)
    assert dx.isnan().all() and dw.isnan().all()
    got = run()
    assert torch.isfinite(want[0].float()).all() and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
