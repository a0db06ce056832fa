"""The norm with the residual's addition, its 8-bit output and its backward pass against the formulas in
64 bits. u = 2^-24 is fp32's rounding. Bounds: a row's sum of squares is a chain of at most 32 terms a
thread, 5 shuffles and 16 warps, all positive, of terms rounded twice: 56 u relative, half of it in rstd,
plus the division and the root: below 64 u. A bf16 output adds half an ulp, 2^-8 relative; an e4m3 code
half a step, 2^-4 relative or 2^-10 scales near zero (e5m2: 2^-3, 2^-17)."""
import numpy as np
import pytest
import torch

from tests.gpu_util import mx_unblock_rows

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-6
FMAX = {3: 448.0, 4: 57344.0}


@pytest.fixture(scope="module")
def fp8():
    import moe_grouped_gemm_absmax_gb300 as m
    return m


def _inputs(T, H, seed, residual=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g)
    x[:, torch.randint(0, H, (max(1, H // 100),), generator=g)] *= 30
    x[T // 2] *= 1e-3  # a row of another magnitude
    r = torch.randn(T, H, generator=g) if residual else None
    w = 1 + 0.3 * torch.randn(H, generator=g)
    return x.bfloat16().cuda(), r.bfloat16().cuda() if residual else None, w.bfloat16().cuda()


def _reference(x, r, w, eps=EPS):
    s = x.double() + (r.double() if r is not None else 0)
    rstd = 1 / (s.square().mean(1) + eps).sqrt()
    return s, rstd, s * rstd[:, None] * w.double()


def _check_codes(deq, y, inv, dt):
    half, tiny = (2.0 ** -4, 2.0 ** -10) if dt == 3 else (2.0 ** -3, 2.0 ** -17)
    bound = torch.maximum(y.abs() * half, inv * tiny) * (1 + 1e-4)
    assert ((deq - y).abs() <= bound).all()


SHAPES = [(1, 8), (3, 264), (9, 512), (130, 520), (5, 2048), (2, 2056), (33, 4096), (1, 7168), (7, 8192), (3, 8200),
          (2, 16384)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("dt", [3, 4])
def test_row_scales(fp8, T, H, residual, dt):
    x, r, w = _inputs(T, H, T + H, residual)
    h, y, q, inv, rstd = fp8.add_rmsnorm_alloc(x, w, EPS, r, fp8.GRAN_ROW, dt, want_y=True, want_rstd=True)
    s, rs, yr = _reference(x, r, w)
    if residual:
        assert torch.equal(h, (x.float() + r.float()).bfloat16())
    assert ((rstd.double() - rs).abs() <= 64 * U * rs).all()
    assert ((y.double() - yr).abs() <= (2.0 ** -8 + 64 * U) * yr.abs()).all()
    want = yr.abs().amax(1).clamp_min(1e-12) / FMAX[dt]
    assert ((inv.double() - want).abs() <= 80 * U * want).all()
    _check_codes(q.double() * inv.double()[:, None], yr, inv.double()[:, None], dt)


@pytest.mark.parametrize("T,H", [(1, 128), (37, 512), (130, 2176), (3, 7168), (2, 16384)])
@pytest.mark.parametrize("dt", [3, 4])
def test_block_scales(fp8, T, H, dt):
    x, r, w = _inputs(T, H, 3 * T + H)
    _, _, q, inv, _ = fp8.add_rmsnorm_alloc(x, w.float(), EPS, r, fp8.GRAN_BLOCK_1x128, dt)
    yr = _reference(x, r, w)[2].view(T, H // 128, 128)
    want = yr.abs().amax(2).clamp_min(1e-12) / FMAX[dt]
    assert ((inv.double() - want).abs() <= 80 * U * want).all()
    _check_codes(q.double().view_as(yr) * inv.double()[..., None], yr, inv.double()[..., None], dt)


@pytest.mark.parametrize("T,H", [(1, 128), (130, 512), (3, 7168), (2, 16384)])
@pytest.mark.parametrize("dt", [3, 4])
def test_mx_scales(fp8, T, H, dt):
    x, r, w = _inputs(T, H, 5 * T + H)
    _, _, q, sf, _ = fp8.add_rmsnorm_alloc(x, w, EPS, r, fp8.GRAN_MX, dt)
    yr = _reference(x, r, w)[2].view(T, H // 32, 32)
    codes = torch.from_numpy(mx_unblock_rows(sf, np.arange(T), H).astype(np.float64)).cuda()
    X = torch.exp2(codes - 127)
    low = X * (2.0 ** 8 if dt == 3 else 2.0 ** 15)  # X = 2^(floor(log2 amax) - emax)
    amax = yr.abs().amax(2)
    assert (low <= amax * (1 + 1e-5)).all() and (amax * (1 - 1e-5) < 2 * low).all()
    clipped = yr.clamp(-FMAX[dt] * X[..., None], FMAX[dt] * X[..., None])
    _check_codes(q.double().view_as(yr) * X[..., None], clipped, X[..., None], dt)


def test_degenerate_rows(fp8):
    """A zero row (rstd = 1 / sqrt(eps), codes zero, the scale's floor), a NaN, an infinity, huge and tiny rows; the other
    rows keep their values."""
    T, H = 8, 1024
    x, _, w = _inputs(T, H, 1, False)
    clean = fp8.add_rmsnorm_alloc(x, w, EPS, None, fp8.GRAN_ROW, want_y=True, want_rstd=True)
    x2 = x.clone()
    x2[1] = 0
    x2[2, 5] = float("nan")
    x2[3, 7] = float("inf")
    x2[5] = x[5] * 1e15
    x2[6] = x[6] * 1e-15
    _, y, q, inv, rstd = fp8.add_rmsnorm_alloc(x2, w, EPS, None, fp8.GRAN_ROW, want_y=True, want_rstd=True)
    for t in (0, 4, 7):
        assert torch.equal(y[t], clean[1][t]) and torch.equal(q[t].view(torch.uint8), clean[2][t].view(torch.uint8))
        assert inv[t] == clean[3][t] and rstd[t] == clean[4][t]
    assert abs(float(rstd[1]) * EPS ** 0.5 - 1) < 1e-6 and not y[1].any() and not q[1].float().any()
    assert float(inv[1]) == pytest.approx(1e-12 / 448)
    assert rstd[2].isnan() and y[2].isnan().all() and q[2].float().isnan().all() and inv[2].isnan()
    assert rstd[3] == 0 and y[3, 7].isnan() and inv[3].isnan()
    assert torch.isfinite(y[5]).all() and torch.isfinite(y[6].float()).all()
    w2 = w.clone()
    w2[9] = float("nan")
    _, y, _, inv, _ = fp8.add_rmsnorm_alloc(x, w2, EPS, None, fp8.GRAN_ROW, want_y=True)
    assert inv.isnan().all() and y[:, 9].isnan().all() and int(y.isnan().sum()) == T


def test_in_place_stream_and_graph(fp8):
    T, H = 19, 4096
    x, r, w = _inputs(T, H, 2)
    want = fp8.add_rmsnorm_alloc(x, w, EPS, r, want_y=True)
    a, b = x.clone(), r.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fp8.fp8_add_rmsnorm(a, w, EPS, residual=b, h=b, y=a)  # both outputs over their inputs
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(b, want[0]) and torch.equal(a, want[1])
    h, y = torch.zeros_like(x), torch.zeros_like(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp8.fp8_add_rmsnorm(x, w, EPS, residual=r, h=h, y=y)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(h, want[0]) and torch.equal(y, want[1])


@pytest.mark.parametrize("T", [4101, 8191, 8195])
@pytest.mark.parametrize("H", [520, 776, 1024, 1032])
def test_many_short_rows(fp8, T, H):
    test_row_scales(fp8, T, H, T % 2 == 0, 3)
    test_row_scales(fp8, T, H, T % 2 == 1, 4)


@pytest.mark.parametrize("T", [8190, 8196])
@pytest.mark.parametrize("H", [640, 896, 1024])
def test_many_short_rows_in_blocks(fp8, T, H):
    test_block_scales(fp8, T, H, 3)
    test_mx_scales(fp8, T, H, 4)


@pytest.mark.parametrize("T,H", [(2051, 5120), (2047, 5128), (2051, 5128), (2048, 8192)])
def test_many_wide_rows(fp8, T, H):
    test_row_scales(fp8, T, H, True, 3)


# ------------------------------------------------------------------------------------------ backward

def _bwd_reference(dy, h, w, rstd, dh):
    xhat = h.double() * rstd.double()[:, None]
    g = dy.double() * w.double()
    dx = rstd.double()[:, None] * (g - xhat * (g * xhat).mean(1, keepdim=True))
    if dh is not None:
        dx = dx + dh.double()
    return dx, (dy.double() * xhat).sum(0)


@pytest.mark.parametrize("T,H", [(1, 8), (2, 264), (77, 520), (305, 2048), (610, 2056), (33, 4096), (5, 8200), (3, 16384),
                                 (2000, 1024)])
@pytest.mark.parametrize("stream_grad", [True, False])
def test_backward_formula(fp8, T, H, stream_grad):
    x, r, w = _inputs(T, H, 7 * T + H)
    h, _, _, _, rstd = fp8.add_rmsnorm_alloc(x, w, EPS, r, want_rstd=True)
    g = torch.Generator(device="cuda").manual_seed(T)
    dy = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    dh = torch.randn(T, H, generator=g, device="cuda").bfloat16() if stream_grad else None
    dx, dw = torch.empty_like(h), torch.empty(H, device="cuda")
    ws = fp8.rmsnorm_bwd_workspace(T, H, "cuda")
    ws.fill_(0xFF)  # the workspace needs no particular contents
    fp8.fp8_add_rmsnorm_bwd(dy, h, w, rstd, dx, dw, dh=dh, workspace=ws)
    rx, rw = _bwd_reference(dy, h, w, rstd, dh)
    # each fp32 term is rounded a few times, the row's mean is a chain of 53 terms of either sign
    xhat = h.double().abs() * rstd.double()[:, None]
    gabs = dy.double().abs() * w.double().abs()
    terms = rstd.double()[:, None] * (gabs + xhat * (gabs * xhat).mean(1, keepdim=True))
    assert ((dx.double() - rx).abs() <= 2.0 ** -8 * rx.abs() + 64 * U * terms + 1e-30).all()
    # a partial sum has ceil(T / 304) rows, and at most 304 partial sums are added
    bound = (T / 304 + 60) * U * (dy.double().abs() * xhat).sum(0) + 1e-30
    assert ((dw.double() - rw).abs() <= bound).all()
    dx2, dw2, dwb = torch.empty_like(dx), torch.empty_like(dw), torch.empty(H, dtype=torch.bfloat16, device="cuda")
    fp8.fp8_add_rmsnorm_bwd(dy, h, w, rstd, dx2, dw2, dh=dh, workspace=ws)
    fp8.fp8_add_rmsnorm_bwd(dy, h, w.float(), rstd, None, dwb, dh=dh, workspace=ws)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(dwb, dw.bfloat16())
    over = dy.clone()  # dx over dy, without dw and so without a workspace
    fp8.fp8_add_rmsnorm_bwd(over, h, w, rstd, over, dh=dh)
    assert torch.equal(over, dx)


@pytest.mark.parametrize("T,H", [(2, 264), (5, 4096)])
def test_backward_against_differences(fp8, T, H):
    """sum(dx v) against the central difference of L(x) = sum(dy y(x)) + sum(dh x) along random v, in 64 bits; the
    same for w. The difference's own error is third order; dx's rounding to bf16 bounds the rest."""
    x, _, w = _inputs(T, H, 11, False)
    _, _, _, _, rstd = fp8.add_rmsnorm_alloc(x, w, EPS, None, want_rstd=True)
    g = torch.Generator(device="cuda").manual_seed(5)
    dy, dh, v = (torch.randn(T, H, generator=g, device="cuda").bfloat16() for _ in range(3))
    dx, dw = torch.empty_like(x), torch.empty(H, device="cuda")
    fp8.fp8_add_rmsnorm_bwd(dy, x, w, rstd, dx, dw, dh=dh, workspace=fp8.rmsnorm_bwd_workspace(T, H, "cuda"))
    vw = torch.randn(H, generator=g, device="cuda").double()

    def loss(a, b):
        y = a / (a.square().mean(1, keepdim=True) + EPS).sqrt() * b
        return (dy.double() * y).sum() + (dh.double() * a).sum()

    a, b, d = x.double(), w.double(), 1e-4
    step = d * a.abs().amax(1, keepdim=True) * v.double() / v.double().abs().amax()
    num = (loss(a + step, b) - loss(a - step, b)) / 2
    got = (dx.double() * step).sum()
    assert abs(got - num) <= 2.0 ** -8 * (dx.double() * step).abs().sum() + 1e-6 * abs(num) + 1e-12
    num = (loss(a, b + d * vw) - loss(a, b - d * vw)) / (2 * d)
    assert abs((dw.double() * vw).sum() - num) <= 128 * U * (dw.double() * vw).abs().sum() + 1e-6 * abs(num)


def test_no_rows(fp8):
    H = 264
    e = torch.empty(0, H, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(H, device="cuda")
    fp8.add_rmsnorm_alloc(e, w, EPS, e, fp8.GRAN_ROW, want_y=True, want_rstd=True)
    dw = torch.full((H,), 3.0, device="cuda")
    fp8.fp8_add_rmsnorm_bwd(e, e, w, torch.empty(0, device="cuda"), e, dw, workspace=fp8.rmsnorm_bwd_workspace(0, H, "cuda"))
    assert not dw.any()


# ------------------------------------------------------------------------------------------ many rows

@pytest.mark.parametrize("T,H,gran", [(5000, 264, "row"), (2500, 1024, "block"), (1300, 4096, "row"), (1217, 2056, "row"),
                                      (1300, 4096, "mx"), (700, 7168, "row"), (700, 7168, "block"), (650, 8200, "row"),
                                      (615, 16384, "block"), (615, 16384, "mx"), (700, 7168, "none")])
@pytest.mark.parametrize("residual", [True, False])
def test_many_rows(fp8, T, H, gran, residual):
    """Enough rows that each CTA takes several groups of them, the last group short: every row as the formula gives it,
    and the same bits as in a call with that row among few."""
    x, r, w = _inputs(T, H, T + 2 * H, residual)
    g = {"row": fp8.GRAN_ROW, "block": fp8.GRAN_BLOCK_1x128, "mx": fp8.GRAN_MX, "none": None}[gran]
    h, y, q, inv, rstd = fp8.add_rmsnorm_alloc(x, w, EPS, r, g, want_y=True, want_rstd=True)
    s, rs, yr = _reference(x, r, w)
    if residual:
        assert torch.equal(h, (x.float() + r.float()).bfloat16())
    assert ((rstd.double() - rs).abs() <= 64 * U * rs).all()
    assert ((y.double() - yr).abs() <= (2.0 ** -8 + 64 * U) * yr.abs()).all()
    if gran == "row":
        want = yr.abs().amax(1).clamp_min(1e-12) / 448
        assert ((inv.double() - want).abs() <= 80 * U * want).all()
        _check_codes(q.double() * inv.double()[:, None], yr, inv.double()[:, None], 3)
    elif gran == "block":
        yb = yr.view(T, H // 128, 128)
        want = yb.abs().amax(2).clamp_min(1e-12) / 448
        assert ((inv.double() - want).abs() <= 80 * U * want).all()
        _check_codes(q.double().view_as(yb) * inv.double()[..., None], yb, inv.double()[..., None], 3)
    elif gran == "mx":
        yb = yr.view(T, H // 32, 32)
        X = torch.exp2(torch.from_numpy(mx_unblock_rows(inv, np.arange(T), H).astype(np.float64)).cuda() - 127)
        amax = yb.abs().amax(2)
        assert (X * 2.0 ** 8 <= amax * (1 + 1e-5)).all() and (amax * (1 - 1e-5) < X * 2.0 ** 9).all()
        clipped = yb.clamp(-448 * X[..., None], 448 * X[..., None])
        _check_codes(q.double().view_as(yb) * X[..., None], clipped, X[..., None], 3)


@pytest.mark.parametrize("T,H", [(5000, 264), (1300, 4096), (700, 7168), (320, 8200), (315, 16384), (9000, 1024)])
def test_many_rows_backward_in_place(fp8, T, H):
    """dx over dy's own buffer, rows loaded ahead of the ones being written."""
    x, r, w = _inputs(T, H, 7 * T + H)
    h, _, _, _, rstd = fp8.add_rmsnorm_alloc(x, w, EPS, r, want_rstd=True)
    g = torch.Generator(device="cuda").manual_seed(T)
    dy, dh = (torch.randn(T, H, generator=g, device="cuda").bfloat16() for _ in range(2))
    rx, rw = _bwd_reference(dy, h, w, rstd, dh)
    xhat = h.double().abs() * rstd.double()[:, None]
    gabs = dy.double().abs() * w.double().abs()
    terms = rstd.double()[:, None] * (gabs + xhat * (gabs * xhat).mean(1, keepdim=True))
    bound = (T / 152 + 60) * U * (dy.double().abs() * xhat).sum(0) + 1e-30
    dw = torch.empty(H, device="cuda")
    fp8.fp8_add_rmsnorm_bwd(dy, h, w, rstd, dy, dw, dh=dh, workspace=fp8.rmsnorm_bwd_workspace(T, H, "cuda"))
    assert ((dy.double() - rx).abs() <= 2.0 ** -8 * rx.abs() + 64 * U * terms + 1e-30).all()
    assert ((dw.double() - rw).abs() <= bound).all()
