"""The gated feed-forward's forward and backward kernels against their formulas in 64 bits (bounds: gated_util.py)."""
import pytest
import torch

from tests.gated_util import (E4, E5, HALF_BF16, act64, check, check_codes, ends, gen, hidden, operand, product, randn,
                              status_word)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8():
    import moe_grouped_gemm_absmax_gb300 as m
    return m


def _act(fp8, name):
    return fp8.ACT_SILU if name == "silu" else fp8.ACT_GELU


def _operands(seed, M, K, rows, counts, kind, a_dt=E4, b_dt=E4, a_size=1.0):
    g = gen(seed)
    A, sA, a = operand(g, (M, K), kind, a_dt, size=a_size)
    shape = (len(counts), rows, K) if counts is not None else (rows, K)
    B, sB, b = operand(g, shape, kind, b_dt, rows=128, size=2.0 / K ** 0.5)  # projections of about 2
    return g, A, sA, a, B, sB, b


# (M, K, I, counts by expert or None)
DENSE = [(1, 16, 8), (1, 4096, 1024), (3, 128, 136), (17, 400, 1000), (128, 128, 128), (130, 1040, 264), (300, 2064, 72),
         (2500, 256, 1288), (2048, 512, 1280),
         (1200, 256, 1920), (1200, 128, 3840), (250, 64, 9600), (250, 64, 19200), (200, 512, 2048)]
EXPERTS = [(1500, 256, 1408, [700, 0, 800]), (1500, 128, 2816, [1, 1400, 99]), (1, 128, 128, [0, 1, 0]), (9, 256, 200, [9]), (77, 144, 264, [0, 30, 0, 46, 1]), (300, 512, 512, [129, 0, 171]),
           (2304, 256, 640, [256, 0, 1, 700, 1300, 47, 0]), (4000, 384, 384, [3999, 1]), (2100, 128, 264, [0] * 1000 + [2000, 77, 23] + [0] * 21)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("kind", ["row", "tensor", "bf16", "block"])
@pytest.mark.parametrize("M,K,I", DENSE)
def test_dense(fp8, M, K, I, kind, act):
    if kind == "block":
        K, I = -(-K // 128) * 128, -(-I // 128) * 128
    _run(fp8, M, K, I, None, kind, act)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("kind", ["row", "block"])
@pytest.mark.parametrize("M,K,I,counts", EXPERTS)
def test_experts(fp8, M, K, I, counts, kind, act):
    if kind == "block":
        K, I = -(-K // 128) * 128, -(-I // 128) * 128
    _run(fp8, M, K, I, counts, kind, act)


def _run(fp8, M, K, I, counts, kind, act):
    _, A, sA, a, B, sB, b = _operands(M + K + I, M, K, 2 * I, counts, kind, E5 if kind == "tensor" else E4)
    y, err = product(a, b, counts)
    h64, eh = hidden(y, err, act)
    off = ends(counts) if counts is not None else None
    flags = fp8.MM_BLOCKWISE if kind == "block" else 0
    st = status_word()
    codes = kind != "bf16" and I % 128 == 0
    h, gu, q, inv = fp8.gated_mm_alloc(A, B, sA, sB, off, _act(fp8, act), flags, want_gu=True,
                                       q_dtype=(fp8.DT_E5M2 if act == "gelu" else fp8.DT_E4M3) if codes else None, status=st)
    assert st.item() == 0
    check(gu, y, err + HALF_BF16 * y.abs(), "projections")
    check(h, h64, eh + HALF_BF16 * (h64.abs() + eh), "hidden layer")
    if codes:
        check_codes(q, inv, h64, eh)
    # each output by itself has the same bits
    for k, ref in (("h", h), ("gu", gu), ("q", q)):
        if ref is None:
            continue
        only = torch.zeros_like(ref)
        kw = {k: only}
        if k == "q":
            kw["inv_scales"] = torch.zeros_like(inv)
        fp8.fp8_gated_mm(A, B, sA, sB, offsets=off, act=_act(fp8, act), flags=flags, **kw)
        assert torch.equal(only.view(torch.uint8), ref.view(torch.uint8)), k
        if k == "q":
            assert torch.equal(kw["inv_scales"], inv)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("kind", ["row", "tensor", "bf16", "bf16-mn", "block"])
@pytest.mark.parametrize("M,K,I", DENSE)
def test_dense_backward(fp8, M, K, I, kind, act):
    if kind == "block":
        K = -(-K // 128) * 128
    _run_backward(fp8, M, K, I, None, kind, act)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("kind", ["row", "block"])
@pytest.mark.parametrize("M,K,I,counts", EXPERTS)
def test_experts_backward(fp8, M, K, I, counts, kind, act):
    if kind == "block":
        K = -(-K // 128) * 128
    _run_backward(fp8, M, K, I, counts, kind, act)


def _run_backward(fp8, M, K, I, counts, kind, act):
    mn = kind == "bf16-mn"
    g, A, sA, a, B, sB, b = _operands(M + K + I + 1, M, K, I, counts, "bf16" if mn else kind, E5, a_size=1e-3)
    dh, err = product(a, b, counts)
    gu = (1.5 * randn(g, M, 2 * I)).to(torch.bfloat16)
    g64, u64 = gu.double().split(I, 1)
    a64, d64, ea, ed = act64(g64, act)
    off = ends(counts) if counts is not None else None
    flags = fp8.MM_BLOCKWISE if kind == "block" else fp8.MM_B_MN_MAJOR if mn else 0
    if mn:
        B = B.T.contiguous()
    st = status_word()
    dgu = torch.full_like(gu, float("nan"))
    h = torch.full((M, I), float("nan"), dtype=torch.bfloat16, device="cuda")
    fp8.fp8_gated_mm_bwd(A, B, sA, sB, gu, dgu, h, off, _act(fp8, act), flags, st)
    assert st.item() == 0
    dg, du, h64 = dh * u64 * d64, dh * a64, a64 * u64
    bound = err * (u64 * d64).abs() + (dh.abs() + err) * u64.abs() * ed + 2.0 ** -22 * dg.abs()
    check(dgu[:, :I], dg, bound + HALF_BF16 * (dg.abs() + bound), "gate's gradient")
    bound = err * a64.abs() + (dh.abs() + err) * ea + 2.0 ** -22 * du.abs()
    check(dgu[:, I:], du, bound + HALF_BF16 * (du.abs() + bound), "up projection's gradient")
    bound = ea * u64.abs() + 2.0 ** -22 * h64.abs()
    check(h, h64, bound + HALF_BF16 * (h64.abs() + bound), "hidden layer")
    same = gu.clone()  # in place, without the hidden layer
    fp8.fp8_gated_mm_bwd(A, B, sA, sB, same, same, None, off, _act(fp8, act), flags, st)
    assert torch.equal(same, dgu)


@pytest.mark.parametrize("kind,M,counts", [("row", 5, None), ("bf16", 5, None), ("block", 5, None), ("row", 2304, [2300, 4]),
                                           ("block", 300, [0, 300])])
def test_not_finite(fp8, kind, M, counts):
    """A NaN or an infinity stays in its row, and the row gives what the formulas give: NaN in a block's largest makes its
    scale and codes NaN; gates of -inf are 0 * -inf = NaN, of +inf infinities with the up projection's sign."""
    K, I = 256, 256
    _, A, sA, a, B, sB, b = _operands(3, M, K, 2 * I, counts, kind, a_dt=E5 if kind != "bf16" else E4)
    A2 = A.clone()
    A2[1, 7] = float("nan")
    A2[3, 9] = float("inf")
    off = ends(counts) if counts is not None else None
    flags = fp8.MM_BLOCKWISE if kind == "block" else 0
    qd = fp8.DT_E4M3 if kind != "bf16" else None
    h, gu, q, inv = fp8.gated_mm_alloc(A, B, sA, sB, off, flags=flags, want_gu=True, q_dtype=qd)
    h2, gu2, q2, inv2 = fp8.gated_mm_alloc(A2, B, sA, sB, off, flags=flags, want_gu=True, q_dtype=qd)
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[1] = keep[3] = False
    assert torch.equal(h2[keep], h[keep]) and torch.equal(gu2[keep], gu[keep])
    assert h2[1].isnan().all() and gu2[1].isnan().all()
    assert not gu2[3].isfinite().any() and not h2[3].isfinite().any()
    g, u = gu2[3].double().split(I)
    ref = g * torch.sigmoid(g) * u
    same = (h2[3].double() == ref) | (h2[3].isnan() & ref.isnan())
    assert same.all()
    if q is not None:
        assert torch.equal(q2.view(torch.uint8)[keep], q.view(torch.uint8)[keep]) and torch.equal(inv2[keep], inv[keep])
        assert inv2[1].isnan().all() and q2[1].float().isnan().all()
        assert not inv2[3].isfinite().any()
    # backward: a row's NaN stays in its row
    g2, D, sD, _, W, sW, _ = _operands(4, M, K, I, counts, kind, a_dt=E5 if kind != "bf16" else E4)
    x = (randn(g2, M, 2 * I)).to(torch.bfloat16)
    x2 = x.clone()
    x2[1, 5] = float("nan")
    D2 = D.clone()
    D2[3, 9] = float("nan")
    d1, d2 = torch.empty_like(x), torch.empty_like(x)
    fp8.fp8_gated_mm_bwd(D, W, sD, sW, x, d1, None, off, flags=flags)
    fp8.fp8_gated_mm_bwd(D2, W, sD, sW, x2, d2, None, off, flags=flags)
    assert torch.equal(d1[keep], d2[keep]) and d2[3].isnan().all()
    assert d2[1, 5].isnan() and d2[1, I + 5].isnan()
    rest = torch.ones(2 * I, dtype=torch.bool, device="cuda")
    rest[5] = rest[I + 5] = False
    assert torch.equal(d1[1][rest], d2[1][rest])


def test_zero_rows_give_floor_scales(fp8):
    """A block of zeros: scale 1e-12 / 448 as the recipe's, codes 0."""
    A = torch.zeros(4, 128, dtype=E4, device="cuda")
    B = torch.ones(512, 128, device="cuda").to(E4)
    one = torch.ones(1, device="cuda")
    _, _, q, inv = fp8.gated_mm_alloc(A, B, one, one, q_dtype=fp8.DT_E4M3)
    assert (q.float() == 0).all() and torch.allclose(inv, torch.full_like(inv, 1e-12 / 448), rtol=1e-6, atol=0)


def test_no_rows_and_no_columns(fp8):
    one = torch.ones(1, device="cuda")
    A, B = torch.zeros(0, 128, dtype=E4, device="cuda"), torch.zeros(512, 128, dtype=E4, device="cuda")
    h, _, _, _ = fp8.gated_mm_alloc(A, B, torch.ones(0, device="cuda"), torch.ones(512, device="cuda"))
    assert h.shape == (0, 256)
    h, _, _, _ = fp8.gated_mm_alloc(torch.zeros(3, 128, dtype=E4, device="cuda"), B[:0], one, one)
    assert h.shape == (3, 0)
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind", ["row", "block"])
@pytest.mark.parametrize("counts", [[5, 3, -1], [5, 4], [7, 1]])
def test_bad_offsets(fp8, kind, counts):
    """Offsets that fall, or that end short of or past the rows: the status word says so and nothing is written."""
    M, K, I = 8, 128, 128
    bad = torch.tensor(counts, device="cuda").cumsum(0).to(torch.int32)
    if counts == [7, 1]:
        bad = torch.tensor([7, 3000], dtype=torch.int32, device="cuda")
    _, A, sA, _, B, sB, _ = _operands(1, M, K, 2 * I, counts, kind)
    flags = fp8.MM_BLOCKWISE if kind == "block" else 0
    st = status_word()
    h = torch.full((M, I), 7.0, dtype=torch.bfloat16, device="cuda")
    fp8.fp8_gated_mm(A, B, sA, sB, h=h, offsets=bad, flags=flags, status=st)
    assert st.item() == fp8.DEV_BAD_OFFSETS and (h == 7).all()
    _, D, sD, _, W, sW, _ = _operands(2, M, K, I, counts, kind)
    st.zero_()
    gu = torch.full((M, 2 * I), 7.0, dtype=torch.bfloat16, device="cuda")
    fp8.fp8_gated_mm_bwd(D, W, sD, sW, gu, gu, None, bad, flags=flags, status=st)
    assert st.item() == fp8.DEV_BAD_OFFSETS and (gu == 7).all()


def test_nothing_beside_the_outputs_is_written(fp8):
    """Outputs inside larger buffers: the bytes before and behind stay."""
    M, K, I = 133, 256, 264
    for kind, counts in (("row", None), ("bf16", None), ("row", [100, 33])):
        _, A, sA, _, B, sB, _ = _operands(9, M, K, 2 * I, counts, kind)
        off = ends(counts) if counts else None
        pad = 4096
        bufs = [torch.full((pad + M * w + pad,), 7.0, dtype=torch.bfloat16, device="cuda") for w in (I, 2 * I)]
        h, gu = (b[pad:pad + M * w].view(M, w) for b, w in zip(bufs, (I, 2 * I)))
        fp8.fp8_gated_mm(A, B, sA, sB, h=h, gu=gu, offsets=off)
        _, D, sD, _, W, sW, _ = _operands(10, M, K, I, counts, kind)
        fp8.fp8_gated_mm_bwd(D, W, sD, sW, gu, gu, h, off)
        for b in bufs:
            assert (b[:pad] == 7).all() and (b[-pad:] == 7).all()


def test_streams_and_graphs(fp8):
    """A call on a side stream, and a captured one replayed on new inputs."""
    M, K, I = 40, 512, 384
    _, A, sA, _, B, sB, _ = _operands(11, M, K, 2 * I, None, "row")
    _, A2, sA2, _, _, _, _ = _operands(12, M, K, 2 * I, None, "row")
    want = [fp8.gated_mm_alloc(x, B, s, sB, q_dtype=fp8.DT_E4M3) for x, s in ((A, sA), (A2, sA2))]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    h = torch.zeros(M, I, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    fp8.fp8_gated_mm(A, B, sA, sB, h=h, stream=s)
    s.synchronize()
    assert torch.equal(h, want[0][0])
    x, sx = A.clone(), sA.clone()
    q, inv = torch.zeros_like(want[0][2]), torch.zeros_like(want[0][3])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp8.fp8_gated_mm(x, B, sx, sB, h=h, q=q, inv_scales=inv)
    for src, ss, w in ((A2, sA2, want[1]), (A, sA, want[0])):
        x.copy_(src)
        sx.copy_(ss)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, w[0]) and torch.equal(q.view(torch.uint8), w[2].view(torch.uint8)) and torch.equal(inv, w[3])


def test_gradient_against_differences(fp8):
    """The backward pass of y = h W2^T against central differences of the forward formulas in 64 bits, at the bf16
    projections: dgu against d(sum(dy * y)) / d(g, u)."""
    M, K, I = 6, 64, 40
    for act in ("silu", "gelu"):
        g, D, _, d, W, _, w = _operands(21, M, K, I, None, "bf16")
        gu = randn(g, M, 2 * I).to(torch.bfloat16)
        dgu = torch.empty_like(gu)
        fp8.fp8_gated_mm_bwd(D, W, None, None, gu, dgu, act=_act(fp8, act))

        def loss(x):  # [M, 2 I] -> each element's own contribution, [M, I]
            return act64(x[:, :I], act)[0] * x[:, I:] * (d @ w.T)

        x, step = gu.double(), 1e-5
        for part in (0, 1):
            e = torch.zeros_like(x)
            e[:, part * I:(part + 1) * I] = step
            num = (loss(x + e) - loss(x - e)) / (2 * step)
            got = dgu[:, part * I:(part + 1) * I].double()
            # half a step of bf16, fp32 sums, and differences' own error (third derivatives below 2, rounding)
            bound = HALF_BF16 * num.abs() + 1e-4 * (d.abs() @ w.abs().T) * (1 + x[:, I:].abs())
            assert ((got - num).abs() <= bound).all()


# the few rows' kernel: rows of a tile (16, 32, 64), one or several CTAs a tile, ragged and empty experts
FEW = [(1, 128, 128, None), (1, 7168, 256, None), (16, 2048, 136, None), (17, 1024, 384, None), (32, 4096, 128, None),
       (33, 512, 640, None), (64, 1536, 264, None), (64, 256, 13000, None), (8, 1024, 256, [0, 3, 0, 4, 1]),
       (64, 512, 200, [1, 0, 40, 23]), (40, 2048, 128, [40]), (64, 384, 384, [1] * 64 + [0] * 200), (5, 640, 2048, [0] * 1023 + [5])]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("kind", ["row", "block"])
@pytest.mark.parametrize("M,K,I,counts", FEW)
def test_few_rows(fp8, M, K, I, counts, kind, act):
    if kind == "block":
        K, I = -(-K // 128) * 128, -(-I // 128) * 128
    _run(fp8, M, K, I, counts, kind, act)
