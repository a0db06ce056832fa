"""The gated feed-forward's training function, the serving block with block scales, and the operators run together as an
expert layer trains: against the same chain in 64 bits with the roundings to 8 bits bounded as they propagate."""
import pytest
import torch

from tests.gated_util import E4, act64, ends, gen, randn, status_word

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8():
    import moe_grouped_gemm_absmax_gb300 as m
    return m


@pytest.fixture(scope="module")
def ag():
    import moe_grouped_gemm_absmax_gb300.autograd as m
    return m


def _inputs(M, H, I, seed):
    g = gen(seed)
    x = randn(g, M, H).to(torch.bfloat16).requires_grad_(True)
    w13 = (randn(g, 2 * I, H) / H ** 0.5).to(torch.bfloat16).requires_grad_(True)
    w2 = (randn(g, H, I) / I ** 0.5).to(torch.bfloat16).requires_grad_(True)
    return x, w13, w2, randn(g, M, H).to(torch.bfloat16)


def _chain64(x, w13, w2, act):
    I = w2.shape[1]
    y = x @ w13.T
    f = torch.nn.functional.silu if act == "silu" else lambda t: torch.nn.functional.gelu(t, approximate="tanh")
    return (f(y[:, :I]) * y[:, I:]) @ w2.T


# An e4m3 rounding moves a value by at most 2^-4 of it, an e5m2 one by 2^-3, independently from value to value: the
# relative error in the 2-norm that one operand brings to a product of many terms stays below that, and those of the
# operands on the way add up. y: x, w13 (both twice: gate and up), h, w2. dW2: h (its two operands' roundings; dY is bf16).
# dx: dY (e5m2), w2, x and w13 through gate and up, dgu (e5m2), w13. dW13: dY, w2, and x and w13 through gate and up.
E4R, E5R = 2.0 ** -4, 2.0 ** -3
BOUND = {"y": 6 * E4R, "dw2": 4 * E4R, "dx": 2 * E5R + 6 * E4R, "dw13": E5R + 5 * E4R}


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("gran", ["row", "block"])
@pytest.mark.parametrize("shape", [(3, 128, 256), (2, 70, 384, 128), (300, 256, 640)])
def test_training_function(fp8, ag, shape, gran, act):
    *lead, H, I = shape
    M = 1
    for n in lead:
        M *= n
    x, w13, w2, c = _inputs(M, H, I, M + H + I)
    xin = x.view(*lead, H)
    granularity = fp8.GRAN_ROW if gran == "row" else fp8.GRAN_BLOCK_1x128
    y = ag.GatedMLPFunction.apply(xin, w13, w2, granularity, fp8.ACT_SILU if act == "silu" else fp8.ACT_GELU)
    assert y.shape == xin.shape and y.dtype == torch.bfloat16
    (y * c.view(y.shape)).float().sum().backward()
    d = [t.detach().double().requires_grad_(True) for t in (x, w13, w2)]
    y64 = _chain64(*d, act)
    (y64 * c.double()).sum().backward()
    for name, got, ref in (("y", y.reshape(M, H), y64), ("dx", x.grad, d[0].grad), ("dw13", w13.grad, d[1].grad),
                           ("dw2", w2.grad, d[2].grad)):
        rel = float((got.double() - ref).norm() / ref.norm())
        assert rel <= BOUND[name], (name, rel)


def test_equals_the_entry_points(fp8, ag):
    """The function only allocates and wires buffers: its results are those of the calls."""
    x, w13, w2, c = _inputs(200, 256, 384, 5)
    y = ag.GatedMLPFunction.apply(x, w13, w2, fp8.GRAN_BLOCK_1x128)
    y.backward(c)
    f = fp8
    B = f.MM_BLOCKWISE
    with torch.no_grad():
        xq, _, xi, _ = f.blk_quantize_alloc(x, f.DT_E4M3)
        q13, q13t, i13, i13t = f.blk_quantize_alloc(w13, f.DT_E4M3, True, f.LAYOUT_BOTH)
        q2, q2t, i2, i2t = f.blk_quantize_alloc(w2, f.DT_E4M3, True, f.LAYOUT_BOTH)
        _, gu, hq, hi = f.gated_mm_alloc(xq, q13, xi, i13, flags=B, want_h=False, want_gu=True, q_dtype=f.DT_E4M3)
        out = torch.empty_like(y)
        f.fp8_scaled_mm(hq, q2, hi, i2, out, B)
        assert torch.equal(out, y)
        dq, _, di, _ = f.blk_quantize_alloc(c, f.DT_E5M2)
        dgu, h = f.gated_mm_bwd_alloc(dq, q2t, di, i2t, gu, flags=B, want_h=True)
        dw2, dw13, dx = torch.empty_like(w2), torch.empty_like(w13), torch.empty_like(x)
        outer = f.MM_A_MN_MAJOR | f.MM_B_MN_MAJOR
        f.fp8_scaled_mm(c, h, None, None, dw2, outer)
        f.fp8_scaled_mm(dgu, x, None, None, dw13, outer)
        gq, _, gi, _ = f.blk_quantize_alloc(dgu, f.DT_E5M2)
        f.fp8_scaled_mm(gq, q13t, gi, i13t, dx, B)
    assert torch.equal(dw2, w2.grad) and torch.equal(dw13, w13.grad) and torch.equal(dx, x.grad)


def test_module_and_gradients_that_are_not_asked_for(fp8, ag):
    torch.manual_seed(0)
    mlp = ag.Fp8GatedMLP(256, 512, device="cuda")
    x = torch.randn(5, 256, device="cuda").bfloat16()
    mlp(x).float().square().sum().backward()
    full = [p.grad.clone() for p in mlp.parameters()]
    assert all(g.isfinite().all() and g.any() for g in full) and "row" in repr(mlp)
    mlp.zero_grad()
    mlp.w13.requires_grad_(False)
    mlp(x).float().square().sum().backward()
    assert mlp.w13.grad is None and torch.equal(mlp.w2.grad, full[1])
    mlp.w2.requires_grad_(False)
    xr = x.clone().requires_grad_(True)
    mlp(xr).float().square().sum().backward()
    assert xr.grad.isfinite().all() and xr.grad.any()
    mlp.zero_grad()
    mlp.w13.requires_grad_(True)
    mlp.w2.requires_grad_(True)
    for gran in (fp8.GRAN_ROW, fp8.GRAN_BLOCK_1x128):  # no rows: zeros
        mlp.granularity = gran
        xr = x[:0].clone().requires_grad_(True)
        y = mlp(xr)
        assert y.shape == (0, 256)
        y.float().sum().backward()
        assert xr.grad.shape == (0, 256) and not mlp.w13.grad.any() and not mlp.w2.grad.any()


def test_refusals(fp8, ag):
    x, w13, w2, _ = _inputs(4, 128, 128, 1)
    with pytest.raises(TypeError):
        ag.GatedMLPFunction.apply(x.float(), w13, w2)
    with pytest.raises(ValueError):
        ag.GatedMLPFunction.apply(x, w13, w2, fp8.GRAN_MX)
    with pytest.raises(ValueError):
        ag.Fp8GatedMLP(100, 128)
    with pytest.raises(ValueError):
        ag.Fp8GatedMLP(144, 128, fp8.GRAN_BLOCK_1x128)
    y = ag.GatedMLPFunction.apply(x, w13, w2)
    gx, = torch.autograd.grad(y.float().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        (gx.float().sum() + x.float().sum()).backward()


def test_captured_training_step(fp8, ag):
    """Forward and backward captured into one graph and replayed on other inputs."""
    x, w13, w2, c = _inputs(130, 256, 256, 9)
    other, _, _, c2 = _inputs(130, 256, 256, 10)

    def step(x, c):
        y = ag.GatedMLPFunction.apply(x, w13, w2)
        return (y,) + torch.autograd.grad(y, (x, w13, w2), c)

    # no eager graph of the weights outlives this: a backward pass cannot be captured beside one (torch's own rule)
    want = [[t.detach().clone() for t in step(a, b)] for a, b in ((x, c), (other, c2))]
    sx, sc = x.detach().clone().requires_grad_(True), c.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            step(sx, sc)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(sx, sc)
    for (a, b), w in zip(((other, c2), (x, c)), (want[1], want[0])):
        with torch.no_grad():
            sx.copy_(a)
            sc.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, w))


@pytest.mark.parametrize("T,E,H,I,k", [(1, 8, 256, 128, 2), (7, 16, 1024, 512, 3), (40, 8, 512, 256, 2), (300, 16, 1024, 512, 4)])
def test_serving_block_with_block_scales(fp8, T, E, H, I, k):
    """Decode and prompts through the gated and the block-scaled grouped product: the norm's output and the hidden layer are
    rounded to e4m3 (2^-4 a value), the hidden layer through both projections of the first."""
    from moe_grouped_gemm_absmax_gb300.moe import Fp8MoEBlock
    g = gen(T)
    norm, router = (1 + 0.1 * randn(g, H)).bfloat16(), (0.05 * randn(g, E, H)).bfloat16()
    w1, w3, w2 = (0.05 * randn(g, E, I, H)).bfloat16(), (0.05 * randn(g, E, I, H)).bfloat16(), (0.05 * randn(g, E, H, I)).bfloat16()
    block = Fp8MoEBlock(norm, router, w1, w3, w2, k, granularity=fp8.GRAN_BLOCK_1x128)
    x, r = randn(g, T, H).bfloat16(), randn(g, T, H).bfloat16()
    st = status_word()
    out, h = block(x, r, st)
    assert st.item() == 0 and torch.equal(h, (x.float() + r.float()).bfloat16())
    s = x.double() + r.double()
    y = s / (s.square().mean(1, keepdim=True) + block.eps).sqrt() * norm.double()
    _, yb, _, _, _ = fp8.add_rmsnorm_alloc(x, norm, block.eps, r, want_y=True)
    logits = torch.empty(T, E, device="cuda")
    fp8.fp8_scaled_mm(yb, router, None, None, logits)
    ids, weights, _, _, _ = fp8.moe_route_alloc(logits, k, table=False)
    up = lambda q, s: q.double() * s.double().repeat_interleave(128, -2).repeat_interleave(128, -1)  # noqa: E731
    v13, v2 = up(block.w13, block.s13), up(block.w2, block.s2)
    ref = torch.zeros_like(y)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            gu = v13[e] @ y[t]
            ref[t] += weights[t, j].double() * (v2[e] @ (act64(gu[:I], "silu")[0] * gu[I:]))
    rel = float((out.double() - ref).norm() / ref.norm())
    assert rel <= 3 * 2.0 ** -4, rel
    # no rows, and a token with a NaN: its own row alone
    assert block(x[:0], r[:0])[0].shape == (0, H)
    if T > 1:
        x[1, 3] = float("nan")
        out2, _ = block(x, r, st)
        assert out2[1].isnan().all()
        keep = torch.arange(T, device="cuda") != 1
        assert torch.equal(out2[keep], out[keep])


def test_block_refusals(fp8):
    from moe_grouped_gemm_absmax_gb300.moe import Fp8MoEBlock
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    with pytest.raises(ValueError):
        Fp8MoEBlock(z(256), z(4, 256), z(4, 136, 256), z(4, 136, 256), z(4, 256, 136), 2, granularity=fp8.GRAN_BLOCK_1x128)
    with pytest.raises(ValueError):
        Fp8MoEBlock(z(256), z(4, 256), z(4, 128, 256), z(4, 128, 256), z(4, 256, 128), 2, granularity=fp8.GRAN_MX)


def test_experts_train_together(fp8):
    """A layer of experts as it trains: route, gated product by expert, second product, then back through both, with the
    weight gradients by the grouped GEMM over each expert's rows; against 64 bits on the same routed rows."""
    T, E, H, I, k = 200, 6, 256, 384, 2
    f = fp8
    g = gen(31)
    x = randn(g, T, H).bfloat16()
    logits = randn(g, T, E)
    ids, weights, order, pos, off = f.moe_route_alloc(logits, k)
    rows = (order // k).long()
    w13, w2 = (randn(g, E, 2 * I, H) / 16).bfloat16(), (randn(g, E, H, I) / 16).bfloat16()
    q13 = [f.blk_quantize_alloc(w13[e], f.DT_E4M3, True, f.LAYOUT_BOTH) for e in range(E)]
    q2 = [f.blk_quantize_alloc(w2[e], f.DT_E4M3, True, f.LAYOUT_BOTH) for e in range(E)]
    st8 = lambda qs, i: torch.stack([t[i].view(torch.uint8) for t in qs]).view(E4)  # noqa: E731
    st = lambda qs, i: torch.stack([t[i] for t in qs])  # noqa: E731
    a = x[rows].contiguous()
    aq, _, ai, _ = f.blk_quantize_alloc(a, f.DT_E4M3)
    B, n, status = f.MM_BLOCKWISE, T * k, status_word()
    _, gu, hq, hi = f.gated_mm_alloc(aq, st8(q13, 0), ai, st(q13, 2), off, flags=B, want_h=False, want_gu=True,
                                     q_dtype=f.DT_E4M3, status=status)
    y = torch.empty(n, H, dtype=torch.bfloat16, device="cuda")
    f.fp8_grouped_mm(hq, st8(q2, 0), off, hi, st(q2, 2), y, f.GROUPED_JAGGED_M, B, status)
    dy = randn(g, n, H).bfloat16()
    dq, _, di, _ = f.blk_quantize_alloc(dy, f.DT_E5M2)
    dgu, h = f.gated_mm_bwd_alloc(dq, st8(q2, 1), di, st(q2, 3), gu, off, flags=B, want_h=True, status=status)
    gq, _, gi, _ = f.blk_quantize_alloc(dgu, f.DT_E5M2)
    dx = torch.empty(n, H, dtype=torch.bfloat16, device="cuda")
    f.fp8_grouped_mm(gq, st8(q13, 1), off, gi, st(q13, 3), dx, f.GROUPED_JAGGED_M, B, status)
    _, dyt, dyi = f.quantize_alloc(dy, f.GRAN_COL, f.DT_E5M2, offsets=off, status=status)
    _, ht, hti = f.quantize_alloc(h, f.GRAN_COL, f.DT_E4M3, offsets=off, status=status)
    dw2 = torch.empty(E, H, I, dtype=torch.bfloat16, device="cuda")
    f.fp8_grouped_mm(dyt, ht, off, dyi, hti, dw2, f.GROUPED_JAGGED_K, 0, status)
    assert status.item() == 0
    ev = torch.cat([torch.zeros(1, dtype=torch.int32), off.cpu()]).tolist()
    v = [t.double().requires_grad_(True) for t in (a, w13, w2)]
    ref = torch.cat([_chain64(v[0][b:c], v[1][e], v[2][e], "silu") for e, (b, c) in enumerate(zip(ev, ev[1:]))])
    (ref * dy.double()).sum().backward()
    for name, got, want in (("y", y, ref), ("dx", dx, v[0].grad), ("dw2", dw2, v[2].grad)):
        rel = float((got.double() - want).norm() / want.norm())
        assert rel <= BOUND[name] + (E5R + E4R if name == "dw2" else 0), (name, rel)
