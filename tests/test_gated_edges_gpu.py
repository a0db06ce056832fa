"""The gated feed-forward and the block-scaled product at the ends of what a call allows: gates so large that the activation's
inner polynomial overflows, outputs that start between sectors, tensors of more than 2^31 elements, two calls at once, and
calls behind whatever else a stream or a captured graph holds."""
import pytest
import torch

from tests.gated_util import E4, E5, HALF_BF16, act64, check, ends, gen, hidden, operand, product, randn, status_word

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8():
    import moe_grouped_gemm_absmax_gb300 as m
    return m


def _act(fp8, name):
    return fp8.ACT_SILU if name == "silu" else fp8.ACT_GELU


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_saturated_gates(fp8, act):
    """Gates up to the type's largest value: the derivative is 1 or 0 there, and a product that a zero derivative ends does
    not overflow on its way."""
    K, I = 64, 64
    gates = torch.tensor([1e10, 1e13, 3e15, 1e19, 5e19, 1e20, 1e25, 3e38], device="cuda")
    gates = torch.cat([gates, -gates]).repeat(4)  # 64 columns
    for size in (1.0, 1e18):
        g = gen(31)
        D, _, d = operand(g, (5, K), "bf16", size=size)
        W, _, w = operand(g, (I, K), "bf16", size=0.25)
        u = (size * randn(g, 5, I)).to(torch.bfloat16)
        gu = torch.cat([gates.to(torch.bfloat16).expand(5, I), u], 1).contiguous()
        dgu, h = fp8.gated_mm_bwd_alloc(D, W, None, None, gu, act=_act(fp8, act), want_h=True)
        dh, err = product(d, w)
        up = gu[:, :I].double() > 0
        u64 = u.double()
        # act' is 1 or 0; act(g) is g or 0
        dg = torch.where(up, dh * u64, 0.0)
        assert dg.abs().max() < 1e38
        bound = torch.where(up, err * u64.abs() + 2.0 ** -20 * dg.abs(), 0.0) + 1e-30 * u64.abs() * dh.abs()
        check(dgu[:, :I], dg, bound + HALF_BF16 * (dg.abs() + bound))
        off = ~up
        assert (dgu[:, I:][off].double().abs() <= 1e-30 * dh[off].abs()).all()
        assert (h[off].double().abs() <= 1e-30 * u64[off].abs()).all()
        low = up & (gu[:, :I].double() < 1e15)
        du = dh * gu[:, :I].double()
        eb = (err * gu[:, :I].double() + 2.0 ** -20 * du.abs())
        check(dgu[:, I:][low], du[low], (eb + HALF_BF16 * (du.abs() + eb))[low])


@pytest.mark.parametrize("kind", ["row", "block"])
@pytest.mark.parametrize("M,counts", [(9, None), (64, None), (65, None), (130, [100, 0, 30]), (2304, [2200, 104])])
def test_outputs_between_sectors(fp8, kind, M, counts):
    """Outputs that start on 16 bytes and not on 32 get the bits of those that do."""
    K, I = 256, 384
    g = gen(M)
    A, sA, _ = operand(g, (M, K), kind)
    lead = (len(counts),) if counts else ()
    B, sB, _ = operand(g, lead + (2 * I, K), kind, rows=128, size=0.1)
    off = ends(counts) if counts else None
    flags = fp8.MM_BLOCKWISE if kind == "block" else 0
    h, gu, q, inv = fp8.gated_mm_alloc(A, B, sA, sB, off, flags=flags, want_gu=True, q_dtype=fp8.DT_E4M3)

    def shifted(t, by=16):
        n = by // t.element_size()
        x = torch.full((t.numel() + 2 * n,), 7.0, device="cuda").to(t.dtype)
        return x, x[n:n + t.numel()].view(t.shape)

    (hb, h2), (gb, gu2), (qb, q2), (ib, inv2) = shifted(h), shifted(gu), shifted(q), shifted(inv)
    fp8.fp8_gated_mm(A, B, sA, sB, h2, gu2, q2, inv2, off, flags=flags)
    for a, b in ((h, h2), (gu, gu2), (q, q2), (inv, inv2)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    D, sD, _ = operand(g, (M, K), kind, E5, size=1e-2)
    W, sW, _ = operand(g, lead + (I, K), kind, rows=128)
    d1, h1 = fp8.gated_mm_bwd_alloc(D, W, sD, sW, gu, off, flags=flags, want_h=True)
    fp8.fp8_gated_mm_bwd(D, W, sD, sW, gu2, gu2, h2, off, flags=flags)
    assert torch.equal(d1, gu2) and torch.equal(h1, h2)
    if counts and kind == "block":
        P, sP, _ = operand(g, (len(counts), 520, I), "block", rows=128)
        out = torch.empty(M, 520, dtype=torch.bfloat16, device="cuda")
        fp8.fp8_grouped_mm(q, P, off, inv, sP, out, fp8.GROUPED_JAGGED_M, fp8.MM_BLOCKWISE)
        ob, out2 = shifted(out)
        fp8.fp8_grouped_mm(q2, P, off, inv2, sP, out2, fp8.GROUPED_JAGGED_M, fp8.MM_BLOCKWISE)
        assert torch.equal(out, out2)
        assert (ob[:8] == 7).all() and (ob[-8:] == 7).all()
    for b in (hb, gb):
        assert (b[:8] == 7).all() and (b[-8:] == 7).all()
    assert (qb[:16].float() == 7).all() and (qb[-16:].float() == 7).all() and (ib[:4] == 7).all() and (ib[-4:] == 7).all()


@pytest.mark.parametrize("M,counts", [(9, None), (130, None), (9, [4, 0, 5]), (300, [120, 180])])
def test_scales_at_any_word(fp8, M, counts):
    """Block scales that start on 4 bytes and not on 16 give the bits of those that do."""
    K, I = 1024, 256
    g = gen(M + 1)
    lead = (len(counts),) if counts else ()
    off = ends(counts) if counts else None

    def word(t):
        x = torch.zeros(t.numel() + 1, device="cuda")
        x[1:] = t.flatten()
        return x[1:].view(t.shape)

    A, sA, _ = operand(g, (M, K), "block")
    B, sB, _ = operand(g, lead + (2 * I, K), "block", rows=128, size=0.1)
    D, sD, _ = operand(g, (M, K), "block", E5)
    W, sW, _ = operand(g, lead + (I, K), "block", rows=128, size=0.1)
    gu = randn(g, M, 2 * I).to(torch.bfloat16)
    got = []
    for f in (lambda t: t, word):
        h, _, q, inv = fp8.gated_mm_alloc(A, B, f(sA), f(sB), off, flags=fp8.MM_BLOCKWISE, q_dtype=fp8.DT_E4M3)
        dgu, h2 = fp8.gated_mm_bwd_alloc(D, W, f(sD), f(sW), gu, off, flags=fp8.MM_BLOCKWISE, want_h=True)
        out = torch.empty(M, I, device="cuda")
        if counts:
            fp8.fp8_grouped_mm(A, W, off, f(sA), f(sW), out, fp8.GROUPED_JAGGED_M, fp8.MM_BLOCKWISE)
        else:
            fp8.fp8_scaled_mm(A, W, f(sA), f(sW), out, fp8.MM_BLOCKWISE)
        got.append([h, q, inv, dgu, h2, out])
    for a, b in zip(*got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("kind", ["row", "block"])
@pytest.mark.parametrize("counts", [None, [69981, 0, 50]])
def test_more_than_2_31_elements(fp8, kind, counts):
    """The rows behind the 2^31st element of the projections, and of the hidden layer's codes beside them."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    M, K, I = 70031, 128, 16384
    g = gen(77)
    A, sA, a = operand(g, (M, K), kind)
    lead = (len(counts),) if counts else ()
    B, sB, b = operand(g, lead + (2 * I, K), kind, rows=128, size=0.2)
    off = ends(counts) if counts else None
    flags = fp8.MM_BLOCKWISE if kind == "block" else 0
    st = status_word()
    h, gu, q, inv = fp8.gated_mm_alloc(A, B, sA, sB, off, flags=flags, want_gu=True, q_dtype=fp8.DT_E4M3, status=st)
    assert gu.numel() > 2 ** 31 and st.item() == 0
    rows = [0, 1, 65535, 65536, 65537, 69980, 69981, M - 33, M - 32, M - 1]
    e_of = [0 if not counts or r < 69981 else 2 for r in rows]
    w = b.unsqueeze(0) if not counts else b
    for r, e in zip(rows, e_of):
        y, err = product(a[r:r + 1], w[e])
        h64, eh = hidden(y, err, "silu")
        check(gu[r:r + 1], y, err + HALF_BF16 * y.abs(), f"row {r}")
        check(h[r:r + 1], h64, eh + HALF_BF16 * (h64.abs() + eh), f"row {r}")
        top = inv[r].double().repeat_interleave(128) * q[r].double()
        check(top[None], h64, 2.0 ** -4 * h64.abs() + 2.0 ** -9 * inv[r].double().repeat_interleave(128) + 2 * eh + 2.0 ** -20 * h64.abs())
    del h, q, inv
    W, sW, wd = operand(g, lead + (I, K), kind, rows=128)
    D, sD, d = operand(g, (M, K), kind, E5, size=1e-2)
    dgu, h = fp8.gated_mm_bwd_alloc(D, W, sD, sW, gu, off, flags=flags, want_h=True, status=st)
    assert st.item() == 0
    wd = wd.unsqueeze(0) if not counts else wd
    for r, e in zip(rows, e_of):
        dh, err = product(d[r:r + 1], wd[e])
        g64, u64 = gu[r:r + 1].double().split(I, 1)
        a64, d64, ea, ed = act64(g64, "silu")
        dg, du, h64 = dh * u64 * d64, dh * a64, a64 * u64
        bound = err * (u64 * d64).abs() + (dh.abs() + err) * u64.abs() * ed + 2.0 ** -22 * dg.abs()
        check(dgu[r:r + 1, :I], dg, bound + HALF_BF16 * (dg.abs() + bound), f"row {r}")
        bound = err * a64.abs() + (dh.abs() + err) * ea + 2.0 ** -22 * du.abs()
        check(dgu[r:r + 1, I:], du, bound + HALF_BF16 * (du.abs() + bound), f"row {r}")
        bound = ea * u64.abs() + 2.0 ** -22 * h64.abs()
        check(h[r:r + 1], h64, bound + HALF_BF16 * (h64.abs() + bound), f"row {r}")


class _Chain:
    """A feed-forward's steps on fixed weights, each call's output the next one's input: dense with row scales, or by expert
    with block scales."""

    def __init__(self, fp8, M, experts, seed=5):
        self.fp8, self.M, self.K, self.I = fp8, M, 512, 640
        g = gen(seed)
        self.kind = "block" if experts else "row"
        lead = (experts,) if experts else ()
        self.x = randn(g, M, self.K).to(torch.bfloat16)
        self.w13, self.s13, _ = operand(g, lead + (2 * self.I, self.K), self.kind, rows=128, size=0.06)
        self.w2, self.s2, _ = operand(g, lead + (self.K, self.I), self.kind, rows=128, size=0.06)
        self.w2t, self.s2t, _ = operand(g, lead + (self.I, self.K), self.kind, rows=128, size=0.06)
        self.ends = None
        if experts:
            cuts = sorted(torch.randint(0, M + 1, (experts - 1,), generator=torch.Generator().manual_seed(seed)).tolist())
            self.ends = torch.tensor(cuts + [M], dtype=torch.int32, device="cuda")
        self.out, self.dgu, self.h = (torch.zeros(M, n, dtype=torch.bfloat16, device="cuda") for n in (self.K, 2 * self.I, self.I))

    def step(self, sync=lambda: None):
        f = self.fp8
        if self.kind == "row":
            q, _, inv = f.quantize_alloc(self.x, f.GRAN_ROW, f.DT_E4M3)
            sync()
            h, gu, _, _ = f.gated_mm_alloc(q, self.w13, inv, self.s13, want_gu=True)
            sync()
            hq, _, hi = f.quantize_alloc(h, f.GRAN_ROW, f.DT_E4M3)
            sync()
            f.fp8_scaled_mm(hq, self.w2, hi, self.s2, self.out)
            sync()
            dq, _, di = f.quantize_alloc(self.out, f.GRAN_ROW, f.DT_E5M2)
            flags = 0
        else:
            q, _, inv, _ = f.blk_quantize_alloc(self.x, f.DT_E4M3)
            sync()
            flags = f.MM_BLOCKWISE
            _, gu, hq, hi = f.gated_mm_alloc(q, self.w13, inv, self.s13, self.ends, flags=flags, want_h=False, want_gu=True,
                                             q_dtype=f.DT_E4M3)
            sync()
            f.fp8_grouped_mm(hq, self.w2, self.ends, hi, self.s2, self.out, f.GROUPED_JAGGED_M, flags)
            sync()
            dq, _, di, _ = f.blk_quantize_alloc(self.out, f.DT_E5M2)
        sync()
        f.fp8_gated_mm_bwd(dq, self.w2t, di, self.s2t, gu, self.dgu, self.h, self.ends, flags=flags)
        sync()
        self.x.copy_((self.x + 0.1 * self.out + self.dgu[:, :self.K] + self.h[:, :self.K]).clamp_(-4, 4))
        sync()

    def state(self):
        return [t.clone() for t in (self.x, self.out, self.dgu, self.h)]


CHAINS = [(1, 0), (40, 0), (300, 0), (2600, 0), (1, 8), (48, 24), (700, 12)]


@pytest.mark.parametrize("M,experts", CHAINS)
def test_back_to_back_and_captured(fp8, M, experts):
    """Without a wait between the calls, and captured and replayed, the results are those of a run that synchronizes after
    every call, bit for bit."""
    want, got, graphed = (_Chain(fp8, M, experts) for _ in range(3))
    for _ in range(8):
        want.step(torch.cuda.synchronize)
    for _ in range(8):
        got.step()
    torch.cuda.synchronize()
    assert torch.isfinite(want.x).all() and want.x.abs().amax() > 0
    for a, b in zip(got.state(), want.state()):
        assert torch.equal(a, b)
    start = graphed.x.clone()
    graphed.step()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for _ in range(4):
            graphed.step()
    graphed.x.copy_(start)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(graphed.state(), want.state()):
        assert torch.equal(a, b)


@pytest.mark.parametrize("M,experts", [(3, 0), (300, 0), (40, 16), (500, 8)])
def test_two_at_once(fp8, M, experts):
    """Two threads of calls on two streams, on buffers of their own, one of them of a few rows."""
    sizes = ((M, experts), (40, 0))
    want = [_Chain(fp8, *s, seed=7 + i) for i, s in enumerate(sizes)]
    got = [_Chain(fp8, *s, seed=7 + i) for i, s in enumerate(sizes)]
    torch.cuda.synchronize()
    for c in want:
        for _ in range(10):
            c.step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in got]
    for _ in range(10):
        for c, s in zip(got, streams):
            with torch.cuda.stream(s):
                c.step()
    torch.cuda.synchronize()
    for c, w in zip(got, want):
        for a, b in zip(c.state(), w.state()):
            assert torch.equal(a, b)


@pytest.mark.parametrize("before", ["memset", "copy", "host copy", "join"])
def test_what_comes_before_in_a_capture(fp8, before):
    """Each kernel as the first call behind a memset, a copy or a join of two streams, captured and replayed."""
    g = gen(4)
    for M, counts in ((5, None), (5, [2, 0, 3]), (300, None), (300, [120, 180]), (2304, None)):
        K, I = 512, 256
        lead = (len(counts),) if counts else ()
        off = ends(counts) if counts else None
        for kind in ("row", "block"):
            flags = fp8.MM_BLOCKWISE if kind == "block" else 0
            A, sA, _ = operand(g, (M, K), kind)
            B, sB, _ = operand(g, lead + (2 * I, K), kind, rows=128, size=0.1)
            D, sD, _ = operand(g, (M, K), kind, E5)
            W, sW, _ = operand(g, lead + (I, K), kind, rows=128, size=0.1)
            gu = randn(g, M, 2 * I).to(torch.bfloat16)
            h, dgu = torch.zeros(M, I, dtype=torch.bfloat16, device="cuda"), torch.zeros_like(gu)
            out = torch.zeros(M, I, dtype=torch.bfloat16, device="cuda")
            calls = [(lambda: fp8.fp8_gated_mm(A, B, sA, sB, h=h, offsets=off, flags=flags), A, h),
                     (lambda: fp8.fp8_gated_mm_bwd(D, W, sD, sW, gu, dgu, None, off, flags=flags), gu, dgu)]
            if kind == "block" and counts:
                calls.append((lambda: fp8.fp8_grouped_mm(A, W, off, sA, sW, out, fp8.GROUPED_JAGGED_M, flags), A, out))
            for call, inp, res in calls:
                inp = inp.view(torch.uint8)
                src = inp.clone()
                host = src.cpu().pin_memory()
                if before == "memset":
                    inp.zero_()
                call()
                torch.cuda.synchronize()
                want = res.clone()
                side = torch.cuda.Stream()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    if before == "memset":
                        inp.zero_()
                    elif before == "copy":
                        inp.copy_(src)
                    elif before == "host copy":
                        inp.copy_(host, non_blocking=True)
                    else:
                        side.wait_stream(torch.cuda.current_stream())
                        with torch.cuda.stream(side):
                            inp.copy_(src)
                        torch.cuda.current_stream().wait_stream(side)
                    call()
                inp.fill_(0x38)  # ordinary values, not the call's
                res.fill_(7.0)
                for _ in range(2):
                    graph.replay()
                torch.cuda.synchronize()
                assert torch.equal(res, want), (before, M, counts, kind)
                inp.copy_(src)
