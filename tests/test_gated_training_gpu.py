"""The gated feed-forward's training function step by step: its results are those of the entry points on the same operands,
bit for bit, and each step is held to 64 bits on the values that its own operands stand for, so that only fp32 sums and the
rounding of the result are left (bounds: gated_util.py); each quantization to half a step of its codes. An experts' layer
with the gradients of both weights, by the same measure."""
import pytest
import torch

from tests.gated_util import E4, E5, HALF_BF16, act64, check, check_codes, ends, gen, hidden, product, randn, status_word

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def f():
    import moe_grouped_gemm_absmax_gb300 as m
    return m


def _full(inv, shape):
    """A scale for each value: of rows [R], of 1 x 128 blocks [R, C / 128], of 128 x 128 blocks [R / 128, C / 128]."""
    R, C = shape
    if inv.dim() == 1:
        return inv.double()[:, None].expand(R, C)
    rows = 1 if inv.shape[0] == R else 128
    return inv.double().repeat_interleave(rows, 0)[:R].repeat_interleave(128, 1)


def _values(q, inv, x, what):
    """The values that codes stand for, held to x: half a step of a code, at least half the smallest one's, and 2^-22 for the
    scale's own roundings."""
    s = _full(inv, q.shape)
    v, x = q.double() * s, x.double()
    half, tiny = (2.0 ** -4, 2.0 ** -10) if q.dtype == E4 else (2.0 ** -3, 2.0 ** -17)
    check(v, x, (half + 2.0 ** -22) * x.abs() + tiny * s, what)
    return v


def _rounded(got, ref, err, what):
    check(got, ref, err + HALF_BF16 * (ref.abs() + err), what)


def _backward64(dh, err, gu, act):
    """(value, bound) of dg, du and h from dh and the projections as they are stored."""
    I = gu.shape[1] // 2
    g, u = gu.double().split(I, 1)
    a, d, ea, ed = act64(g, act)
    dg, du, h = dh * u * d, dh * a, a * u
    return ((dg, err * (u * d).abs() + (dh.abs() + err) * u.abs() * ed + 2.0 ** -22 * dg.abs()),
            (du, err * a.abs() + (dh.abs() + err) * ea + 2.0 ** -22 * du.abs()), (h, ea * u.abs() + 2.0 ** -22 * h.abs()))


def _quantizers(f, gran):
    """(activations, weights, weights transposed, flags): each gives codes and scales."""
    if gran == "row":
        def rows(t, dt):
            q, _, inv = f.quantize_alloc(t, f.GRAN_ROW, dt)
            return q, inv

        def columns(t):
            _, q, inv = f.quantize_alloc(t, f.GRAN_COL, f.DT_E4M3)
            return q, inv
        return rows, lambda t: rows(t, f.DT_E4M3), columns, 0

    def blocks(t, dt):
        q, _, inv, _ = f.blk_quantize_alloc(t, dt)
        return q, inv

    def tiles(t):
        q, _, inv, _ = f.blk_quantize_alloc(t, f.DT_E4M3, True)
        return q, inv

    def tiles_t(t):
        _, q, _, inv = f.blk_quantize_alloc(t, f.DT_E4M3, True, f.LAYOUT_COL_MAJOR)
        return q, inv
    return blocks, tiles, tiles_t, f.MM_BLOCKWISE


CASES = [("row", 200, 256, 384), ("row", 65, 144, 272), ("row", 1, 512, 256), ("row", 2100, 256, 640),
         ("block", 200, 256, 384), ("block", 1, 512, 256), ("block", 300, 128, 640)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("gran,M,H,I", CASES)
def test_steps(f, gran, M, H, I, act):
    import moe_grouped_gemm_absmax_gb300.autograd as ag
    g = gen(M + H + I)
    x = (randn(g, M, H) * (0.25 + 4 * torch.rand(M, 1, generator=g, device="cuda"))).to(torch.bfloat16).requires_grad_(True)
    w13 = (randn(g, 2 * I, H) * (0.25 + torch.rand(2 * I, 1, generator=g, device="cuda")) / H ** 0.5).to(torch.bfloat16).requires_grad_(True)
    w2 = (randn(g, H, I) * (0.25 + torch.rand(H, 1, generator=g, device="cuda")) / I ** 0.5).to(torch.bfloat16).requires_grad_(True)
    dy = (randn(g, M, H) * (0.25 + 4 * torch.rand(M, 1, generator=g, device="cuda"))).to(torch.bfloat16)
    code = f.ACT_SILU if act == "silu" else f.ACT_GELU
    y = ag.GatedMLPFunction.apply(x, w13, w2, f.GRAN_ROW if gran == "row" else f.GRAN_BLOCK_1x128, code)
    kept = y.grad_fn.saved_tensors[3]
    y.backward(dy)
    x, w13, w2, gx, g13, g2 = x.detach(), w13.detach(), w2.detach(), x.grad, w13.grad, w2.grad
    rows, weights, transposed, flags = _quantizers(f, gran)

    # forward
    xq, xi = rows(x, f.DT_E4M3)
    wq, wi = weights(w13)
    h, gu, hq, hi = f.gated_mm_alloc(xq, wq, xi, wi, act=code, flags=flags, want_h=gran == "row", want_gu=True,
                                     q_dtype=f.DT_E4M3 if gran == "block" else None)
    assert torch.equal(gu, kept)
    gu64, e_gu = product(_values(xq, xi, x, "x"), _values(wq, wi, w13, "w13"))
    _rounded(gu, gu64, e_gu, "projections")
    h64, e_h = hidden(gu64, e_gu, act)
    if gran == "row":
        _rounded(h, h64, e_h, "hidden layer")
        hq, hi = rows(h, f.DT_E4M3)
        hv = _values(hq, hi, h, "hidden layer's codes")
    else:
        check_codes(hq, hi, h64, e_h, "hidden layer")
        hv = hq.double() * _full(hi, hq.shape)
    wq, wi = weights(w2)
    out = torch.empty_like(x)
    f.fp8_scaled_mm(hq, wq, hi, wi, out, flags)
    assert torch.equal(out, y.detach())
    _rounded(out, *product(hv, _values(wq, wi, w2, "w2")), "y")

    # backward
    dq, di = rows(dy, f.DT_E5M2)
    wq, wi = transposed(w2)
    dgu, h = f.gated_mm_bwd_alloc(dq, wq, di, wi, gu, act=code, flags=flags, want_h=True)
    dh64, e_dh = product(_values(dq, di, dy, "dy"), _values(wq, wi, w2.T, "w2 transposed"))
    for name, got, (ref, err) in zip(("dg", "du", "h"), (dgu[:, :I], dgu[:, I:], h), _backward64(dh64, e_dh, gu, act)):
        _rounded(got, ref, err, name)
    outer = f.MM_A_MN_MAJOR | f.MM_B_MN_MAJOR
    for name, got, a, b in (("dw2", g2, dy, h), ("dw13", g13, dgu, x)):
        w = torch.empty_like(got)
        f.fp8_scaled_mm(a, b, None, None, w, outer)
        assert torch.equal(w, got), name
        _rounded(w, *product(a.double().T, b.double().T), name)
    gq, gi = rows(dgu, f.DT_E5M2)
    wq, wi = transposed(w13)
    f.fp8_scaled_mm(gq, wq, gi, wi, out, flags)
    assert torch.equal(out, gx)
    _rounded(out, *product(_values(gq, gi, dgu, "dgu"), _values(wq, wi, w13.T, "w13 transposed")), "dx")


def _segments(q, inv, counts):
    """Each expert's values from the segment-padded column-major codes [C, P] with scales [E, C]."""
    at, out = 0, []
    for e, n in enumerate(counts):
        out.append(q[:, at:at + n].double() * inv[e].double()[:, None])
        at += -(-n // 128) * 128
    return out


@pytest.mark.parametrize("gran", ["row", "block"])
@pytest.mark.parametrize("counts", [[70, 0, 129, 1], [300, 128, 5, 0], [0, 2, 1900, 260]])
def test_experts_weight_gradients(f, counts, gran):
    """By expert: the projections' gradients from the output's, the input's, and both weights', each against 64 bits."""
    M, E, H, I = sum(counts), len(counts), 256, 384
    g, off, status = gen(M), ends(counts), status_word()
    x, dy = randn(g, M, H).to(torch.bfloat16), randn(g, M, H).to(torch.bfloat16)
    w13, w2 = (randn(g, E, 2 * I, H) / 16).to(torch.bfloat16), (randn(g, E, H, I) / 16).to(torch.bfloat16)
    rows, weights, transposed, flags = _quantizers(f, gran)
    each = lambda fn, w: [fn(w[e].contiguous()) for e in range(E)]  # noqa: E731
    codes = lambda qs: torch.stack([q.view(torch.uint8) for q, _ in qs]).view(E4)  # noqa: E731
    scales = lambda qs: torch.stack([i for _, i in qs])  # noqa: E731
    values = lambda qs, w: torch.stack([_values(q, i, w[e], "weights") for e, (q, i) in enumerate(qs)])  # noqa: E731
    aq, ai = rows(x, f.DT_E4M3)
    q13 = each(weights, w13)
    h, gu, _, _ = f.gated_mm_alloc(aq, codes(q13), ai, scales(q13), off, flags=flags, want_gu=True, status=status)
    gu64, e_gu = product(_values(aq, ai, x, "x"), values(q13, w13), counts)
    _rounded(gu, gu64, e_gu, "projections")
    _rounded(h, *hidden(gu64, e_gu, "silu"), "hidden layer")
    dq, di = rows(dy, f.DT_E5M2)
    q2 = each(transposed, w2)
    dgu, h = f.gated_mm_bwd_alloc(dq, codes(q2), di, scales(q2), gu, off, flags=flags, want_h=True, status=status)
    dh64, e_dh = product(_values(dq, di, dy, "dy"), values(q2, w2.transpose(1, 2)), counts)
    for name, got, (ref, err) in zip(("dg", "du", "h"), (dgu[:, :I], dgu[:, I:], h), _backward64(dh64, e_dh, gu, "silu")):
        _rounded(got, ref, err, name)
    gq, gi = rows(dgu, f.DT_E5M2)
    q13 = each(transposed, w13)
    dx = torch.empty_like(x)
    f.fp8_grouped_mm(gq, codes(q13), off, gi, scales(q13), dx, f.GROUPED_JAGGED_M, flags, status)
    _rounded(dx, *product(_values(gq, gi, dgu, "dgu"), values(q13, w13.transpose(1, 2)), counts), "dx")
    for name, left, right in (("dw2", dy, h), ("dw13", dgu, x)):  # over each expert's rows, in 8 bits
        _, lq, li = f.quantize_alloc(left, f.GRAN_COL, f.DT_E5M2, offsets=off, status=status)
        _, rq, ri = f.quantize_alloc(right, f.GRAN_COL, f.DT_E4M3, offsets=off, status=status)
        dw = torch.full((E, left.shape[1], right.shape[1]), float("nan"), dtype=torch.bfloat16, device="cuda")
        f.fp8_grouped_mm(lq, rq, off, li, ri, dw, f.GROUPED_JAGGED_K, 0, status)
        at = 0
        for e, (a, b) in enumerate(zip(_segments(lq, li, counts), _segments(rq, ri, counts))):
            n = counts[e]
            for v, t, s, half, tiny in ((a, left, li, 2.0 ** -3, 2.0 ** -17), (b, right, ri, 2.0 ** -4, 2.0 ** -10)):
                ref = t[at:at + n].double().T
                if n:
                    check(v, ref, (half + 2.0 ** -22) * ref.abs() + tiny * s[e].double()[:, None], f"{name} operand")
            at += n
            if n == 0:
                assert not dw[e].any() and dw[e].isfinite().all()
            else:
                _rounded(dw[e], *product(a, b), f"{name} of expert {e}")
    assert status.item() == 0
