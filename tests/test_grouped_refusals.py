"""The argument checks of the grouped product: each refusal's code, found before any device work, so without a GPU too.
The descriptors point at addresses that nothing reads; a call that every check lets pass would then be launched, so those
have no rows or, without a device, end with the device's error."""
import pytest

INVALID, UNSUPPORTED, ALIGNMENT, DEVICE = 1, 2, 3, 6
BF16, F32, E4M3, E5M2, I32, E8M0 = 1, 2, 3, 4, 5, 6
FAST, A_MN, B_MN, BLOCK = 1, 2, 4, 8
ROWS, CONTRACTION = 0, 1


@pytest.fixture(scope="module")
def fp8():
    import moe_grouped_gemm_absmax_gb300 as m
    return m


def _d(fp8, dt, *shape, ptr=4096):
    return fp8._PACK(ptr, dt, len(shape), *(list(shape) + [0, 0])[:3])


def _call(fp8, scales="row", mode=ROWS, flags=0, M=4, K=256, N=128, E=3, **kw):
    """JAGGED_K: N and M rows of the operands, K padded token columns."""
    d = lambda *a: _d(fp8, *a)  # noqa: E731
    mx = fp8.fp8_mx_scale_bytes
    a = dict(off=d(I32, E), A=d(E4M3, M, K))
    if mode == ROWS:
        P = -(-(M + 127 * E) // 128) * 128
        a.update(B=d(E4M3, E, N, K), out=d(BF16, M, N))
        a.update({"row": dict(sA=d(F32, M), sB=d(F32, E, N)),
                  "block": dict(sA=d(F32, M, K // 128), sB=d(F32, E, -(-N // 128), K // 128)),
                  "mx": dict(sA=d(E8M0, mx(P, K)), sB=d(E8M0, E * mx(N, K)))}[scales])
    else:
        a.update(B=d(E4M3, N, K), out=d(BF16, E, M, N))
        a.update({"row": dict(sA=d(F32, E, M), sB=d(F32, E, N)),
                  "block": dict(sA=d(F32, E, M), sB=d(F32, E, N)),
                  "mx": dict(sA=d(E8M0, mx(M, K)), sB=d(E8M0, mx(N, K)))}[scales])
    a.update(kw)
    p = {k: None if v is None else fp8.Fp8Tensor.from_buffer_copy(v) for k, v in a.items()}
    return fp8.lib.fp8_grouped_mm(p["A"], p["B"], p["off"], p["sA"], p["sB"], p["out"], mode, flags, None, None)


def _taken(fp8, **kw):
    """Every check lets the call pass: without a device its error, with one an empty result."""
    import torch
    if torch.cuda.is_available():
        kw.update({"M": 0})
        return _call(fp8, **kw) == 0
    return _call(fp8, **kw) == DEVICE


@pytest.mark.parametrize("mode", [ROWS, CONTRACTION])
@pytest.mark.parametrize("scales", ["row", "mx"])
def test_flags(fp8, scales, mode):
    """A flag that the call would not follow is refused."""
    for flags in (0, FAST):
        assert _taken(fp8, scales=scales, mode=mode, flags=flags)
    for flags in (A_MN, B_MN, 16, 1 << 20, FAST | A_MN, -1 << 31):
        assert _call(fp8, scales=scales, mode=mode, flags=flags) == UNSUPPORTED
    if scales == "mx" or mode == CONTRACTION:
        for flags in (BLOCK, BLOCK | FAST):
            assert _call(fp8, scales=scales, mode=mode, flags=flags) == UNSUPPORTED


def test_flags_with_block_scales(fp8):
    assert _taken(fp8, scales="block", flags=BLOCK) and _taken(fp8, scales="block", flags=BLOCK | FAST)
    assert _call(fp8, scales="block", flags=BLOCK | A_MN) == UNSUPPORTED
    assert _call(fp8, scales="block", flags=0) == INVALID and _call(fp8, scales="row", flags=BLOCK) == INVALID


def test_shapes_and_types(fp8):
    d = lambda *a, **k: _d(fp8, *a, **k)  # noqa: E731
    for kw in (dict(A=None), dict(B=None), dict(off=None), dict(sA=None), dict(sB=None), dict(out=None), dict(mode=2),
               dict(A=d(BF16, 4, 256)), dict(out=d(E4M3, 4, 128)), dict(out=d(BF16, 4, 129)), dict(B=d(E4M3, 2, 128, 256)),
               dict(B=d(E4M3, 3, 128, 240)), dict(off=d(F32, 3)), dict(off=d(I32, 0)), dict(sA=d(F32, 5)), dict(sB=d(F32, 3)),
               dict(sA=d(E8M0, 4)), dict(sB=d(E8M0, 4)), dict(A=d(E4M3, 4, 256, ptr=0))):
        assert _call(fp8, **kw) == INVALID, kw
    assert _call(fp8, A=d(E5M2, 4, 256), B=d(E5M2, 3, 128, 256)) == UNSUPPORTED
    assert _call(fp8, K=272, scales="block", flags=BLOCK, sA=d(F32, 4, 2), sB=d(F32, 3, 1, 2)) == UNSUPPORTED
    assert _call(fp8, K=264) == ALIGNMENT
    for name, shape in (("A", (E4M3, 4, 256)), ("B", (E4M3, 3, 128, 256)), ("out", (BF16, 4, 128))):
        assert _call(fp8, **{name: d(*shape, ptr=4104)}) == ALIGNMENT
