"""The argument checks of the gated feed-forward and of the block-scaled grouped product: each refusal's code, found
before any device work (so without a GPU, except for the grouped product, whose first check is the device's). The
descriptors point at addresses that nothing reads."""
import pytest

INVALID, UNSUPPORTED, ALIGNMENT, DEVICE = 1, 2, 3, 6
BF16, F32, E4M3, E5M2, I32, E8M0 = 1, 2, 3, 4, 5, 6
BLOCK, B_MN, A_MN = 8, 4, 2


@pytest.fixture(scope="module")
def fp8():
    import moe_grouped_gemm_absmax_gb300 as m
    return m


def _d(fp8, dt, *shape, ptr=4096):
    return fp8._PACK(ptr, dt, len(shape), *(list(shape) + [0, 0])[:3])


def _fwd(fp8, M=4, K=256, I=128, act=0, flags=0, E=0, **kw):
    lead = (E,) if E else ()
    a = dict(A=_d(fp8, E4M3, M, K), B=_d(fp8, E4M3, *lead, 2 * I, K), off=_d(fp8, I32, E) if E else None,
             sA=_d(fp8, F32, M), sB=_d(fp8, F32, *lead, 2 * I), h=_d(fp8, BF16, M, I), gu=_d(fp8, BF16, M, 2 * I),
             q=_d(fp8, E4M3, M, I), inv=_d(fp8, F32, M, max(I // 128, 0)))
    if flags & BLOCK:
        a.update(sA=_d(fp8, F32, M, K // 128), sB=_d(fp8, F32, *lead, 2 * I // 128, K // 128))
    a.update(kw)
    return fp8.lib.fp8_gated_mm(a["A"], a["B"], a["off"], a["sA"], a["sB"], act, flags, a["h"], a["gu"], a["q"], a["inv"],
                                None, None)


def _bwd(fp8, M=4, K=256, I=128, act=0, flags=0, E=0, **kw):
    lead = (E,) if E else ()
    a = dict(A=_d(fp8, E5M2, M, K), B=_d(fp8, E4M3, *lead, I, K), off=_d(fp8, I32, E) if E else None,
             sA=_d(fp8, F32, M), sB=_d(fp8, F32, *lead, I), gu=_d(fp8, BF16, M, 2 * I), dgu=_d(fp8, BF16, M, 2 * I),
             h=_d(fp8, BF16, M, I))
    if flags & BLOCK:
        a.update(sA=_d(fp8, F32, M, K // 128), sB=_d(fp8, F32, *lead, -(-I // 128), K // 128))
    a.update(kw)
    return fp8.lib.fp8_gated_mm_bwd(a["A"], a["B"], a["off"], a["sA"], a["sB"], act, flags, a["gu"], a["dgu"], a["h"], None,
                                    None)


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_operands(fp8, call):
    d = lambda *a, **k: _d(fp8, *a, **k)  # noqa: E731
    per = 2 if call is _fwd else 1
    rows = 128 * per
    assert call(fp8, A=None) == INVALID and call(fp8, B=None) == INVALID and call(fp8, A=d(F32, 4, 256)) == INVALID
    assert call(fp8, A=d(E4M3, 4, 256, ptr=0)) == INVALID and call(fp8, A=d(E4M3, 1024)) == INVALID
    assert call(fp8, B=d(BF16, rows, 256)) == INVALID  # FP8 with bf16
    assert call(fp8, A=d(E5M2, 4, 256), B=d(E5M2, rows, 256)) == UNSUPPORTED
    assert call(fp8, act=2) == INVALID and call(fp8, act=-1) == INVALID
    assert call(fp8, flags=A_MN) == UNSUPPORTED and call(fp8, flags=B_MN) == UNSUPPORTED and call(fp8, flags=32) == UNSUPPORTED
    assert call(fp8, B=d(E4M3, rows, 240)) == INVALID  # another K
    assert call(fp8, B=d(E4M3, 2, rows, 256)) == INVALID  # experts without offsets
    assert call(fp8, A=d(E4M3, 4, 264), B=d(E4M3, rows, 264)) == ALIGNMENT
    assert call(fp8, A=d(E4M3, 4, 0), B=d(E4M3, rows, 0)) == UNSUPPORTED
    assert call(fp8, A=d(E4M3, 4, 256, ptr=4104)) == ALIGNMENT and call(fp8, B=d(E4M3, rows, 256, ptr=4104)) == ALIGNMENT
    assert call(fp8, A=d(E4M3, 1 << 31, 256)) == UNSUPPORTED and call(fp8, B=d(E4M3, 1 << 31, 256)) == UNSUPPORTED
    assert call(fp8, B=d(E4M3, 1 << 40, 256)) == UNSUPPORTED
    assert call(fp8, sA=None) == INVALID and call(fp8, sB=None) == INVALID
    assert call(fp8, sA=d(F32, 5)) == INVALID and call(fp8, sB=d(F32, rows + 1)) == INVALID
    assert call(fp8, sA=d(F32, 4, ptr=4098)) == ALIGNMENT and call(fp8, sB=d(F32, rows, ptr=4098)) == ALIGNMENT
    assert call(fp8, sA=d(E8M0, 1024), sB=d(E8M0, 1024)) == UNSUPPORTED  # MX scales
    assert call(fp8, sA=d(BF16, 4)) == INVALID
    # bf16
    bf = dict(A=d(BF16, 4, 256), B=d(BF16, rows, 256), sA=None, sB=None)
    assert call(fp8, **{**bf, "sA": d(F32, 4)}) == INVALID
    assert call(fp8, **{**bf, "flags": BLOCK}) == UNSUPPORTED
    assert call(fp8, **{**bf, "A": d(BF16, 4, 252), "B": d(BF16, rows, 252)}) == ALIGNMENT
    assert call(fp8, **{**bf, "off": d(I32, 2), "B": d(BF16, 2, rows, 256)}) == UNSUPPORTED
    # experts
    assert call(fp8, E=3, off=d(I32, 2)) == INVALID and call(fp8, E=3, off=d(F32, 3)) == INVALID
    assert call(fp8, E=3, B=d(E4M3, rows, 256)) == INVALID and call(fp8, E=3, sA=d(F32, 1)) == INVALID
    assert call(fp8, E=3, sB=d(F32, 1)) == INVALID and call(fp8, E=3, sB=d(F32, 3, rows + 1)) == INVALID
    assert call(fp8, E=1025) == UNSUPPORTED and call(fp8, E=3, off=d(I32, 0)) == INVALID
    assert call(fp8, E=3, off=d(I32, 3, ptr=4098)) == ALIGNMENT
    # blockwise
    assert call(fp8, flags=BLOCK, K=272) == UNSUPPORTED
    assert call(fp8, flags=BLOCK, sA=d(F32, 4)) == INVALID and call(fp8, flags=BLOCK, sB=d(F32, rows)) == INVALID
    assert call(fp8, flags=BLOCK, E=3, sB=d(F32, rows // 128, 2)) == INVALID


def test_forward_outputs(fp8):
    d = lambda *a, **k: _d(fp8, *a, **k)  # noqa: E731
    assert _fwd(fp8, h=None, gu=None, q=None, inv=None) == INVALID  # nothing asked for
    assert _fwd(fp8, q=None) == INVALID and _fwd(fp8, inv=None) == INVALID
    assert _fwd(fp8, h=d(F32, 4, 128)) == INVALID and _fwd(fp8, h=d(BF16, 4, 256)) == INVALID
    assert _fwd(fp8, gu=d(BF16, 4, 128)) == INVALID and _fwd(fp8, gu=d(BF16, 4, 256, ptr=4104)) == ALIGNMENT
    assert _fwd(fp8, q=d(BF16, 4, 128)) == INVALID and _fwd(fp8, inv=d(F32, 4)) == INVALID
    assert _fwd(fp8, I=136, inv=d(F32, 4, 1)) == UNSUPPORTED  # no whole blocks of 128
    assert _fwd(fp8, B=d(E4M3, 255, 256)) == INVALID and _fwd(fp8, I=132) == ALIGNMENT
    assert _fwd(fp8, flags=BLOCK, I=136, q=None, inv=None) == UNSUPPORTED
    bf = dict(A=d(BF16, 4, 256), B=d(BF16, 256, 256), sA=None, sB=None)
    assert _fwd(fp8, flags=B_MN, **bf) == UNSUPPORTED


def test_backward_outputs(fp8):
    d = lambda *a, **k: _d(fp8, *a, **k)  # noqa: E731
    assert _bwd(fp8, gu=None) == INVALID and _bwd(fp8, dgu=None) == INVALID
    assert _bwd(fp8, gu=d(BF16, 4, 128)) == INVALID and _bwd(fp8, dgu=d(F32, 4, 256)) == INVALID
    assert _bwd(fp8, h=d(BF16, 4, 256)) == INVALID and _bwd(fp8, h=d(BF16, 4, 128, ptr=4104)) == ALIGNMENT
    assert _bwd(fp8, I=132) == ALIGNMENT
    bf = dict(A=d(BF16, 4, 256), sA=None, sB=None, flags=B_MN)
    assert _bwd(fp8, B=d(BF16, 128, 256), **bf) == INVALID  # K and I the other way round
    assert _bwd(fp8, B=d(BF16, 256, 132), I=132, gu=d(BF16, 4, 264), dgu=d(BF16, 4, 264), h=None, **bf) == ALIGNMENT


def test_grouped_product(fp8):
    """On a machine without a device every call says so; with one, the checks."""
    import torch
    d = lambda *a, **k: _d(fp8, *a, **k)  # noqa: E731

    def call(M=4, K=256, N=128, E=3, mode=0, flags=BLOCK, **kw):
        a = dict(A=d(E4M3, M, K), B=d(E4M3, E, N, K), off=d(I32, E), sA=d(F32, M, K // 128),
                 sB=d(F32, E, -(-N // 128), K // 128), out=d(BF16, M, N))
        a.update(kw)
        p = {k: fp8.Fp8Tensor.from_buffer_copy(v) for k, v in a.items()}
        return fp8.lib.fp8_grouped_mm(p["A"], p["B"], p["off"], p["sA"], p["sB"], p["out"], mode, flags, None, None)

    if not torch.cuda.is_available():
        assert call() == DEVICE
        return
    assert call(K=272, sA=d(F32, 4, 2), sB=d(F32, 3, 1, 2)) == UNSUPPORTED
    assert call(sA=d(F32, 4)) == INVALID and call(sB=d(F32, 3, 128)) == INVALID and call(sB=d(F32, 1, 2)) == INVALID
    assert call(flags=0) == INVALID  # block scales where row scales belong
    assert call(M=8, E=2049) == UNSUPPORTED and call(M=300, E=2049) == UNSUPPORTED
    assert call(mode=1, A=d(E4M3, 128, 256), B=d(E4M3, 128, 256), out=d(BF16, 3, 128, 128)) == UNSUPPORTED
