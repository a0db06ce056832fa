"""Scales, maxima and offsets are read and written word by word at least: a pointer between words is refused by every
entry point, ahead of any device work (so without a GPU too). The descriptors point at addresses that nothing reads."""
import ctypes

import pytest

ALIGNMENT = 3
BF16, F32, E4M3, E5M2, I32, E8M0 = 1, 2, 3, 4, 5, 6
BLOCK = 8


@pytest.fixture(scope="module")
def fp8():
    import moe_grouped_gemm_absmax_gb300 as m
    return m


def _calls(f, odd):
    """One call of each entry point for each of its tensors of words, that one at an address `odd` off its word."""
    keep = []

    def d(dt, *shape, ptr=4096):
        keep.append(f.Fp8Tensor.from_buffer_copy(f._PACK(ptr, dt, len(shape), *(list(shape) + [0, 0])[:3])))
        return ctypes.byref(keep[-1])

    def w(dt, *shape):
        return d(dt, *shape, ptr=4096 + odd)

    L, M, N, K, E = f.lib, 128, 128, 256, 3
    x, A, B, out = d(BF16, M, K), d(E4M3, M, K), d(E4M3, N, K), d(BF16, M, N)
    inv, off = d(F32, M), d(I32, E)
    ws = 4096
    calls = []
    calls.append(("quantize: scales", L.fp8_quantize(x, 1, E4M3, 1, A, None, w(F32, M), None, None, 0, None, None)))
    P = f.fp8_jagged_padded_rows(M, E)
    n = f.fp8_workspace_size(f.OP_QUANTIZE, E, K, M, f.GRAN_COL)
    calls.append(("quantize: offsets", L.fp8_quantize(x, f.GRAN_COL, E4M3, 2, None, d(E4M3, K, P), d(F32, E, K), w(I32, E), ws, n,
                                                      None, None)))
    calls.append(("from amax: scales", L.fp8_quantize_from_amax(x, f.GRAN_TENSOR, E4M3, 1, A, None, w(F32, 1), d(F32, 1), None, None)))
    calls.append(("from amax: maxima", L.fp8_quantize_from_amax(x, f.GRAN_TENSOR, E4M3, 1, A, None, d(F32, 1), w(F32, 1), None, None)))
    calls.append(("noalloc", L.fp8_quantize_tensor_noalloc(x, E4M3, 1, A, None, w(F32, 1), None)))
    for flags, sA, sB in ((0, (M,), (N,)), (0, (1,), (1,)), (BLOCK, (M, K // 128), (N // 128, K // 128))):
        calls.append(("scaled: sA", L.fp8_scaled_mm(A, B, w(F32, *sA), d(F32, *sB), out, flags, None, None)))
        calls.append(("scaled: sB", L.fp8_scaled_mm(A, B, d(F32, *sA), w(F32, *sB), out, flags, None, None)))
    sb = d(F32, N)
    for i, name in enumerate(("sA", "sB", "row maxima", "column maxima")):
        t = [inv, sb, inv, sb]
        t[i] = w(F32, M)
        calls.append(("amax: " + name, L.fp8_scaled_mm_amax(A, B, t[0], t[1], out, 0, t[2], t[3], None, None)))
    for i, name in enumerate(("sA", "sB", "scales")):
        t = [inv, sb, d(F32, M, 1)]
        t[i] = w(F32, M) if i < 2 else w(F32, M, 1)
        calls.append(("quant: " + name, L.fp8_scaled_mm_quant(A, B, t[0], t[1], 0, f.GRAN_BLOCK_1x128, d(E4M3, M, N), t[2], None, None)))
    W = d(E4M3, E, N, K)
    for flags, sA, sB in ((0, (M,), (E, N)), (BLOCK, (M, K // 128), (E, 1, K // 128))):
        for i, name in enumerate(("offsets", "sA", "sB")):
            t = [off, d(F32, *sA), d(F32, *sB)]
            t[i] = w(I32, E) if i == 0 else w(F32, *(sA if i == 1 else sB))
            calls.append(("grouped: " + name, L.fp8_grouped_mm(A, W, t[0], t[1], t[2], out, 0, flags, None, None)))
    G, X, o3 = d(E5M2, M, 512), d(E4M3, N, 512), d(BF16, E, M, N)
    for i, name in enumerate(("offsets", "sA", "sB")):
        t = [off, d(F32, E, M), d(F32, E, N)]
        t[i] = w(I32, E) if i == 0 else w(F32, E, M)
        calls.append(("grouped by the contraction: " + name, L.fp8_grouped_mm(G, X, t[0], t[1], t[2], o3, 1, 0, None, None)))
    for name in ("x_inv", "w_inv"):
        saved = f.Fp8LinearSaved()
        for field, dt, shape in (("x_q", E4M3, (M, K)), ("w_q", E4M3, (N, K)), ("x_inv", F32, (M,)), ("w_inv", F32, (N,))):
            at = 4096 + (odd if field == name else 0)
            setattr(saved, field, f.Fp8Tensor.from_buffer_copy(f._PACK(at, dt, len(shape), *(list(shape) + [0, 0])[:3])))
        keep.append(saved)
        p = ctypes.byref(saved)
        calls.append(("linear: " + name, L.fp8_linear_fwd(x, d(BF16, N, K), f.GRAN_ROW, 0, out, p, None, 0, None, None)))
        n = f.fp8_workspace_size(f.OP_LINEAR_BWD, M, K, N, f.GRAN_ROW, f.WGRAD_BF16)
        calls.append(("linear backward: " + name, L.fp8_linear_bwd(out, p, x, d(BF16, N, K), f.GRAN_ROW, f.WGRAD_BF16, d(BF16, M, K),
                                                                   d(BF16, N, K), ws, n, None, None)))
    return calls


@pytest.mark.parametrize("odd", [1, 2, 3])
def test_between_words(fp8, odd):
    for name, rc in _calls(fp8, odd):
        assert rc == ALIGNMENT, (name, rc)


def test_any_word_is_taken(fp8):
    """Words that are not at 16 bytes pass the check: without a device, its error is what is left."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are nobody's: for a machine without a device")
    for name, rc in _calls(fp8, 4):
        assert rc == 6, (name, rc)
