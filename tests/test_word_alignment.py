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

    def saved(gran, name):
        block, s = gran == f.GRAN_BLOCK_1x128, f.Fp8LinearSaved()
        rows = gran == f.GRAN_ROW
        for field, dt, shape in (("x_q", E4M3, (M, K)), ("w_q", E4M3, (N, K)), ("wt_q", E4M3, (K, N)), ("xt_q", E4M3, (K, M)),
                                 ("x_inv", F32, (M, K // 128) if block else (M,) if rows else (1,)),
                                 ("w_inv", F32, (N // 128, K // 128) if block else (N,) if rows else (1,)),
                                 ("wt_inv", F32, (K // 128, N // 128))):
            at = 4096 + (odd if field == name else 0)
            setattr(s, field, f.Fp8Tensor.from_buffer_copy(f._PACK(at, dt, len(shape), *(list(shape) + [0, 0])[:3])))
        keep.append(s)
        return ctypes.byref(s)

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
    # the Linear: the scales that a call writes or reads, of those that it saves
    T, B, R, F8, BF = f.GRAN_TENSOR, f.GRAN_BLOCK_1x128, f.GRAN_ROW, f.WGRAD_FP8, f.WGRAD_BF16
    for backward, gran, wgrad, names in ((False, T, BF, ("x_inv", "w_inv")), (False, R, BF, ("x_inv", "w_inv")),
                                         (False, B, BF, ("x_inv", "w_inv", "wt_inv")), (True, T, F8, ("x_inv", "w_inv")),
                                         (True, T, BF, ("w_inv",)), (True, B, BF, ("wt_inv",))):
        for name in names:
            p = saved(gran, name)
            if backward:
                n = f.fp8_workspace_size(f.OP_LINEAR_BWD, M, K, N, gran, wgrad)
                rc = L.fp8_linear_bwd(out, p, x, d(BF16, N, K), gran, wgrad, d(BF16, M, K), d(BF16, N, K), ws, n, None, None)
            else:
                rc = L.fp8_linear_fwd(x, d(BF16, N, K), gran, 0, out, p, ws, 256, None, None)
            calls.append((f"linear {'backward' if backward else 'forward'} {gran}: {name}", rc))
    return calls


@pytest.mark.parametrize("odd", [1, 2, 3])
def test_between_words(fp8, odd):
    for name, rc in _calls(fp8, odd):
        assert rc == ALIGNMENT, (name, rc)


def test_what_a_linear_does_not_use(fp8):
    """Saved scales that a call neither writes nor reads may be left unset."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are nobody's: for a machine without a device")
    f, M, N, K = fp8, 128, 128, 256
    keep = []

    def d(dt, *shape, ptr=4096):
        keep.append(f.Fp8Tensor.from_buffer_copy(f._PACK(ptr, dt, len(shape), *(list(shape) + [0, 0])[:3])))
        return keep[-1]

    s = f.Fp8LinearSaved()
    s.x_q, s.w_q, s.x_inv, s.w_inv = d(E4M3, M, K), d(E4M3, N, K), d(F32, M), d(F32, N)
    s.xt_inv, s.wt_inv = d(F32, 1, ptr=1), d(F32, 1, ptr=3)
    x, w, y = (ctypes.byref(d(BF16, *t)) for t in ((M, K), (N, K), (M, N)))
    assert f.lib.fp8_linear_fwd(x, w, f.GRAN_ROW, 0, y, ctypes.byref(s), None, 0, None, None) == 6
    s.x_inv, s.w_inv = d(F32, M, ptr=1), d(F32, N, ptr=1)
    n = f.fp8_workspace_size(f.OP_LINEAR_BWD, M, K, N, f.GRAN_ROW, f.WGRAD_BF16)
    assert f.lib.fp8_linear_bwd(y, ctypes.byref(s), x, w, f.GRAN_ROW, f.WGRAD_BF16, x, w, 4096, n, None, None) == 6


def test_any_word_is_taken(fp8):
    """Words that are not at 16 bytes pass the check: without a device, its error is what is left."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are nobody's: for a machine without a device")
    for name, rc in _calls(fp8, 4):
        assert rc == 6, (name, rc)
