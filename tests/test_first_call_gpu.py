"""A host thread whose first CUDA call is one of the library's: it has no context yet, and the call is taken all the same,
captured calls of another thread beside it included. Its result is that of the same call from the main thread."""
import ctypes
import threading

import pytest
import torch

from tests.gated_util import E4, E5, ends, gen, operand, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8():
    import moe_grouped_gemm_absmax_gb300 as m
    return m


def _calls(f):
    """name -> (function of the library with every argument but the last, the stream, its outputs)."""
    g = gen(3)
    keep = []

    def c(fn, *args):
        packed = []
        for a in args:
            if isinstance(a, torch.Tensor):
                d = f.desc(a)
                keep.append((a, d))
                packed.append(ctypes.byref(d))
            else:
                packed.append(a)
        return lambda stream: fn(*packed, stream)

    new = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    L, B, M, K, N = f.lib, f.MM_BLOCKWISE, 132, 256, 256
    A, sA, _ = operand(g, (M, K), "row")
    W, sW, _ = operand(g, (2, N, K), "row")
    Ab, sAb, _ = operand(g, (M, K), "block")
    Wb, sWb, _ = operand(g, (2, N, K), "block", rows=128)
    D, sD, _ = operand(g, (M, K), "row", E5)
    x, w = randn(g, M, K).to(torch.bfloat16), randn(g, N, K).to(torch.bfloat16)
    gu, off = randn(g, M, 2 * N).to(torch.bfloat16), ends([100, 32])
    calls = {}
    o = new(M, N)
    calls["scaled"] = c(L.fp8_scaled_mm, A, W[0], sA, sW[0], o, 0, None), o
    o = new(M, N)
    calls["bf16"] = c(L.fp8_scaled_mm, x, w, None, None, o, 0, None), o
    o = new(M, N)
    calls["blockwise"] = c(L.fp8_scaled_mm, Ab, Wb[0], sAb, sWb[0], o, B, None), o
    o = new(M, N)
    calls["grouped"] = c(L.fp8_grouped_mm, A, W, off, sA, sW, o, 0, 0, None), o
    o = new(M, N)
    calls["grouped blockwise"] = c(L.fp8_grouped_mm, Ab, Wb, off, sAb, sWb, o, 0, B, None), o
    o = new(32, N)
    calls["few rows"] = c(L.fp8_grouped_mm, Ab[:32], Wb, ends([20, 12]), sAb[:32], sWb, o, 0, B, None), o
    o = new(M, N // 2)
    calls["gated"] = c(L.fp8_gated_mm, A, W, off, sA, sW, 0, 0, o, None, None, None, None), o
    o = new(M, 2 * N)
    calls["gated backward"] = c(L.fp8_gated_mm_bwd, D, W, off, sD, sW, 0, 0, gu, o, None, None), o
    y = randn(g, 256, K).to(torch.bfloat16)
    o, inv = new(256, K, dt=E4), torch.zeros(1, device="cuda")
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    calls["quantize, tensor"] = c(L.fp8_quantize, y, f.GRAN_TENSOR, f.DT_E4M3, 1, o, None, inv, None, ws.data_ptr(), 16, None), o
    ot, invc = new(K, 256, dt=E4), torch.zeros(K, device="cuda")
    n = f.fp8_workspace_size(f.OP_QUANTIZE, 1, K, 256, f.GRAN_COL)
    wc = torch.zeros(n, dtype=torch.uint8, device="cuda")
    calls["quantize, columns"] = c(L.fp8_quantize, y, f.GRAN_COL, f.DT_E4M3, 2, None, ot, invc, None, wc.data_ptr(), n, None), ot
    keep += [ws, wc, inv, invc]
    return calls, keep


def test_first_call_of_a_thread(fp8):
    calls, _keep = _calls(fp8)
    main = torch.cuda.current_stream().cuda_stream
    for name, (call, out) in calls.items():
        assert call(main) == 0, name
        torch.cuda.synchronize()
        want = out.clone()
        out.view(torch.uint8).fill_(0x5A)
        torch.cuda.synchronize()
        codes = []
        t = threading.Thread(target=lambda: codes.append(call(main)))
        t.start()
        t.join()
        assert codes == [0], (name, codes)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.uint8), want.view(torch.uint8)), name


def test_beside_a_capture(fp8):
    """While the main thread captures, a new thread's first call goes to another stream; both give their results."""
    calls, _keep = _calls(fp8)
    (call, out), (other, res) = calls["grouped"], calls["gated"]
    main = torch.cuda.current_stream().cuda_stream
    assert call(main) == 0 and other(main) == 0
    torch.cuda.synchronize()
    want, want_res = out.clone(), res.clone()
    out.zero_(), res.zero_()
    side, graph, codes = torch.cuda.Stream(), torch.cuda.CUDAGraph(), []
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, capture_error_mode="thread_local"):
        assert call(torch.cuda.current_stream().cuda_stream) == 0
        t = threading.Thread(target=lambda: codes.append(other(side.cuda_stream)))
        t.start()
        t.join()
    assert codes == [0]
    torch.cuda.synchronize()
    assert torch.equal(res, want_res) and not out.any()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
