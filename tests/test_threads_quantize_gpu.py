"""The column-wise quantize from several host threads at once, on streams and buffers of their own, by segments of very
different numbers: the segments' tables share a CTA's memory with its rings. Every call is accepted and its codes and
scales are those of the call alone, bit for bit."""
import ctypes
import threading

import pytest
import torch

from tests.gated_util import E4, E5, ends, gen, randn

pytestmark = pytest.mark.gpu

CALLS = 4000


def _make(f, E, dt):
    R, C = 256, 128
    x = randn(gen(E), R, C).to(torch.bfloat16)
    off = ends([R // 2] + [0] * (E - 2) + [R // 2])
    P = f.fp8_jagged_padded_rows(R, E)
    out, inv = torch.zeros(C, P, dtype=dt, device="cuda"), torch.zeros(E, C, device="cuda")
    n = f.fp8_workspace_size(f.OP_QUANTIZE, E, C, R, f.GRAN_COL)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    keep = [(t, f.desc(t)) for t in (x, out, inv, off)] + [ws]
    p = [ctypes.byref(d) for _, d in keep[:4]]
    fmt = f.DT_E4M3 if dt == E4 else f.DT_E5M2
    return lambda s: f.lib.fp8_quantize(p[0], f.GRAN_COL, fmt, 2, None, p[1], p[2], p[3], ws.data_ptr(), n, None, s), (out, inv), keep


@pytest.mark.parametrize("dt", [E4, E5])
def test_other_numbers_of_segments(dt):
    import moe_grouped_gemm_absmax_gb300 as f
    made = [_make(f, E, dt) for E in (4, 1000, 5, 7)]
    want = []
    for call, outs, _ in made:
        assert call(torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
        for t in outs:
            t.view(torch.uint8).zero_()  # as before the call: what lies behind the last segment is left as it was
    torch.cuda.synchronize()
    gate, codes = threading.Barrier(len(made)), [None] * len(made)

    def work(i, call):
        s = torch.cuda.Stream()
        handle, seen = s.cuda_stream, {}
        torch.cuda.synchronize()
        gate.wait()
        for j in range(CALLS):
            rc = call(handle)
            if rc:
                seen[rc] = seen.get(rc, 0) + 1
            if j % 250 == 249:
                s.synchronize()
        s.synchronize()
        codes[i] = seen

    threads = [threading.Thread(target=work, args=(i, m[0])) for i, m in enumerate(made)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert codes == [{}] * len(made), codes  # code: how many calls
    torch.cuda.synchronize()
    for (_, outs, _), w in zip(made, want):
        for a, b in zip(outs, w):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
