"""Calls of several host threads at once, each on a stream and buffers of its own: the same kernel with very different
numbers of experts, whose offsets share a CTA's memory with the ring, so that the calls ask for different amounts of it.
Every call is accepted and its result is that of the call alone, bit for bit."""
import ctypes
import threading

import pytest
import torch

from tests.gated_util import E4, E5, ends, gen, operand, randn

pytestmark = pytest.mark.gpu

CALLS = 8000


@pytest.fixture(scope="module")
def fp8():
    import moe_grouped_gemm_absmax_gb300 as m
    return m


def _at_once(makers):
    """Each maker gives (call, outputs): call(stream handle) -> return code. The descriptors are ready beforehand and ctypes
    lets go of the interpreter's lock, so that the threads are inside the library together."""
    made = [m() for m in makers]
    main = torch.cuda.current_stream().cuda_stream
    want = []
    for call, outs, _ in made:
        assert call(main) == 0
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
        for t in outs:
            t.view(torch.uint8).fill_(0x5A)
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


def _counts(E, M):
    c = [0] * E
    c[0], c[E // 2], c[-1] = M // 2, M // 4, M - M // 2 - M // 4
    return c


def _call(fn, args):
    """args: tensors, None, or plain ints; keeps them and their descriptors alive."""
    keep, packed = [], []
    for a in args:
        if isinstance(a, torch.Tensor):
            import moe_grouped_gemm_absmax_gb300 as m
            keep.append((a, m.desc(a)))
            packed.append(ctypes.byref(keep[-1][1]))
        else:
            packed.append(a)
    return (lambda stream: fn(*packed, None, stream)), keep


def _grouped(fp8, E, M, kind):
    g = gen(E)
    A, sA, _ = operand(g, (M, 256), kind)
    B, sB, _ = operand(g, (E, 256, 256), kind, rows=128)
    out = torch.empty(M, 256, dtype=torch.bfloat16, device="cuda")
    call, keep = _call(fp8.lib.fp8_grouped_mm, (A, B, ends(_counts(E, M)), sA, sB, out, fp8.GROUPED_JAGGED_M,
                                                fp8.MM_BLOCKWISE if kind == "block" else 0))
    return call, [out], keep


def _forward(fp8, E, M, kind):
    g = gen(E)
    A, sA, _ = operand(g, (M, 128), kind)
    B, sB, _ = operand(g, (E, 256, 128), kind, rows=128)
    h, gu = (torch.empty(M, n, dtype=torch.bfloat16, device="cuda") for n in (128, 256))
    call, keep = _call(fp8.lib.fp8_gated_mm, (A, B, ends(_counts(E, M)), sA, sB, fp8.ACT_SILU,
                                              fp8.MM_BLOCKWISE if kind == "block" else 0, h, gu, None, None))
    return call, [h, gu], keep


def _backward(fp8, E, M, kind):
    g = gen(E + 1)
    D, sD, _ = operand(g, (M, 128), kind, E5)
    W, sW, _ = operand(g, (E, 128, 128), kind, rows=128)
    gu = randn(g, M, 256).to(torch.bfloat16)
    dgu = torch.empty_like(gu)
    call, keep = _call(fp8.lib.fp8_gated_mm_bwd, (D, W, ends(_counts(E, M)), sD, sW, fp8.ACT_GELU,
                                                  fp8.MM_BLOCKWISE if kind == "block" else 0, gu, dgu, None))
    return call, [dgu], keep


# rows enough for the tile kernels, on single CTAs and (row scales) on pairs
@pytest.mark.parametrize("M", [132, 2052])
@pytest.mark.parametrize("kind", ["row", "block"])
@pytest.mark.parametrize("op,most", [(_grouped, 2000), (_forward, 1000), (_backward, 1000)])
def test_other_numbers_of_experts(fp8, op, most, kind, M):
    _at_once([lambda E=E: op(fp8, E, M, kind) for E in (4, most, 5, 7)])


def test_weight_gradients(fp8):
    def make(E):
        g = gen(E)
        P = 128 * E
        G, X = randn(g, 16, P).to(E5), randn(g, 16, P).to(E4)
        one = torch.ones(E, 16, device="cuda")
        out = torch.empty(E, 16, 16, dtype=torch.bfloat16, device="cuda")
        call, keep = _call(fp8.lib.fp8_grouped_mm, (G, X, ends([64] * E), one, one, out, fp8.GROUPED_JAGGED_K, 0))
        return call, [out], keep

    _at_once([lambda E=E: make(E) for E in (4, 2000, 5, 7)])


def test_few_rows_and_many(fp8):
    """The few rows' kernel, the tiles' and the backward pass, each in a thread."""
    _at_once([lambda: _forward(fp8, 4, 7, "row"), lambda: _forward(fp8, 1000, 132, "row"),
              lambda: _backward(fp8, 300, 132, "block"), lambda: _grouped(fp8, 2000, 33, "block")])
