"""The gated feed-forward's and the block-scaled grouped product's kernels when a wait runs out: the test hook lets the MMA
issuer wait for what nothing signals, the wait ends after 2 ms, the status word says so, loads in flight land, and the
next call on the same buffers is right, bit for bit."""
import pytest
import torch

from tests.gated_util import E4, E5, ends, gen, operand, randn, status_word

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8():
    import moe_grouped_gemm_absmax_gb300 as m
    return m


def _stalled(fp8, run):
    want, st = run()
    assert st.item() == 0
    old = fp8.fp8_set_wait_limit_ns(2_000_000)  # 2 ms
    fp8.fp8_set_test_stall(True)
    try:
        _, st = run()
    finally:
        fp8.fp8_set_test_stall(False)
        fp8.fp8_set_wait_limit_ns(old)
    assert st.item() & fp8.DEV_TIMEOUT
    got, st = run()
    assert st.item() == 0
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# few rows (one CTA a tile, a cluster), single CTAs, pairs; experts
SIZES = [(3, 512, 13056, None), (40, 2048, 256, None), (20, 512, 256, [7, 0, 13]), (200, 512, 384, None), (2048, 512, 1280, None),
         (300, 256, 640, [129, 0, 171]), (2304, 256, 640, [2300, 0, 4])]


@pytest.mark.parametrize("kind", ["row", "block", "bf16"])
@pytest.mark.parametrize("M,K,I,counts", SIZES)
def test_forward(fp8, M, K, I, counts, kind):
    if kind == "bf16" and counts:
        counts = None
    g = gen(M)
    A, sA, _ = operand(g, (M, K), kind)
    B, sB, _ = operand(g, (len(counts), 2 * I, K) if counts else (2 * I, K), kind, rows=128)
    off = ends(counts) if counts else None

    def run():
        st = status_word()
        out = fp8.gated_mm_alloc(A, B, sA, sB, off, flags=fp8.MM_BLOCKWISE if kind == "block" else 0, want_gu=True,
                                 q_dtype=fp8.DT_E4M3 if kind != "bf16" else None, status=st)
        torch.cuda.synchronize()
        return [t for t in out if t is not None], st

    _stalled(fp8, run)


@pytest.mark.parametrize("kind", ["row", "block", "bf16"])
@pytest.mark.parametrize("M,K,I,counts", SIZES)
def test_backward(fp8, M, K, I, counts, kind):
    if kind == "bf16" and counts:
        counts = None
    g = gen(M + 1)
    A, sA, _ = operand(g, (M, K), kind, E5)
    B, sB, _ = operand(g, (len(counts), I, K) if counts else (I, K), kind, E4, rows=128)
    gu = randn(g, M, 2 * I).bfloat16()
    off = ends(counts) if counts else None

    def run():
        st = status_word()
        out = fp8.gated_mm_bwd_alloc(A, B, sA, sB, gu, off, flags=fp8.MM_BLOCKWISE if kind == "block" else 0, want_h=True,
                                     status=st)
        torch.cuda.synchronize()
        return out, st

    _stalled(fp8, run)


@pytest.mark.parametrize("counts,K,N", [([3, 0, 5], 1024, 640), ([40], 2048, 256), ([100, 0, 300], 512, 1000), ([1900], 256, 2560)])
def test_block_product(fp8, counts, K, N):
    M = sum(counts)
    g = gen(M)
    A, sA, _ = operand(g, (M, K), "block")
    B, sB, _ = operand(g, (len(counts), N, K), "block", rows=128)
    off = ends(counts)

    def run():
        st = status_word()
        out = torch.empty(M, N, device="cuda")
        fp8.fp8_grouped_mm(A, B, off, sA, sB, out, fp8.GROUPED_JAGGED_M, fp8.MM_BLOCKWISE, st)
        torch.cuda.synchronize()
        return [out], st

    _stalled(fp8, run)
