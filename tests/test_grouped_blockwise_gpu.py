"""The experts' products with a scale for each block of 128 (grouped GEMM, FP8_MM_BLOCKWISE) against 64 bits (bounds:
gated_util.py): ragged and empty experts, few and many rows, odd widths, both formats and outputs."""
import pytest
import torch

from tests.gated_util import E4, E5, HALF_BF16, check, ends, gen, operand, product, status_word

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8():
    import moe_grouped_gemm_absmax_gb300 as m
    return m


FEW = [([0, 0, 1], 7168, 128), ([16], 2048, 520), ([1] * 17, 1024, 128), ([33], 4096, 264), ([0, 40, 0, 24], 512, 1000),
       ([64], 384, 7168), ([2, 0] * 16, 1152, 384), ([0] * 2000 + [3], 640, 136)]
CASES = FEW + [([1900], 256, 2560), ([100] * 9, 512, 1300), ([1], 128, 8), ([0, 1, 0], 256, 128), ([8] * 1, 2048, 7168), ([3, 0, 0, 5], 384, 200), ([1] * 9, 1024, 520),
         ([17, 33, 0, 64, 65], 512, 264), ([129, 0, 171], 640, 1000), ([0, 0, 0, 700], 256, 129 * 8),
         ([256, 0, 1, 700, 1300, 47, 0], 256, 640), ([1, 2, 4000], 384, 384), ([2] * 300, 128, 136), ([64, 64], 7168, 24)]


@pytest.mark.parametrize("out_dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("a_dt", [E4, E5])
@pytest.mark.parametrize("counts,K,N", CASES)
def test_product(fp8, counts, K, N, a_dt, out_dt):
    M = sum(counts)
    g = gen(M + K + N)
    A, sA, a = operand(g, (M, K), "block", a_dt)
    B, sB, b = operand(g, (len(counts), N, K), "block", E4, rows=128)
    ref, err = product(a, b, counts)
    out = torch.full((M, N), float("nan"), dtype=out_dt, device="cuda")
    st = status_word()
    fp8.fp8_grouped_mm(A, B, ends(counts), sA, sB, out, fp8.GROUPED_JAGGED_M, fp8.MM_BLOCKWISE, st)
    assert st.item() == 0
    check(out, ref, err + (HALF_BF16 * (ref.abs() + err) if out_dt == torch.bfloat16 else 0.0))


def test_odd_width(fp8):
    """A width whose rows are not whole 16-byte words."""
    counts, K, N = [5, 0, 140], 256, 131
    g = gen(5)
    A, sA, a = operand(g, (145, K), "block")
    B, sB, b = operand(g, (3, N, K), "block", rows=128)
    ref, err = product(a, b, counts)
    for dt in (torch.bfloat16, torch.float32):
        out = torch.full((145, N), float("nan"), dtype=dt, device="cuda")
        fp8.fp8_grouped_mm(A, B, ends(counts), sA, sB, out, fp8.GROUPED_JAGGED_M, fp8.MM_BLOCKWISE)
        check(out, ref, err + HALF_BF16 * (ref.abs() + err))


def test_equals_the_dense_product(fp8):
    """One expert with all rows: the dense blockwise GEMM's values, within both sums' errors."""
    M, K, N = 300, 768, 512
    g = gen(8)
    A, sA, a = operand(g, (M, K), "block")
    B, sB, b = operand(g, (1, N, K), "block", rows=128)
    _, err = product(a, b[0])
    dense, grouped = (torch.empty(M, N, device="cuda") for _ in range(2))
    fp8.fp8_scaled_mm(A, B[0], sA, sB[0], dense, fp8.MM_BLOCKWISE)
    fp8.fp8_grouped_mm(A, B, ends([M]), sA, sB, grouped, fp8.GROUPED_JAGGED_M, fp8.MM_BLOCKWISE)
    assert ((dense.double() - grouped.double()).abs() <= 2 * err).all()


def test_not_finite_stays_in_its_row(fp8):
    for M, counts in ((9, [4, 5]), (400, [399, 1])):
        K, N = 256, 256
        g = gen(6)
        A, sA, _ = operand(g, (M, K), "block")
        B, sB, _ = operand(g, (2, N, K), "block", rows=128)
        A2, sA2 = A.clone(), sA.clone()
        A2[2, 3] = float("nan")
        sA2[5, 1] = float("inf")
        run = lambda x, s: _call(fp8, x, B, s, sB, counts, N)  # noqa: E731
        o, o2 = run(A, sA), run(A2, sA2)
        keep = torch.ones(M, dtype=torch.bool, device="cuda")
        keep[2] = keep[5] = False
        assert torch.equal(o[keep], o2[keep]) and o2[2].isnan().all() and not o2[5].isfinite().any()


def _call(fp8, A, B, sA, sB, counts, N):
    out = torch.full((A.shape[0], N), float("nan"), device="cuda")
    fp8.fp8_grouped_mm(A, B, ends(counts), sA, sB, out, fp8.GROUPED_JAGGED_M, fp8.MM_BLOCKWISE)
    return out


def test_no_rows(fp8):
    B = torch.zeros(2, 128, 128, dtype=E4, device="cuda")
    out = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    fp8.fp8_grouped_mm(torch.zeros(0, 128, dtype=E4, device="cuda"), B, ends([0, 0]), torch.zeros(0, 1, device="cuda"),
                       torch.ones(2, 1, 1, device="cuda"), out, fp8.GROUPED_JAGGED_M, fp8.MM_BLOCKWISE)
    torch.cuda.synchronize()


@pytest.mark.parametrize("M", [8, 3000])
def test_bad_offsets(fp8, M):
    g = gen(7)
    A, sA, _ = operand(g, (M, 128), "block")
    B, sB, _ = operand(g, (2, 128, 128), "block", rows=128)
    for bad in ([M + 1, M], [1, M - 1], [0, M + 5], [-3, M]):
        out = torch.full((M, 128), 7.0, device="cuda")
        st = status_word()
        fp8.fp8_grouped_mm(A, B, torch.tensor(bad, dtype=torch.int32, device="cuda"), sA, sB, out, fp8.GROUPED_JAGGED_M,
                           fp8.MM_BLOCKWISE, st)
        assert st.item() == fp8.DEV_BAD_OFFSETS and (out == 7).all(), bad


def test_same_bits_on_every_run_and_in_a_graph(fp8):
    counts = [3, 0, 29, 1]
    g = gen(13)
    A, sA, _ = operand(g, (33, 1024), "block")
    B, sB, _ = operand(g, (4, 640, 1024), "block", rows=128)
    off = ends(counts)
    first = _call(fp8, A, B, sA, sB, counts, 640)
    out = torch.zeros_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp8.fp8_grouped_mm(A, B, off, sA, sB, out, fp8.GROUPED_JAGGED_M, fp8.MM_BLOCKWISE)
    for _ in range(20):
        out.zero_()
        graph.replay()
        assert torch.equal(out, first)
