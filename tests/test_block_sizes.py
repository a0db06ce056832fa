"""The workspace sizes of the norm's backward, the router and the experts of a few tokens for any arguments, refused
ones among them: a number, never a crash, so each query runs in a process of its own."""
import os
import subprocess
import sys

import pytest

QUERIES = {
    # widths that are no multiple of 8, below 8, above 16384, past 32 bits
    "rmsnorm_bwd": [(4, H) for H in (-8, 0, 1, 4, 7, 12, 16385, 16392, 1 << 28, 1 << 30, (1 << 31) - 8, 1 << 31, 1 << 40)] +
                   [(T, 256) for T in (-1, 0, 1 << 31, 1 << 62)],
    "moe_route": [(T, E) for T, E in ((4, 0), (4, -1), (4, 1025), (0, 8), (-5, 8), (1 << 31, 8), (1 << 62, 8))],
    "moe_tokens": [(65, 2, 256, 128), (0, 2, 256, 128), (4, 0, 256, 128), (4, 17, 256, 128), (4, 2, 0, 128), (4, 2, 256, -16),
                   (4, 2, 1 << 31, 128), (4, 2, 256, 1 << 40)],
}


@pytest.mark.parametrize("name", QUERIES)
def test_refused_shapes_need_no_workspace(name):
    code = ("import moe_grouped_gemm_absmax_gb300 as m\n"
            f"for a in {QUERIES[name]!r}:\n    print(getattr(m, 'fp8_{name}_workspace_size')(*a))\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.returncode
    assert [int(v) for v in r.stdout.split()] == [0] * len(QUERIES[name])


@pytest.mark.parametrize("H", [8, 16, 2056, 8192, 8200, 12288, 16384])
def test_every_width_that_the_call_takes_has_one(H):
    import moe_grouped_gemm_absmax_gb300 as m
    assert all(m.fp8_rmsnorm_bwd_workspace_size(T, H) >= 4 * H for T in (1, 7, 4096))
