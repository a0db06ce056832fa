"""The score argument of the router with the bias on the score. (No call here gets past the checks: a missing workspace is
what an accepted score is refused for.)"""
from tests.test_block_refusals import F32, I32, INVALID, WORKSPACE, _d, _route, fp8  # noqa: F401


def test_score_and_flag(fp8):  # noqa: F811
    assert fp8.SCORE_BIASED == 16
    for score in (0, 1, 16, 17):
        assert _route(fp8, score=score, ws=None) == WORKSPACE
    for score in (2, 4, 8, 15, 18, 19, 32, 48, -1, -16, 1 << 30):
        assert _route(fp8, score=score, ws=None) == INVALID
        assert fp8.lib.fp8_moe_route_bwd(_d(fp8, F32, 4, 32), _d(fp8, I32, 4, 2), _d(fp8, F32, 4, 2), score, 0, 1.0,
                                         _d(fp8, F32, 4, 32), None, None) == INVALID
