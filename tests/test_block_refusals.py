"""The argument checks of the norm, the router and the experts of a few tokens: each refusal's code, found before any
device work (so without a GPU). The descriptors point at addresses that nothing reads."""
import pytest

INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 1, 2, 3, 4
BF16, F32, E4M3, E5M2, I32, E8M0 = 1, 2, 3, 4, 5, 6


@pytest.fixture(scope="module")
def fp8():
    import moe_grouped_gemm_absmax_gb300 as m
    return m


def _d(fp8, dt, *shape, ptr=4096):
    return fp8._PACK(ptr, dt, len(shape), *(list(shape) + [0, 0])[:3])


def _norm(fp8, T=4, H=256, eps=1e-6, gran=1, **kw):
    a = dict(x=_d(fp8, BF16, T, H), residual=_d(fp8, BF16, T, H), weight=_d(fp8, BF16, H), h=_d(fp8, BF16, T, H),
             y=None, q=_d(fp8, E4M3, T, H), inv=_d(fp8, F32, T), rstd=None)
    a.update(kw)
    return fp8.lib.fp8_add_rmsnorm(a["x"], a["residual"], a["weight"], eps, gran, a["h"], a["y"], a["q"], a["inv"],
                                   a["rstd"], None)


def test_norm(fp8):
    d = lambda *a, **k: _d(fp8, *a, **k)  # noqa: E731
    assert _norm(fp8, x=None) == INVALID and _norm(fp8, x=d(F32, 4, 256)) == INVALID
    assert _norm(fp8, x=d(BF16, 256)) == INVALID and _norm(fp8, x=d(BF16, 4, 256, ptr=0)) == INVALID
    assert _norm(fp8, x=d(BF16, 4, 252)) == ALIGNMENT and _norm(fp8, x=d(BF16, 4, 256, ptr=4104)) == ALIGNMENT
    assert _norm(fp8, x=d(BF16, 4, 16392)) == UNSUPPORTED and _norm(fp8, x=d(BF16, 1 << 40, 256)) == UNSUPPORTED
    assert _norm(fp8, x=d(BF16, 4, 0)) == UNSUPPORTED
    assert _norm(fp8, weight=d(BF16, 128)) == INVALID and _norm(fp8, weight=d(E4M3, 256)) == INVALID
    assert _norm(fp8, residual=d(BF16, 3, 256)) == INVALID and _norm(fp8, h=d(F32, 4, 256)) == INVALID
    assert _norm(fp8, eps=-1.0) == INVALID and _norm(fp8, eps=float("nan")) == INVALID
    assert _norm(fp8, inv=None) == INVALID and _norm(fp8, q=None) == INVALID
    assert _norm(fp8, q=None, inv=None, h=None) == INVALID  # nothing asked for
    assert _norm(fp8, q=d(BF16, 4, 256)) == INVALID and _norm(fp8, inv=d(F32, 5)) == INVALID
    assert _norm(fp8, gran=0) == UNSUPPORTED and _norm(fp8, gran=2) == UNSUPPORTED and _norm(fp8, gran=5) == UNSUPPORTED
    assert _norm(fp8, gran=4) == INVALID  # row scales where block scales belong
    assert _norm(fp8, gran=3, inv=d(E8M0, 128 * 8 - 1)) == INVALID
    assert _norm(fp8, H=264, gran=4, inv=d(F32, 4, 2)) == UNSUPPORTED
    assert _norm(fp8, rstd=d(F32, 3)) == INVALID and _norm(fp8, rstd=d(F32, 4, ptr=4100)) == ALIGNMENT


def _norm_bwd(fp8, T=4, H=256, ws=4096, ws_bytes=1 << 20, **kw):
    a = dict(dy=_d(fp8, BF16, T, H), h=_d(fp8, BF16, T, H), weight=_d(fp8, BF16, H), rstd=_d(fp8, F32, T), dh=None,
             dx=_d(fp8, BF16, T, H), dw=_d(fp8, F32, H))
    a.update(kw)
    return fp8.lib.fp8_add_rmsnorm_bwd(a["dy"], a["h"], a["weight"], a["rstd"], a["dh"], a["dx"], a["dw"], ws, ws_bytes,
                                       None)


def test_norm_bwd(fp8):
    d = lambda *a, **k: _d(fp8, *a, **k)  # noqa: E731
    need = fp8.fp8_rmsnorm_bwd_workspace_size(4, 256)
    assert need > 0 and fp8.fp8_rmsnorm_bwd_workspace_size(-1, 256) == 0
    assert _norm_bwd(fp8, ws_bytes=need - 1) == WORKSPACE and _norm_bwd(fp8, ws=None) == WORKSPACE
    assert _norm_bwd(fp8, ws=4104) == WORKSPACE
    assert _norm_bwd(fp8, dx=None, dw=None) == INVALID and _norm_bwd(fp8, dw=d(E4M3, 256)) == INVALID
    assert _norm_bwd(fp8, rstd=None) == INVALID and _norm_bwd(fp8, h=d(BF16, 4, 264)) == INVALID
    assert _norm_bwd(fp8, dh=d(BF16, 4, 128)) == INVALID and _norm_bwd(fp8, dy=d(BF16, 4, 260)) == ALIGNMENT


def _route(fp8, T=4, E=32, k=2, score=0, ws=4096, ws_bytes=1 << 20, **kw):
    a = dict(logits=_d(fp8, F32, T, E), bias=None, ids=_d(fp8, I32, T, k), weights=_d(fp8, F32, T, k),
             order=_d(fp8, I32, T * k), pos=_d(fp8, I32, T, k), ends=_d(fp8, I32, E))
    a.update(kw)
    return fp8.lib.fp8_moe_route(a["logits"], a["bias"], score, 1, 1.0, a["ids"], a["weights"], a["order"], a["pos"],
                                 a["ends"], ws, ws_bytes, None, None)


def test_route(fp8):
    d = lambda *a, **k: _d(fp8, *a, **k)  # noqa: E731
    assert _route(fp8, score=2) == INVALID and _route(fp8, logits=d(E4M3, 4, 32)) == INVALID
    assert _route(fp8, k=33) == INVALID and _route(fp8, k=17) == UNSUPPORTED and _route(fp8, E=1025) == UNSUPPORTED
    assert _route(fp8, T=1 << 30) == UNSUPPORTED  # T * k past 32 bits
    assert _route(fp8, ids=d(I32, 5, 2)) == INVALID and _route(fp8, ids=d(F32, 4, 2)) == INVALID
    assert _route(fp8, weights=d(F32, 4, 3)) == INVALID and _route(fp8, bias=d(F32, 31)) == INVALID
    assert _route(fp8, order=None) == INVALID and _route(fp8, ends=None) == INVALID and _route(fp8, pos=None) == INVALID
    assert _route(fp8, order=d(I32, 7)) == INVALID and _route(fp8, logits=d(F32, 4, 32, ptr=4100)) == ALIGNMENT
    need = fp8.fp8_moe_route_workspace_size(4, 32)
    assert need > 0 and _route(fp8, ws_bytes=need - 1) == WORKSPACE and _route(fp8, ws=None) == WORKSPACE


def test_route_bwd(fp8):
    d = lambda *a, **k: _d(fp8, *a, **k)  # noqa: E731
    f = fp8.lib.fp8_moe_route_bwd
    lg, ids, dw = d(F32, 4, 32), d(I32, 4, 2), d(F32, 4, 2)
    assert f(lg, ids, dw, 0, 0, 1.0, d(BF16, 4, 32), None, None) == INVALID  # another type than the logits'
    assert f(lg, ids, d(F32, 4, 3), 0, 0, 1.0, d(F32, 4, 32), None, None) == INVALID
    assert f(lg, ids, dw, 5, 0, 1.0, d(F32, 4, 32), None, None) == INVALID
    assert f(lg, ids, dw, 0, 0, 1.0, d(F32, 4, 32, ptr=4100), None, None) == ALIGNMENT


def _moe(fp8, T=4, k=2, E=8, H=256, I=128, ws=4096, ws_bytes=1 << 40, **kw):
    a = dict(x=_d(fp8, BF16, T, H), ids=_d(fp8, I32, T, k), weights=_d(fp8, F32, T, k), w13=_d(fp8, E4M3, E, 2 * I, H),
             s13=_d(fp8, F32, E, 2 * I), w2=_d(fp8, E4M3, E, H, I), s2=_d(fp8, F32, E, H), out=_d(fp8, BF16, T, H))
    a.update(kw)
    return fp8.lib.fp8_moe_tokens(a["x"], a["ids"], a["weights"], a["w13"], a["s13"], a["w2"], a["s2"], a["out"], ws,
                                  ws_bytes, None, None)


def test_moe_tokens(fp8):
    d = lambda *a, **k: _d(fp8, *a, **k)  # noqa: E731
    assert _moe(fp8, T=65) == UNSUPPORTED and _moe(fp8, k=17) == UNSUPPORTED and _moe(fp8, E=1025) == UNSUPPORTED
    assert _moe(fp8, H=264) == ALIGNMENT and _moe(fp8, I=136) == ALIGNMENT and _moe(fp8, H=65552) == UNSUPPORTED
    assert _moe(fp8, H=0) == UNSUPPORTED and _moe(fp8, I=0) == UNSUPPORTED and _moe(fp8, E=0) == INVALID
    assert _moe(fp8, w13=d(E5M2, 8, 256, 256)) == INVALID and _moe(fp8, w13=d(E4M3, 8, 255, 256)) == INVALID
    assert _moe(fp8, w2=d(E4M3, 8, 256, 144)) == INVALID and _moe(fp8, s13=d(F32, 8, 128)) == INVALID
    assert _moe(fp8, s2=d(F32, 7, 256)) == INVALID and _moe(fp8, out=d(F32, 4, 256)) == INVALID
    assert _moe(fp8, ids=d(I32, 3, 2)) == INVALID and _moe(fp8, weights=d(F32, 4, 3)) == INVALID
    assert _moe(fp8, x=d(BF16, 4, 256, ptr=4104)) == ALIGNMENT
    need = fp8.fp8_moe_tokens_workspace_size(4, 2, 256, 128)
    assert need > 0 and _moe(fp8, ws_bytes=need - 1) == WORKSPACE and _moe(fp8, ws=None) == WORKSPACE
    assert fp8.fp8_moe_tokens_workspace_size(65, 2, 256, 128) == 0


def test_workspace_for_many_serves_fewer(fp8):
    """A workspace sized for the most tokens is large enough for any smaller number of them."""
    counts = sorted({1, 2, 8, 16, 17, 32, 33, 63, 64, 65, 100, 1216, 1217, 1218, 2432, 2433, 5000, 16384, 10 ** 6, 10 ** 7, 10 ** 8})
    for E in (1, 8, 32, 33, 256, 257, 1024):
        sizes = [fp8.fp8_moe_route_workspace_size(T, E) for T in counts]
        assert sizes == sorted(sizes) and sizes[0] > 0
    for H in (8, 264, 2056, 4096, 7168, 8200, 12296, 16384):
        sizes = [fp8.fp8_rmsnorm_bwd_workspace_size(T, H) for T in counts]
        assert sizes == sorted(sizes) and sizes[0] > 0
    for k, H, I in ((1, 512, 256), (8, 7168, 2048), (16, 1040, 528)):
        sizes = [fp8.fp8_moe_tokens_workspace_size(T, k, H, I) for T in range(1, 65)]
        assert sizes == sorted(sizes) and sizes[0] > 0


def test_binding_refuses_strided_tensors(fp8):
    import torch
    x = torch.zeros(8, 512, dtype=torch.bfloat16)[:, ::2]
    with pytest.raises(ValueError):
        fp8.fp8_add_rmsnorm(x, torch.zeros(256), 1e-6, y=x)
    with pytest.raises(ValueError):
        fp8.fp8_add_rmsnorm(torch.zeros(1, 1, 1, 8, dtype=torch.bfloat16), torch.zeros(8), 1e-6)
