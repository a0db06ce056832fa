"""The experts of a few tokens against the formula in 64 bits. The kernels hold the activations to
2^-20 of their row's largest value or better, the hidden layer to 2^-12 of its value and 2^-20 of its
row's largest, sums are fp32 in any order ((n + 64) u of the sum of magnitudes, u = 2^-24), the output
is rounded once to bf16 (2^-8), and a result below fp32's normal range (2^-126) may be zero. The bound follows each through silu (slope below 1.1) and the products."""
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def fp8():
    import moe_grouped_gemm_absmax_gb300 as m
    return m


def _layer(E, H, I, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def quantized(n, k):
        w = 0.05 * torch.randn(E, n, k, generator=g, device="cuda")
        s = w.abs().amax(2) / 448
        return (w / s[..., None]).to(torch.float8_e4m3fn), s

    return (*quantized(2 * I, H), *quantized(H, I)), g


def _tokens(g, T, H, E, k):
    x = torch.randn(T, H, generator=g, device="cuda")
    x[:, torch.randint(0, H, (max(1, H // 100),), generator=g, device="cuda")] *= 50
    x *= torch.exp2(torch.randint(-12, 4, (T, 1), generator=g, device="cuda").float())
    ids = torch.stack([torch.randperm(E, generator=g, device="cuda")[:k] for _ in range(T)]).int() if T else \
        torch.empty(0, k, dtype=torch.int32, device="cuda")
    return x.bfloat16(), ids.contiguous(), torch.randn(T, k, generator=g, device="cuda")


def _reference(x, ids, wt, w13, s13, w2, s2):
    """(out, bound) in 64 bits, expert by expert."""
    T, H = x.shape
    I = w2.shape[2]
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    err = torch.zeros_like(out)
    for e in range(w13.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if not len(t):
            continue
        a13 = w13[e].double() * s13[e].double()[:, None]
        a2 = w2[e].double() * s2[e].double()[:, None]
        xt = x[t].double()
        gu = xt @ a13.T
        mag = xt.abs() @ a13.abs().T
        d = (H + 64) * U * mag + 2.0 ** -20 * xt.abs().amax(1, keepdim=True) * a13.abs().sum(1)
        g, u = gu[:, :I], gu[:, I:]
        a = torch.nn.functional.silu(g) * u
        da = 1.1 * d[:, :I] * (u.abs() + d[:, I:]) + torch.nn.functional.silu(g).abs() * d[:, I:] + 16 * U * a.abs()
        da = da + 2.0 ** -12 * a.abs() + 2.0 ** -20 * a.abs().amax(1, keepdim=True)
        w = wt[t, j].double()[:, None]
        out.index_add_(0, t, w * (a @ a2.T))
        err.index_add_(0, t, w.abs() * (da @ a2.abs().T + (I + 64) * U * (a.abs() @ a2.abs().T)))
    return out, err + 16 * U * out.abs() + 2.0 ** -8 * (out.abs() + err) + 2.0 ** -126


def _check(fp8, x, ids, wt, layer):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = fp8.moe_tokens_alloc(x, ids, wt, *layer, status=st)
    assert int(st) == 0
    ref, bound = _reference(x, ids, wt, *layer)
    assert ((out.double() - ref).abs() <= bound).all(), float(((out.double() - ref).abs() / bound.clamp_min(1e-300)).max())
    return out


@pytest.mark.parametrize("T,E,k,H,I", [
    (1, 1, 1, 16, 16), (1, 8, 2, 1040, 528), (2, 4, 4, 48, 112), (3, 5, 1, 128, 64), (5, 16, 3, 272, 1040),
    (7, 6, 2, 2048, 16), (8, 3, 3, 16, 2048), (9, 32, 8, 512, 256), (16, 40, 4, 1024, 384), (17, 2, 2, 656, 144),
    (33, 8, 2, 400, 720), (64, 64, 8, 256, 128), (64, 3, 2, 1024, 1024), (1, 256, 8, 2048, 512)])
def test_sizes(fp8, T, E, k, H, I):
    layer, g = _layer(E, H, I, T + H)
    _check(fp8, *_tokens(g, T, H, E, k), layer)


def test_wide_layer(fp8):
    """Rows of 7168 and 2048 codes, a batch whose tokens share experts."""
    layer, g = _layer(12, 7168, 2048, 4)
    _check(fp8, *_tokens(g, 21, 7168, 12, 8), layer)


def test_every_token_to_one_expert(fp8):
    for T in (8, 12, 64):
        layer, g = _layer(4, 528, 272, T)
        x, ids, wt = _tokens(g, T, 528, 4, 1)
        ids.fill_(2)
        _check(fp8, x, ids, wt, layer)


def test_unused_slots(fp8):
    """-1 slots: their weights are not read, a token with none used gives zeros; an expert named twice by a token counts
    twice; no slot used at all."""
    layer, g = _layer(6, 272, 144, 1)
    x, ids, wt = _tokens(g, 9, 272, 6, 4)
    ids[0, 1] = -1
    ids[3] = -1
    ids[5, :3] = -1
    ids[6] = 4
    wt[ids < 0] = float("nan")
    out = _check(fp8, x, ids, torch.where(ids < 0, 0.0, wt), layer)
    assert torch.equal(fp8.moe_tokens_alloc(x, ids, wt, *layer), out) and not out[3].any()
    ids.fill_(-1)
    assert not fp8.moe_tokens_alloc(x, ids, wt, *layer).any()


def test_bad_ids_set_the_status(fp8):
    layer, g = _layer(4, 128, 64, 2)
    x, ids, wt = _tokens(g, 3, 128, 4, 2)
    used = ids.clone()
    ids[1, 0], used[1, 0] = 4, -1
    ids[2, 1], used[2, 1] = -2, -1
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = fp8.moe_tokens_alloc(x, ids, wt, *layer, status=st)
    assert int(st) == fp8.DEV_BAD_IDS
    assert torch.equal(out, fp8.moe_tokens_alloc(x, used, wt, *layer))


def test_nan_stays_where_it_belongs(fp8):
    """A NaN or an infinity in a token reaches that token only; a NaN code in an expert reaches its tokens only, and in
    the last columns of a row (a width that is no multiple of 128) not the next row."""
    H, I = 272, 144
    layer, g = _layer(5, H, I, 3)
    x, ids, wt = _tokens(g, 6, H, 5, 2)
    ids[:] = torch.tensor([[0, 1], [1, 2], [2, 3], [3, 4], [4, 0], [0, 2]], dtype=torch.int32)
    clean = _check(fp8, x, ids, wt, layer)
    y = x.clone()
    y[2, 5] = float("nan")
    y[4, 7] = float("inf")
    out = fp8.moe_tokens_alloc(y, ids, wt, *layer)
    assert out[2].isnan().all() and not torch.isfinite(out[4].float()).any()
    assert all(torch.equal(out[t], clean[t]) for t in (0, 1, 3, 5))
    w13, s13, w2, s2 = (t.clone() for t in layer)
    w2.view(torch.uint8)[3, 10, I - 1] = 0x7F  # NaN in row 10 of expert 3's last projection
    out = fp8.moe_tokens_alloc(x, ids, wt, w13, s13, w2, s2)
    for t in range(6):
        bad = out[t].isnan()
        assert bad.tolist() == [t in (2, 3) and n == 10 for n in range(H)]
    w13.view(torch.uint8)[1, 2 * I - 1, H - 1] = 0x7F  # the last row of expert 1: before expert 2's first row
    w2.copy_(layer[2])
    out = fp8.moe_tokens_alloc(x, ids, wt, w13, s13, w2, s2)
    assert out[:2].isnan().all() and all(torch.equal(out[t], clean[t]) for t in range(2, 6))


def test_zero_and_extreme_rows(fp8):
    layer, g = _layer(3, 272, 144, 5)
    x, ids, wt = _tokens(g, 4, 272, 3, 2)
    x[0] = 0
    x[1] = x[1].float().div(x[1].float().abs().max()).mul(1e-30).bfloat16()
    x[2] = x[2].float().div(x[2].float().abs().max()).mul(1e12).bfloat16()
    out = _check(fp8, x, ids, wt, layer)
    assert not out[0].any()


def test_same_bits_streams_graph(fp8):
    layer, g = _layer(16, 1040, 528, 6)
    x, ids, wt = _tokens(g, 11, 1040, 16, 4)
    want = fp8.moe_tokens_alloc(x, ids, wt, *layer)
    for _ in range(3):
        assert torch.equal(fp8.moe_tokens_alloc(x, ids, wt, *layer), want)
    ws = fp8.moe_tokens_workspace(11, 4, 1040, 528, "cuda")
    ws.fill_(0xFF)  # the workspace needs no particular contents
    out = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fp8.fp8_moe_tokens(x, ids, wt, *layer, out, ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)
    out.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp8.fp8_moe_tokens(x, ids, wt, *layer, out, ws)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_no_tokens(fp8):
    layer, g = _layer(2, 64, 32, 7)
    out = fp8.moe_tokens_alloc(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"),
                               torch.empty(0, 2, dtype=torch.int32, device="cuda"), torch.empty(0, 2, device="cuda"), *layer)
    assert out.shape == (0, 64)


@pytest.mark.parametrize("T,E,k,H,I", [(1, 4, 2, 256, 128), (20, 8, 4, 2048, 1024)])
def test_wait_limit_expiry_reports_timeout_and_context_survives(fp8, T, E, k, H, I):
    """The MMA issuer waits on a barrier that nothing signals; the wait runs out, the kernel reports it, drains and
    returns, and the next call is right."""
    layer, g = _layer(E, H, I, 8)
    x, ids, wt = _tokens(g, T, H, E, k)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    old = fp8.fp8_set_wait_limit_ns(2_000_000)  # 2 ms
    fp8.fp8_set_test_stall(True)
    try:
        fp8.moe_tokens_alloc(x, ids, wt, *layer, status=st)
        torch.cuda.synchronize()
    finally:
        fp8.fp8_set_test_stall(False)
        fp8.fp8_set_wait_limit_ns(old)
    assert int(st) & fp8.DEV_TIMEOUT
    _check(fp8, x, ids, wt, layer)


@pytest.mark.parametrize("T,E,k,H,I", [(64, 1024, 16, 48, 32), (40, 1000, 16, 272, 48), (3, 1024, 16, 144, 64), (33, 2, 1, 256, 128),
                                       (9, 300, 5, 1040, 272)])
def test_many_experts_and_slots(fp8, T, E, k, H, I):
    """The counting of slots by expert at its limits, and a token's unused slots in between."""
    layer, g = _layer(E, H, I, T * E)
    x, ids, wt = _tokens(g, T, H, E, k)
    _check(fp8, x, ids, wt, layer)
    ids[torch.rand(T, k, generator=g, device="cuda") < 0.3] = -1
    _check(fp8, x, ids, wt, layer)


def test_one_expert_takes_every_slot(fp8):
    """64 tokens that name one expert 16 times each: 1024 slots, in entries of 40."""
    layer, g = _layer(3, 272, 144, 9)
    x, ids, wt = _tokens(g, 64, 272, 3, 1)
    _check(fp8, x, torch.full((64, 16), 1, dtype=torch.int32, device="cuda"), torch.randn(64, 16, generator=g, device="cuda"),
           layer)
