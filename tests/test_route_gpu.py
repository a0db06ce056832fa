"""The router against a plain implementation: the choice is compared exactly (it is a comparison of fp32
sums that both sides form with one rounding), the weights and gradients against 64 bits. u = 2^-24.
Bounds: exp is good to 2 ulp, a row's sum of E positive terms is a chain of E / 32 + 5, the rest a few
roundings: 64 u relative for E <= 1024. A gradient's terms of either sign add up: 64 u of their sum."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def fp8():
    import moe_grouped_gemm_absmax_gb300 as m
    return m


def _choose(logits, bias, k):
    """ids by a stable sort of each row, on the host."""
    sel = logits.float().cpu().numpy()
    if bias is not None:
        sel = sel + bias.cpu().numpy()[None]
    sel = np.where(np.isnan(sel), -np.inf, sel)
    order = np.argsort(-sel, axis=1, kind="stable")[:, :k]
    ok = np.take_along_axis(sel, order, 1) > -np.inf
    return np.where(ok, order, -1)


def _weights(logits, ids, softmax, renorm, scale):
    """64-bit weights of the ids given, differentiable."""
    taken = ids >= 0
    at = ids.clamp_min(0).long()
    if softmax and renorm:
        v = torch.softmax(torch.where(taken, logits.gather(1, at), -torch.inf), 1)
    else:
        v = (torch.softmax(logits, 1) if softmax else torch.sigmoid(logits)).gather(1, at)
        if renorm:
            z = torch.where(taken, v, 0.0).sum(1, keepdim=True)
            v = v / (z + 1e-20)
    return torch.where(taken, scale * v, 0.0)


def _check_table(ids, order, pos, ends, E):
    ids, order, pos, ends = (t.cpu().numpy() for t in (ids, order, pos, ends))
    flat = ids.ravel()
    want = np.concatenate([np.flatnonzero(flat == e) for e in range(E)])
    counts = np.array([(flat == e).sum() for e in range(E)])
    assert np.array_equal(ends, np.cumsum(counts))
    assert np.array_equal(order[:want.size], want) and (order[want.size:] == -1).all()
    place = np.full(flat.size, -1)
    place[want] = np.arange(want.size)
    assert np.array_equal(pos.ravel(), place)


def _run(fp8, logits, k, bias=None, softmax=True, renorm=True, scale=1.0):
    score = fp8.SCORE_SOFTMAX if softmax else fp8.SCORE_SIGMOID
    ids, w, order, pos, ends = fp8.moe_route_alloc(logits, k, bias, score, renorm, scale)
    want = _choose(logits, bias, k)
    assert np.array_equal(ids.cpu().numpy(), want)
    _check_table(ids, order, pos, ends, logits.shape[1])
    return ids, w


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (5, 7, 7), (8, 33, 3), (64, 64, 6), (129, 100, 16), (1000, 256, 8),
                                   (5003, 256, 8), (37, 1000, 10), (300, 500, 4), (20000, 17, 2)])
@pytest.mark.parametrize("softmax,renorm", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_choice_weights_table(fp8, T, E, k, softmax, renorm, dtype):
    g = torch.Generator(device="cuda").manual_seed(T + E)
    logits = (2 * torch.randn(T, E, generator=g, device="cuda")).to(dtype)
    bias = torch.randn(E, generator=g, device="cuda") if (T + k) % 2 else None
    ids, w = _run(fp8, logits, k, bias, softmax, renorm, 2.5)
    ref = _weights(logits.double(), ids, softmax, renorm, 2.5)
    assert ((w.double() - ref).abs() <= 64 * U * ref).all()


@pytest.mark.parametrize("T,E,k", [(33, 600, 5), (60, 1024, 16), (17, 257, 4), (16, 900, 2), (320, 64, 6), (321, 65, 6), (700, 64, 8), (4000, 1000, 3), (9000, 512, 16), (499000, 4, 2), (700001, 9, 1)])
def test_many_experts_and_long_chunks(fp8, T, E, k):
    """Chunks of several batches of slots, and of thousands of tokens; most slots at one expert."""
    g = torch.Generator(device="cuda").manual_seed(T)
    logits = torch.randn(T, E, generator=g, device="cuda")
    logits[: T // 2, E - 1] += 8
    _run(fp8, logits, k)


def test_ties_take_the_lowest_index(fp8):
    g = torch.Generator(device="cuda").manual_seed(1)
    logits = torch.randint(-2, 3, (777, 200), generator=g, device="cuda").float()
    logits[::2] *= -0.0  # rows of zeros of either sign: level
    _run(fp8, logits, 9)
    _run(fp8, torch.zeros(40, 1024, device="cuda"), 16, softmax=False)


@pytest.mark.parametrize("softmax,renorm", [(True, True), (True, False), (False, True), (False, False)])
def test_masks(fp8, softmax, renorm):
    """-inf logits, a row without any expert, NaN, experts masked by the bias, the types' extremes."""
    T, E, k = 41, 40, 4
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.randn(T, E, generator=g, device="cuda")
    logits[1] = -torch.inf
    logits[2, 3:] = -torch.inf       # fewer left than k
    logits[3, ::2] = -torch.inf
    logits[4] = torch.finfo(torch.float32).min
    logits[5, 7] = torch.finfo(torch.float32).max
    logits[6, :] = 300.0             # far past exp's range
    logits[7, :] = -300.0
    bias = torch.zeros(E, device="cuda")
    bias[10:20] = -torch.inf
    ids, w = _run(fp8, logits, k, bias, softmax, renorm)
    ids_h = ids.cpu()
    assert (ids_h[1] == -1).all() and not w[1].any() and (ids_h[2] >= 0).sum() == 3
    assert not torch.isin(ids_h, torch.arange(10, 20)).any()
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[1] = False
    keep[7] = softmax  # sigmoid(-300): zero in fp32, 1e-131 in 64 bits
    ref = _weights(logits.double()[keep], ids[keep], softmax, renorm, 1.0)
    assert ((w[keep].double() - ref).abs() <= 64 * U * ref + 2.0 ** -126).all()
    logits[8, 0] = float("nan")
    logits[9] = float("nan")
    ids, w = _run(fp8, logits, k, bias, softmax, renorm)
    assert (ids[9] == -1).all() and not w[9].any() and (ids[8] > 0).all()
    if not softmax or renorm:
        assert torch.isfinite(w).all()  # a NaN that is not taken does not reach the weights


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 8, 2), (65, 33, 5), (500, 256, 8), (17, 1000, 16)])
@pytest.mark.parametrize("softmax,renorm", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_backward(fp8, T, E, k, softmax, renorm, dtype):
    g = torch.Generator(device="cuda").manual_seed(E + k)
    logits = (2 * torch.randn(T, E, generator=g, device="cuda")).to(dtype)
    ids = torch.from_numpy(_choose(logits, None, k).astype(np.int32)).cuda()
    if T > 2:
        ids[1, 0] = -1
        ids[2] = -1  # a token without experts
    dw = torch.randn(T, k, generator=g, device="cuda")
    d = torch.full((T, E), float("nan"), dtype=dtype, device="cuda")
    score = fp8.SCORE_SOFTMAX if softmax else fp8.SCORE_SIGMOID
    fp8.fp8_moe_route_bwd(logits, ids, dw, d, score, renorm, 2.5)
    # the formula, by autograd in 64 bits (tokens without experts apart: their weights are constant)
    some = (ids >= 0).any(1)
    l64 = logits.double()[some].requires_grad_(True)
    ref = torch.zeros(T, E, dtype=torch.float64, device="cuda")
    ref[some] = torch.autograd.grad(_weights(l64, ids[some], softmax, renorm, 2.5), l64, dw.double()[some])[0]
    v = torch.softmax(logits.double(), 1) if softmax else torch.sigmoid(logits.double())
    taken = ids >= 0
    if softmax and renorm:
        v = torch.zeros_like(v).scatter_add_(1, ids.clamp_min(0).long(), _weights(logits.double(), ids, True, True, 1.0))
        v = torch.where(taken.any(1, keepdim=True), v, 0.0)
    gv = torch.where(taken, 2.5 * dw.double().abs() * v.gather(1, ids.clamp_min(0).long()), 0.0)
    z = gv.new_ones(())
    if renorm and not softmax:
        z = torch.where(taken, v.gather(1, ids.clamp_min(0).long()), 0.0).sum(1, keepdim=True).clamp_min(1e-20)
    size = torch.zeros_like(v).scatter_add_(1, ids.clamp_min(0).long(), gv / z) + v * (gv / z).sum(1, keepdim=True) / z
    bound = 64 * U * size + (2.0 ** -8 * ref.abs() if dtype == torch.bfloat16 else 0) + 1e-38
    assert ((d.double() - ref).abs() <= bound).all()
    # central differences of the 64-bit formula along a random direction
    dirn = torch.randn(T, E, generator=g, device="cuda").double()
    h = 1e-5

    def f(a):
        return (_weights(a, ids, softmax, renorm, 2.5)[some] * dw.double()[some]).sum()

    num = (f(logits.double() + h * dirn) - f(logits.double() - h * dirn)) / (2 * h)
    got = (d.double() * dirn).sum()
    assert abs(got - num) <= (bound * dirn.abs()).sum() + 1e-7 * (ref * dirn).abs().sum() + 1e-9


def test_backward_named_twice_and_bad_ids(fp8):
    """An expert named twice in a row gets both slots' gradients; an id out of range sets the status and counts as unused."""
    g = torch.Generator(device="cuda").manual_seed(9)
    logits = torch.randn(2, 20, generator=g, device="cuda")
    ids = torch.tensor([[3, 3, 5], [4, 25, -7]], dtype=torch.int32, device="cuda")
    dw = torch.randn(2, 3, generator=g, device="cuda")
    used = ids.clone()
    used[1, 1:] = -1
    for softmax, renorm in [(True, False), (False, False)]:
        d = torch.empty_like(logits)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        fp8.fp8_moe_route_bwd(logits, ids, dw, d, fp8.SCORE_SOFTMAX if softmax else fp8.SCORE_SIGMOID, renorm, 1.0, st)
        l64 = logits.double().requires_grad_(True)
        ref = torch.autograd.grad(_weights(l64, used, softmax, renorm, 1.0), l64, dw.double())[0]
        assert int(st) == fp8.DEV_BAD_IDS
        assert ((d.double() - ref).abs() <= 128 * U * dw.abs().sum(1, keepdim=True)).all()


def test_streams_graph_no_rows(fp8):
    g = torch.Generator(device="cuda").manual_seed(2)
    logits = torch.randn(3001, 64, generator=g, device="cuda")
    want = fp8.moe_route_alloc(logits, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = fp8.moe_route_alloc(logits, 4)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = [torch.zeros_like(t) for t in want]
    ws = fp8.route_workspace(3001, 64, "cuda")
    ws.fill_(0xFF)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp8.fp8_moe_route(logits, *out, workspace=ws)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    ids, w, order, pos, ends = fp8.moe_route_alloc(torch.empty(0, 6, device="cuda"), 2)
    assert not ends.any() and ids.shape == (0, 2)
