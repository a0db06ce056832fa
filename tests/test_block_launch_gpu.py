"""The kernels around a mixture-of-experts layer begin before the kernel before them has ended and wait for it on the
device: whatever comes before (a torch kernel, a copy, a memset, another of these calls on the same buffers,
work on another stream), the results are those of a run that synchronizes after every call, bit for bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu
T, E, k, H, I = 6, 16, 3, 1040, 528


@pytest.fixture(scope="module")
def fp8():
    import moe_grouped_gemm_absmax_gb300 as m
    return m


class _Chain:
    """Steps of a decode loop on fixed buffers: every call's output is the next one's input."""

    def __init__(self, fp8, tokens=T):
        g = torch.Generator(device="cuda").manual_seed(3)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.fp8, self.T = fp8, tokens
        self.x, self.h = r(tokens, H).bfloat16(), torch.zeros(tokens, H, dtype=torch.bfloat16, device="cuda")
        self.w, self.router = (1 + 0.1 * r(H)).bfloat16(), 0.05 * r(H, E)
        q = lambda *s: ((0.05 * r(*s)) / 1e-3).to(torch.float8_e4m3fn)  # noqa: E731
        self.w13, self.w2 = q(E, 2 * I, H), q(E, H, I)
        self.s13, self.s2 = torch.full((E, 2 * I), 1e-3, device="cuda"), torch.full((E, H), 1e-3, device="cuda")
        self.y, self.out = torch.empty_like(self.x), torch.empty_like(self.x)
        self.rstd = torch.empty(tokens, device="cuda")
        self.ids, self.pos = (torch.empty(tokens, k, dtype=torch.int32, device="cuda") for _ in range(2))
        self.weights, self.order = torch.empty(tokens, k, device="cuda"), torch.empty(tokens * k, dtype=torch.int32, device="cuda")
        self.ends = torch.empty(E, dtype=torch.int32, device="cuda")
        self.dw, self.dx, self.dl = torch.empty(H, device="cuda"), torch.empty_like(self.x), torch.empty(tokens, E, device="cuda")
        self.wr, self.wm = fp8.route_workspace(tokens, E, "cuda"), fp8.moe_tokens_workspace(min(tokens, 64), k, H, I, "cuda")
        self.wn = fp8.rmsnorm_bwd_workspace(tokens, H, "cuda")

    def step(self, sync):
        f = self.fp8
        f.fp8_add_rmsnorm(self.x, self.w, 1e-6, residual=self.h, h=self.h, y=self.y, rstd=self.rstd)
        sync()
        logits = self.y.float() @ self.router
        sync()
        f.fp8_moe_route(logits, self.ids, self.weights, self.order, self.pos, self.ends, workspace=self.wr)
        sync()
        if self.T <= 64:
            f.fp8_moe_tokens(self.y, self.ids, self.weights, self.w13, self.s13, self.w2, self.s2, self.out, self.wm)
        else:
            self.out.copy_(self.y * self.weights.sum(1, keepdim=True))
        sync()
        f.fp8_add_rmsnorm_bwd(self.out, self.h, self.w, self.rstd, self.dx, self.dw, dh=self.y, workspace=self.wn)
        sync()
        f.fp8_moe_route_bwd(logits, self.ids, self.weights, self.dl)
        sync()
        # the next step's input and residual stream, by torch
        self.x.copy_((self.out + 0.01 * self.dx + 1e-3 * self.dw + self.dl.sum()).clamp_(-4, 4))
        self.h.mul_(0.5)
        sync()

    def state(self):
        return [t.clone() for t in (self.x, self.h, self.y, self.rstd, self.ids, self.weights, self.order, self.pos, self.ends,
                                    self.out, self.dx, self.dw, self.dl)]


@pytest.mark.parametrize("tokens", [1, T, 23, 700, 3000])
def test_back_to_back_calls(fp8, tokens):
    want, got = _Chain(fp8, tokens), _Chain(fp8, tokens)
    for _ in range(12):
        want.step(torch.cuda.synchronize)
    for _ in range(12):
        got.step(lambda: None)
    torch.cuda.synchronize()
    assert torch.isfinite(want.x).all()
    for a, b in zip(got.state(), want.state()):
        assert torch.equal(a, b)


def test_graph_of_steps(fp8):
    want, got = _Chain(fp8), _Chain(fp8)
    start = [t.clone() for t in (got.x, got.h)]
    got.step(lambda: None)  # the first torch matmul outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(4):
            got.step(lambda: None)
    got.x.copy_(start[0])
    got.h.copy_(start[1])
    for _ in range(3):
        graph.replay()
    for _ in range(12):
        want.step(torch.cuda.synchronize)
    torch.cuda.synchronize()
    for a, b in zip(got.state(), want.state()):
        assert torch.equal(a, b)


@pytest.mark.parametrize("before", ["nothing", "memset", "copy", "host copy", "join"])
def test_what_comes_before_in_a_capture(fp8, before):
    """Each entry point as the first call after a memset, a copy or a join of two streams, captured and replayed."""
    c = _Chain(fp8)
    c.step(torch.cuda.synchronize)
    logits = torch.randn(T, E, device="cuda")
    calls = [
        (lambda: fp8.fp8_add_rmsnorm(c.x, c.w, 1e-6, y=c.y), c.x, lambda: c.y),
        (lambda: fp8.fp8_add_rmsnorm_bwd(c.x, c.h, c.w, c.rstd, c.dx, c.dw, workspace=c.wn), c.x, lambda: c.dx),
        (lambda: fp8.fp8_moe_route(logits, c.ids, c.weights, c.order, c.pos, c.ends, workspace=c.wr), logits, lambda: c.weights),
        (lambda: fp8.fp8_moe_route_bwd(logits, c.ids, c.weights, c.dl), logits, lambda: c.dl),
        (lambda: fp8.fp8_moe_tokens(c.x, c.ids, c.weights, c.w13, c.s13, c.w2, c.s2, c.out, c.wm), c.x, lambda: c.out),
    ]
    for call, inp, out in calls:
        src = torch.randn_like(inp.float()).to(inp.dtype)
        host = src.cpu().pin_memory()
        inp.copy_(src)
        if before == "memset":
            inp.zero_()
        call()
        torch.cuda.synchronize()
        want = out().clone()
        side = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            if before == "memset":
                inp.zero_()
            elif before == "copy":
                inp.copy_(src)
            elif before == "host copy":
                inp.copy_(host, non_blocking=True)
            elif before == "join":
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(side):
                    inp.copy_(src)
                    inp.mul_(1.0)
                torch.cuda.current_stream().wait_stream(side)
            call()
        if before != "nothing":
            inp.fill_(7.0)
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out(), want), before


def test_other_stream(fp8):
    """The input is written on another stream, which the call's stream waits for by an event."""
    c = _Chain(fp8)
    big = torch.randn(8192, 4096, device="cuda")
    fp8.fp8_add_rmsnorm(c.x, c.w, 1e-6, y=c.y)
    torch.cuda.synchronize()
    want, src = c.y.clone(), c.x.clone()
    side = torch.cuda.Stream()
    for _ in range(10):
        c.x.zero_()
        c.y.zero_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(3):
                big.mul_(1.0)
            c.x.copy_(src)
        torch.cuda.current_stream().wait_stream(side)
        fp8.fp8_add_rmsnorm(c.x, c.w, 1e-6, y=c.y)
        torch.cuda.synchronize()
        assert torch.equal(c.y, want)
