"""Each operator of a mixture-of-experts block as the first call after something else in a captured graph, with every
buffer that a call could wrongly read or leave unwritten poisoned before each replay: the inputs hold other random
values until the graph's own copy, memset or other stream writes them, the outputs a pattern. All outputs count."""
import pytest
import torch

from tests.test_block_launch_gpu import E, T, _Chain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8():
    import moe_grouped_gemm_absmax_gb300 as m
    return m


def _calls(fp8, c, logits):
    """(call, the input that is written in the graph, its outputs)"""
    return [
        (lambda: fp8.fp8_add_rmsnorm(c.x, c.w, 1e-6, y=c.y, rstd=c.rstd), c.x, [c.y, c.rstd]),
        (lambda: fp8.fp8_add_rmsnorm_bwd(c.x, c.h, c.w, c.rstd, c.dx, c.dw, workspace=c.wn), c.x, [c.dx, c.dw]),
        (lambda: fp8.fp8_moe_route(logits, c.ids, c.weights, c.order, c.pos, c.ends, workspace=c.wr), logits,
         [c.ids, c.weights, c.order, c.pos, c.ends]),
        (lambda: fp8.fp8_moe_route_bwd(logits, c.ids, c.weights, c.dl), logits, [c.dl]),
        (lambda: fp8.fp8_moe_tokens(c.x, c.ids, c.weights, c.w13, c.s13, c.w2, c.s2, c.out, c.wm), c.x, [c.out]),
    ]


@pytest.mark.parametrize("before", ["memset", "copy", "host copy", "join"])
@pytest.mark.parametrize("which", range(5))
@pytest.mark.parametrize("tokens", [T, 3000])
def test_poisoned_buffers(fp8, before, which, tokens):
    if which == 4 and tokens > fp8.MOE_MAX_TOKENS:
        pytest.skip("up to MOE_MAX_TOKENS tokens")
    c = _Chain(fp8, tokens)
    c.step(torch.cuda.synchronize)
    g = torch.Generator(device="cuda").manual_seed(which)
    logits = torch.empty(tokens, E, device="cuda")
    call, inp, outs = _calls(fp8, c, logits)[which]
    fresh = lambda: torch.randn(inp.shape, generator=g, device="cuda").to(inp.dtype)  # noqa: E731
    src = torch.zeros_like(inp) if before == "memset" else fresh()
    host = src.cpu().pin_memory()
    inp.copy_(src)
    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        if before == "memset":
            inp.zero_()
        elif before == "copy":
            inp.copy_(src)
        elif before == "host copy":
            inp.copy_(host, non_blocking=True)
        else:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                inp.copy_(src)
                inp.mul_(1.0)
            torch.cuda.current_stream().wait_stream(side)
        call()
    # the poison itself gives other outputs, so a call that read it would show
    inp.copy_(fresh())
    call()
    torch.cuda.synchronize()
    assert any(not torch.equal(a, b) for a, b in zip(outs, want))
    for _ in range(3):
        inp.copy_(fresh())
        for t in outs:
            t.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b), before
