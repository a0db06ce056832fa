"""Inputs of the gated feed-forward and of block-scaled products, their formulas in 64 bits, and the bounds that the
kernels' results have to keep: products are exact in fp32, a sum of K of them is off by at most K steps of 2^-23 of the
sum of their magnitudes (an adder that cuts off instead of rounding included), each rounding to a type by half a step."""
import math

import torch

HALF_BF16 = 2.0 ** -8
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
FMAX = {E4: 448.0, E5: 57344.0}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def operand(g, shape, kind, dt=E4, rows=1, size=1.0):
    """Random codes or bf16 values of `shape` with scales by kind ("bf16", "tensor", "row", "block" with blocks of rows x
    128), such that the values are about `size`. Returns the operand, its scales, and its values in 64 bits."""
    x = randn(g, *shape)
    if kind == "bf16":
        v = (x * size).to(torch.bfloat16)
        return v, None, v.double()
    q = (x * (FMAX[dt] / 4.0)).clamp(-FMAX[dt], FMAX[dt]).to(dt)  # the clamp acts past four deviations
    unit = size / (FMAX[dt] / 4.0)
    lead = shape[:-1]
    if kind == "tensor":
        s = torch.full((1,), unit, device="cuda")
        return q, s, q.double() * s.double()
    if kind == "row":
        s = unit * (0.5 + torch.rand(*lead, generator=g, device="cuda"))
        return q, s, q.double() * s.double()[..., None]
    n = -(-shape[-2] // rows)
    s = unit * (0.5 + torch.rand(*lead[:-1], n, shape[-1] // 128, generator=g, device="cuda"))
    full = s.double().repeat_interleave(rows, -2)[..., :shape[-2], :].repeat_interleave(128, -1)
    return q, s, q.double() * full


def product(a, b, counts=None):
    """a b^T in 64 bits (rows by expert with counts), and the bound of an fp32 sum's error."""
    K = a.shape[1]
    if counts is None:
        y, mag = a @ b.T, a.abs() @ b.abs().T
    else:
        y = torch.zeros(a.shape[0], b.shape[1], dtype=torch.float64, device=a.device)
        mag, at = torch.zeros_like(y), 0
        for e, n in enumerate(counts):
            y[at:at + n] = a[at:at + n] @ b[e].T
            mag[at:at + n] = a[at:at + n].abs() @ b[e].abs().T
            at += n
    # K additions and the scales' two products
    return y, (K * 2.0 ** -23 + 2.0 ** -21) * mag + 1e-36


def act64(g, act):
    """act(g), its derivative, and bounds of the errors that fp32 arithmetic and the fast exponential add to them: the
    logistic function is off by (|w| + 8) 2^-23 of itself, its complement by 2^-23."""
    if act == "silu":
        w, dw = g, torch.ones_like(g)
    else:
        c = 2 * math.sqrt(2 / math.pi)
        w, dw = c * (g + 0.044715 * g ** 3), c * (1 + 3 * 0.044715 * g ** 2)
    s = torch.sigmoid(w)
    a, d = g * s, s + g * s * (1 - s) * dw
    e = (w.abs() + 8) * 2.0 ** -23
    return a, d, e * a.abs() + 1e-30, 4 * e * (s + (a * (1 - s) * dw).abs()) + 2.0 ** -22 * (a * dw).abs() + 1e-30


def hidden(y, err, act):
    """(h, its bound before rounding) from both projections [M, 2 I]."""
    I = y.shape[1] // 2
    g, u = y[:, :I], y[:, I:]
    eg, eu = err[:, :I], err[:, I:]
    a, _, ea, _ = act64(g, act)
    ea = ea + 1.13 * eg  # |act'| stays below 1.13
    return a * u, ea * (u.abs() + eu) + a.abs() * eu + 2.0 ** -22 * (a * u).abs()


def check(got, ref, bound, what=""):
    assert got.isfinite().all(), what
    over = (got.double() - ref).abs() - bound
    assert (over <= 0).all(), f"{what}: {(over > 0).sum().item()} of {over.numel()} outside, worst excess {over.max().item():.3e}"


def check_codes(q, inv, h, err, what=""):
    """8-bit codes and inverse scales of h's 1 x 128 blocks against h in 64 bits."""
    fmax = FMAX[q.dtype]
    half, tiny = (2.0 ** -4, 2.0 ** -10) if q.dtype == E4 else (2.0 ** -3, 2.0 ** -17)
    M, I = h.shape
    b = h.view(M, I // 128, 128).abs().amax(2).clamp_min(1e-12) / fmax
    eb = err.view(M, I // 128, 128).amax(2) / fmax
    check(inv, b, eb + 2.0 ** -21 * b, what + " scales")
    s = inv.double().repeat_interleave(128, 1)
    check(q.double() * s, h, half * h.abs() + tiny * s + 2 * err + 2.0 ** -20 * h.abs(), what + " codes")
    top = q.double().abs().view(M, I // 128, 128).amax(2)
    assert (top[b > 1e-12] == fmax).all(), what  # the largest of a block takes the largest code


def ends(counts):
    return torch.tensor(counts, device="cuda").cumsum(0).to(torch.int32)


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")
