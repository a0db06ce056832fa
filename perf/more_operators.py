"""The gated feed-forward of dense layers and of experts, and products with a scale for each block of 128: what is
timed, on which inputs, and their plain forms.

Three operators:

- gated_mm: h = act(x W1^T) * (x W3^T), both projections, the activation and the product in one call; dense, or
  with the rows routed to experts by offsets; on FP8 operands with a scale per row or per block of 128, or on bf16.
  The result in bf16, or in 8 bits with a scale per 1 x 128 block; for training also the projections themselves.
- gated_mm_bwd: from the gradient of the block's output and the projections, the gradient of the projections:
  dh = dy W2, du = dh act(g), dg = dh u act'(g); and h again, for the gradient of W2.
- grouped_mm: the experts' products on FP8 operands with a scale for each block of 128 (1 x 128 of the rows,
  128 x 128 of the weights).

`own` False: plain torch in 32 bits, each output rounded once. `own` True: the package's calls.
"""
import math
import random

import torch

own = False

DEV = "cuda"
F8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}


# ------------------------------------------------------------------------------------------
# cases: M rows; E experts (0: a dense layer), `active` of them with rows; K the contraction's length
# (of gated_mm_bwd: the model's width), I the hidden layer's, N the output's

def listed():
    return [
        # one decoded token of a dense layer (Llama3-8B-shaped): the weights' bytes and the call's latency
        dict(name="gate-token", op="gate", kind="row", M=1, E=0, K=4096, I=14336, act="silu", out="h", fmt="e4m3"),
        # one decoded token routed to 8 of 256 experts (DeepSeek-V3-shaped), blockwise, codes for the second product
        dict(name="gate-token-experts", op="gate", kind="block", M=8, E=256, active=8, K=7168, I=2048, act="silu",
             out="q", fmt="e4m3"),
        # a training batch of a dense layer, a scale per row: the hidden layer and what the backward pass needs
        dict(name="gate-train", op="gate", kind="row", M=8192, E=0, K=4096, I=14336, act="silu", out="train",
             fmt="e4m3"),
        # a long prompt on 16 large experts (Llama4-shaped), blockwise, codes for the second product
        dict(name="gate-experts", op="gate", kind="block", M=16384, E=16, active=16, K=5120, I=8192, act="silu",
             out="q", fmt="e4m3"),
        # high-precision training of an odd layer with GELU, ragged batch
        dict(name="gate-odd", op="gate", kind="bf16", M=1021, E=0, K=2056, I=5128, act="gelu", out="train"),
        # the backward pass of the training batch, the hidden layer made again
        dict(name="gategrad-train", op="gate_bwd", kind="row", M=8192, E=0, K=4096, I=14336, act="silu", h=True,
             fmt="e5m2"),
        # experts' backward pass on a ragged batch, blockwise
        dict(name="gategrad-experts", op="gate_bwd", kind="block", M=4099, E=32, active=31, K=7168, I=2048, act="silu",
             h=False, fmt="e5m2"),
        # a short odd batch in bf16: latency
        dict(name="gategrad-odd", op="gate_bwd", kind="bf16", M=77, E=0, K=1032, I=2056, act="gelu", h=True),
        # the second product of one token's 8 experts
        dict(name="block-token", op="block", M=8, E=256, active=8, K=2048, N=7168, fmt="e4m3", out="bf16"),
        # of a decode batch of 32 tokens
        dict(name="block-batch", op="block", M=256, E=256, active=144, K=2048, N=7168, fmt="e4m3", out="bf16"),
        # of a long prompt on 64 experts
        dict(name="block-prefill", op="block", M=32768, E=64, active=63, K=2048, N=7168, fmt="e4m3", out="bf16"),
        # a gradient's product on few odd experts, fp32 out
        dict(name="block-grad", op="block", M=5003, E=5, active=4, K=5120, N=1000, fmt="e5m2", out="f32"),
    ]


MOST_FLOPS = 4 * 16384 * 8192 * 5120      # of the largest listed case
MOST_WEIGHTS = 256 * 2 * 2048 * 7168      # bytes of one operand's weights


def _size(rng, lo, hi):
    """A whole number of lo .. hi, spread over its logarithm: an odd one, or a power of two."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))
    if rng.random() < 0.4:
        n = 1 << int(round(math.log2(v)))
        if lo <= n <= hi:
            return n
    n = int(v) | 1
    return n if lo <= n <= hi else max(lo, n - 2)


def draw(rng):
    op = rng.choice(["gate", "gate", "gate_bwd", "gate_bwd", "block", "block"])
    E = 0 if op != "block" and rng.random() < 0.5 else _size(rng, 1, 256)
    kind = "block" if op == "block" else rng.choice(["row", "block"] if E else ["row", "block", "bf16"])
    M = _size(rng, 1, 16384 if op != "block" else 32768)
    K = 128 * _size(rng, 2, 56) if kind == "block" else 16 * _size(rng, 16, 448)
    case = dict(op=op, M=M, E=E)
    if op == "block":
        N = 8 * _size(rng, 8, 1024)
        case.update(K=K, N=N, fmt=rng.choice(["e4m3", "e4m3", "e5m2"]), out=rng.choice(["bf16", "bf16", "f32"]))
    else:
        I = 128 * _size(rng, 2, 112) if kind == "block" else 8 * _size(rng, 32, 1792)
        N = 2 * I
        outs = ["h", "train"] + (["q"] if I % 128 == 0 and kind != "bf16" else [])
        case.update(kind=kind, K=K, I=I, act=rng.choice(["silu", "silu", "gelu"]))
        if op == "gate":
            case.update(out=rng.choice(outs), fmt="e4m3")
        else:
            case.update(h=rng.random() < 0.5, fmt=rng.choice(["e5m2", "e5m2", "e4m3"]))
    while case["E"] * N * K > MOST_WEIGHTS:
        case["E"] = max(1, case["E"] // 2)
    while 2 * case["M"] * N * K > MOST_FLOPS:
        case["M"] = max(1, case["M"] // 2)
    if E:
        case["active"] = rng.randint(1, min(case["E"], case["M"]))
    return case


# ------------------------------------------------------------------------------------------
# inputs

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _hidden(g, M, K):
    """Hidden states as layers make them: normal, with one channel in a hundred 20 times larger."""
    x = _randn(g, M, K)
    x[:, torch.randint(0, K, (max(1, K // 100),), generator=g, device=DEV)] *= 20.0
    return x


def _quantize(x, rows, cols, fmt):
    """Codes of x [R, C] and a scale for each block of rows x cols (0: the whole row), [ceil(R / rows), ceil(C / cols)]."""
    dt, fmax = F8[fmt]
    R, C = x.shape
    cols = cols or C
    r, c = -(-R // rows), -(-C // cols)
    pad = torch.nn.functional.pad(x, (0, c * cols - C, 0, r * rows - R)).view(r, rows, c, cols)
    inv = pad.abs().amax((1, 3)).clamp_min_(1e-12) / fmax
    return (pad / inv[:, None, :, None]).clamp_(-fmax, fmax).to(dt).view(r * rows, c * cols)[:R, :C].contiguous(), inv


def _weights(g, E, N, K, kind):
    """The weights of E matrices [N, K] (E 0: one, without that dimension), N(0, 0.02^2): bf16, or e4m3 codes with a
    scale per row or per 128 x 128 block."""
    n = max(E, 1)
    if kind == "bf16":
        return (0.02 * _randn(g, N, K)).to(torch.bfloat16), None
    q = torch.empty(n, N, K, dtype=torch.float8_e4m3fn, device=DEV)
    inv = torch.empty((n, N) if kind == "row" else (n, -(-N // 128), K // 128), dtype=torch.float32, device=DEV)
    for e in range(n):
        w = _randn(g, N, K).mul_(0.02)
        q[e], s = _quantize(w, *((1, 0) if kind == "row" else (128, 128)), "e4m3")
        inv[e] = s[:, 0] if kind == "row" else s
    return (q, inv) if E else (q[0], inv[0])


def _rows(x, kind, fmt):
    if kind == "bf16":
        return x.to(torch.bfloat16), None
    q, inv = _quantize(x, 1, 0 if kind == "row" else 128, fmt)
    return q, inv[:, 0].contiguous() if kind == "row" else inv


def _counts(seed, M, E, active):
    """Rows of each expert: `active` of them with one at least, the rest by a popularity that falls off as a trained
    layer's routing does."""
    rng = random.Random(seed)
    experts = rng.sample(range(E), active)
    counts = [0] * E
    for e in experts + rng.choices(experts, [1.0 / (r + 4) for r in range(active)], k=M - active):
        counts[e] += 1
    return counts


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c, op, M, E, K = case, case["op"], case["M"], case["E"], case["K"]
    s = dict(case=case, ends=None, counts=None)
    if E:
        s["counts"] = _counts(seed, M, E, c["active"])
        s["ends"] = torch.tensor(s["counts"], device=DEV).cumsum(0).to(torch.int32)
    if op == "block":
        s["A"], s["sA"] = _rows(_hidden(g, M, K) if c["fmt"] == "e4m3" else 1e-3 * _randn(g, M, K), "block", c["fmt"])
        s["B"], s["sB"] = _weights(g, E, c["N"], K, "block")
        s["o"] = torch.empty(M, c["N"], dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32, device=DEV)
        return s
    kind, I = c["kind"], c["I"]
    if op == "gate":
        s["A"], s["sA"] = _rows(_hidden(g, M, K), kind, "e4m3")
        s["B"], s["sB"] = _weights(g, E, 2 * I, K, kind)
        if c["out"] == "q":
            s["q"] = torch.empty(M, I, dtype=F8[c["fmt"]][0], device=DEV)
            s["inv"] = torch.empty(M, I // 128, dtype=torch.float32, device=DEV)
        else:
            s["h"] = torch.empty(M, I, dtype=torch.bfloat16, device=DEV)
        if c["out"] == "train":
            s["gu"] = torch.empty(M, 2 * I, dtype=torch.bfloat16, device=DEV)
        return s
    s["A"], s["sA"] = _rows(1e-3 * _randn(g, M, K), kind, c.get("fmt"))
    s["B"], s["sB"] = _weights(g, E, I, K, kind)  # W2 transposed: a row for each column of the hidden layer
    s["gu"] = (1.5 * _randn(g, M, 2 * I)).to(torch.bfloat16)
    s["dgu"] = torch.empty(M, 2 * I, dtype=torch.bfloat16, device=DEV)
    if c["h"]:
        s["h"] = torch.empty(M, I, dtype=torch.bfloat16, device=DEV)
    return s


# ------------------------------------------------------------------------------------------
# one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import moe_grouped_gemm_absmax_gb300 as fp8
    c = s["case"]
    if c["op"] == "block":
        fp8.fp8_grouped_mm(s["A"], s["B"], s["ends"], s["sA"], s["sB"], s["o"], fp8.GROUPED_JAGGED_M, fp8.MM_BLOCKWISE)
        return s["o"]
    act = fp8.ACT_SILU if c["act"] == "silu" else fp8.ACT_GELU
    flags = fp8.MM_BLOCKWISE if c["kind"] == "block" else 0
    if c["op"] == "gate":
        fp8.fp8_gated_mm(s["A"], s["B"], s["sA"], s["sB"], h=s.get("h"), gu=s.get("gu"), q=s.get("q"),
                         inv_scales=s.get("inv"), offsets=s["ends"], act=act, flags=flags)
        return [s[k] for k in ("h", "gu", "q", "inv") if k in s]
    fp8.fp8_gated_mm_bwd(s["A"], s["B"], s["sA"], s["sB"], s["gu"], s["dgu"], h=s.get("h"), offsets=s["ends"], act=act,
                         flags=flags)
    return [s[k] for k in ("dgu", "h") if k in s]


def _wide(codes, inv, kind):
    """An operand in 32 bits."""
    if kind == "bf16":
        return codes.float()
    if kind == "row":
        return codes.float() * inv[:, None]
    rows = 128 if inv.shape[0] != codes.shape[0] else 1  # the rows' blocks have one row, the weights' 128
    full = inv.repeat_interleave(rows, 0)[:codes.shape[0]].repeat_interleave(128, 1)
    return codes.float() * full


def _product(s, kind):
    """A B^T in 32 bits, by expert where there are experts."""
    A = _wide(s["A"], s["sA"], kind)
    if s["counts"] is None:
        return A @ _wide(s["B"], s["sB"], kind).T
    out = torch.empty(A.shape[0], s["B"].shape[1], dtype=torch.float32, device=A.device)
    at = 0
    for e, n in enumerate(s["counts"]):
        if n:
            torch.mm(A[at:at + n], _wide(s["B"][e], s["sB"][e], kind).T, out=out[at:at + n])
        at += n
    return out


def _act(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        sig = 1.0 / (1.0 + torch.exp(-g))
        return g * sig, sig * (1.0 + g * (1.0 - sig))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g)


def _run_plain(s):
    c = s["case"]
    if c["op"] == "block":
        return _product(s, "block").to(s["o"].dtype)
    y = _product(s, c["kind"])
    I = c["I"]
    if c["op"] == "gate":
        h = _act(y[:, :I], c["act"])[0] * y[:, I:]
        if c["out"] == "q":
            dt, fmax = F8[c["fmt"]]
            blocks = h.view(c["M"], -1, 128)
            amax = blocks.abs().amax(-1).clamp_min(1e-12)
            return [(blocks * (fmax / amax)[..., None]).clamp(-fmax, fmax).to(dt).view(h.shape), amax / fmax]
        return [h.to(torch.bfloat16)] + ([y.to(torch.bfloat16)] if c["out"] == "train" else [])
    g, u = s["gu"][:, :I].float(), s["gu"][:, I:].float()
    a, d = _act(g, c["act"])
    return [torch.cat([y * u * d, y * a], 1).to(torch.bfloat16)] + ([(a * u).to(torch.bfloat16)] if c["h"] else [])


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op, M, K, kind = case["op"], case["M"], case["K"], case.get("kind", "block")
    parts, at = [], 0
    for e, n in enumerate(s["counts"] or [M]):
        if n == 0:
            continue
        a, b = s["A"][at:at + n].double(), (s["B"][e] if case["E"] else s["B"]).double()
        if kind == "bf16":
            parts.append(torch.einsum("mk,nk->mn", a, b))
        else:
            sa, sb = s["sA"][at:at + n].double(), (s["sB"][e] if case["E"] else s["sB"]).double()
            if kind == "row":
                parts.append(torch.einsum("mk,nk->mn", a, b) * torch.outer(sa, sb))
            else:
                acc = torch.zeros(n, b.shape[0], dtype=torch.float64, device=DEV)
                column = torch.arange(b.shape[0], device=DEV) // 128
                for k in range(K // 128):
                    ka = a[:, 128 * k:128 * k + 128] * sa[:, k, None]
                    acc.addmm_(ka, (b[:, 128 * k:128 * k + 128] * sb[column, k, None]).T)
                parts.append(acc)
        at += n
    y = torch.cat(parts)
    if op == "block":
        return y
    I = case["I"]

    def act(v):
        return torch.nn.functional.silu(v) if case["act"] == "silu" else torch.nn.functional.gelu(v, approximate="tanh")

    if op == "gate":
        h = act(y[:, :I]) * y[:, I:]
        if case["out"] != "q":
            return [h] + ([y] if case["out"] == "train" else [])
        dt, fmax = F8[case["fmt"]]
        inv = torch.stack([b.abs().amax(1) for b in h.split(128, 1)], 1).clamp_min(1e-12) / fmax
        scaled = torch.cat([b / inv[:, i, None] for i, b in enumerate(h.split(128, 1))], 1)
        return [scaled.clamp(-fmax, fmax).to(dt).double(), inv]
    # the derivative of sum(dh * act(g) * u)
    gate, up = (t.double().requires_grad_(True) for t in s["gu"].split(I, 1))
    h = act(gate) * up
    dg, du = torch.autograd.grad(h, (gate, up), y)
    return [torch.cat([dg, du], 1)] + ([h.detach()] if case["h"] else [])


# ------------------------------------------------------------------------------------------

def work(case):
    """Bytes that a pass cannot do without (each input once, each output once) and its operations."""
    op, M, E, K = case["op"], case["M"], case["E"], case["K"]
    kind = case.get("kind", "block")
    n = case["active"] if E else 1
    N = case["N"] if op == "block" else 2 * case["I"] if op == "gate" else case["I"]
    size = 2 if kind == "bf16" else 1
    total = M * K * size + n * N * K * size + 4 * E
    if kind == "row":
        total += 4 * (M + n * N)
    elif kind == "block":
        total += 4 * (M * (K // 128) + n * -(-N // 128) * (K // 128))
    if op == "block":
        total += M * N * (2 if case["out"] == "bf16" else 4)
    elif op == "gate":
        total += {"h": 2 * M * N // 2, "train": 3 * M * N, "q": M * N // 2 + 4 * M * (N // 256)}[case["out"]]
    else:
        total += 8 * M * N + (2 * M * N if case["h"] else 0)
    return {"bytes": total, "flops": 2 * M * N * K}
