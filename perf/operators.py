"""The operators around a mixture-of-experts layer: what is timed, on which inputs, and their plain forms.

Three operators, five calls:

- add_rmsnorm: s = x + residual, h = bf16(s), y = s * rstd * weight, and y in 8 bits with one scale
  per row or per 1 x 128 block; its backward pass.
- moe_route: top-k experts of each token with their weights, and the table of the (token, expert)
  slots sorted by expert that the grouped GEMM's offsets need; its backward pass.
- moe_tokens: the experts of a few tokens, from the bf16 hidden state to the weighted sum of the
  experts' outputs, on FP8 weights with a scale per row.

`own` False: plain torch in 32 bits, each output rounded once. `own` True: the package's calls.
"""
import math

import torch

own = False

EPS = 1e-6
DEV = "cuda"
F8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}


# ------------------------------------------------------------------------------------------
# cases

def listed():
    return [
        # the norm before the router and the experts of one decoded token: latency
        dict(name="norm-decode", op="norm", T=1, H=7168, residual=True, gran="row", fmt="e4m3"),
        # the norm before the up projection of a training batch (Llama3-8B-shaped), a scale per row
        dict(name="norm-train", op="norm", T=8192, H=4096, residual=True, gran="row", fmt="e4m3"),
        # a first layer without a residual branch, ragged batch, blockwise scales
        dict(name="norm-block", op="norm", T=1021, H=5120, residual=False, gran="block", fmt="e4m3"),
        # the backward pass of a training batch with the residual stream's own gradient
        dict(name="normgrad-train", op="norm_bwd", T=8192, H=7168, residual=True),
        # a short odd batch, a width that no power of two divides far, no residual gradient
        dict(name="normgrad-odd", op="norm_bwd", T=77, H=2056, residual=False),
        # routing of a decode batch
        dict(name="route-decode", op="route", T=8, E=256, k=8, score="softmax", renorm=True, bias=False, logits="f32"),
        # routing of a training or prefill batch: 131072 routed rows over 256 experts, with the balancing bias
        dict(name="route-prefill", op="route", T=16384, E=256, k=8, score="sigmoid", renorm=True, bias=True,
             logits="f32"),
        # its gradient for the router's own training
        dict(name="routegrad-train", op="route_bwd", T=16384, E=256, k=8, score="softmax", renorm=False, logits="f32"),
        # a small layer and a single token: launches and waits, not bytes
        dict(name="moe-small", op="moe", T=1, E=8, H=1040, I=528, k=2, active=2),
        # one decoded token of a wide layer (256 experts, 8 of them)
        dict(name="moe-token", op="moe", T=1, E=256, H=7168, I=2048, k=8, active=8),
        # an odd few tokens of a layer with few, large experts
        dict(name="moe-large", op="moe", T=7, E=16, H=5120, I=8192, k=1, active=5),
        # a decode batch: experts with one to a dozen tokens each
        dict(name="moe-batch", op="moe", T=32, E=256, H=7168, I=2048, k=8, active=144),
    ]


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
    op = rng.choice(["norm", "norm", "norm_bwd", "norm_bwd", "route", "route", "route_bwd", "moe", "moe", "moe", "moe"])
    if op in ("norm", "norm_bwd"):
        gran = rng.choice(["row", "block"])
        H = 128 * _size(rng, 4, 96) if op == "norm" and gran == "block" else 8 * _size(rng, 32, 1536)
        T = _size(rng, 1, max(1, min(16384, 8192 * 7168 // H)))
        case = dict(op=op, T=T, H=H, residual=rng.random() < 0.6)
        if op == "norm":
            case.update(gran=gran, fmt=rng.choice(["e4m3", "e4m3", "e5m2"]))
        return case
    if op in ("route", "route_bwd"):
        E = _size(rng, 8, 512)
        case = dict(op=op, T=_size(rng, 1, min(16384, 16384 * 256 // E)), E=E, k=rng.randint(1, min(E, 10)),
                    score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.5,
                    logits=rng.choice(["f32", "f32", "bf16"]))
        if op == "route":
            case["bias"] = rng.random() < 0.5
        return case
    E = _size(rng, 4, 256)
    H = 16 * _size(rng, 32, 448)
    I = 16 * _size(rng, 16, 512)
    while E * H * I > 256 * 7168 * 2048:
        E = max(4, E // 2)
    k = rng.randint(1, min(E, 8))
    T = _size(rng, 1, 32)
    while T * k * H * I > 32 * 8 * 7168 * 2048:
        T = max(1, T // 2)
    most = 140 * 7168 * 2048 // (H * I)  # experts read: no more bytes than the largest listed case
    return dict(op=op, T=T, E=E, H=H, I=I, k=k, active=rng.randint(k, min(E, T * k, most)))


# ------------------------------------------------------------------------------------------
# inputs

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _hidden(g, T, H):
    """Hidden states as layers make them: normal, with one channel in a hundred 20 times larger."""
    x = _randn(g, T, H)
    x[:, torch.randint(0, H, (max(1, H // 100),), generator=g, device=DEV)] *= 20.0
    return x.to(torch.bfloat16)


def _expert_weights(g, E, N, K):
    """FP8 codes [E, N, K] and a scale per row [E, N] of N(0, 0.02^2) weights, an expert at a time."""
    q = torch.empty(E, N, K, dtype=torch.float8_e4m3fn, device=DEV)
    inv = torch.empty(E, N, dtype=torch.float32, device=DEV)
    for e in range(E):
        w = _randn(g, N, K).mul_(0.02)
        inv[e] = w.abs().amax(1) / 448.0
        q[e] = w.div_(inv[e][:, None]).to(torch.float8_e4m3fn)
    return q, inv


def _slots(g, T, E, k, active):
    """Experts of each token: k different ones of `active`, each of the `active` taken at least once,
    the rest by a popularity that falls off as the routing of a trained layer does."""
    experts = torch.randperm(E, generator=g, device=DEV)[:active]
    pop = torch.arange(1, active + 1, device=DEV, dtype=torch.float32).reciprocal()
    score = pop.log()[None] - torch.rand(T, active, generator=g, device=DEV).clamp_(1e-6, 1 - 1e-6).log().neg_().log_()
    # expert a belongs to token a % T whatever its popularity: active <= T * k, so at most k fall on one token
    a = torch.arange(active, device=DEV)
    score[a % T, a] += 1e4
    ids = experts[score.topk(k, dim=1).indices]
    return ids.to(torch.int32).contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, T = case["op"], case["T"]
    s = dict(case=case)
    if op in ("norm", "norm_bwd"):
        H = case["H"]
        s["weight"] = (1.0 + 0.1 * _randn(g, H)).to(torch.bfloat16)
        if op == "norm":
            s["x"] = _hidden(g, T, H)
            s["residual"] = _hidden(g, T, H) if case["residual"] else None
            s["h"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV) if case["residual"] else None
            s["q"] = torch.empty(T, H, dtype=F8[case["fmt"]][0], device=DEV)
            s["inv"] = torch.empty((T,) if case["gran"] == "row" else (T, H // 128), dtype=torch.float32, device=DEV)
            s["rstd"] = torch.empty(T, dtype=torch.float32, device=DEV)
        else:
            s["h"] = _hidden(g, T, H)
            s["rstd"] = (s["h"].float().square().mean(1) + EPS).rsqrt()
            s["dy"] = (1e-3 * _randn(g, T, H)).to(torch.bfloat16)
            s["dh"] = (1e-3 * _randn(g, T, H)).to(torch.bfloat16) if case["residual"] else None
            s["dx"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
            s["dw"] = torch.empty(H, dtype=torch.float32, device=DEV)
    elif op in ("route", "route_bwd"):
        E, k = case["E"], case["k"]
        dt = torch.float32 if case["logits"] == "f32" else torch.bfloat16
        # a router's logits: a popularity of each expert plus what the token adds
        s["logits"] = (1.5 * _randn(g, T, E) + 0.5 * _randn(g, 1, E)).to(dt)
        s["scale"] = 2.5 if case["score"] == "sigmoid" else 1.0
        if op == "route":
            s["bias"] = 0.1 * _randn(g, E) if case["bias"] else None
            s["ids"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
            s["weights"] = torch.empty(T, k, dtype=torch.float32, device=DEV)
            s["order"] = torch.empty(T * k, dtype=torch.int32, device=DEV)
            s["pos"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
            s["ends"] = torch.empty(E, dtype=torch.int32, device=DEV)
        else:
            s["ids"] = s["logits"].float().sort(dim=1, descending=True, stable=True).indices[:, :k].int().contiguous()
            s["dweights"] = 1e-2 * _randn(g, T, k)
            s["dlogits"] = torch.empty(T, E, dtype=dt, device=DEV)
    else:
        E, H, I, k = case["E"], case["H"], case["I"], case["k"]
        s["x"] = _hidden(g, T, H)
        s["ids"] = _slots(g, T, E, k, case["active"])
        s["weights"] = torch.softmax(_randn(g, T, k), 1)
        s["w13"], s["s13"] = _expert_weights(g, E, 2 * I, H)
        s["w2"], s["s2"] = _expert_weights(g, E, H, I)
        s["out"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    return s


# ------------------------------------------------------------------------------------------
# one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import moe_grouped_gemm_absmax_gb300 as fp8
    c = s["case"]
    op = c["op"]
    if op == "norm":
        gran = fp8.GRAN_ROW if c["gran"] == "row" else fp8.GRAN_BLOCK_1x128
        fp8.fp8_add_rmsnorm(s["x"], s["weight"], EPS, residual=s["residual"], h=s["h"], q=s["q"], inv_scales=s["inv"],
                            granularity=gran, rstd=s["rstd"])
        return [s["h"], s["q"], s["inv"], s["rstd"]]
    if op == "norm_bwd":
        if "ws" not in s:
            s["ws"] = fp8.rmsnorm_bwd_workspace(c["T"], c["H"], DEV)
        fp8.fp8_add_rmsnorm_bwd(s["dy"], s["h"], s["weight"], s["rstd"], s["dx"], s["dw"], dh=s["dh"],
                                workspace=s["ws"])
        return [s["dx"], s["dw"]]
    if op in ("route", "route_bwd"):
        score = fp8.SCORE_SOFTMAX if c["score"] == "softmax" else fp8.SCORE_SIGMOID
        if op == "route_bwd":
            fp8.fp8_moe_route_bwd(s["logits"], s["ids"], s["dweights"], s["dlogits"], score=score,
                                  renormalize=c["renorm"], scale=s["scale"])
            return s["dlogits"]
        if "ws" not in s:
            s["ws"] = fp8.route_workspace(c["T"], c["E"], DEV)
        fp8.fp8_moe_route(s["logits"], s["ids"], s["weights"], order=s["order"], pos=s["pos"], ends=s["ends"],
                          bias=s["bias"], score=score, renormalize=c["renorm"], scale=s["scale"], workspace=s["ws"])
        return [s["ids"], s["weights"], s["order"], s["pos"], s["ends"]]
    if "ws" not in s:
        s["ws"] = fp8.moe_tokens_workspace(c["T"], c["k"], c["H"], c["I"], DEV)
    fp8.fp8_moe_tokens(s["x"], s["ids"], s["weights"], s["w13"], s["s13"], s["w2"], s["s2"], s["out"],
                       workspace=s["ws"])
    return s["out"]


def _plain_scores(logits, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-logits))
    e = torch.exp(logits - logits.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_route(s, c):
    logits, k, E = s["logits"].float(), c["k"], c["E"]
    sel = logits if s["bias"] is None else logits + s["bias"]
    sel = torch.where(sel.isnan(), -torch.inf, sel)
    best, at = sel.sort(dim=1, descending=True, stable=True)
    best, at = best[:, :k], at[:, :k]
    there = best > -torch.inf
    w = _plain_scores(logits, c["score"]).gather(1, at)
    w = torch.where(there, w, 0.0)
    if c["renorm"]:
        w = w / (w.sum(1, keepdim=True) + (1e-20 if c["score"] == "sigmoid" else 0.0))
    ids = torch.where(there, at, -1)
    key = torch.where(there, at, E).reshape(-1)
    keys, order = key.sort(stable=True)
    ends = torch.searchsorted(keys, torch.arange(E, device=DEV), right=True)
    place = torch.arange(key.numel(), device=DEV)
    pos = torch.empty_like(place)
    pos[order] = torch.where(keys < E, place, -1)
    order = torch.where(keys < E, order, -1)
    return [ids.int(), w * s["scale"], order.int(), pos.int().view(-1, k), ends.int()]


def _plain_route_bwd(s, c):
    logits, ids = s["logits"].float(), s["ids"].long()
    p = _plain_scores(logits, c["score"])
    v = p.gather(1, ids)
    g = s["dweights"] * s["scale"]
    if c["renorm"]:  # w = v / sum(v)
        z = v.sum(1, keepdim=True) + (1e-20 if c["score"] == "sigmoid" else 0.0)
        g = (g - (g * v).sum(1, keepdim=True) / z) / z
    if c["score"] == "sigmoid":
        d = torch.zeros_like(p).scatter_add_(1, ids, g * v * (1.0 - v))
    else:
        d = torch.zeros_like(p).scatter_add_(1, ids, g * v) - p * (g * v).sum(1, keepdim=True)
    return d.to(s["logits"].dtype)


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "norm":
        a = s["x"].float()
        if c["residual"]:
            a = a + s["residual"].float()
        rstd = 1.0 / torch.sqrt((a * a).mean(1) + EPS)
        y = a * rstd[:, None] * s["weight"].float()
        dt, fmax = F8[c["fmt"]]
        blocks = y if c["gran"] == "row" else y.view(c["T"], -1, 128)
        amax = blocks.abs().amax(-1).clamp_min(1e-12)
        q = (blocks * (fmax / amax)[..., None]).clamp(-fmax, fmax).to(dt).view(y.shape)
        return [a.to(torch.bfloat16) if c["residual"] else None, q, amax / fmax, rstd]
    if op == "norm_bwd":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xhat = s["h"].float() * rstd
        g = dy * s["weight"].float()
        dx = rstd * (g - xhat * (g * xhat).mean(1, keepdim=True))
        if c["residual"]:
            dx = dx + s["dh"].float()
        return [dx.to(torch.bfloat16), (dy * xhat).sum(0)]
    if op == "route":
        return _plain_route(s, c)
    if op == "route_bwd":
        return _plain_route_bwd(s, c)
    ids = s["ids"].reshape(-1).long()
    slots = s["x"].float().repeat_interleave(c["k"], 0)[..., None]  # [T k, H, 1]
    codes = s["w13"].view(torch.uint8)[ids].view(torch.float8_e4m3fn)
    gu = (codes.float() @ slots)[..., 0] * s["s13"][ids]
    gate, up = gu[:, :c["I"]], gu[:, c["I"]:]
    a = gate / (1.0 + torch.exp(-gate)) * up
    codes = s["w2"].view(torch.uint8)[ids].view(torch.float8_e4m3fn)
    y = (codes.float() @ a[..., None])[..., 0] * s["s2"][ids]
    return (y.view(c["T"], c["k"], -1) * s["weights"][..., None]).sum(1).to(torch.bfloat16)


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op, T = case["op"], case["T"]
    d = {k: v.double() for k, v in s.items()
         if torch.is_tensor(v) and k in ("x", "residual", "weight", "h", "dy", "dh", "rstd", "logits", "bias",
                                         "dweights", "weights")}
    if op == "norm":
        a = d["x"] + d["residual"] if case["residual"] else d["x"]
        mean_square = torch.einsum("th,th->t", a, a) / case["H"]
        rstd = (mean_square + EPS) ** -0.5
        y = torch.einsum("th,t,h->th", a, rstd, d["weight"])
        dt, fmax = F8[case["fmt"]]
        width = case["H"] if case["gran"] == "row" else 128
        inv = torch.maximum(y.reshape(T, -1, width).abs().amax(2), torch.tensor(1e-12, device=DEV, dtype=y.dtype)) / fmax
        q = (y.reshape(T, -1, width) / inv[..., None]).clamp(-fmax, fmax).reshape(y.shape)
        return [a if case["residual"] else None, q.to(dt).double(), inv[:, 0] if case["gran"] == "row" else inv, rstd]
    if op == "norm_bwd":
        # the derivative of sum(dy * w * h * r(h)) with r's own derivative, -r^3 h / H
        inner = torch.einsum("th,th,h->t", d["dy"], d["h"], d["weight"])
        dx = d["dy"] * d["weight"] * d["rstd"][:, None] - d["h"] * (inner * d["rstd"] ** 3 / case["H"])[:, None]
        return [dx + d["dh"] if case["residual"] else dx, torch.einsum("th,th,t->h", d["dy"], d["h"], d["rstd"])]
    if op == "route":
        lg, k = d["logits"], case["k"]
        sel = s["logits"].float() if s["bias"] is None else s["logits"].float() + s["bias"]
        # the place of each expert in its row: how many are above it, or level with it and before it
        chosen = []
        left = sel.clone()
        rows = torch.arange(T, device=DEV)
        for _ in range(k):
            top = left.amax(1, keepdim=True)
            e = (left == top).to(torch.uint8).argmax(1)
            chosen.append(e)
            left[rows, e] = -torch.inf
        ids = torch.stack(chosen, 1)
        v = torch.softmax(lg, 1) if case["score"] == "softmax" else torch.sigmoid(lg)
        v = torch.stack([v[rows, ids[:, j]] for j in range(k)], 1)
        return [None, s["scale"] * (v / v.sum(1, keepdim=True) if case["renorm"] else v), None, None, None]
    if op == "route_bwd":
        lg = d["logits"].clone().requires_grad_(True)
        v = torch.softmax(lg, 1) if case["score"] == "softmax" else torch.sigmoid(lg)
        v = torch.gather(v, 1, s["ids"].long())
        w = s["scale"] * (v / v.sum(1, keepdim=True) if case["renorm"] else v)
        return torch.autograd.grad(w, lg, d["dweights"])[0]
    if T * case["k"] * case["H"] * case["I"] > 2 ** 32:
        return None  # a matrix of each slot in 64 bits takes too long
    out = torch.zeros(T, case["H"], dtype=torch.float64, device=DEV)
    for e in torch.unique(s["ids"]).tolist():
        t, j = torch.nonzero(s["ids"] == e, as_tuple=True)
        w13 = s["w13"][e].double() * s["s13"][e].double()[:, None]
        gate, up = (d["x"][t] @ w13.T).chunk(2, 1)
        y = (torch.nn.functional.silu(gate) * up) @ (s["w2"][e].double() * s["s2"][e].double()[:, None]).T
        out.index_add_(0, t, y * d["weights"][t, j][:, None])
    return out


# ------------------------------------------------------------------------------------------

def work(case):
    """Bytes that a pass cannot do without (each input once, each output once) and its operations."""
    op, T = case["op"], case["T"]
    if op == "norm":
        H = case["H"]
        scales = T if case["gran"] == "row" else T * (H // 128)
        per = 2 + 1 + (4 if case["residual"] else 0)
        return {"bytes": T * H * per + 2 * H + 4 * scales + 4 * T, "flops": 6 * T * H}
    if op == "norm_bwd":
        H = case["H"]
        return {"bytes": T * H * (8 if case["residual"] else 6) + 2 * H + 4 * T + 4 * H, "flops": 10 * T * H}
    if op in ("route", "route_bwd"):
        E, k = case["E"], case["k"]
        size = 4 if case["logits"] == "f32" else 2
        if op == "route":
            return {"bytes": T * E * size + T * k * 16 + 4 * E * (2 if case["bias"] else 1), "flops": 4 * T * E}
        return {"bytes": 2 * T * E * size + T * k * 8, "flops": 6 * T * E}
    H, I, k = case["H"], case["I"], case["k"]
    return {"bytes": case["active"] * (3 * H * I + 4 * (2 * I + H)) + 4 * T * H + 8 * T * k,
            "flops": 6 * T * k * H * I}
