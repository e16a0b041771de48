"""Operators around a trained expert layer and its dense neighbour, as cases to measure: routing of
tokens to experts (forward and backward), the movement of token rows into the experts' order and
back (dispatch, combine, and combine's gradient), and the matrix product with bias, activation and
residual in its epilogue (forward, and the whole backward pass of such a layer).

A route gives every token the k experts of highest score + bias (without a bias: of highest logit),
ties to the lowest index, within the best groups of experts where there are groups.  Its choices
are sorted by expert and, within one, by token: expert e owns rows [offsets[e], offsets[e + 1]).
Padded tokens choose nobody: their experts and rows are -1, their weights zero, and rows behind the
last offset belong to nobody.

`run` computes in elementary torch operations, or with `own` through the package.
"""
import math
import random

import torch

own = False


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------
def listed():
    def route(name, tokens, experts, k, score, op="route", dtype="fp32", bias=False, groups=1, top_groups=1, group_top=1, renorm=True,
              scale=1.0, padded=0.0):
        return dict(name=name, op=op, tokens=tokens, experts=experts, k=k, score=score, dtype=dtype, bias=bias, groups=groups,
                    top_groups=top_groups, group_top=group_top, renorm=renorm, scale=scale, padded=padded)

    def move(name, op, tokens, experts, k, d, ys="bf16", out="bf16", residual=False, padded=0.0):
        return dict(name=name, op=op, tokens=tokens, experts=experts, k=k, d=d, ys=ys, out=out, residual=residual, padded=padded)

    def gemm(name, rows, d, n, act, out="bf16", bias=True, residual="", pre=False):
        return dict(name=name, op="gemm", rows=rows, d=d, n=n, act=act, out=out, bias=bias, residual=residual, pre=pre)

    return [
        # one token of a served model, two experts of 16: latency
        route("route 1 token", 1, 16, 2, "softmax"),
        # a padded training batch, bf16 logits, weights as the softmax gives them
        route("route 3001 tokens", 3001, 40, 3, "softmax", dtype="bf16", renorm=False, padded=0.06),
        # a training batch over many small experts: sigmoid scores, a balance bias, 4 of 8 groups
        route("route 16384 tokens", 16384, 256, 8, "sigmoid", bias=True, groups=8, top_groups=4, group_top=2, scale=2.5),
        # the gradient of that batch's logits
        route("route bwd 16384 tokens", 16384, 256, 8, "sigmoid", op="route_bwd", bias=True, groups=8, top_groups=4, group_top=2, scale=2.5),
        # a training batch's rows into the experts' order
        move("dispatch 8192 tokens", "dispatch", 8192, 16, 2, 5120),
        # a served batch of 24 tokens: fp32 rows of the experts' last product
        move("combine 24 tokens", "combine", 24, 16, 2, 5120, ys="fp32"),
        # the training batch's rows back, onto the residual stream
        move("combine 8192 tokens", "combine", 8192, 16, 2, 5120, residual=True),
        # the gradient of a padded batch of odd size
        move("combine bwd 3001 tokens", "combine_bwd", 3001, 40, 3, 1032, padded=0.06),
        # one token through the first product of the 5120 x 20480 feed-forward layer
        gemm("gemm 1 token", 1, 5120, 20480, "gelu"),
        # a ragged batch of a fine-tuning step onto an fp32 residual stream
        gemm("gemm 333 rows", 333, 5120, 1288, "silu", out="fp32", residual="fp32"),
        # that layer's training step at 8192 tokens, the pre-activation kept
        gemm("gemm 8192 rows", 8192, 5120, 20480, "gelu", pre=True),
        # the backward pass of a squared-ReLU layer: gradients of input, weight and bias
        dict(name="linear bwd 4096 rows", op="linear_bwd", rows=4096, d=5120, n=5120, act="relu2"),
    ]


def draw(rng: random.Random):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("route", "route", "route_bwd", "dispatch", "combine", "combine_bwd", "gemm", "gemm", "linear_bwd"))
    if op in ("route", "route_bwd"):
        groups = rng.choice((1, 1, 2, 4, 8))
        experts = groups * max(1, spread(8, 512) // groups)
        size = experts // groups
        top_groups = rng.randint(1, groups)
        tokens = spread(1, 16384)
        while tokens * experts > 16384 * 256:
            tokens //= 2
        return dict(op=op, tokens=tokens, experts=experts, k=rng.randint(1, min(12, top_groups * size)),
                    score=rng.choice(("softmax", "sigmoid")), dtype=rng.choice(("fp32", "bf16")), bias=rng.random() < 0.5,
                    groups=groups, top_groups=top_groups, group_top=min(size, rng.choice((1, 2))), renorm=rng.random() < 0.6,
                    scale=rng.choice((1.0, 2.5)), padded=rng.choice((0.0, 0.0, 0.1)))
    if op in ("dispatch", "combine", "combine_bwd"):
        d, k = 8 * spread(8, 640), rng.randint(1, 8)
        tokens = spread(1, 8192)
        while tokens * k * d > 8192 * 2 * 5120:
            tokens //= 2
        return dict(op=op, tokens=tokens, experts=spread(8, 128), k=k, d=d, ys="bf16" if op != "combine" else rng.choice(("bf16", "fp32")),
                    out="bf16" if op != "combine" else rng.choice(("bf16", "fp32")), residual=op == "combine" and rng.random() < 0.5,
                    padded=rng.choice((0.0, 0.0, 0.1)))
    act = rng.choice(("none", "relu", "relu2", "gelu", "silu"))
    d, n, rows = 8 * spread(8, 640), 8 * spread(8, 2560), spread(1, 8192)
    if op == "linear_bwd":
        n = min(n, 5120)
        rows = min(rows, 4096)
        return dict(op=op, rows=rows, d=d, n=n, act=act)
    return dict(op=op, rows=rows, d=d, n=n if rng.random() < 0.7 else n - rng.randrange(8), act=act, out=rng.choice(("bf16", "bf16", "fp32")),
                bias=rng.random() < 0.7, residual=rng.choice(("", "bf16", "fp32")), pre=rng.random() < 0.3)


def size_of(dtype):
    return 4 if dtype == "fp32" else 2


def work(case):
    op = case["op"]
    if op in ("route", "route_bwd"):
        t, e, k = case["tokens"], case["experts"], case["k"]
        logits = t * e * size_of(case["dtype"])
        if op == "route":
            return {"bytes": logits + 16 * t * k + 4 * e * (2 if case["bias"] else 1), "flops": 4 * t * e}
        if case["score"] == "softmax" and not case["renorm"]:
            return {"bytes": 2 * logits + 8 * t * k, "flops": 6 * t * e}
        return {"bytes": logits + 8 * t * k + min(logits, 4 * t * k), "flops": t * e + 8 * t * k}
    if op in ("dispatch", "combine", "combine_bwd"):
        t, k, d = case["tokens"], case["k"], case["d"]
        t = t - int(t * case["padded"])
        if op == "dispatch":
            return {"bytes": 2 * t * d * (1 + k) + 4 * t * k, "flops": 0}
        if op == "combine":
            out = size_of(case["out"]) * case["tokens"] * d
            return {"bytes": size_of(case["ys"]) * t * k * d + out * (2 if case["residual"] else 1) + 8 * t * k, "flops": 2 * t * k * d}
        return {"bytes": 2 * t * d * (1 + 2 * k) + 12 * t * k, "flops": 3 * t * k * d}
    m, d, n = case["rows"], case["d"], case["n"]
    if op == "linear_bwd":
        pre = 0 if case["act"] == "none" else 2 * m * n
        return {"bytes": 2 * m * n + pre + 4 * m * d + 6 * n * d + 4 * n, "flops": 4 * m * n * d}
    out = size_of(case["out"]) * m * n + (2 * m * n if case["pre"] else 0) + (size_of(case["residual"]) * m * n if case["residual"] else 0)
    return {"bytes": 2 * m * d + 2 * n * d + out + (4 * n if case["bias"] else 0), "flops": 2 * m * n * d}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype="bf16"):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std).to(DTYPES[dtype])

    op, s = case["op"], {"case": case}
    if op in ("gemm", "linear_bwd"):
        m, d, n = case["rows"], case["d"], case["n"]
        s |= {"x": normal(m, d), "w": normal(n, d, std=1.5 / math.sqrt(d))}
        if op == "linear_bwd":
            s |= {"dy": normal(m, n, std=1e-3), "pre": normal(m, n, std=1.5),
                  "dx": torch.zeros(m, d, device="cuda", dtype=torch.bfloat16), "dw": torch.zeros(n, d, device="cuda"), "db": torch.zeros(n, device="cuda")}
            return s
        s["bias"] = normal(n, std=0.5, dtype="fp32") if case["bias"] else None
        s["residual"] = normal(m, n, dtype=case["residual"]) if case["residual"] else None
        s["pre"] = torch.zeros(m, n, device="cuda", dtype=torch.bfloat16) if case["pre"] else None
        s["out"] = torch.zeros(m, n, device="cuda", dtype=DTYPES[case["out"]])
        return s
    t, e, k = case["tokens"], case["experts"], case["k"]
    valid = None
    if case["padded"]:
        valid = torch.ones(t, device="cuda", dtype=torch.bool)
        valid[t - int(t * case["padded"]):] = False
    s["valid"] = valid
    if op in ("route", "route_bwd"):
        s["logits"] = normal(t, e, std=1.5, dtype=case["dtype"])
        s["bias"] = normal(e, std=0.1, dtype="fp32") if case["bias"] else None
        if op == "route_bwd":
            s["routes"] = plain_route(s, case)
            s["dweights"] = normal(t, k, dtype="fp32")
            s["out"] = torch.zeros_like(s["logits"])
        return s
    d = case["d"]
    experts = torch.rand(t, e, generator=gen, device="cuda").argsort(1)[:, :k].int()
    weights = torch.rand(t, k, generator=gen, device="cuda") + 0.05
    weights = weights / weights.sum(1, keepdim=True)
    if valid is not None:
        experts[~valid] = -1
        weights[~valid] = 0
    s["routes"] = (experts, weights, *layout(experts, e))
    if op == "dispatch":
        s |= {"x": normal(t, d), "out": torch.zeros(t * k, d, device="cuda", dtype=torch.bfloat16)}
    elif op == "combine":
        s |= {"ys": normal(t * k, d, dtype=case["ys"]), "out": torch.zeros(t, d, device="cuda", dtype=DTYPES[case["out"]])}
        s["residual"] = normal(t, d, dtype=case["out"]) if case["residual"] else None
    else:
        s |= {"ys": normal(t * k, d), "dy": normal(t, d, std=1e-3), "dys": torch.zeros(t * k, d, device="cuda", dtype=torch.bfloat16),
              "dweights": torch.zeros(t, k, device="cuda")}
    return s


def layout(experts, count):
    """Rows of the choices sorted by expert, the choice of each row (-1 behind the last) and the experts' offsets."""
    flat = experts.reshape(-1).long()
    key = torch.where(flat < 0, count, flat)
    order = torch.sort(key, stable=True)[1]
    place = torch.empty_like(order)
    place[order] = torch.arange(len(order), device=order.device)
    rows = torch.where(flat < 0, -1, place).int().view(experts.shape)
    held = torch.zeros(count + 1, device=order.device, dtype=torch.long).scatter_add_(0, key, torch.ones_like(key))[:count]
    offsets = torch.cat([torch.zeros(1, device=order.device, dtype=torch.long), held.cumsum(0)]).int()
    sources = torch.where(torch.arange(len(order), device=order.device) < offsets[-1], order, -1).int()
    return rows, sources, offsets


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------
def run(s):
    case = s["case"]
    if own:
        return run_own(s, case)
    return PLAIN[case["op"]](s, case)


def run_own(s, case):
    import nvfp4_bit_quantized_02_b200 as nv
    op = case["op"]
    if op == "gemm":
        y = nv.nvfp4_bf16_gemm_act(s["x"], s["w"], s["bias"], act=getattr(nv, "ACT_" + case["act"].upper()), residual=s["residual"],
                                   pre=s["pre"], out=s["out"])
        return [y, s["pre"]] if case["pre"] else [y]
    if op == "linear_bwd":
        if "layer" not in s:   # a training run keeps its layers
            s["layer"] = nv.LinearActBF16(case["rows"], case["d"], case["n"], act=getattr(nv, "ACT_" + case["act"].upper()))
        return list(s["layer"].bwd(s["x"], s["w"], s["dy"], s["pre"], dx=s["dx"], dw=s["dw"], dbias=s["db"]))
    if op in ("route", "route_bwd"):
        score = nv.SCORE_SOFTMAX if case["score"] == "softmax" else nv.SCORE_SIGMOID
        if op == "route":
            if "held" not in s:   # a program's buffers of a route
                s["held"] = nv.Routes.empty(case["tokens"], case["experts"], case["k"])
            r = nv.nvfp4_route(s["logits"], case["k"], score=score, bias=s["bias"], groups=case["groups"], top_groups=case["top_groups"],
                               group_top=case["group_top"], renormalize=case["renorm"], scale=case["scale"], valid=s["valid"], out=s["held"])
            return [r.experts, r.weights, r.rows, r.sources, r.offsets]
        return nv.nvfp4_route_bwd(s["dweights"], s["logits"], own_routes(nv, s), score=score, renormalize=case["renorm"],
                                  scale=case["scale"], out=s["out"])
    if op == "dispatch":
        return nv.nvfp4_dispatch(s["x"], own_routes(nv, s), out=s["out"])
    if op == "combine":
        # an fp32 residual is the running sum itself, as in the plain form
        out = s["residual"] if case["residual"] and case["out"] == "fp32" else s["out"]
        return nv.nvfp4_combine(s["ys"], own_routes(nv, s), residual=s["residual"], out=out)
    return list(nv.nvfp4_combine_bwd(s["dy"], s["ys"], own_routes(nv, s), dys=s["dys"], dweights=s["dweights"]))


def own_routes(nv, s):
    if "held" not in s:
        s["held"] = nv.Routes(*s["routes"])
    return s["held"]


def plain_route(s, case):
    x = s["logits"].float()
    t, e = x.shape
    k, g = case["k"], case["groups"]
    size = e // g
    wide = x.double()                                  # scores next to one another are told apart in 64 bits
    if case["score"] == "softmax":
        top = torch.exp(wide - wide.amax(1, keepdim=True))
        score = top / top.sum(1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-wide))
    plain_order = s["bias"] is None and case["group_top"] == 1
    choice = wide if plain_order else score if s["bias"] is None else score + s["bias"].double()
    if g > 1:
        best = torch.sort(choice.view(t, g, size), dim=2, descending=True)[0][:, :, :case["group_top"]].sum(2)
        keep = torch.sort(best, dim=1, descending=True, stable=True)[1][:, :case["top_groups"]]
        mask = torch.zeros(t, g, device=x.device, dtype=torch.bool).scatter_(1, keep, True)
        if s["bias"] is None:
            choice = wide
        choice = torch.where(mask.repeat_interleave(size, 1), choice, -math.inf)
    elif s["bias"] is None:
        choice = wide
    experts = torch.sort(choice, dim=1, descending=True, stable=True)[1][:, :k]
    weights = score.gather(1, experts)
    if case["renorm"]:
        weights = weights / weights.sum(1, keepdim=True)
    weights = (weights * case["scale"]).float()
    experts = experts.int()
    if s["valid"] is not None:
        experts = torch.where(s["valid"][:, None], experts, -1)
        weights = torch.where(s["valid"][:, None], weights, 0.0)
    return [experts, weights, *layout(experts, e)]


def plain_route_bwd(s, case):
    x, g = s["logits"].float(), s["dweights"]
    experts, weights = s["routes"][:2]
    held = experts >= 0
    at = experts.clamp(min=0).long()
    g = torch.where(held, g, 0.0) * case["scale"]
    if case["score"] == "softmax":
        p = torch.exp(x - x.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-x))
    chosen = p.gather(1, at)
    if case["renorm"]:
        share = weights / case["scale"]
        d = share * (g - (g * share).sum(1, keepdim=True))
        if case["score"] == "sigmoid":
            d = d * (1.0 - chosen)
        d = torch.where(held, d, 0.0)
        return s["out"].copy_(torch.zeros_like(x).scatter_add_(1, at, d))
    if case["score"] == "sigmoid":
        return s["out"].copy_(torch.zeros_like(x).scatter_add_(1, at, g * chosen * (1.0 - chosen)))
    dp = torch.zeros_like(x).scatter_add_(1, at, g)
    return s["out"].copy_(p * (dp - (dp * p).sum(1, keepdim=True)))


def choices(s):
    """Tokens, places and rows of the choices that have a row."""
    rows = s["routes"][2]
    token, j = torch.nonzero(rows >= 0, as_tuple=True)
    return token, j, rows[token, j].long()


def plain_dispatch(s, case):
    token, _, row = choices(s)
    s["out"][row] = s["x"][token]
    return s["out"]


def plain_combine(s, case):
    token, j, row = choices(s)
    y = torch.zeros(s["out"].shape, device="cuda") if s["residual"] is None else s["residual"].float()
    experts, weights = s["routes"][:2]
    for place in range(case["k"]):                    # one choice after the other, so that no order is left open
        at = j == place
        y[token[at]] += weights[token[at], place, None] * s["ys"][row[at]].float()
    return s["out"].copy_(y)


def plain_combine_bwd(s, case):
    token, j, row = choices(s)
    dy, weights = s["dy"][token].float(), s["routes"][1][token, j]
    s["dys"][row] = (dy * weights[:, None]).to(s["dys"].dtype)
    s["dweights"].zero_()
    s["dweights"][token, j] = (dy * s["ys"][row].float()).sum(1)
    return [s["dys"], s["dweights"]]


def act_of(name, h):
    if name == "relu":
        return torch.clamp(h, min=0)
    if name == "relu2":
        return torch.clamp(h, min=0) ** 2
    if name == "gelu":
        return 0.5 * h * torch.erfc(h * -math.sqrt(0.5))
    if name == "silu":
        return h / (1.0 + torch.exp(-h))
    return h


def slope_of(name, h):
    if name == "relu":
        return (h > 0).to(h.dtype)
    if name == "relu2":
        return 2 * torch.clamp(h, min=0)
    if name == "gelu":
        return 0.5 * torch.erfc(h * -math.sqrt(0.5)) + h * torch.exp(-0.5 * h * h) / math.sqrt(2 * math.pi)
    if name == "silu":
        p = 1.0 / (1.0 + torch.exp(-h))
        return p * (1.0 + h * (1.0 - p))
    return torch.ones_like(h)


def plain_gemm(s, case):
    h = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        h = h + s["bias"]
    if case["pre"]:
        s["pre"].copy_(h)
    y = act_of(case["act"], h)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    s["out"].copy_(y)
    return [s["out"], s["pre"]] if case["pre"] else [s["out"]]


def plain_linear_bwd(s, case):
    dh = s["dy"].float() * slope_of(case["act"], s["pre"].float())
    s["db"].copy_(dh.sum(0))
    held = dh.bfloat16().float()                      # what the two products take
    s["dx"].copy_(held @ s["w"].float())
    s["dw"].copy_(held.t() @ s["x"].float())
    return [s["dx"], s["dw"], s["db"]]


PLAIN = {"route": plain_route, "route_bwd": plain_route_bwd, "dispatch": plain_dispatch, "combine": plain_combine,
         "combine_bwd": plain_combine_bwd, "gemm": plain_gemm, "linear_bwd": plain_linear_bwd}


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gemm":
        h = torch.einsum("md,nd->mn", s["x"].double(), s["w"].double())
        if s["bias"] is not None:
            h += s["bias"].double()
        y = exact_act(case["act"], h)
        if s["residual"] is not None:
            y = y + s["residual"].double()
        return [y, h] if case["pre"] else [y]
    if op == "linear_bwd":
        h = s["pre"].double().requires_grad_()
        slope, = torch.autograd.grad(exact_act(case["act"], h).sum(), h)
        dh = s["dy"].double() * slope
        held = dh.bfloat16().double()
        return [torch.einsum("mn,nd->md", held, s["w"].double()), torch.einsum("mn,md->nd", held, s["x"].double()), dh.sum(0)]
    if op == "route":
        return exact_route(s, case)
    if op == "route_bwd":
        return exact_route_bwd(s, case)
    experts, weights, rows, sources, offsets = s["routes"]
    live = int(offsets[-1])
    source = sources[:live].long()
    token = source // case["k"]
    if op == "dispatch":
        out = s["out"].double()
        out[:live] = s["x"].double()[token]
        return out
    if op == "combine":
        y = torch.zeros(s["out"].shape, device="cuda", dtype=torch.float64)
        y.index_add_(0, token, s["ys"][:live].double() * weights.double().view(-1)[source][:, None])
        return y if s["residual"] is None else y + s["residual"].double()
    dys = s["dys"].double()
    dys[:live] = s["dy"].double()[token] * weights.double().view(-1)[source][:, None]
    dw = torch.zeros(weights.numel(), device="cuda", dtype=torch.float64)
    dw[source] = torch.einsum("rd,rd->r", s["dy"].double()[token], s["ys"][:live].double())
    return [dys, dw.view(weights.shape)]


def exact_act(name, h):
    if name == "gelu":
        return h * torch.special.ndtr(h)
    if name == "silu":
        return h * torch.special.expit(h)
    return {"none": lambda v: v, "relu": torch.relu, "relu2": lambda v: torch.relu(v).square()}[name](h)


def exact_score(case, x):
    return torch.softmax(x, 1) if case["score"] == "softmax" else torch.special.expit(x)


def exact_route(s, case):
    x = s["logits"].double()
    t, e = x.shape
    score = exact_score(case, x)
    value = score if s["bias"] is None else score + s["bias"].double()
    left = x.clone() if s["bias"] is None else value.clone()          # what a choice goes by
    if case["groups"] > 1:
        group = (value if case["group_top"] > 1 else left).view(t, case["groups"], -1).topk(case["group_top"], 2)[0].sum(2)
        shut = torch.ones_like(group, dtype=torch.bool)
        for _ in range(case["top_groups"]):
            at = first_of_max(group.masked_fill(~shut, -math.inf))
            shut[torch.arange(t, device=x.device), at] = False
        left = left.view(t, case["groups"], -1).masked_fill(shut[:, :, None], -math.inf).view(t, e)
    picked = []
    for _ in range(case["k"]):
        at = first_of_max(left)
        left[torch.arange(t, device=x.device), at] = -math.inf
        picked.append(at)
    experts = torch.stack(picked, 1)
    weights = score.gather(1, experts)
    if case["renorm"]:
        weights = weights / weights.sum(1, keepdim=True)
    weights = weights * case["scale"]
    if s["valid"] is not None:
        experts[~s["valid"]] = -1
        weights[~s["valid"]] = 0
    # each expert's choices, one expert after the other
    flat, rows, sources, ends = experts.view(-1), torch.full((t * case["k"],), -1, device=x.device), [], [0]
    for i in range(e):
        own_choices = torch.nonzero(flat == i).view(-1)
        rows[own_choices] = ends[-1] + torch.arange(len(own_choices), device=x.device)
        sources.append(own_choices)
        ends.append(ends[-1] + len(own_choices))
    sources = torch.cat(sources + [torch.full((t * case["k"] - ends[-1],), -1, device=x.device)])
    return [experts.int(), weights, rows.int().view(t, -1), sources.int(), torch.tensor(ends, device=x.device, dtype=torch.int32)]


def first_of_max(x):
    """The lowest index of each row's largest value."""
    index = torch.arange(x.shape[1], device=x.device).expand(x.shape)
    return torch.where(x == x.amax(1, keepdim=True), index, x.shape[1]).amin(1)


def exact_route_bwd(s, case):
    x = s["logits"].double().requires_grad_()
    experts = s["routes"][0].long()
    w = exact_score(case, x).gather(1, experts.clamp(min=0))
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    grad, = torch.autograd.grad((w * case["scale"] * torch.where(experts >= 0, s["dweights"].double(), 0.0)).sum(), x)
    return grad
