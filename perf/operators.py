"""Operators of a trained expert layer, as cases to measure: the products grouped by expert
(forward, input gradient, weight gradient) and the AdamW step over many tensors.

Rows of tokens are sorted by expert: expert e owns rows [offsets[e], offsets[e + 1]) and has a
weight of its own.  Some experts own no row (`idle`), the others own at least one each; rows
behind the last offset belong to nobody.

The AdamW step updates fp32 master weights from fp32 or bf16 gradients and writes the bf16 weights
of the next forward pass.  Its moments are held in fp32, or in 8 bits: E4M3 codes with one fp32
scale per 256 elements, the second moment as its square root, rounded stochastically from
Philox4x32-10 under a given seed.

`run` computes in elementary torch operations, or with `own` through the package.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 256                          # elements per scale of an 8-bit moment
BETA1, BETA2, EPS, DECAY = 0.9, 0.95, 1e-8, 0.1
STREAM_M, STREAM_V = 4, 5            # Philox counter word 2 of the two moments


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------
def listed():
    def fwd(name, rows, experts, idle, d, n, out="bf16", behind=0, skew=0.6):
        return dict(name=name, op="fwd", rows=rows, behind=behind, experts=experts, idle=idle, d=d, n=n, out=out, skew=skew)

    def grad(name, op, rows, experts, idle, d, n, out, behind=0, skew=0.6, add=False):
        return dict(name=name, op=op, rows=rows, behind=behind, experts=experts, idle=idle, d=d, n=n, out=out, skew=skew, add=add)

    def adamw(name, state, tensors, lo, hi, odd, grad):
        return dict(name=name, op="adamw", state=state, tensors=tensors, lo=lo, hi=hi, odd=odd, grad=grad)

    return [
        # one token, two experts of 16: the answer of a served model, where latency counts
        fwd("fwd 1 token top 2", 2, 16, 14, 2048, 704),
        # a served batch of 24 tokens, two experts each, over the 5120 x 20480 projection cut in 16 experts
        fwd("fwd 48 rows", 48, 16, 2, 5120, 1280),
        # that projection's training step at 16384 rows
        fwd("fwd 16384 rows", 16384, 16, 0, 5120, 1280),
        # many small experts, a padded batch, odd sizes, fp32 logits of a gate's second product
        fwd("fwd ragged fp32", 3001, 40, 3, 1032, 712, "fp32", behind=95, skew=1.0),
        # wide experts at the largest batch
        fwd("fwd 32768 rows wide", 32768, 8, 0, 5120, 5120),
        # the input gradient of the 16384-row step
        grad("dgrad 16384 rows", "dgrad", 16384, 16, 0, 5120, 1280, "bf16"),
        # the weight gradient of the 16384-row step
        grad("wgrad 16384 rows", "wgrad", 16384, 16, 0, 5120, 1280, "fp32"),
        # a micro-batch's weight gradients added onto those of the ones before it, short ragged runs of tokens
        grad("wgrad ragged added", "wgrad", 2003, 40, 3, 1032, 712, "fp32", behind=45, skew=1.0, add=True),
        # the norms and biases of a small model: latency
        adamw("adamw small", "fp32", 24, 320, 40960, True, "fp32"),
        # both projections of the 5120 x 20480 feed-forward layer, moments in fp32
        adamw("adamw ffn fp32", "fp32", 2, 5120 * 20480, 5120 * 20480, False, "fp32"),
        # one layer's tensors, moments in 8 bits: latency
        adamw("adamw small fp8", "fp8", 9, 257, 65536, True, "fp32"),
        # a model's two hundred tensors of odd sizes, gradients in bf16, moments in 8 bits
        adamw("adamw model fp8", "fp8", 200, 1000, 4800000, True, "bf16"),
    ]


def draw(rng: random.Random):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("fwd", "fwd", "dgrad", "wgrad", "adamw", "adamw"))
    if op == "adamw":
        tensors, hi = spread(1, 300), spread(300, 20000000)
        while tensors * hi > 150000000:
            tensors = max(1, tensors // 2)
        return dict(op=op, state=rng.choice(("fp32", "fp8")), tensors=tensors, lo=max(1, hi // spread(1, 300)), hi=hi, odd=rng.random() < 0.7,
                    grad=rng.choice(("fp32", "bf16")))
    experts = spread(1, 64)
    d, n = 8 * spread(8, 640), 8 * spread(8, 640)
    while experts * d * n > 160000000:
        experts = max(1, experts // 2)
        if experts == 1:
            break
    idle = rng.randrange(experts) if rng.random() < 0.4 else 0
    rows = spread(1, 24000)
    idle = max(idle, experts - rows)
    c = dict(op=op, rows=rows, behind=rng.choice((0, 0, 1, 77)), experts=experts, idle=idle, d=d, n=n,
             out="fp32" if op == "wgrad" else rng.choice(("bf16", "fp32")), skew=rng.choice((0.0, 0.6, 1.0)))
    if op != "fwd":
        c["add"] = op == "wgrad" and rng.random() < 0.5
    return c


def sizes_of(case):
    t, lo, hi = case["tensors"], case["lo"], case["hi"]
    ns = [int(round(lo * (hi / lo) ** (i / max(1, t - 1)))) for i in range(t)]
    return [n | 1 for n in ns] if case["odd"] else ns


def work(case):
    if case["op"] == "adamw":
        n = sum(sizes_of(case))
        blocks = sum(-(-k // BLOCK) for k in sizes_of(case))
        state = 2 * 2 * (4 * n) if case["state"] == "fp32" else 2 * 2 * (n + 4 * blocks)   # both moments, read and written
        return {"bytes": 8 * n + (4 if case["grad"] == "fp32" else 2) * n + 2 * n + state, "flops": 14 * n}
    rows, d, n = case["rows"], case["d"], case["n"]
    w = (case["experts"] - case["idle"]) * d * n
    size = 2 if case["out"] == "bf16" else 4
    flops = 2 * rows * d * n
    if case["op"] == "wgrad":
        # every expert's gradient is written (that of an idle one is zero); an added one is read too, where it changes
        out = w * 8 if case["add"] else case["experts"] * d * n * 4
        return {"bytes": 2 * rows * (d + n) + out, "flops": flops}
    k, m = (d, n) if case["op"] == "fwd" else (n, d)
    return {"bytes": 2 * rows * k + 2 * w + size * rows * m, "flops": flops}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def rows_of_experts(case, seed):
    """How many rows each expert owns: `idle` experts none, the others one and a skewed share of the rest."""
    r = np.random.default_rng(seed)
    e, busy = case["experts"], case["experts"] - case["idle"]
    share = np.exp(case["skew"] * r.standard_normal(busy))
    counts = np.zeros(e, np.int64)
    counts[np.sort(r.permutation(e)[:busy])] = 1 + r.multinomial(case["rows"] - busy, share / share.sum())
    return counts


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std).to(dtype)

    if case["op"] == "adamw":
        ns = sizes_of(case)
        starts = np.concatenate([[0], np.cumsum([-(-n // BLOCK) * BLOCK for n in ns])])
        total = int(starts[-1])
        at = torch.arange(total, device="cuda")
        tensor = torch.searchsorted(torch.tensor(starts[1:], device="cuda"), at, right=True)
        start = torch.tensor(starts, device="cuda")[tensor]
        inside = at - start < torch.tensor(ns, device="cuda")[tensor]     # the flat buffers are zero between the tensors
        del at
        p = normal(total, std=0.02, dtype=torch.float32).mul_(inside)
        g = normal(total, std=1e-4, dtype=torch.float32).mul_(inside)
        m = normal(total, std=3e-5, dtype=torch.float32).mul_(inside)
        v = normal(total, std=1e-4, dtype=torch.float32).square_().add_(1e-10).mul_(inside)
        s = {"case": case, "ns": ns, "starts": starts.tolist(), "p": p, "g": g if case["grad"] == "fp32" else g.bfloat16(), "w": p.bfloat16(),
             "lr": 3e-4, "step": 500, "sr_seed": (seed * 0x9E3779B97F4A7C15 + 1) % 2 ** 63}
        if case["state"] == "fp32":
            s |= {"m": m, "v": v}
        else:
            for name, x in (("m", m), ("v", v.sqrt())):
                b = x.view(-1, BLOCK)
                scale = b.abs().amax(1) / 448
                s[name] = (b / scale.clamp(min=1e-30)[:, None]).to(torch.float8_e4m3fn).view(-1)
                s[name + "_scale"] = scale
            s |= {"tensor": tensor[::8].clone(), "group": (torch.arange(total, device="cuda")[::8] - start[::8]) // 8}
        return s

    counts = rows_of_experts(case, seed)
    rows, e, d, n = case["rows"], case["experts"], case["d"], case["n"]
    every = rows + case["behind"]
    s = {"case": case, "offsets": torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda"), "most": int(counts.max())}
    if case["op"] == "wgrad":
        s |= {"dy": normal(every, n, std=1e-4), "x": normal(every, d)}
        s["out"] = normal(e, n, d, std=1e-3, dtype=torch.float32) if case["add"] else torch.zeros(e, n, d, device="cuda")
        return s
    s["a"] = normal(every, d) if case["op"] == "fwd" else normal(every, n, std=1e-4)
    s["w"] = normal(e, n, d, std=0.02)
    s["out"] = torch.zeros(every, n if case["op"] == "fwd" else d, device="cuda", dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32)
    return s


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------
def run(s):
    case = s["case"]
    if own:
        return run_own(s, case)
    if case["op"] == "adamw":
        return plain_adamw(s, case)
    return plain_grouped(s, case)


def run_own(s, case):
    import nvfp4_bit_quantized_02_b200 as nv
    if case["op"] == "fwd":
        return nv.nvfp4_bf16_gemm_grouped(s["a"], s["w"], s["offsets"], out=s["out"])
    if case["op"] == "dgrad":
        return nv.nvfp4_bf16_gemm_grouped(s["a"], s["w"], s["offsets"], b_kn=True, out=s["out"])
    if case["op"] == "wgrad":
        return nv.nvfp4_bf16_wgrad_grouped(s["dy"], s["x"], s["offsets"], out=s["out"], accumulate=case["add"])
    fp8 = case["state"] == "fp8"
    if "ctx" not in s:   # the tensors of a training run stay where they are from step to step
        def cut(name, per=1):
            return [s[name][a // per:a // per + -(-n // per)] for a, n in zip(s["starts"], s["ns"])]

        scales = {"m_scale": cut("m_scale", BLOCK), "v_scale": cut("v_scale", BLOCK)} if fp8 else {}
        s["ctx"] = nv.AdamWContext(cut("p"), cut("g"), cut("w"), m=cut("m"), v=cut("v"), state=nv.STATE_FP8 if fp8 else nv.STATE_FP32, **scales)
    nv.nvfp4_adamw_step(s["ctx"], s["lr"], s["step"], beta1=BETA1, beta2=BETA2, eps=EPS, weight_decay=DECAY, mode=nv.SR, sr_seed=s["sr_seed"])
    return outputs(s, fp8)


def outputs(s, fp8):
    """8-bit moments as float8 numbers, in units of their blocks' scales, and the scales."""
    return [s[k] for k in ("p", "w", "m", "v") + (("m_scale", "v_scale") if fp8 else ())]


def padded(x, expert, place, experts, most):
    """The rows of x [rows][k] by expert, as fp32 [experts][most][k] with zeros behind each expert's rows."""
    out = torch.zeros(experts, most, x.shape[1], device=x.device)
    out[expert, place] = x.float()
    return out


def plain_grouped(s, case):
    rows, experts, out = case["rows"], case["experts"], s["out"]
    at = torch.arange(rows, device=out.device)
    expert = torch.searchsorted(s["offsets"][1:].contiguous(), at, right=True)
    place = at - s["offsets"][expert]
    if case["op"] == "wgrad":
        dy, x = (padded(s[k][:rows], expert, place, experts, s["most"]) for k in ("dy", "x"))
        dw = torch.bmm(dy.transpose(1, 2), x)
        return out.add_(dw) if case["add"] else out.copy_(dw)
    a = padded(s["a"][:rows], expert, place, experts, s["most"])
    w = s["w"].float()
    y = torch.bmm(a, w.transpose(1, 2) if case["op"] == "fwd" else w)
    out[:rows] = y[expert, place].to(out.dtype)
    return out


def factors(s):
    """The step's scalars: the weight decay's factor, the step size and the second moment's correction."""
    return 1.0 - s["lr"] * DECAY, s["lr"] / (1.0 - BETA1 ** s["step"]), 1.0 / math.sqrt(1.0 - BETA2 ** s["step"])


def plain_adamw(s, case):
    keep, size, fix = factors(s)
    fp8 = case["state"] == "fp8"
    g = s["g"].float()
    if fp8:
        m, r = decoded(s, "m"), decoded(s, "v")
        v = r * r
    else:
        m, v = s["m"], s["v"]
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + (g * (1.0 - BETA2)) * g
    r = torch.sqrt(v)
    s["p"].copy_(s["p"] * keep - (m / (r * fix + EPS)) * size)
    s["w"].copy_(s["p"])
    if fp8:
        encode(s, "m", m, STREAM_M)
        encode(s, "v", r, STREAM_V)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    return outputs(s, fp8)


def decoded(s, name):
    return (s[name].float().view(-1, BLOCK) * s[name + "_scale"][:, None]).view(-1)


def encode(s, name, x, stream):
    """x into E4M3 codes with a scale per block, rounded up where the element's 16 random bits are below the
    fraction of the step that is cut off."""
    b = x.view(-1, BLOCK)
    top = b.abs().amax(1)
    held = top >= 2.0 ** -100          # a block below that is held as zero
    scale = torch.where(held, top / 448, 0.0)
    per = torch.where(held, 448 / torch.where(held, top, 1.0), 0.0)
    u = (b.abs() * per[:, None]).view(-1)
    low = u < 2.0 ** -6                # below the normal numbers: one step, that of the binade above 2^-6
    t = torch.where(low, u + 2.0 ** -6, u).view(torch.int32)
    t = t + (0xFFFFF - (fields(s, stream) << 4))
    code = ((t >> 20) - 960 - 8 * low.int()).clamp(max=0x7E)
    code = code | torch.where(torch.signbit(x), 128, 0)
    s[name].copy_(code.to(torch.uint8).view(torch.float8_e4m3fn))
    s[name + "_scale"].copy_(scale)


def fields(s, stream):
    """The 16 random bits of each element: eight fields, low halves first, of the Philox4x32-10 block with key
    sr_seed and counter (element / 8, stream, tensor)."""
    def times(a, b):                   # the high and low words of a product of 32-bit words
        low, high = (b & 0xFFFF) * a, (b >> 16) * a
        mid = (low >> 16) + high
        return mid >> 16, ((mid & 0xFFFF) << 16) | (low & 0xFFFF)

    c = [s["group"] & 0xFFFFFFFF, s["group"] >> 32, torch.full_like(s["group"], stream), s["tensor"]]
    key = [s["sr_seed"] & 0xFFFFFFFF, s["sr_seed"] >> 32]
    for _ in range(10):
        (h0, l0), (h1, l1) = times(0xD2511F53, c[0]), times(0xCD9E8D57, c[2])
        c = [h1 ^ c[1] ^ key[0], l1, h0 ^ c[3] ^ key[1], l0]
        key = [(key[0] + 0x9E3779B9) & 0xFFFFFFFF, (key[1] + 0xBB67AE85) & 0xFFFFFFFF]
    words = torch.stack(c, 1)
    return torch.stack([words & 0xFFFF, words >> 16], 2).view(-1).int()


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adamw":
        return exact_adamw(s, case)
    out = s["out"].double()
    ends = s["offsets"].tolist()
    for e in range(case["experts"]):
        a, b = ends[e], ends[e + 1]
        if case["op"] == "wgrad":
            dw = s["dy"][a:b].double().t() @ s["x"][a:b].double()
            out[e] = out[e] + dw if case["add"] else dw
        elif b > a:
            w = s["w"][e].double()
            out[a:b] = s["a"][a:b].double() @ (w.t() if case["op"] == "fwd" else w)
    return out


def exact_adamw(s, case):
    keep, size, fix = factors(s)
    g, p, t = s["g"].double(), s["p"].double(), {}
    if case["state"] == "fp8":
        for k in ("m", "v"):
            t[k] = s[k].double() * s[k + "_scale"].double().repeat_interleave(BLOCK)
        t["v"] = t["v"] ** 2
    else:
        t = {k: s[k].double() for k in ("m", "v")}
    m = BETA1 * t["m"] + (1 - BETA1) * g
    v = BETA2 * t["v"] + (1 - BETA2) * g * g
    p = keep * p - size * m / (v.sqrt() * fix + EPS)
    if case["state"] == "fp32":
        return [p, p, m, v]
    (mq, ms), (vq, vs) = exact_fp8(s, m, STREAM_M), exact_fp8(s, v.sqrt(), STREAM_V)
    return [p, p, mq, vq, ms, vs]


def exact_fp8(s, x, stream):
    top = x.view(-1, BLOCK).abs().amax(1)
    unit = (top / 448).repeat_interleave(BLOCK)
    u = torch.where(unit > 0, x.abs() / unit, 0.0)
    step = torch.ldexp(torch.ones_like(u), (torch.frexp(u.clamp(min=2.0 ** -6))[1] - 1 - 3).int())
    lo = torch.floor(u / step)
    word = 0xFFFFFFFF
    c0, c1, c2, c3 = s["group"] & word, s["group"] >> 32, torch.full_like(s["group"], stream), s["tensor"].clone()
    k0, k1 = s["sr_seed"] & word, s["sr_seed"] >> 32
    for _ in range(10):                # a product's 64 bits in a wrapping 64-bit integer
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((p1 >> 32) & word) ^ c1 ^ k0, p1 & word, ((p0 >> 32) & word) ^ c3 ^ k1, p0 & word
        k0, k1 = (k0 + 0x9E3779B9) & word, (k1 + 0xBB67AE85) & word
    r16 = torch.stack([h for c in (c0, c1, c2, c3) for h in (c & 0xFFFF, c >> 16)], 1).view(-1)
    up = r16 < (u / step - lo) * 65536
    return torch.copysign(((lo + up) * step).clamp(max=448), x), top / 448
