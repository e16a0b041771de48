"""Routing (nvfp4_route, nvfp4_route_bwd) against its definition in 64 bits.

The choices, rows, sources and offsets have to be equal.  Tolerances of the weights, in units of u = 2^-24:
expf errs by at most 4 u relative and its argument, a difference, by u |l - max|; a sum of 32 positive terms over
five steps by 5 u; a quotient and the scale by u each, and the sigmoid's 1 + e^-|l| and quotient by 6 u: renormalised
weights within (32 + 4 D) u, D the largest distance |l - max| among the chosen.  The softmax's sum over all takes
__expf, 2 + 1.173 |x| ulp of 2 u, weighted by the terms (sum p |x| <= 1 + ln E <= 8), so 24 u, and at most 37 adds:
(96 + 4 D) u.  The gradient n (g - sum g n) multiplies and subtracts such weights: three of them and
a sum of 32 terms, relative to n (|g| + sum |g| n).  A bf16 gradient adds half a step, 2^-8."""
import numpy as np
import pytest
import torch

from gpu_helpers import nv

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
INF = float("inf")


def _score(x, sigmoid):
    """s and the logits as they count: NaN and -inf are none, +inf is the largest number"""
    x = torch.where(torch.isnan(x), -INF, x.double()).clamp(max=float(np.finfo(np.float32).max))
    if sigmoid:
        return torch.where(x > -INF, 1.0 / (1.0 + torch.exp(-x)), 0.0), x
    top = x.amax(1, keepdim=True)
    e = torch.where(x > -INF, torch.exp(x - torch.where(top > -INF, top, 0.0)), 0.0)
    return e / e.sum(1, keepdim=True).clamp(min=1e-300), x


def reference(logits, k, sigmoid=False, bias=None, groups=1, top_groups=1, group_top=1, renormalize=True, scale=1.0, valid=None):
    s, x = _score(logits, sigmoid)
    T, E = x.shape
    c = x if bias is None else torch.where(x > -INF, s + bias.double(), -INF)
    c = torch.where(torch.isnan(c), -INF, c)
    if groups > 1:
        by = c if bias is not None or group_top == 1 else torch.where(x > -INF, s, -INF)
        score = by.view(T, groups, -1).topk(group_top, 2)[0].sum(2)
        order = torch.sort(score, dim=1, descending=True, stable=True)[1][:, :top_groups]
        stays = torch.zeros(T, groups, dtype=torch.bool).scatter_(1, order, True) & (score > -INF)
        c = torch.where(stays.repeat_interleave(E // groups, 1), c, -INF)
    value, chosen = torch.sort(c, dim=1, descending=True, stable=True)
    value, chosen = value[:, :k], chosen[:, :k].clone()
    held = value > -INF
    if valid is not None:
        held &= valid[:, None]
    w = torch.where(held, s.gather(1, chosen), 0.0)
    if renormalize:
        # from the logits, so that scores that underflow together keep their shares
        z = x.gather(1, chosen).clamp(max=0.0) if sigmoid else x.gather(1, chosen)
        z = torch.where(held, z, -INF)
        top = z.amax(1, keepdim=True)
        v = torch.where(held, torch.exp(z - torch.where(top > -INF, top, 0.0)), 0.0)
        if sigmoid:
            v = v / (1 + torch.exp(-x.gather(1, chosen).abs()))
        w = v / v.sum(1, keepdim=True).clamp(min=1e-300)
    chosen = torch.where(held, chosen, -1).int()
    flat = chosen.view(-1).long()
    order = torch.sort(torch.where(flat < 0, E, flat), stable=True)[1]
    rows = torch.empty(T * k, dtype=torch.long)
    rows[order] = torch.arange(T * k)
    rows[flat < 0] = -1
    offsets = torch.cat([torch.zeros(1, dtype=torch.long), torch.bincount(flat[flat >= 0], minlength=E).cumsum(0)])
    sources = torch.where(torch.arange(T * k) < offsets[-1], order, -1)
    return dict(experts=chosen, weights=w * scale, rows=rows.view(T, k).int(), sources=sources.int(), offsets=offsets.int(), held=held, x=x)


def check(logits, k, out=None, valid=None, bias=None, want=0, ws=None, **args):
    m = nv()
    ref = reference(logits, k, bias=bias, valid=valid, **args)
    sigmoid = args.pop("sigmoid", False)
    ws = ws or m.Workspace()
    r = m.nvfp4_route(logits.cuda(), k, score=m.SCORE_SIGMOID if sigmoid else m.SCORE_SOFTMAX, bias=None if bias is None else bias.cuda(),
                      valid=None if valid is None else valid.cuda(), ws=ws, out=out, **args)
    assert m.nvfp4_poll(ws) == want
    for name in ("experts", "offsets", "rows", "sources"):
        got = getattr(r, name).cpu()
        bad = torch.nonzero(got != ref[name])
        assert len(bad) == 0, f"{name}: {len(bad)} differ, first at {bad[0].tolist()}"
    got = r.weights.cpu().double()
    assert ((got == 0) | ref["held"]).all()
    x = ref["x"].gather(1, ref["experts"].clamp(min=0).long())
    whole = not args.get("renormalize", True)
    top = ref["x"].amax(1, keepdim=True) if whole else torch.where(ref["held"], x, -INF).amax(1, keepdim=True)
    far = torch.where(ref["held"], (x - top).abs(), 0.0).clamp(max=1e4)
    tol = ((96 if whole else 32) + 4 * far) * U * ref["weights"].abs() + 2.0 ** -125
    err = (got - ref["weights"]).abs()
    assert (err <= tol).all(), f"weights: worst {float((err / tol).max()):.3g} of the tolerance"
    return r, ref


def _logits(T, E, seed, dtype=torch.float32, std=1.5):
    return (torch.randn(T, E, generator=torch.Generator().manual_seed(seed)) * std).to(dtype)


def _bias(E, seed, std=0.1):
    return torch.randn(E, generator=torch.Generator().manual_seed(seed + 99)) * std


SHAPES = [(1, 16, 2), (2, 1, 1), (5, 7, 7), (3, 33, 32), (31, 40, 3), (64, 96, 6), (255, 256, 8), (256, 64, 1), (257, 64, 4), (300, 512, 12),
          (1000, 1024, 32), (3001, 72, 5), (7000, 10, 3)]


@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_route_sizes(shape, sigmoid):
    T, E, k = shape
    for n, (dtype, bias, renormalize) in enumerate([(torch.float32, False, True), (torch.float32, True, False), (torch.bfloat16, True, True),
                                                    (torch.bfloat16, False, False)]):
        check(_logits(T, E, T + n, dtype), k, sigmoid=sigmoid, bias=_bias(E, n) if bias else None, renormalize=renormalize, scale=2.5 if n else 1.0)


GROUPS = [(8, 64, 4, 8, 2, 1), (300, 256, 8, 8, 4, 2), (300, 96, 5, 3, 2, 2), (40, 1020, 9, 17, 4, 2), (33, 1024, 32, 32, 8, 1), (9, 30, 2, 5, 1, 2),
          (500, 24, 4, 12, 3, 2), (70, 32, 6, 32, 6, 1), (257, 160, 8, 4, 4, 1), (64, 1023, 7, 3, 1, 2), (20, 1008, 6, 9, 5, 2)]


@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("shape", GROUPS, ids=lambda s: "x".join(map(str, s)))
def test_route_groups(shape, sigmoid):
    T, E, k, groups, top_groups, group_top = shape
    for n, (dtype, bias) in enumerate([(torch.float32, True), (torch.float32, False), (torch.bfloat16, True), (torch.bfloat16, False)]):
        check(_logits(T, E, T + n, dtype), k, sigmoid=sigmoid, bias=_bias(E, n) if bias else None, groups=groups, top_groups=top_groups,
              group_top=group_top, renormalize=n % 2 == 0)


@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [(1, 1, 1), (8, 3, 1), (8, 3, 2)], ids=["whole", "best", "two"])
def test_ties_go_to_the_lowest_index(groups, sigmoid):
    g, tg, gt = groups
    gen = torch.Generator().manual_seed(5)
    few = torch.randint(-1, 2, (400, 64), generator=gen).float()   # three values: ties everywhere
    for bias in (None, torch.zeros(64), torch.randint(0, 2, (64,), generator=gen).float() * 0.25):
        for x in (few, few.bfloat16(), torch.zeros(400, 64), -torch.zeros(400, 64), torch.where(few > 0, 0.0, -0.0)):
            check(x, 6, sigmoid=sigmoid, bias=bias, groups=g, top_groups=tg, group_top=gt)


@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
def test_close_choices_are_told_apart(sigmoid):
    """Scores plus biases that differ by less than fp32 can hold: the bias takes back what the score gives, but
    for a few parts in 2^24."""
    gen = torch.Generator().manual_seed(6)
    x = torch.randn(600, 32, generator=gen)
    s, _ = _score(x[:1], sigmoid)
    bias = (0.75 - s[0]).float()             # every c of the first row next to 0.75
    near = x[:1] + torch.randint(-3, 4, (600, 32), generator=gen) * 2.0 ** -23
    for groups in ((1, 1, 1), (4, 2, 1), (4, 2, 2)):
        check(near, 8, sigmoid=sigmoid, bias=bias, groups=groups[0], top_groups=groups[1], group_top=groups[2])


@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_masked_experts(dtype, sigmoid):
    gen = torch.Generator().manual_seed(7)
    x = _logits(300, 48, 8, dtype)
    x[torch.rand(300, 48, generator=gen) < 0.6] = -INF
    x[3] = -INF                                        # nothing left
    x[4, 5:] = -INF                                    # fewer than k
    x[5] = torch.finfo(dtype).min                      # the lowest value: eligible, all alike
    x[6, 1:] = torch.finfo(dtype).min
    for bias in (None, _bias(48, 1)):
        for groups in ((1, 1, 1), (6, 2, 1), (6, 2, 2)):
            for renormalize in (False, True):
                check(x, 7, sigmoid=sigmoid, bias=bias, groups=groups[0], top_groups=groups[1], group_top=groups[2], renormalize=renormalize)
    bias = _bias(48, 2)
    bias[::5] = -INF
    check(x, 7, sigmoid=sigmoid, bias=bias)
    bias[3] = float("nan")
    check(x, 7, sigmoid=sigmoid, bias=bias)


@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
def test_non_finite_logits_are_flagged(sigmoid):
    m = nv()
    x = _logits(300, 40, 9)
    x[7, 3] = float("nan")
    check(x, 4, sigmoid=sigmoid, want=7)
    x[7, 3] = 0.5
    x[299, 39] = INF
    x[100, 2] = x[100, 30] = INF
    for bias in (None, _bias(40, 3)):
        for renormalize in (False, True):
            check(x, 4, sigmoid=sigmoid, bias=bias, renormalize=renormalize, want=7)
    # a padded token's logits are not read
    x = _logits(300, 40, 9)
    x[100:] = float("nan")
    check(x, 4, sigmoid=sigmoid, valid=torch.arange(300) < 100)


@pytest.mark.parametrize("T", [1, 90, 256, 2000])
def test_padded_tokens(T):
    gen = torch.Generator().manual_seed(T)
    for share in (0.0, 0.5, 1.0):
        valid = torch.rand(T, generator=gen) >= share
        check(_logits(T, 40, T), 3, valid=valid)
        check(_logits(T, 40, T), 3, valid=valid, sigmoid=True, bias=_bias(40, T))


def test_no_tokens():
    m = nv()
    r = m.nvfp4_route(torch.zeros(0, 40, device="cuda"), 3)
    assert r.offsets.tolist() == [0] * 41 and r.experts.shape == (0, 3)
    assert m.nvfp4_route_bwd(r.weights, torch.zeros(0, 40, device="cuda"), r).shape == (0, 40)


@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
def test_far_logits_keep_their_shares(sigmoid):
    # scores that underflow fp32 together: the renormalised weights do not
    x = _logits(64, 32, 11) - 200.0
    x[:, 20:] += 195.0
    bias = torch.zeros(32)
    bias[20:] = -5.0                      # the bias takes the choice to the far ones
    check(x, 4, sigmoid=sigmoid, bias=bias)
    check(_logits(64, 32, 12) * 1e4, 4, sigmoid=sigmoid)


@pytest.mark.parametrize("T", [3, 700])
def test_strides(T):
    for dtype in (torch.float32, torch.bfloat16):
        for E, ld in ((40, 41), (64, 72), (256, 260), (256, 300)):
            wide = torch.full((T, ld), 9.0, dtype=dtype)
            wide[:, :E] = _logits(T, E, E, dtype)
            m = nv()
            ref = reference(wide[:, :E], 4)
            x = wide.cuda()[:, :E]
            r = m.nvfp4_route(x, 4)
            assert torch.equal(r.experts.cpu(), ref["experts"]) and torch.equal(r.rows.cpu(), ref["rows"])
            out = torch.full((T, ld), 3.0, dtype=dtype, device="cuda")
            m.nvfp4_route_bwd(torch.ones(T, 4, device="cuda"), x, r, renormalize=False, out=out[:, :E])
            want = m.nvfp4_route_bwd(torch.ones(T, 4, device="cuda"), x.contiguous(), r, renormalize=False)
            assert torch.equal(out[:, :E], want) and (out[:, E:] == 3).all()


def test_captured_calls_and_streams():
    """Two graphs with routes of their own, replayed on two streams at once on changing logits; a call on a stream
    that is not the current one."""
    m = nv()
    T, E, k = 2000, 64, 4
    x = [_logits(T, E, s).cuda() for s in (1, 2)]
    bias = _bias(E, 1)
    routes = [m.Routes.empty(T, E, k) for _ in x]
    ws = [m.Workspace() for _ in x]
    graphs, streams = [], [torch.cuda.Stream() for _ in x]
    b = bias.cuda()
    for i in range(2):
        m.nvfp4_route(x[i], k, bias=b, out=routes[i], ws=ws[i])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.nvfp4_route(x[i], k, bias=b, out=routes[i], ws=ws[i])
        graphs.append(g)
    for seed in (10, 20, 30):
        data = [_logits(T, E, seed + i) for i in range(2)]
        for i in range(2):
            x[i].copy_(data[i])
        torch.cuda.synchronize()
        for _ in range(5):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            ref = reference(data[i], k, bias=bias)
            for name in ("experts", "rows", "sources", "offsets"):
                assert torch.equal(getattr(routes[i], name).cpu(), ref[name]), name
    s = torch.cuda.Stream()
    r = m.nvfp4_route(x[0], k, bias=b, stream=s)
    s.synchronize()
    assert torch.equal(r.rows.cpu(), routes[0].rows.cpu())


# ---------------------------------------------------------------------------------------
# gradient
# ---------------------------------------------------------------------------------------
def grad_formula(x, chosen, g, sigmoid, renormalize, scale):
    """dlogits, and the size of what its terms cancel from"""
    s, x = _score(x, sigmoid)
    held = (chosen >= 0) & (x.gather(1, chosen.clamp(min=0).long()) > -INF)
    at = chosen.clamp(min=0).long()
    g = torch.where(held, g.double() * scale, 0.0)
    p = torch.where(held, s.gather(1, at), 0.0)
    d, size = torch.zeros_like(x), torch.zeros_like(x)
    if renormalize:
        z = x.gather(1, at).clamp(max=0.0) if sigmoid else x.gather(1, at)
        z = torch.where(held, z, -INF)
        top = z.amax(1, keepdim=True)
        v = torch.where(held, torch.exp(z - torch.where(top > -INF, top, 0.0)), 0.0)
        if sigmoid:
            v = v / (1 + torch.exp(-x.gather(1, at).abs()))
        n = v / v.sum(1, keepdim=True).clamp(min=1e-300)
        dn, sn = n * (g - (g * n).sum(1, keepdim=True)), n * (g.abs() + (g * n).abs().sum(1, keepdim=True))
        if sigmoid:
            xa = x.gather(1, at)
            rest = torch.where(held, torch.where(xa >= 0, torch.exp(-xa.abs()), 1.0) / (1 + torch.exp(-xa.abs())), 0.0)
            dn, sn = dn * rest, sn * rest
        return d.scatter_add_(1, at, torch.where(held, dn, 0.0)), size.scatter_add_(1, at, torch.where(held, sn, 0.0))
    if sigmoid:
        xa = x.gather(1, at)
        rest = torch.where(xa >= 0, torch.exp(-xa.abs()), 1.0) / (1 + torch.exp(-xa.abs()))
        dn = torch.where(held, g * p * rest, 0.0)
        return d.scatter_add_(1, at, dn), size.scatter_add_(1, at, dn.abs())
    full = d.scatter_add(1, at, g)
    mean, most = (full * s).sum(1, keepdim=True), (full * s).abs().sum(1, keepdim=True)
    return s * (full - mean), s * (full.abs() + most)


@pytest.mark.parametrize("renormalize", [False, True], ids=["scores", "shares"])
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("shape", [(1, 16, 2), (2, 1, 1), (31, 40, 3), (64, 33, 32), (300, 256, 8), (500, 1024, 12), (1000, 10, 3)],
                         ids=lambda s: "x".join(map(str, s)))
def test_gradient(shape, sigmoid, renormalize):
    m = nv()
    T, E, k = shape
    for dtype in (torch.float32, torch.bfloat16):
        x = _logits(T, E, T, dtype)
        if E > 4:
            x[0, 1::2] = -INF
            x[T - 1] = -INF
        valid = torch.arange(T) % 5 != 4
        score = m.SCORE_SIGMOID if sigmoid else m.SCORE_SOFTMAX
        r = m.nvfp4_route(x.cuda(), k, score=score, renormalize=renormalize, scale=2.5, valid=valid.cuda())
        g = torch.randn(T, k, generator=torch.Generator().manual_seed(T))
        out = torch.full((T, E), 7.0, dtype=dtype, device="cuda")
        got = m.nvfp4_route_bwd(g.cuda(), x.cuda(), r, score=score, renormalize=renormalize, scale=2.5, out=out).cpu().double()
        want, size = grad_formula(x, r.experts.cpu(), g, sigmoid, renormalize, 2.5)
        far = torch.where(x > -INF, x.double(), 0.0)
        far = (far.amax(1, keepdim=True) - far.amin(1, keepdim=True)).abs()
        tol = (400 + 16 * far) * U * size + (2.0 ** -8 * want.abs() if dtype == torch.bfloat16 else 0.0) + 2.0 ** -120
        err = (got - want).abs()
        assert (err <= tol).all(), f"worst {float((err / tol).max()):.3g} of the tolerance"
        assert (got[~valid] == 0).all()


@pytest.mark.parametrize("renormalize", [False, True], ids=["scores", "shares"])
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
def test_gradient_against_differences(sigmoid, renormalize):
    """The kernel's gradient beside central differences of the 64-bit weights (step h: their error is of
    the order of h^2 = 1e-10 and of 1e-16 / h = 1e-11, far below fp32's)."""
    m = nv()
    T, E, k, h = 4, 24, 5, 1e-5
    x = _logits(T, E, 3)
    score = m.SCORE_SIGMOID if sigmoid else m.SCORE_SOFTMAX
    r = m.nvfp4_route(x.cuda(), k, score=score, renormalize=renormalize, scale=1.5)
    chosen = r.experts.cpu().long()
    g = torch.randn(T, k, generator=torch.Generator().manual_seed(1))

    def loss(v):
        w = _score(v, sigmoid)[0].gather(1, chosen)
        if renormalize:
            w = w / w.sum(1, keepdim=True)
        return (1.5 * w * g.double()).sum(1)

    want = torch.zeros(T, E, dtype=torch.float64)
    for e in range(E):
        step = torch.zeros(E, dtype=torch.float64)
        step[e] = h
        want[:, e] = (loss(x.double() + step) - loss(x.double() - step)) / (2 * h)
    got = m.nvfp4_route_bwd(g.cuda(), x.cuda(), r, score=score, renormalize=renormalize, scale=1.5).cpu().double()
    assert (got - want).abs().max() <= 1e-5 * float(g.abs().max()) * 1.5


def test_gradient_skips_what_is_no_expert():
    m = nv()
    x = _logits(6, 16, 4)
    r = m.nvfp4_route(x.cuda(), 3)
    r.experts[2] = torch.tensor([16, -7, 2 ** 31 - 1], dtype=torch.int32)
    got = m.nvfp4_route_bwd(torch.ones(6, 3, device="cuda"), x.cuda(), r)
    assert (got[2] == 0).all() and torch.isfinite(got).all()
