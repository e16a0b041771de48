"""An expert layer as a program strings it together: router product, route, dispatch, the experts' two products with GeLU between
them, combine onto the residual stream; then its backward pass down to the router's weights.  Against 64-bit autograd
of the same formulas, captured into a graph, and with padded tokens.

Tolerance: every tensor on the way is rounded to bf16 at most once, which moves it by at most 2^-8 of its values, so of
its norm; no path from an input to a result has more than ten of them, and products with random matrices carry a relative error on
as it is, on average: 10 * 2^-8, and as much again for where the average does not hold."""
import pytest
import torch

from gpu_helpers import nv

pytestmark = pytest.mark.gpu

E, K, GROUPS, SCALE = 16, 3, 4, 1.5
BF = torch.bfloat16


class Layer:
    """The buffers and weights that a program keeps."""

    def __init__(self, T, d, n, seed):
        m = nv()
        g = torch.Generator().manual_seed(seed)
        rand = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std)
        self.T, self.d, self.n = T, d, n
        self.router = rand(E, d, std=d ** -0.5).to(BF).cuda()
        self.up = rand(E, n, d, std=d ** -0.5).to(BF).cuda()
        self.down = rand(E, d, n, std=n ** -0.5).to(BF).cuda()
        self.bias = rand(E, std=0.05).cuda()
        self.x, self.dy = rand(T, d).to(BF).cuda(), rand(T, d).to(BF).cuda()
        self.valid = torch.ones(T, dtype=torch.bool, device="cuda")
        self.routes = m.Routes.empty(T, E, K)
        self.gate = m.LinearActBF16(T, d, E, act=m.ACT_NONE)
        self.ups, self.downs = m.GroupedLinearBF16(E, d, n), m.GroupedLinearBF16(E, n, d)
        self.ws = m.Workspace()
        # what nobody's rows hold must not matter
        self.xs = torch.full((T * K, d), float("nan"), dtype=BF, device="cuda")
        self.dys = torch.full((T * K, d), float("nan"), dtype=BF, device="cuda")

    def step(self):
        m, r = nv(), self.routes
        logits = m.nvfp4_bf16_gemm_act(self.x, self.router, out_dtype=torch.float32, ws=self.ws)
        m.nvfp4_route(logits, K, score=m.SCORE_SIGMOID, bias=self.bias, groups=GROUPS, top_groups=2, group_top=2, scale=SCALE,
                      valid=self.valid, out=r, ws=self.ws)
        xs = m.nvfp4_dispatch(self.x, r, out=self.xs)
        h = self.ups.fwd(xs, self.up, r.offsets)
        a = m.nvfp4_gelu_fwd(h)
        ys = self.downs.fwd(a, self.down, r.offsets)
        y = m.nvfp4_combine(ys, r, residual=self.x)
        # backward: the residual's gradient is dy
        dys, dw = m.nvfp4_combine_bwd(self.dy, ys, r, dys=self.dys)
        da, ddown = self.downs.bwd(a, self.down, dys, r.offsets)
        dh = m.nvfp4_gelu_bwd(h, da)
        dxs, dup = self.ups.bwd(xs, self.up, dh, r.offsets)
        dx = m.nvfp4_combine(dxs, r, residual=self.dy, weighted=False)
        dlogits = m.nvfp4_route_bwd(dw, logits, r, score=m.SCORE_SIGMOID, scale=SCALE)
        dgate, drouter, _ = self.gate.bwd(self.x, self.router, dlogits.to(BF))
        return y, dx, dgate, drouter, dup, ddown

    def expected(self):
        """(y, the gradients) in 64 bits for the experts that were chosen"""
        x, router, up, down = (t.double().requires_grad_() for t in (self.x, self.router, self.up, self.down))
        x_gate = self.x.double().requires_grad_()
        s = torch.special.expit(x_gate @ router.t())
        at = self.routes.experts.long()
        held = at >= 0
        w = torch.where(held, s.gather(1, at.clamp(min=0)), 0.0)
        w = SCALE * w / w.sum(1, keepdim=True).clamp(min=1e-30)
        y = x
        for e in range(E):
            token, j = torch.nonzero(at == e, as_tuple=True)
            h = x[token] @ up[e].t()
            out = (h * torch.special.ndtr(h)) @ down[e].t()
            y = y.index_add(0, token, out * w[token, j, None])
        return (y, *torch.autograd.grad(y, (x, x_gate, router, up, down), self.dy.double()))

    def choice(self):
        """the route in 64 bits"""
        s = torch.special.expit((self.x.double() @ self.router.double().t()))
        c = s + self.bias.double()
        keep = c.view(self.T, GROUPS, -1).topk(2, 2)[0].sum(2).topk(2, 1)[1]
        mask = torch.zeros(self.T, GROUPS, dtype=torch.bool, device="cuda").scatter_(1, keep, True).repeat_interleave(E // GROUPS, 1)
        return torch.where(mask, c, -1.0).topk(K, 1)[1]


def _far(a, b):
    a, b = a.double(), b.detach()
    return float((a - b).norm() / b.norm().clamp(min=1e-300))


@pytest.mark.parametrize("T,d,n,padded", [(1, 64, 40, 0), (37, 136, 200, 5), (500, 264, 328, 100), (3001, 520, 1032, 0), (2500, 1032, 264, 400)])
def test_step(T, d, n, padded):
    m = nv()
    layer = Layer(T, d, n, T)
    if padded:
        layer.valid[T - padded:] = False
    got = layer.step()
    assert m.nvfp4_poll(layer.ws) == m.nvfp4_poll(layer.gate.ws) == m.nvfp4_poll(layer.ups.ws) == m.nvfp4_poll(layer.downs.ws) == 0
    live = T - padded
    assert (layer.routes.experts[live:] == -1).all()
    same = (layer.routes.experts[:live].long() == layer.choice()[:live]).all(1)
    # the logits are sums in fp32: a choice may differ where two scores are as close as those
    assert float((~same).float().mean()) <= 1e-3
    for name, a, b in zip(("y", "dx", "dx of the router", "drouter", "dup", "ddown"), got, layer.expected()):
        assert torch.isfinite(a).all(), name
        assert _far(a, b) <= 20 * 2.0 ** -8, name
    assert torch.equal(got[0][live:], layer.x[live:]) and torch.equal(got[1][live:], layer.dy[live:])


def test_step_of_padding_alone():
    layer = Layer(40, 64, 72, 1)
    layer.valid.zero_()
    y, dx, dgate, drouter, dup, ddown = layer.step()
    assert torch.equal(y, layer.x) and torch.equal(dx, layer.dy)
    assert not any(t.any() for t in (dgate, drouter, dup, ddown))


def test_captured_steps_side_by_side():
    """Two layers' steps, each captured and replayed on a stream of its own on changing inputs: bit for bit the eager ones."""
    layers = [Layer(600, 136, 264, 3), Layer(2100, 520, 136, 4)]
    held, streams = [], [torch.cuda.Stream() for _ in layers]
    for layer in layers:
        layer.step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = layer.step()
        held.append((g, out))
    for seed in (11, 12):
        for layer in layers:
            gen = torch.Generator().manual_seed(seed)
            layer.x.copy_(torch.randn(layer.T, layer.d, generator=gen))
            layer.valid.copy_(torch.rand(layer.T, generator=gen) < 0.9)
        torch.cuda.synchronize()
        for _ in range(3):
            for (g, _), s in zip(held, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        results = [[t.clone() for t in out] for _, out in held]
        for layer, result in zip(layers, results):
            for a, b in zip(layer.step(), result):
                assert torch.equal(a, b)
