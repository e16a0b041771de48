"""A layer's weight gradient (nvfp4_bf16_wgrad): dy^T x in fp32 against 64 bits.

Tolerance: bf16 products are exact in fp32; runs of at most 512 of them, whose sum errs by gamma_512 of the magnitudes at most (u =
2^-23, the tensor core may truncate), are joined by rounded adds, one per run and 8 parts of K at most beyond; what is added to
rounds once more."""
import pytest
import torch

from gpu_helpers import nv

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _tol(rows, sabs, total):
    u = 2.0 ** -23
    run = min(rows, 512)
    return (run * u / (1 - run * u) + (-(-rows // run) + 9) * u) * sabs + u * total.abs() + 1e-30


def _wide(t, gap):
    w = torch.full((t.shape[0], (t.shape[1] + 7) // 8 * 8 + gap), float("nan"), dtype=t.dtype)
    w[:, :t.shape[1]] = t
    return w.cuda()[:, :t.shape[1]]


def _check(rows, n, d, gap=0, seed=0):
    m = nv()
    g = torch.Generator().manual_seed(seed + rows)
    dy, x = (_wide(torch.randn(rows, c, generator=g).to(BF), gap) for c in (n, d))
    ws = m.Workspace()
    back = torch.full((n, d + 5), 7.0, device="cuda")
    out = m.nvfp4_bf16_wgrad(dy, x, out=back[:, :d], ws=ws)
    assert m.nvfp4_poll(ws) == 0 and (back[:, d:] == 7).all()
    want, sabs = dy.double().t() @ x.double(), dy.double().abs().t() @ x.double().abs()
    bad = ~((out.double() - want).abs() <= _tol(rows, sabs, want))
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist())
    assert torch.equal(out, m.nvfp4_bf16_wgrad(dy, x, ws=ws))
    before = torch.randn(n, d, generator=g).cuda()
    added = before.clone()
    m.nvfp4_bf16_wgrad(dy, x, out=added, accumulate=True, ws=ws)
    total = want + before.double()
    assert ((added.double() - total).abs() <= _tol(rows, sabs, total) + 2.0 ** -23 * sabs).all()


@pytest.mark.parametrize("rows", [1, 2, 7, 8, 15, 16, 17, 63, 64, 65, 127, 500, 513, 1025, 4099])
def test_rows(rows):
    _check(rows, 264, 136)
    _check(rows, 40, 520, gap=16)


@pytest.mark.parametrize("n,d", [(1, 1), (1, 200), (3, 5), (8, 8), (15, 17), (16, 64), (17, 63), (33, 129), (64, 127), (65, 128), (80, 255), (96, 256),
                                 (112, 257), (127, 65), (128, 300), (129, 72), (160, 513), (192, 264), (224, 136), (255, 40), (257, 1000), (513, 385)])
def test_edges(n, d):
    _check(333, n, d, gap=8)
    _check(70, n, d)


@pytest.mark.parametrize("rows,n,d", [(600, 2056, 1288), (264, 5128, 2504), (2000, 1032, 1032), (300, 96, 5120), (9000, 72, 200), (40, 4096, 4096)])
def test_many_tiles(rows, n, d):
    _check(rows, n, d)


def test_exact_on_small_integers():
    g = torch.Generator().manual_seed(1)
    for rows, n, d in ((777, 130, 70), (1500, 520, 264)):
        dy, x = (_wide(torch.randint(-3, 4, (rows, c), generator=g).to(BF), 0) for c in (n, d))   # strides of whole 16 bytes
        assert torch.equal(nv().nvfp4_bf16_wgrad(dy, x).double(), dy.double().t() @ x.double())


def test_no_rows_and_streams():
    m = nv()
    z = lambda c: torch.zeros(0, c, dtype=BF, device="cuda")
    out = torch.full((24, 45), 7.0, device="cuda")
    m.nvfp4_bf16_wgrad(z(24), z(40), out=out[:, :40], accumulate=True)
    assert (out == 7).all()
    m.nvfp4_bf16_wgrad(z(24), z(40), out=out[:, :40])
    assert not out[:, :40].any() and (out[:, 40:] == 7).all()
    dy, x = (torch.randn(300, c, device="cuda").to(BF) for c in (136, 264))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    side = m.nvfp4_bf16_wgrad(dy, x, stream=s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    total = torch.zeros(136, 264, device="cuda")
    with torch.cuda.graph(g):
        m.nvfp4_bf16_wgrad(dy, x, out=total, accumulate=True)
    assert torch.equal(side, m.nvfp4_bf16_wgrad(dy, x))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(total, side)


def test_expired_waits():
    m = nv()
    ws = m.Workspace()
    for rows, n, d in ((4000, 1280, 1288), (5000, 40, 264)):
        dy, x = (torch.randn(rows, c, device="cuda").to(BF) for c in (n, d))
        want = m.nvfp4_bf16_wgrad(dy, x)
        for ns in (1, 500, 3000):
            m.nvfp4_set_wait_budget_ns(ns)
            try:
                m.nvfp4_bf16_wgrad(dy, x, ws=ws)
                assert m.nvfp4_poll(ws) in (0, 8)
            finally:
                m.nvfp4_set_wait_budget_ns(0)
        assert torch.equal(m.nvfp4_bf16_wgrad(dy, x, ws=ws), want) and m.nvfp4_poll(ws) == 0


@pytest.mark.parametrize("T,d,n", [(0, 64, 40), (130, 1032, 2032), (130, 1032, 2040), (1, 2056, 1032), (700, 2056, 1288)])
def test_layer_on_both_sides_of_the_rule(T, d, n):
    """LinearActBF16's gradients where its weight has up to 2^21 elements, and more."""
    m = nv()
    g = torch.Generator().manual_seed(T + n)
    x, w, dy = (torch.randn(*s, generator=g).to(BF).cuda() for s in ((T, d), (n, d), (T, n)))
    layer = m.LinearActBF16(T, d, n, act=m.ACT_NONE)
    dx, dw, db = layer.bwd(x, w, dy)
    want, sabs = dy.double().t() @ x.double(), dy.double().abs().t() @ x.double().abs()
    assert ((dw.double() - want).abs() <= _tol(max(T, 1), sabs, want)).all()
    back, babs = dy.double() @ w.double(), dy.double().abs() @ w.double().abs()
    u = 2.0 ** -23
    run = min(n, 4096)
    tol = (run * u / (1 - run * u) + (-(-n // run) + 8) * u) * babs
    assert ((dx.double() - back).abs() <= tol + 2.0 ** -8 * (back.abs() + tol)).all()
    total = dw.clone()
    layer.bwd(x, w, dy, dw=total, dbias=db, accumulate=True)
    assert ((total.double() - 2 * want).abs() <= _tol(max(T, 1), 2 * sabs, 2 * want) + 2.0 ** -23 * sabs).all()
    assert m.nvfp4_poll(layer.ws) == 0
