"""The product with bias, activation and residual, and the weight gradient: long sums with bf16 outputs, and waits that run out, in
each of the kernels."""
import pytest
import torch

from gpu_helpers import nv

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("M", [5, 16, 40, 200, 700])
@pytest.mark.parametrize("K", [4096, 5120, 20480, 65544])
def test_bf16_output_of_a_long_sum_of_one_sign(M, K):
    """An fp32 residual takes the sum back but for its error, which bf16 would hide.

    Tolerance: an accumulator holds at most 4096 products, 256 MMAs of 16, each of which truncates by at most 2^-23 of the sum: 2^-15.
    The runs of a part of K and the parts (8 at most) are joined by rounded adds, 2^-24 of the sum each, and the residual by one;
    the output rounds by 2^-8 of itself."""
    m = nv()
    g = torch.Generator().manual_seed(M)
    a, b = (torch.rand(r, K, generator=g).add_(0.5).bfloat16().cuda() for r in (M, 264))
    h = a.double() @ b.double().t()
    back = -h.float()
    want = h + back.double()
    tol = (2.0 ** -15 + (-(-K // 4096) + 16) * 2.0 ** -24) * h
    for w, kn in ((b, False), (b.t().contiguous(), True)):
        out = m.nvfp4_bf16_gemm_act(a, w, residual=back, out_dtype=BF, b_kn=kn).double()
        assert ((out - want).abs() <= tol + 2.0 ** -8 * out.abs()).all(), float(((out - want).abs() / h).max())


def _expires(call, ws):
    """`call` with a budget that its first wait for a copy exceeds: the flag is raised, and the next call is whole."""
    m = nv()
    want = call().clone()
    assert m.nvfp4_poll(ws) == 0
    m.nvfp4_set_wait_budget_ns(1)
    try:
        call()
        assert m.nvfp4_poll(ws) == 8
    finally:
        m.nvfp4_set_wait_budget_ns(0)
    assert torch.equal(call(), want) and m.nvfp4_poll(ws) == 0


# SM pairs; pairs that cut K in two; one CTA per tile; one CTA per tile, K cut in five
@pytest.mark.parametrize("kn", [False, True], ids=["nk", "kn"])
@pytest.mark.parametrize("M,N,K", [(3000, 2048, 4096), (1000, 1280, 5120), (2088, 376, 504), (200, 1280, 5120)])
def test_waits_of_the_product_run_out(M, N, K, kn):
    m = nv()
    g = torch.Generator().manual_seed(M)
    a, b = (torch.randn(r, K, generator=g).bfloat16().cuda() for r in (M, N))
    b = b.t().contiguous() if kn else b
    ws = m.Workspace()
    out = torch.empty(M, N, dtype=BF, device="cuda")
    _expires(lambda: m.nvfp4_bf16_gemm_act(a, b, act=m.ACT_RELU, out=out, ws=ws, b_kn=kn), ws)


# SM pairs; pairs that cut the rows in four; one CTA per tile, the rows cut in eight
@pytest.mark.parametrize("rows,n,d", [(4000, 1280, 1288), (8192, 1000, 1000), (16384, 256, 256)])
def test_waits_of_the_weight_gradient_run_out(rows, n, d):
    m = nv()
    dy, x = (torch.randn(rows, c, device="cuda").bfloat16() for c in (n, d))
    ws = m.Workspace()
    out = torch.empty(n, d, device="cuda")
    _expires(lambda: m.nvfp4_bf16_wgrad(dy, x, out=out, ws=ws), ws)


@pytest.mark.parametrize("T,d,n", [(40, 72, 64), (40, 1288, 2048)])
def test_refused_backward_calls_add_nothing(T, d, n):
    """On both sides of the rule that chooses the weight gradient's kernel."""
    m = nv()
    g = torch.Generator().manual_seed(1)
    x, w, dy = (torch.randn(*s, generator=g).bfloat16().cuda() for s in ((T, d), (n, d), (T, n)))
    layer = m.LinearActBF16(T, d, n, act=m.ACT_RELU)
    pre = torch.randn(T, n, generator=g).bfloat16().cuda()
    shifted = lambda t, by: torch.zeros(t.shape[0], t.shape[1] + 16, dtype=t.dtype, device="cuda")[:, by:by + t.shape[1]]
    odd = lambda t: torch.zeros(t.shape[0], t.shape[1] + 3, dtype=t.dtype, device="cuda")[:, :t.shape[1]]
    f32 = torch.zeros(n, d, device="cuda")
    cases = [dict(x=x.float()), dict(w=w.float()), dict(dy=dy.float()), dict(pre=pre.float()), dict(x=odd(x)), dict(w=odd(w)), dict(dy=odd(dy)),
             dict(pre=odd(pre)), dict(x=shifted(x, 1)), dict(w=shifted(w, 3)), dict(dy=shifted(dy, 1)), dict(x=x.cpu()), dict(w=w.cpu()),
             dict(dw=f32.bfloat16()), dict(dw=f32.cpu()), dict(dw=shifted(f32, 1)), dict(dw=f32.t()), dict(dx=x.half()), dict(dx=x[:, 8:]),
             dict(dx=shifted(x, 1)), dict(dx=x.cpu())]
    if n * d > 1 << 21:
        cases.append(dict(dw=odd(f32)))
    for change in cases:
        dw, db = torch.full((n, d), 3.0, device="cuda"), torch.full((n,), 5.0, device="cuda")
        args = dict(x=x, w=w, dy=dy, pre=pre, dw=dw, dbias=db, accumulate=True) | change
        with pytest.raises((TypeError, ValueError, m.NVFP4Error)):
            layer.bwd(**args)
        assert (dw == 3).all() and (db == 5).all(), list(change)
    layer.bwd(x, w, dy, pre, dx=shifted(x, 8), dw=shifted(f32, 4))
    assert m.nvfp4_poll(layer.ws) == 0
