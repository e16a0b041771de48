"""The product with bias, activation and residual for B [K][N] (nvfp4_bf16_gemm_act with b_kn), which is a layer's input gradient:
against 64 bits, with the tolerances of the product for B [N][K] (the sums are the same, in the same order), and beyond 16 rows
bit for bit against that product of the transposed operand."""
import pytest
import torch

from gpu_helpers import nv
from test_gpu_gemm_act import ACTS, BF, F32, _code, _half, _inputs, _sum_error, act64

pytestmark = pytest.mark.gpu


def _both(M, N, K, act="none", dtype=BF, bias=True, residual=None, pre=False, seed=0, gap=0):
    m = nv()
    a, b, c, r = (None if t is None else t.cuda() for t in _inputs(M, N, K, seed, bias, residual))
    ldb = (N + 7) // 8 * 8 + gap
    kn = torch.full((K, ldb), float("nan"), dtype=BF, device="cuda")[:, :N]
    kn.copy_(b.t())
    ws = m.Workspace()
    outs = []
    for w, flag in ((kn, True), (b, False)):
        p = torch.full((M, N), 7.0, dtype=BF, device="cuda") if pre else None
        y = m.nvfp4_bf16_gemm_act(a, w, c, act=_code(act), residual=r, pre=p, out_dtype=dtype, ws=ws, b_kn=flag)
        outs.append((y, p))
    assert m.nvfp4_poll(ws) == 0
    (y, p), (y0, p0) = outs
    if M > 16:
        assert torch.equal(y, y0) and (not pre or torch.equal(p, p0))
    h = a.double() @ b.double().t()
    sabs = a.double().abs() @ b.double().abs().t()
    h = h + c.double() if bias else h
    dh = _sum_error(K, dtype == F32, sabs, h) + 1e-30
    slope = {"none": 1.0, "relu": 1.0, "relu2": 2 * h.abs() + dh, "gelu": 1.13, "silu": 1.1}[act]
    own = {"none": 0.0, "relu": 0.0, "relu2": 2.0 ** -23 * h * h}.get(act, (2.0 ** -19 if dtype == BF else 2.0 ** -20) * h.abs())
    want, tol = act64(act, h), slope * dh + own
    if residual:
        want = want + r.double()
        tol = tol + 2.0 ** -23 * (want.abs() + tol)
    tol = tol + _half(dtype) * (want.abs() + tol)
    assert ((y.double() - want).abs() <= tol).all()
    if pre:
        assert ((p.double() - h).abs() <= dh + 2.0 ** -8 * (h.abs() + dh)).all()


@pytest.mark.parametrize("M", [1, 2, 8, 9, 16, 17, 31, 33, 64, 65, 100, 128, 129, 255, 257, 513, 700])
def test_rows(M):
    _both(M, 264, 520, seed=M)
    _both(M, 1032, 2056, bias=False, seed=M + 1)


@pytest.mark.parametrize("N,K", [(1, 8), (3, 72), (7, 64), (8, 8), (63, 136), (65, 128), (127, 200), (129, 1032), (200, 40), (255, 5128),
                                 (257, 264), (385, 4104)])
def test_edges(N, K):
    for M in (5, 70, 300):
        _both(M, N, K, seed=N, gap=8)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_activations(act, dtype):
    for M, N, K in ((3, 72, 136), (90, 264, 520), (600, 712, 1288)):
        _both(M, N, K, act, dtype, residual=F32 if dtype == BF else BF, pre=True, seed=M)


@pytest.mark.parametrize("M,N,K", [(4096, 520, 1032), (2500, 2056, 264), (40, 20480, 264), (1100, 3976, 2504)])
def test_many_tiles(M, N, K):
    _both(M, N, K, "gelu", pre=True, seed=7)


def test_captured_on_another_stream():
    m = nv()
    a, b, c, r = (None if t is None else t.cuda() for t in _inputs(200, 264, 1032, 1))
    kn = b.t().contiguous()
    out = torch.empty(200, 264, dtype=BF, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    m.nvfp4_bf16_gemm_act(a, kn, c, out=out, stream=s, b_kn=True)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.nvfp4_bf16_gemm_act(a, kn, c, out=out, b_kn=True)
    for seed in (2, 3):
        a.copy_(_inputs(200, 264, 1032, seed)[0])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, m.nvfp4_bf16_gemm_act(a, b, c))


def test_no_rows():
    m = nv()
    y = m.nvfp4_bf16_gemm_act(torch.zeros(0, 16, dtype=BF, device="cuda"), torch.zeros(16, 24, dtype=BF, device="cuda"), b_kn=True)
    assert y.shape == (0, 24)
