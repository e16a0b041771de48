"""The product with bias, activation and residual (nvfp4_bf16_gemm_act), its backward pass (nvfp4_act_bwd,
LinearActBF16) against 64-bit evaluations of the same bf16 values.

Tolerances (from the arithmetic).  Sums: bf16 products are exact in fp32; a running sum of k errs by at most gamma_k *
sum |a b|, gamma_k = k u / (1 - k u), u = 2^-23 (the tensor core may truncate); runs of at most 512 (bf16 output: 1024)
are joined by rounded adds, one per run and part of K, 8 at most beyond, and the bias adds one.  The activation passes on an
error with its slope: at most 1 (relu), 1.13 (gelu), 1.1 (silu), 2 |h| + the error (relu2).  Its own evaluation errs, for
bf16 outputs, by |h| / 2 erfc(|h| / sqrt 2) times 1e-6 (gelu) or by |h| 2^-20 (silu), below 2^-19 |h| both; with fp32
outputs by normcdff's 5 ulp or expf's 2 and a quotient, below 2^-20 |h|; relu2 by one rounding.  The residual's addition rounds in fp32
(2^-24), the output by half a step (bf16 2^-8, fp32 2^-24)."""
import math

import pytest
import torch

from gpu_helpers import nv

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "relu2", "gelu", "silu"]
BF, F32 = torch.bfloat16, torch.float32


def _code(act):
    return getattr(nv(), "ACT_" + act.upper())


def act64(name, h):
    if name == "relu":
        return h.clamp(min=0)
    if name == "relu2":
        return h.clamp(min=0) ** 2
    if name == "gelu":
        return h * 0.5 * torch.special.erfc(-h / math.sqrt(2))
    if name == "silu":
        return h * torch.special.expit(h)
    return h


def slope64(name, h):
    if name == "relu":
        return (h > 0).double()
    if name == "relu2":
        return 2 * h.clamp(min=0)
    if name == "gelu":
        return 0.5 * torch.special.erfc(-h / math.sqrt(2)) + h * torch.exp(-h * h / 2) / math.sqrt(2 * math.pi)
    if name == "silu":
        s = torch.special.expit(h)
        return s * (1 + h * (1 - s))
    return torch.ones_like(h)


def _half(dtype):
    return 2.0 ** -8 if dtype == BF else 2.0 ** -24


def _sum_error(K, fp32, sabs, h):
    u = 2.0 ** -23
    run = min(K, 512 if fp32 else 1024)
    return (run * u / (1 - run * u) + (-(-K // run) + 8) * u) * sabs + u * h.abs()


def _inputs(M, N, K, seed, bias=True, residual=None, scale=None):
    g = torch.Generator().manual_seed(seed)
    a = torch.randn(M, K, generator=g).bfloat16()
    b = (torch.randn(N, K, generator=g) * (1.5 / math.sqrt(K) if scale is None else scale)).bfloat16()
    c = torch.randn(N, generator=g) * 0.5 if bias else None
    r = torch.randn(M, N, generator=g).to(residual) if residual else None
    return a, b, c, r


def _check(M, N, K, act="none", dtype=BF, bias=True, residual=None, pre=False, seed=0, scale=None):
    m = nv()
    a, b, c, r = _inputs(M, N, K, seed, bias, residual, scale)
    ws = m.Workspace()
    cuda = lambda t: None if t is None else t.cuda()
    out = torch.full((M, N), 7.0, dtype=dtype, device="cuda")
    p = torch.full((M, N), 7.0, dtype=BF, device="cuda") if pre else None
    got = m.nvfp4_bf16_gemm_act(a.cuda(), b.cuda(), cuda(c), act=_code(act), residual=cuda(r), pre=p, out=out, ws=ws)
    assert got is out and m.nvfp4_poll(ws) == 0
    h = a.cuda().double() @ b.cuda().double().t()
    sabs = a.cuda().double().abs() @ b.cuda().double().abs().t()
    if bias:
        h = h + c.cuda().double()
    dh = _sum_error(K, dtype == F32, sabs, h) + 1e-30
    if pre:
        err = (p.double() - h).abs()
        assert (err <= dh + 2.0 ** -8 * (h.abs() + dh)).all(), "pre"
    slope = {"none": 1.0, "relu": 1.0, "relu2": 2 * h.abs() + dh, "gelu": 1.13, "silu": 1.1}[act]
    own = {"none": 0.0, "relu": 0.0, "relu2": 2.0 ** -23 * h * h}.get(act, (2.0 ** -19 if dtype == BF else 2.0 ** -20) * h.abs())
    y, tol = act64(act, h), slope * dh + own
    if residual:
        y = y + r.cuda().double()
        tol = tol + 2.0 ** -23 * (y.abs() + tol)
    tol = tol + _half(dtype) * (y.abs() + tol)
    err = (out.double() - y).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside, worst {float((err / tol).max()):.3g}, first {bad.nonzero()[0].tolist()}"
    return out


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 40, 136), (16, 712, 1032), (17, 712, 1032), (130, 264, 520), (333, 1288, 2056)])
def test_activations(M, N, K, act, dtype):
    _check(M, N, K, act, dtype, pre=True, seed=M)
    _check(M, N, K, act, dtype, bias=False, residual=dtype, seed=M + 1)
    _check(M, N, K, act, dtype, residual=F32 if dtype == BF else BF, pre=True, seed=M + 2)


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 15, 16, 17, 24, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 255, 256, 257, 300, 511, 513, 700])
def test_rows(M):
    # past every size at which another kernel, tile or cut of K may take over
    _check(M, 520, 1096, "gelu", residual=BF, seed=M)
    _check(M, 1280, 5120, "none", F32, seed=M)
    _check(M, 264, 72, "silu", seed=M)


@pytest.mark.parametrize("N,K", [(1, 8), (2, 16), (7, 24), (9, 64), (255, 72), (256, 128), (257, 136), (513, 8), (1000, 4104), (37, 20480), (4097, 264)])
def test_odd_features(N, K):
    for M in (1, 5, 16, 40, 200):
        for dtype in (BF, F32):
            _check(M, N, K, "relu2", dtype, residual=dtype, pre=True, seed=N + K)


@pytest.mark.parametrize("M,N,K", [(2000, 2568, 1288), (4096, 1024, 256), (1500, 5000, 712), (8192, 264, 8), (300, 20480, 520), (3000, 3000, 3000)])
def test_many_tiles(M, N, K):
    # several waves of tiles, bands and runs
    _check(M, N, K, "gelu", residual=F32, pre=True, seed=1)
    _check(M, N, K, "relu", F32, residual=BF, seed=2)


@pytest.mark.parametrize("M", [3, 16, 40, 200, 1000])
def test_exact_on_small_integers(M):
    # |a|, |b| <= 8, K <= 256: every partial sum is a whole number below 2^24
    m = nv()
    g = torch.Generator().manual_seed(M)
    a, b = (torch.randint(-8, 9, (r, 256), generator=g).bfloat16() for r in (M, 392))
    c, r = torch.randint(-99, 99, (392,), generator=g).float(), torch.randint(-99, 99, (M, 392), generator=g).float()
    got = m.nvfp4_bf16_gemm_act(a.cuda(), b.cuda(), c.cuda(), act=m.ACT_RELU, residual=r.cuda(), out_dtype=F32)
    assert torch.equal(got.cpu().double(), (a.double() @ b.double().t() + c).clamp(min=0) + r)


@pytest.mark.parametrize("M", [3, 12, 40, 130])
def test_long_runs_are_joined_by_rounding(M):
    """Positive whole numbers whose products add to at most 512 * 2^14 < 2^24 in a run of 512: only the adds that join the
    runs err, by 2^-24 of the sum each: one per run and one per part of a cut K (16 at most)."""
    m = nv()
    K, N = 65536 + 8, 24
    g = torch.Generator().manual_seed(M)
    a, b = (torch.randint(1, 129, (r, K), generator=g).bfloat16() for r in (M, N))
    got = m.nvfp4_bf16_gemm_act(a.cuda(), b.cuda(), out_dtype=F32).cpu().double()
    ref = a.double() @ b.double().t()
    assert float(((got - ref).abs() / ref).max()) <= (-(-K // 512) + 16) * 2.0 ** -24


@pytest.mark.parametrize("M", [5, 40, 500])
def test_strides_in_place_and_streams(M):
    m = nv()
    N, K = 265, 200
    a, b, c, r = _inputs(M, N, K, 3, residual=BF)
    wide = lambda t, left, right: torch.nn.functional.pad(t, (left, right), value=float("nan")).cuda()[:, left:left + t.shape[1]]
    want = m.nvfp4_bf16_gemm_act(a.cuda(), b.cuda(), c.cuda(), act=m.ACT_SILU, residual=r.cuda())
    for ld in (N, N + 7, N + 8):
        res = torch.full((M, ld), 5.0, dtype=BF, device="cuda")
        res[:, :N] = r.cuda()
        pre = torch.full((M, ld), 5.0, dtype=BF, device="cuda")
        x, w = wide(a, 8, 16), wide(b, 24, 8)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        m.nvfp4_bf16_gemm_act(x, w, c.cuda(), act=m.ACT_SILU, residual=res[:, :N], pre=pre[:, :N], out=res[:, :N], stream=s)
        s.synchronize()
        assert torch.equal(res[:, :N], want) and (res[:, N:] == 5).all() and (pre[:, N:] == 5).all()


@pytest.mark.parametrize("M", [2, 40, 700])
def test_non_finite_rows_stay_to_themselves(M):
    m = nv()
    a, b, c, _ = _inputs(M, 300, 264, 4)
    want = m.nvfp4_bf16_gemm_act(a.cuda(), b.cuda(), c.cuda(), act=m.ACT_GELU)
    a[1, 7] = float("nan")
    got = m.nvfp4_bf16_gemm_act(a.cuda(), b.cuda(), c.cuda(), act=m.ACT_GELU)
    keep = torch.arange(M) != 1
    assert torch.isnan(got[1]).all() and torch.equal(got[keep.cuda()], want[keep.cuda()])
    for act in ACTS:   # what the activations make of the ends
        bias = torch.tensor([math.inf, -math.inf, math.nan, 1e30, -1e30, 40.0, -40.0] + [0.0] * 293).cuda()
        zero = torch.zeros(M, 264, dtype=BF, device="cuda")
        for dtype in (BF, F32):
            y = m.nvfp4_bf16_gemm_act(zero, b.cuda(), bias, act=_code(act), out_dtype=dtype)[M - 1].double().cpu()
            assert y[0] == math.inf and torch.isnan(y[2]) and y[5] == (1600 if act == "relu2" else 40) and (y[7:] == 0).all()
            if act != "none":
                assert (y[4] == 0 or act == "silu") and abs(y[6]) < 1e-15


def test_captured_and_side_by_side():
    """Two graphs on two streams, replayed at once on changing inputs, at a size whose K is cut over a cluster."""
    m = nv()
    sizes = [(200, 1280, 5120), (12, 2048, 2048), (1000, 1024, 512)]
    for M, N, K in sizes:
        a, b, c, r = _inputs(M, N, K, 5, residual=BF)
        b, c, r = b.cuda(), c.cuda(), r.cuda()
        xs = [torch.zeros(M, K, dtype=BF, device="cuda") for _ in range(2)]
        outs = [torch.zeros(M, N, dtype=BF, device="cuda") for _ in range(2)]
        wss, streams, graphs = [m.Workspace() for _ in range(2)], [torch.cuda.Stream() for _ in range(2)], []
        for i in range(2):
            m.nvfp4_bf16_gemm_act(xs[i], b, c, act=m.ACT_GELU, residual=r, out=outs[i], ws=wss[i])
            torch.cuda.synchronize()
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[i]):
                m.nvfp4_bf16_gemm_act(xs[i], b, c, act=m.ACT_GELU, residual=r, out=outs[i], ws=wss[i])
        for seed in (1, 2):
            data = [_inputs(M, 8, K, seed + 10 * i)[0].cuda() for i in range(2)]
            want = [m.nvfp4_bf16_gemm_act(d, b, c, act=m.ACT_GELU, residual=r) for d in data]
            for i in range(2):
                xs[i].copy_(data[i])
            torch.cuda.synchronize()
            for _ in range(4):
                for i in range(2):
                    with torch.cuda.stream(streams[i]):
                        graphs[i].replay()
            torch.cuda.synchronize()
            assert all(torch.equal(outs[i], want[i]) for i in range(2))


def test_no_rows():
    m = nv()
    b = torch.zeros(16, 64, dtype=BF, device="cuda")
    assert m.nvfp4_bf16_gemm_act(torch.zeros(0, 64, dtype=BF, device="cuda"), b).shape == (0, 16)
    db = torch.full((16,), 3.0, device="cuda")
    e = torch.zeros(0, 16, dtype=BF, device="cuda")
    m.nvfp4_act_bwd(e, e, m.ACT_GELU, dbias=db, accumulate=True)
    assert (db == 3).all()
    m.nvfp4_act_bwd(e, e, m.ACT_GELU, dbias=db)
    assert (db == 0).all()


# ---------------------------------------------------------------------------------------
# backward
# ---------------------------------------------------------------------------------------
def _slope_error(act, h):
    """Of the slope itself: gelu's terms err by 1e-6 of Phi and of |h| phi <= 0.25; silu's by 2^-20 (1 + |h| s (1 - s) ...)."""
    return {"gelu": 2.0 ** -18, "silu": 2.0 ** -18}.get(act, 0.0) * torch.ones_like(h)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,n", [(1, 8), (3, 72), (33, 64), (500, 712), (3001, 1032), (9000, 136), (64, 20480)])
def test_act_gradient(rows, n, act):
    m = nv()
    g = torch.Generator().manual_seed(rows)
    dy, pre = torch.randn(rows, n, generator=g).bfloat16().cuda(), (torch.randn(rows, n, generator=g) * 3).bfloat16().cuda()
    pre[0, :3] = torch.tensor([0.0, 25.0, -25.0])
    db = torch.full((n,), 2.0, device="cuda")
    dh = m.nvfp4_act_bwd(dy, pre if act != "none" else None, _code(act), dbias=db)
    s, e = slope64(act, pre.double()), _slope_error(act, pre.double())
    want, err = dy.double() * s, dy.double().abs() * (e + 2.0 ** -23 * s.abs())
    assert ((dh.double() - want).abs() <= err + 2.0 ** -8 * (want.abs() + err) + 2.0 ** -130).all()
    sums = want.sum(0)
    tol = err.sum(0) + (rows + 100) * 2.0 ** -24 * want.abs().sum(0) + 2.0 ** -120
    assert ((db.double() - sums).abs() <= tol).all()
    again = db.clone()
    m.nvfp4_act_bwd(dy, pre, _code(act), out=dy, dbias=again, accumulate=True)    # in place, added
    assert torch.equal(dy, dh) and ((again.double() - 2 * sums).abs() <= 2 * tol + 2.0 ** -22 * sums.abs()).all()


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_slopes_over_every_bf16(act):
    m = nv()
    h = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF).cuda()
    h = h[torch.isfinite(h)]
    h = torch.nn.functional.pad(h, (0, -len(h) % 8)).view(1, -1)
    d = m.nvfp4_act_bwd(torch.ones_like(h), h, _code(act))
    want = slope64(act, h.double())
    assert ((d.double() - want).abs() <= 2.0 ** -18 + 2.0 ** -8 * want.abs()).all()


def test_slopes_against_differences():
    """The slopes beside central differences of the 64-bit activations (their error: h^2 = 1e-8)."""
    m = nv()
    x = torch.linspace(-6, 6, 4096).bfloat16().view(8, 512).cuda()
    for act in ACTS[3:]:
        d = m.nvfp4_act_bwd(torch.ones_like(x), x, _code(act)).double()
        want = (act64(act, x.double() + 1e-4) - act64(act, x.double() - 1e-4)) / 2e-4
        assert ((d - want).abs() <= 2.0 ** -18 + 1e-7 + 2.0 ** -8 * want.abs()).all()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,d,n", [(1, 72, 40), (37, 264, 136), (700, 520, 712)])
def test_layer(T, d, n, act):
    """A layer's step: forward with the pre-activation kept, then all its gradients, twice, the second added."""
    m = nv()
    x, w, c, r = (None if t is None else t.cuda() for t in _inputs(T, n, d, T, residual=BF))
    layer = m.LinearActBF16(T, d, n, act=_code(act))
    pre = torch.empty(T, n, dtype=BF, device="cuda")
    y = layer.fwd(x, w, c, residual=r, pre=pre)
    h = x.double() @ w.double().t() + c.double()
    assert (y.double() - act64(act, h) - r.double()).abs().max() <= 2.0 ** -7 * (h.abs().max() ** (2 if act == "relu2" else 1) + r.double().abs().max())
    dy = torch.randn(T, n, generator=torch.Generator().manual_seed(9)).bfloat16().cuda()
    dx, dw, db = layer.bwd(x, w, dy, pre)
    held = m.nvfp4_act_bwd(dy, pre, _code(act)).double()     # tested above
    tol = lambda k, a, b: (k * 2.0 ** -23 + 2.0 ** -8) * (a.abs() @ b.abs())
    assert ((dx.double() - held @ w.double()).abs() <= tol(n, held, w.double())).all()
    assert ((dw.double() - held.t() @ x.double()).abs() <= tol(T, held.t(), x.double())).all()
    dw2, db2 = dw.clone(), db.clone()
    layer.bwd(x, w, dy, pre, dw=dw2, dbias=db2, accumulate=True)
    assert torch.allclose(dw2, 2 * dw, rtol=1e-6, atol=0) and torch.allclose(db2, 2 * db, rtol=1e-5, atol=1e-5)
    assert m.nvfp4_poll(layer.ws) == 0


def test_expired_waits():
    """A budget that runs out at once ends the call with the flag and leaves the device usable."""
    m = nv()
    ws = m.Workspace()
    for M, N, K in ((200, 1280, 5120), (40, 264, 20480), (3000, 2048, 4096)):
        a, b, c, _ = (None if t is None else t.cuda() for t in _inputs(M, N, K, 6))
        want = m.nvfp4_bf16_gemm_act(a, b, c)
        for ns in (1, 500, 3000):
            m.nvfp4_set_wait_budget_ns(ns)
            try:
                m.nvfp4_bf16_gemm_act(a, b, c, ws=ws)
                assert m.nvfp4_poll(ws) in (0, 8)
            finally:
                m.nvfp4_set_wait_budget_ns(0)
        assert torch.equal(m.nvfp4_bf16_gemm_act(a, b, c, ws=ws), want) and m.nvfp4_poll(ws) == 0
