"""Token rows into the experts' order and back (nvfp4_dispatch, nvfp4_combine, nvfp4_combine_bwd) against 64-bit
sums of the same values.

Tolerances: combine adds k + 1 terms in fp32 by fused multiply-adds, gamma_(k+1) of the sum of their magnitudes, u =
2^-24, then rounds (bf16 2^-8, fp32 2^-24 of the value); a gradient's row is one product, rounded twice; its weight's is
a sum of d products in any order, gamma_d of their magnitudes."""
import pytest
import torch

from gpu_helpers import nv

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _gamma(n):
    return n * U / (1 - n * U)


def _half(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24


def _routes(T, E, k, seed, padded=0.0):
    """Routes on the CPU with random distinct experts and weights"""
    g = torch.Generator().manual_seed(seed)
    experts = torch.rand(T, max(E, k), generator=g).argsort(1)[:, :k].int()
    weights = torch.randn(T, k, generator=g)
    off = torch.rand(T, k, generator=g) < padded
    experts[off] = -1
    flat = experts.reshape(-1).long()
    order = torch.sort(torch.where(flat < 0, E, flat), stable=True)[1]
    rows = torch.empty(T * k, dtype=torch.long)
    rows[order] = torch.arange(T * k)
    rows[flat < 0] = -1
    held = torch.bincount(flat[flat >= 0], minlength=max(E, k))
    offsets = torch.cat([torch.zeros(1, dtype=torch.long), held.cumsum(0)]).int()
    sources = torch.where(torch.arange(T * k) < int(offsets[-1]), order, -1).int()
    return nv().Routes(experts, weights, rows.int().view(T, k), sources, offsets)


def _cuda(r):
    return nv().Routes(*(t.cuda() for t in (r.experts, r.weights, r.rows, r.sources, r.offsets)))


def _rand(shape, seed, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


SIZES = [(1, 1, 8), (1, 8, 5120), (2, 3, 1032), (7, 32, 72), (24, 2, 5120), (100, 5, 4104), (333, 4, 264), (1500, 8, 520), (4000, 1, 64)]


@pytest.mark.parametrize("padded", [0.0, 0.3, 1.0])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_dispatch(size, padded):
    m = nv()
    T, k, d = size
    r = _routes(T, 40, k, T, padded)
    x = _rand((T, d), 1)
    out = torch.full((T * k, d), 7.0, dtype=torch.bfloat16, device="cuda")
    assert m.nvfp4_dispatch(x.cuda(), _cuda(r), out=out) is out
    want = torch.full((T * k, d), 7.0, dtype=torch.bfloat16)
    live = int(r.offsets[-1])
    want[:live] = x[r.sources[:live].long() // k]
    assert torch.equal(out.cpu(), want)


def _combined(r, ys, residual, weighted):
    T, k = r.rows.shape
    held = r.rows >= 0
    w = torch.where(held, r.weights.double() if weighted else torch.ones(T, k, dtype=torch.float64), 0.0)
    terms = w[:, :, None] * torch.where(held[:, :, None], ys.double()[r.rows.clamp(min=0).long()], 0.0)
    y, size = terms.sum(1), terms.abs().sum(1)
    if residual is not None:
        y, size = y + residual.double(), size + residual.double().abs()
    return y, size


@pytest.mark.parametrize("types", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32),
                                   (torch.float32, torch.float32)], ids=["b-b", "f-b", "b-f", "f-f"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_combine(size, types):
    m = nv()
    T, k, d = size
    r = _routes(T, 40, k, T, 0.2)
    ys = _rand((T * k, d), 2, types[0])
    ys[int(r.offsets[-1]):] = float("nan")            # nobody's rows
    for residual, weighted in ((None, True), (_rand((T, d), 3, types[1]), True), (None, False)):
        want, size_ = _combined(r, ys, residual, weighted)
        out = torch.full((T, d), 7.0, dtype=types[1], device="cuda")
        res = None if residual is None else residual.cuda()
        m.nvfp4_combine(ys.cuda(), _cuda(r), residual=res, out=out, weighted=weighted)
        tol = _gamma(k + 1) * size_ + _half(types[1]) * (want.abs() + _gamma(k + 1) * size_) + 2.0 ** -130
        assert ((out.cpu().double() - want).abs() <= tol).all()
        if residual is not None:                      # in place
            m.nvfp4_combine(ys.cuda(), _cuda(r), residual=res, out=res)
            assert torch.equal(res, out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_combine_gradient(size, dtype):
    m = nv()
    T, k, d = size
    r = _routes(T, 40, k, T, 0.2)
    live = int(r.offsets[-1])
    ys, dy = _rand((T * k, d), 4, dtype), _rand((T, d), 5)
    ys[live:] = float("nan")
    dys = torch.full((T * k, d), 7.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((T, k), 7.0, device="cuda")
    m.nvfp4_combine_bwd(dy.cuda(), ys.cuda(), _cuda(r), dys=dys, dweights=dw)
    dys, dw = dys.cpu(), dw.cpu().double()
    assert (dys[live:] == 7).all() and (dw[r.rows < 0] == 0).all()
    choice = r.sources[:live].long()
    want = r.weights.double().view(-1)[choice][:, None] * dy.double()[choice // k]
    assert ((dys[:live].double() - want).abs() <= 2.0 ** -8 * (1 + 2.0 ** -8) * want.abs() + 2.0 ** -130).all()
    products = dy.double()[choice // k] * ys.double()[:live]
    got = dw.view(-1)[choice]
    assert ((got - products.sum(1)).abs() <= _gamma(d) * products.abs().sum(1) + 2.0 ** -130).all()


def test_gradients_against_differences():
    """combine is linear in its rows and weights, so differences are exact up to fp32 rounding: the change of
    sum(dy * y) when one row or one weight changes by a power of two."""
    m = nv()
    T, k, d = 5, 3, 40
    r = _routes(T, 8, k, 1)
    ys, dy = _rand((T * k, d), 6, torch.float32), _rand((T, d), 7)
    rc = _cuda(r)
    base = m.nvfp4_combine(ys.cuda(), rc, out_dtype=torch.float32).cpu().double()
    dys, dw = m.nvfp4_combine_bwd(dy.cuda(), ys.cuda(), rc)
    for t, j in ((0, 0), (4, 2), (2, 1)):
        row = int(r.rows[t, j])
        moved = ys.clone()
        moved[row, 11] += 4.0
        y = m.nvfp4_combine(moved.cuda(), rc, out_dtype=torch.float32).cpu().double()
        want = ((y - base) * dy.double()).sum() / 4
        assert abs(float(dys[row, 11]) - float(want)) <= 2.0 ** -7 * abs(float(want)) + 1e-5
        other = _cuda(r)
        other.weights[t, j] += 4.0
        y = m.nvfp4_combine(ys.cuda(), other, out_dtype=torch.float32).cpu().double()
        want = ((y - base) * dy.double()).sum() / 4
        assert abs(float(dw[t, j]) - float(want)) <= 1e-4 * d


def test_rows_out_of_range_are_skipped():
    m = nv()
    T, k, d = 6, 2, 64
    r = _cuda(_routes(T, 8, k, 2))
    r.rows[1, 0], r.rows[2, 1], r.rows[3, 0] = 12, -5, 2 ** 31 - 1
    x = _rand((T, d), 8).cuda()
    guard = torch.full((T * k + 4, d), 7.0, dtype=torch.bfloat16, device="cuda")
    m.nvfp4_dispatch(x, r, out=guard[:T * k])
    assert (guard[T * k:] == 7).all()
    y = m.nvfp4_combine(torch.ones(T * k, d, dtype=torch.bfloat16, device="cuda"), r, out_dtype=torch.float32, weighted=False)
    assert y[:, 0].tolist() == [2, 1, 1, 1, 2, 2]
    dys, dw = m.nvfp4_combine_bwd(x, torch.ones(T * k, d, dtype=torch.bfloat16, device="cuda"), r, dys=guard[:T * k])
    assert (guard[T * k:] == 7).all() and dw[1, 0] == 0 and dw[2, 1] == 0 and dw[3, 0] == 0


def test_strides_and_streams():
    m = nv()
    T, k, d = 50, 3, 136
    r = _routes(T, 8, k, 3)
    rc = _cuda(r)
    wide = lambda t, cols: torch.cat([t, torch.full((t.shape[0], cols), 9.0, dtype=t.dtype)], 1).cuda()
    x, ys, dy, res = _rand((T, d), 1), _rand((T * k, d), 2), _rand((T, d), 3), _rand((T, d), 4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    args = [wide(x, 8)[:, :d], wide(ys, 24)[:, :d], wide(dy, 16)[:, :d], wide(res, 40)[:, :d]]
    out = torch.full((T * k, d + 8), 9.0, dtype=torch.bfloat16, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    m.nvfp4_dispatch(args[0], rc, out=out[:, :d], stream=s)
    y = m.nvfp4_combine(args[1], rc, residual=args[3], stream=s)
    dys, dw = m.nvfp4_combine_bwd(args[2], args[1], rc, stream=s)
    s.synchronize()
    assert torch.equal(out[:, :d], m.nvfp4_dispatch(x.cuda(), rc)) and (out[:, d:] == 9).all()
    assert torch.equal(y, m.nvfp4_combine(ys.cuda(), rc, residual=res.cuda()))
    want = m.nvfp4_combine_bwd(dy.cuda(), ys.cuda(), rc)
    assert torch.equal(dys, want[0]) and torch.equal(dw, want[1])


def test_no_tokens():
    m = nv()
    r = _cuda(_routes(0, 8, 2, 1))
    e = torch.zeros(0, 16, dtype=torch.bfloat16, device="cuda")
    assert m.nvfp4_dispatch(e, r).shape == (0, 16) and m.nvfp4_combine(e, r).shape == (0, 16)
    dys, dw = m.nvfp4_combine_bwd(e, e, r)
    assert dys.shape == (0, 16) and dw.shape == (0, 2)


# (24 MB and more for combine, 16 for its gradient: warps that stay, where a call of 400 tokens goes by blocks)
LARGE = [(2100, 2, 2056), (13003, 1, 520), (4001, 4, 1288), (2900, 3, 1032), (2300, 2, 2816), (601, 2, 10504)]


@pytest.mark.parametrize("padded", [0.0, 0.25])
@pytest.mark.parametrize("size", LARGE, ids=lambda s: "x".join(map(str, s)))
def test_combine_of_many_tokens(size, padded):
    """Many tokens against 64 bits and, bit for bit, against the same tokens a few hundred at a time."""
    m = nv()
    T, k, d = size
    r = _routes(T, 40, k, T, padded)
    rc = _cuda(r)
    live = int(r.offsets[-1])
    wide = torch.full((T * k, d + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:live, :d] = _rand((live, d), 2).cuda()
    ys = wide[:, :d]
    for dtype in (torch.bfloat16, torch.float32):
        residual = _rand((T, d), 3, dtype).cuda()
        for res, weighted in ((residual, True), (None, False)):
            terms = torch.zeros(T, d, dtype=torch.float64, device="cuda") if res is None else res.double()
            size_ = terms.abs()
            for j in range(k):
                held = rc.rows[:, j] >= 0
                term = torch.where(held[:, None], ys[rc.rows[:, j].clamp(min=0).long()].double(), 0.0)
                term = term * rc.weights[:, j, None].double() if weighted else term
                terms, size_ = terms + term, size_ + term.abs()
            back = torch.full((T, d + 8), 7.0, dtype=dtype, device="cuda")
            y = m.nvfp4_combine(ys, rc, residual=res, out=back[:, :d], weighted=weighted)
            assert (back[:, d:] == 7).all()
            tol = _gamma(k + 1) * size_ + _half(dtype) * (terms.abs() + _gamma(k + 1) * size_) + 2.0 ** -130
            assert ((y.double() - terms).abs() <= tol).all()
            for t in range(0, T, 400):
                part = [v[t:t + 400].contiguous() for v in (rc.experts, rc.weights, rc.rows)]
                part = m.Routes(*part, rc.sources[:part[0].numel()], rc.offsets)
                few = m.nvfp4_combine(ys, part, residual=None if res is None else res[t:t + 400], out_dtype=dtype, weighted=weighted)
                assert torch.equal(few, y[t:t + 400])
            if res is not None:
                held = res.clone()
                assert torch.equal(m.nvfp4_combine(ys, rc, residual=held, out=held), y)


@pytest.mark.parametrize("padded", [0.0, 0.25])
@pytest.mark.parametrize("size", LARGE + [(530, 8, 1032), (900, 5, 2064)], ids=lambda s: "x".join(map(str, s)))
def test_combine_gradient_of_many_tokens(size, padded):
    m = nv()
    T, k, d = size
    r = _routes(T, 40, k, T, padded)
    rc = _cuda(r)
    live = int(r.offsets[-1])
    ys = torch.full((T * k, d + 8), float("nan"), dtype=torch.bfloat16, device="cuda")[:, :d]
    ys[:live] = _rand((live, d), 4).cuda()
    dy = torch.zeros(T, d + 16, dtype=torch.bfloat16, device="cuda")[:, :d]
    dy.copy_(_rand((T, d), 5))
    dys = torch.full((T * k, d + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((T, k), 7.0, device="cuda")
    m.nvfp4_combine_bwd(dy, ys, rc, dys=dys[:, :d], dweights=dw)
    assert (dys[live:] == 7).all() and (dys[:, d:] == 7).all() and (dw[rc.rows < 0] == 0).all()
    choice = rc.sources[:live].long()
    want = rc.weights.double().view(-1)[choice][:, None] * dy.double()[choice // k]
    assert ((dys[:live, :d].double() - want).abs() <= 2.0 ** -8 * (1 + 2.0 ** -8) * want.abs() + 2.0 ** -130).all()
    products = dy.double()[choice // k] * ys[:live].double()
    assert ((dw.double().view(-1)[choice] - products.sum(1)).abs() <= _gamma(d) * products.abs().sum(1) + 2.0 ** -130).all()
    again = torch.full((T * k, d), 7.0, dtype=torch.bfloat16, device="cuda"), torch.empty(T, k, device="cuda")
    m.nvfp4_combine_bwd(dy, ys, rc, dys=again[0], dweights=again[1])
    assert torch.equal(again[0][:live], dys[:live, :d]) and torch.equal(again[1], dw)
