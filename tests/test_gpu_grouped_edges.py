"""Products grouped by expert: launches behind one another, expired waits, wide tiles, long
reductions and offsets out of order.

Operands are small integers where nothing else is said: products and partial sums below 2^24 are
exact in fp32 in any order, so results are compared for equality."""
import numpy as np
import pytest
import torch

from gpu_helpers import nv

pytestmark = pytest.mark.gpu


def _off(counts, first=0):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]) + first, dtype=torch.int32)


def _ints(g, *shape, top=3):
    return torch.randint(-top, top + 1, shape, generator=g).bfloat16()


def _products(a, w, off, kn):
    """fp64 rows of a by their expert's weight; rows that no expert owns are zero."""
    out = torch.zeros(a.shape[0], w.shape[2] if kn else w.shape[1], dtype=torch.float64)
    for e in range(w.shape[0]):
        lo, hi = int(off[e]), int(off[e + 1])
        out[lo:hi] = a[lo:hi].double() @ (w[e].double() if kn else w[e].double().t())
    return out


def _wgrads(dy, x, off):
    return torch.stack([dy[lo:hi].double().t() @ x[lo:hi].double() for lo, hi in zip(off[:-1].tolist(), off[1:].tolist())])


def test_short_launches_behind_one_another():
    # launches of a few tiles, each of which starts while the one before it ends: none leaves an arrival
    # behind that a later one's barriers would count
    m = nv()
    g = torch.Generator().manual_seed(1)
    counts, K, N = [70, 0, 9, 121], 200, 264
    off = _off(counts)
    a, w, dy = _ints(g, sum(counts), K), _ints(g, 4, N, K), _ints(g, sum(counts), N)
    want = (_products(a, w, off, False), _products(dy, w, off, True), _wgrads(dy, a, off))
    a, w, dy, off = (t.cuda() for t in (a, w, dy, off))
    ws = m.Workspace()
    runs = []
    for _ in range(200):
        runs.append((m.nvfp4_bf16_gemm_grouped(a, w, off, out_dtype=torch.float32, ws=ws),
                     m.nvfp4_bf16_gemm_grouped(dy, w, off, b_kn=True, out_dtype=torch.float32, ws=ws),
                     m.nvfp4_bf16_wgrad_grouped(dy, a, off, ws=ws)))
    assert m.nvfp4_poll(ws) == 0
    for got, ref in zip(runs[0], want):
        assert torch.equal(got.cpu().double(), ref)
    assert all(torch.equal(p, q) for r in runs[1:] for p, q in zip(runs[0], r))


def test_offsets_written_by_the_kernel_before():
    # the call's set-up overlaps the end of the kernel that writes its offsets: they are read behind it
    m = nv()
    g = torch.Generator().manual_seed(2)
    K, N = 72, 136
    a, w = _ints(g, 200, K), _ints(g, 3, N, K)
    offs = [_off(c) for c in ([200, 0, 0], [0, 150, 50], [20, 60, 120])]
    want = [_products(a, w, o, False) for o in offs]
    a, w, offs = a.cuda(), w.cuda(), [o.cuda() for o in offs]
    off = torch.zeros_like(offs[0])
    ws = m.Workspace()
    outs = []
    for i in range(60):
        off.copy_(offs[i % 3])
        outs.append(m.nvfp4_bf16_gemm_grouped(a, w, off, out_dtype=torch.float32, ws=ws))
    assert m.nvfp4_poll(ws) == 0
    for i, out in enumerate(outs):
        assert torch.equal(out.cpu().double(), want[i % 3]), i


def _expired(m, ws, call):
    """The status of a call whose waits have a nanosecond."""
    m.nvfp4_set_wait_budget_ns(1)
    try:
        call()
        return m.nvfp4_poll(ws)
    finally:
        m.nvfp4_set_wait_budget_ns(0)     # back to the default


@pytest.mark.parametrize("op", ["fprop", "dgrad", "wgrad"])
@pytest.mark.parametrize("counts", [[300, 0, 77, 1], [129] * 90], ids=["few tiles", "many tiles"])
def test_an_expired_call_drains_and_the_next_is_right(op, counts):
    # the first wait for a load takes far more than a nanosecond: the call stops with copies in flight and
    # lets them land.  fp32 output, i.e. short accumulators; wgrad's tails land on barriers of their own
    m = nv()
    g = torch.Generator().manual_seed(3)
    K, N, off = 520, 264, _off(counts)
    w, x, dy = _ints(g, len(counts), N, K), _ints(g, sum(counts), K), _ints(g, sum(counts), N)
    want = {"fprop": lambda: _products(x, w, off, False), "dgrad": lambda: _products(dy, w, off, True), "wgrad": lambda: _wgrads(dy, x, off)}[op]()
    w, x, dy, off = (t.cuda() for t in (w, x, dy, off))
    ws = m.Workspace()
    call = {"fprop": lambda: m.nvfp4_bf16_gemm_grouped(x, w, off, out_dtype=torch.float32, ws=ws),
            "dgrad": lambda: m.nvfp4_bf16_gemm_grouped(dy, w, off, b_kn=True, out_dtype=torch.float32, ws=ws),
            "wgrad": lambda: m.nvfp4_bf16_wgrad_grouped(dy, x, off, ws=ws)}[op]
    assert torch.equal(call().cpu().double(), want) and m.nvfp4_poll(ws) == 0
    for _ in range(10):
        assert _expired(m, ws, call) == 8 and m.nvfp4_poll(ws) == 0
        assert torch.equal(call().cpu().double(), want) and m.nvfp4_poll(ws) == 0


def test_an_expired_wgrad_of_a_long_run():
    m = nv()
    g = torch.Generator().manual_seed(4)
    rows = 2 ** 18 + 77
    dy, x = _ints(g, rows, 256, top=1), _ints(g, rows, 256, top=1)
    want = (dy.float().t() @ x.float()).double()[None]        # |sums| <= 2^19: exact
    dy, x, off = dy.cuda(), x.cuda(), torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    ws = m.Workspace()
    call = lambda: m.nvfp4_bf16_wgrad_grouped(dy, x, off, ws=ws)
    for _ in range(3):
        assert _expired(m, ws, call) == 8
        assert torch.equal(call().cpu().double(), want) and m.nvfp4_poll(ws) == 0


def test_a_tail_behind_a_long_run_is_waited_for():
    # Two experts of 64 tiles: the first one's are over a millisecond long and end at a whole stage, most
    # pairs then take one of the second's, whose single stage is a tail.  No single load or product takes
    # long, so a budget of 0.25 ms suffices.
    m = nv()
    g = torch.Generator(device="cuda").manual_seed(5)
    counts = [2 ** 19, 17]
    dy, x = (torch.randint(-1, 2, (sum(counts), 2048), generator=g, device="cuda", dtype=torch.int8).bfloat16() for _ in range(2))
    off = _off(counts).cuda()
    ws = m.Workspace()
    out = torch.empty(2, 2048, 2048, device="cuda")
    m.nvfp4_bf16_wgrad_grouped(dy, x, off, out=out, ws=ws)
    assert m.nvfp4_poll(ws) == 0
    out.zero_()
    m.nvfp4_set_wait_budget_ns(250000)
    try:
        m.nvfp4_bf16_wgrad_grouped(dy, x, off, out=out, ws=ws)
        assert m.nvfp4_poll(ws) == 0
    finally:
        m.nvfp4_set_wait_budget_ns(0)
    for e, (lo, hi) in enumerate(((0, counts[0]), (counts[0], sum(counts)))):
        assert torch.equal(out[e], dy[lo:hi].float().t() @ x[lo:hi].float()), e     # integers up to 2^19


@pytest.mark.parametrize("rows", [5, 40, 65, 300])
@pytest.mark.parametrize("kn", [False, True], ids=["nk", "kn"])
def test_bf16_output_of_a_long_reduction(rows, kn):
    """Positive operands, K = 2^20, on both sides of the rule for few rows.  A run of 1024 products takes
    64 adds of 16; each truncates by less than 2^-23 of the partial sum, half of the run's on
    average: 32 * 2^-23.  The K / 512 joins at most, rounded, add K / 512 / 2 * 2^-24.  The rest is half
    a bf16 step of the sum itself.  (In one accumulator the sums come out some 6e-3 low, up to two
    steps.)"""
    m = nv()
    g = torch.Generator(device="cuda").manual_seed(rows)
    K, N = 2 ** 20, 8
    a = torch.rand(rows, K, generator=g, device="cuda").bfloat16()
    w = torch.rand(*((2, K, N) if kn else (2, N, K)), generator=g, device="cuda").bfloat16()
    off = _off([rows // 2, rows - rows // 2])
    ws = m.Workspace()
    got = m.nvfp4_bf16_gemm_grouped(a, w, off.cuda(), b_kn=kn, ws=ws)
    assert got.dtype == torch.bfloat16 and m.nvfp4_poll(ws) == 0
    for e in range(2):
        lo, hi = int(off[e]), int(off[e + 1])
        ref = a[lo:hi].double() @ (w[e].double() if kn else w[e].double().t())
        half = torch.ldexp(torch.ones_like(ref), torch.frexp(ref)[1] - 9)       # of a step: 8 bits from the leading one
        bound = half + ref * (32 * 2.0 ** -23 + K / 1024 * 2.0 ** -24)
        err = (got[lo:hi].double() - ref).abs()
        assert (err <= bound).all(), f"{int((err > bound).sum())} of {err.numel()}, worst {float((err / half).max()):.3f} half steps"


def test_added_gradients_near_the_subnormal_range():
    # exact but where D, the product or the sum is subnormal, each of which may become zero: two of them at
    # most (D and the product, or one and the sum), each below the smallest normal number
    m = nv()
    tiny = 2.0 ** -126
    start = torch.tensor([0.0, 0.5, 1.5, -0.25, -1.0, 3.0, -3.0, 2.0 ** -23], dtype=torch.float64) * tiny
    dy = torch.full((1, 8), 2.0 ** -63).bfloat16()
    x = torch.tensor([[-1.0, 1.0, -0.75, 0.0, 2.0, 1.0, 0.5, -2.0]]).mul(2.0 ** -63).bfloat16()
    out = start[:, None].expand(8, 8).float().contiguous()[None].cuda()
    assert torch.equal(out[0].cpu().double(), start[:, None].expand(8, 8))
    off = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    m.nvfp4_bf16_wgrad_grouped(dy.cuda(), x.cuda(), off, out=out, accumulate=True)
    want = start[:, None] + dy.double().t() @ x.double()
    err = (out[0].cpu().double() - want).abs()
    held = lambda t: (t.abs() >= tiny) | (t == 0)
    exact = held(start)[:, None] & held(x.double() * 2.0 ** -63) & held(want)
    assert (err < 2 * tiny).all() and (err[exact] == 0).all() and exact.any()


@pytest.mark.parametrize("rows,K,N", [(6, 520, 264), (24, 4104, 72), (64, 2056, 4104), (65, 520, 264), (700, 1160, 2056)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_a_row_does_not_depend_on_the_offsets_or_other_rows(rows, K, N, dtype):
    # one weight for all of four experts: however the rows are dealt out, in whatever order, each comes out
    # with the same bits
    m = nv()
    g = torch.Generator(device="cuda").manual_seed(rows)
    a = torch.randn(rows, K, generator=g, device="cuda").bfloat16()
    w = torch.randn(1, N, K, generator=g, device="cuda").bfloat16().expand(4, N, K).contiguous()
    for kn in (False, True):
        b = w.transpose(1, 2).contiguous() if kn else w
        run = lambda x, counts: m.nvfp4_bf16_gemm_grouped(x, b, _off(counts).cuda(), b_kn=kn, out_dtype=dtype)
        first = run(a, [rows, 0, 0, 0])
        for counts in ([0, 0, 0, rows], [rows // 3, 0, rows - rows // 3, 0], [1, rows - 3, 1, 1], [rows // 4] * 3 + [rows - 3 * (rows // 4)]):
            assert torch.equal(run(a, counts), first), (kn, counts)
            order = torch.randperm(rows, generator=g, device="cuda")
            assert torch.equal(run(a[order], counts), first[order]), (kn, counts)


@pytest.mark.parametrize("budget", [2 ** 62, 2 ** 63, 2 ** 64 - 1])
def test_the_longest_budgets_do_not_run_out_at_once(budget):
    # a GEMM whose epilogue waits about a millisecond for its accumulator, and a product grouped by expert
    from test_gpu_wait_budget import _long_k_operand
    m = nv()
    a, b = _long_k_operand(m, 128, 1 << 19, 1), _long_k_operand(m, 256, 1 << 19, 2)
    g = torch.Generator(device="cuda").manual_seed(6)
    x, w = torch.randn(256, 2 ** 17, generator=g, device="cuda").bfloat16(), torch.randn(1, 256, 2 ** 17, generator=g, device="cuda").bfloat16()
    off = torch.tensor([0, 256], dtype=torch.int32, device="cuda")
    ws = m.Workspace()
    m.nvfp4_set_wait_budget_ns(budget)
    try:
        m.nvfp4_gemm(a, b, out_dtype=torch.float32, ws=ws)
        assert m.nvfp4_poll(ws) == 0
        m.nvfp4_bf16_gemm_grouped(x, w, off, ws=ws)
        assert m.nvfp4_poll(ws) == 0
    finally:
        m.nvfp4_set_wait_budget_ns(0)
