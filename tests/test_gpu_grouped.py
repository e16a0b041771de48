"""Products grouped by expert (nvfp4_bf16_gemm_grouped, nvfp4_bf16_wgrad_grouped) against fp64
products of the same bf16 values.

Tolerances (from the arithmetic): bf16 x bf16 products are exact in fp32.  A running fp32 sum of k
products errs by at most gamma_k * sum |a b|, gamma_k = k u / (1 - k u), u = 2^-23 (one fp32 ulp per
add: the tensor core may truncate).  With fp32 output the runs are at most 512 products long and
are joined by rounded fp32 adds: gamma_512 + (number of runs) * 2^-23 covers both.  A bf16 output
adds half a bf16 step, 2^-8 |D| (relative to the value, 2^-9 at best and 2^-8 at worst in a binade)."""
import types

import numpy as np
import pytest
import torch

from gpu_helpers import nv

pytestmark = pytest.mark.gpu

NAN = float("nan")


def _offsets(counts, first=0):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]) + first, dtype=torch.int32)


def _inputs(counts, K, N, E=None, before=0, behind=0, seed=0):
    """a [rows][K] (NaN in rows that no expert owns), w [E][N][K], offsets"""
    g = torch.Generator().manual_seed(seed)
    rows = before + sum(counts) + behind
    a = torch.randn(rows, K, generator=g).bfloat16()
    a[:before] = NAN
    a[before + sum(counts):] = NAN
    w = (torch.randn(len(counts), N, K, generator=g) * 0.1).bfloat16()
    return a, w, _offsets(counts, before)


def _gamma(K, fp32):
    u = 2.0 ** -23
    run = min(K, 512) if fp32 else K
    return run * u / (1 - run * u) + (-(-K // run)) * u


def _within(got, ref, sabs, K, what):
    fp32 = got.dtype == torch.float32
    tol = _gamma(K, fp32) * sabs + (0.0 if fp32 else 2.0 ** -8) * ref.abs() + 1e-30
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst ratio {float((err / tol).max()):.3g}, first {bad.nonzero()[0].tolist()}"


def _reference(a, w, off, kn):
    N = w.shape[2] if kn else w.shape[1]
    ref = torch.zeros(a.shape[0], N, dtype=torch.float64)
    sabs = torch.zeros_like(ref)
    for e in range(w.shape[0]):
        lo, hi = int(off[e]), int(off[e + 1])
        we = w[e].double() if kn else w[e].double().t()
        ref[lo:hi] = a[lo:hi].double() @ we
        sabs[lo:hi] = a[lo:hi].double().abs() @ we.abs()
    return ref, sabs


def _check_gemm(counts, K, N, kn, dtype, before=0, behind=0, seed=0):
    m = nv()
    a, w, off = _inputs(counts, K, N, before=before, behind=behind, seed=seed)
    if kn:
        w = w.transpose(1, 2).contiguous()
    out = torch.full((a.shape[0], N), 7.0, dtype=dtype, device="cuda")
    ws = m.Workspace()
    got = m.nvfp4_bf16_gemm_grouped(a.cuda(), w.cuda(), off.cuda(), b_kn=kn, out=out, ws=ws)
    assert got is out and m.nvfp4_poll(ws) == 0
    got = out.cpu()
    lo, hi = before, before + sum(counts)
    assert (got[:lo] == 7).all() and (got[hi:] == 7).all(), "rows that no expert owns were written"
    ref, sabs = _reference(a, w, off, kn)
    _within(got[lo:hi], ref[lo:hi], sabs[lo:hi], K, f"{counts} K {K} N {N} kn {kn}")


COUNTS = [[1], [0, 3, 0, 0, 1], [63, 64, 65, 1], [0, 127, 128, 129, 0], [255, 256, 257], [700, 0, 31, 5], [1] * 40]


@pytest.mark.parametrize("kn", [False, True], ids=["nk", "kn"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{sum(c)}")
def test_gemm_ragged_rows(counts, dtype, kn):
    _check_gemm(counts, 136, 264, kn, dtype, before=3, behind=6, seed=len(counts))


@pytest.mark.parametrize("kn", [False, True], ids=["nk", "kn"])
@pytest.mark.parametrize("K,N", [(8, 8), (16, 520), (64, 256), (72, 40), (1032, 128), (2056, 8), (520, 1000)])
@pytest.mark.parametrize("counts", [[2, 0, 5], [130, 7, 300]], ids=["few", "more"])
def test_gemm_sizes(counts, K, N, kn):
    _check_gemm(counts, K, N, kn, torch.float32, seed=K + N)
    _check_gemm(counts, K, N, kn, torch.bfloat16, behind=1, seed=K + N + 1)


@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 47, 63, 64, 65, 66, 127, 128, 129, 130, 200])
@pytest.mark.parametrize("spread", ["one", "even"])
def test_gemm_few_rows(rows, spread):
    # from a single token up, past every size at which another kernel may take over
    counts = [0, rows, 0] if spread == "one" else [rows // 3, 0, rows - rows // 3 - rows // 4, rows // 4]
    for kn in (False, True):
        _check_gemm(counts, 520, 328, kn, torch.float32, behind=2, seed=rows)
    _check_gemm(counts, 264, 72, False, torch.bfloat16, seed=rows + 1)


@pytest.mark.parametrize("kn", [False, True], ids=["nk", "kn"])
def test_gemm_exact_on_small_integers(kn):
    # |a|, |b| <= 8 and K <= 256: every partial sum is an integer below 2^24
    m = nv()
    g = torch.Generator().manual_seed(3)
    counts, K, N = [37, 0, 300, 1, 62], 256, 392
    off = _offsets(counts)
    a = torch.randint(-8, 9, (sum(counts), K), generator=g).bfloat16()
    w = torch.randint(-8, 9, (len(counts),) + ((K, N) if kn else (N, K)), generator=g).bfloat16()
    got = m.nvfp4_bf16_gemm_grouped(a.cuda(), w.cuda(), off.cuda(), b_kn=kn, out_dtype=torch.float32)
    assert torch.equal(got.cpu().double(), _reference(a, w, off, kn)[0])


@pytest.mark.parametrize("counts", [[1], [8], [24], [25], [64], [1, 0, 7], [9, 5]], ids=lambda c: f"{len(c)}x{sum(c)}")
@pytest.mark.parametrize("K,N", [(1032, 712), (2040, 40), (2056, 264), (5000, 136), (136, 4104)])
def test_gemm_few_rows_of_a_long_reduction(counts, K, N):
    for dtype in (torch.bfloat16, torch.float32):
        _check_gemm(counts, K, N, False, dtype, before=1, behind=1, seed=K + sum(counts))


@pytest.mark.parametrize("kn", [False, True], ids=["nk", "kn"])
@pytest.mark.parametrize("rows", [3, 11, 40, 100])
def test_gemm_long_runs_are_joined_by_rounding(rows, kn):
    """Positive integers whose products add to at most 512 * 2^14 < 2^24 in a run of 512: the runs
    are exact, so only the fp32 adds that join them err, by 2^-24 of the sum each: one per run of
    512 and one per part of a cut K (8 at most)."""
    m = nv()
    K, N, E = 65536 + 8, 24, 2
    g = torch.Generator().manual_seed(rows)
    a = torch.randint(1, 129, (rows, K), generator=g).bfloat16()
    w = torch.randint(1, 129, (E, K, N) if kn else (E, N, K), generator=g).bfloat16()
    off = _offsets([rows // 2, rows - rows // 2])
    got = m.nvfp4_bf16_gemm_grouped(a.cuda(), w.cuda(), off.cuda(), b_kn=kn, out_dtype=torch.float32).cpu()
    ref, _ = _reference(a, w, off, kn)
    worst = float(((got.double() - ref).abs() / ref).max())
    assert worst <= (-(-K // 512) + 8) * 2.0 ** -24, worst


@pytest.mark.parametrize("rows", [3, 300])
def test_gemm_strides(rows):
    # leading dimensions past the widths, experts apart from one another, an output inside a wider one
    m = nv()
    g = torch.Generator().manual_seed(5)
    K, N, E = 72, 136, 3
    abig = torch.randn(rows, K + 24, generator=g).bfloat16()
    wbig = torch.randn(E, N + 5, K + 16, generator=g).bfloat16()
    dbig = torch.full((rows, N + 16), -3.0, device="cuda")
    off = _offsets([rows // 3, 0, rows - rows // 3])
    a, w = abig[:, 8:8 + K], wbig[:, 2:2 + N, 8:8 + K]
    ag, wg = abig.cuda()[:, 8:8 + K], wbig.cuda()[:, 2:2 + N, 8:8 + K]
    m.nvfp4_bf16_gemm_grouped(ag, wg, off.cuda(), out=dbig[:, 8:8 + N])
    got = dbig.cpu()
    assert (got[:, :8] == -3).all() and (got[:, 8 + N:] == -3).all()
    ref, sabs = _reference(a, w, off, False)
    _within(got[:, 8:8 + N], ref, sabs, K, "strided")
    m.nvfp4_bf16_gemm_grouped(ag, wg.transpose(1, 2).contiguous(), off.cuda(), b_kn=True, out=dbig[:, 8:8 + N])
    _within(dbig.cpu()[:, 8:8 + N], ref, sabs, K, "strided kn")
    # one weight for every expert: stride 0
    shared = wbig.cuda()[:1, 2:2 + N, 8:8 + K].expand(E, N, K)
    m.nvfp4_bf16_gemm_grouped(ag, shared, off.cuda(), out=dbig[:, 8:8 + N])
    ref, sabs = _reference(a, w[:1].expand(E, N, K), off, False)
    _within(dbig.cpu()[:, 8:8 + N], ref, sabs, K, "one weight")


def test_gemm_nonfinite_rows_stay_apart():
    # an Inf or NaN in a row or in an expert's weight reaches the outputs it belongs to, no others
    m = nv()
    for counts in ([2, 3, 1], [70, 200, 131]):
        a, w, off = _inputs(counts, 136, 72, seed=9)
        bad = counts[0] + counts[1] // 2
        a[bad, 5] = NAN
        a[0, 7] = float("inf")
        w[2, 9, 3] = float("inf")
        out = m.nvfp4_bf16_gemm_grouped(a.cuda(), w.cuda(), off.cuda()).cpu().float()
        finite = torch.isfinite(out)
        want = torch.ones_like(finite)
        want[bad] = False
        want[0] = False
        want[counts[0] + counts[1]:, 9] = False
        assert torch.equal(finite, want)


def _check_wgrad(counts, M, N, add=False, before=0, behind=0, seed=0, pad=0):
    m = nv()
    g = torch.Generator().manual_seed(seed)
    E, rows = len(counts), before + sum(counts) + behind
    dy = torch.randn(rows, M, generator=g).bfloat16()
    x = torch.randn(rows, N, generator=g).bfloat16()
    for t in (dy, x):
        t[:before] = NAN
        t[before + sum(counts):] = NAN
    off = _offsets(counts, before)
    big = torch.randn(E, M + pad, N + 4 * pad, generator=g) if add else torch.full((E, M + pad, N + 4 * pad), 5.0)
    dev = big.cuda()
    ws = m.Workspace()
    out = dev[:, :M, :N]
    assert m.nvfp4_bf16_wgrad_grouped(dy.cuda(), x.cuda(), off.cuda(), out=out, accumulate=add, ws=ws) is out
    assert m.nvfp4_poll(ws) == 0
    got = dev.cpu()
    if pad:
        assert torch.equal(got[:, M:], big[:, M:]) and torch.equal(got[:, :, N:], big[:, :, N:])
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        a, b = dy[lo:hi].double(), x[lo:hi].double()
        ref, sabs = a.t() @ b, a.abs().t() @ b.abs()
        if lo == hi:
            assert torch.equal(got[e, :M, :N], big[e, :M, :N] if add else torch.zeros(M, N)), f"expert {e} owns no row"
            continue
        if add:
            ref = ref + big[e, :M, :N].double()
            sabs = sabs + big[e, :M, :N].double().abs()
        _within(got[e, :M, :N], ref, sabs, hi - lo + 1, f"wgrad expert {e} of {counts}")


@pytest.mark.parametrize("add", [False, True], ids=["store", "add"])
@pytest.mark.parametrize("counts", COUNTS + [[5, 0, 1500], [512, 513, 1025]], ids=lambda c: f"{len(c)}x{sum(c)}")
def test_wgrad_ragged_rows(counts, add):
    _check_wgrad(counts, 136, 264, add, before=2, behind=9, seed=len(counts))


@pytest.mark.parametrize("M,N", [(8, 8), (8, 520), (520, 8), (256, 256), (264, 40), (1000, 72)])
def test_wgrad_sizes(M, N):
    _check_wgrad([3, 0, 130, 64], M, N, seed=M + N)
    _check_wgrad([3, 0, 130, 64], M, N, add=True, behind=3, seed=M + N, pad=3)
    _check_wgrad([1], M, N, seed=1, pad=1)


def test_wgrad_nonfinite_rows_stay_with_their_expert():
    m = nv()
    counts = [70, 1, 63, 130]
    g = torch.Generator().manual_seed(2)
    dy = torch.randn(sum(counts), 72, generator=g).bfloat16()
    x = torch.randn(sum(counts), 136, generator=g).bfloat16()
    dy[70] = NAN      # the only row of expert 1, behind expert 0's last and before expert 2's first
    x[70] = float("inf")
    out = m.nvfp4_bf16_wgrad_grouped(dy.cuda(), x.cuda(), _offsets(counts).cuda()).cpu()
    for e in range(4):
        assert torch.isfinite(out[e]).all() if e != 1 else torch.isnan(out[e]).all(), e


def test_wgrad_long_runs_keep_fp32_accuracy():
    # 20000 products of one sign: a truncating running sum would be off by some 1e-4.  A run of 512 takes
    # 32 adds of 16 products; each loses less than 2^-23 of the partial sum, which is half of the run's
    # on average: 32 / 2 * 2^-23 = 1.9e-6; the 40 joins add at most 40 / 2 * 2^-24 = 1.2e-6
    m = nv()
    g = torch.Generator().manual_seed(4)
    dy = torch.rand(20000, 64, generator=g).bfloat16()
    x = torch.rand(20000, 64, generator=g).bfloat16()
    out = m.nvfp4_bf16_wgrad_grouped(dy.cuda(), x.cuda(), _offsets([20000]).cuda()).cpu()[0]
    ref = dy.double().t() @ x.double()
    _within(out, ref, ref, 20000, "long run")
    assert float(((out.double() - ref) / ref).abs().max()) < 4e-6


@pytest.mark.parametrize("values", [[0, 9, 5, 20], [4, 2, 30, 20], [-5, 3, 10, 20], [0, 25, 26, 27], [20, 0, 0, 20], [0, -7, 2 ** 31 - 1, 5]])
def test_offsets_out_of_order_are_reported_and_stay_in_bounds(values):
    m = nv()
    K, N, rows = 64, 72, 20
    g = torch.Generator().manual_seed(1)
    a = torch.randn(rows, K, generator=g).bfloat16()
    w = torch.randn(3, N, K, generator=g).bfloat16()
    off = torch.tensor(values, dtype=torch.int32)
    run = np.maximum.accumulate(np.clip(values, 0, rows))
    ref, sabs = _reference(a, w, run, False)
    out = torch.full((rows + 40, N), 7.0, device="cuda")
    ws = m.Workspace()
    m.nvfp4_bf16_gemm_grouped(a.cuda(), w.cuda(), off.cuda(), out=out[20:40], ws=ws)
    assert m.nvfp4_poll(ws) == 4 and m.nvfp4_poll(ws) == 0
    got = out.cpu()
    assert (got[:20] == 7).all() and (got[40:] == 7).all()
    lo, hi = int(run[0]), int(run[-1])
    _within(got[20 + lo:20 + hi], ref[lo:hi], sabs[lo:hi], K, "rows as the running maximum gives them")
    assert (got[20:20 + lo] == 7).all() and (got[20 + hi:40] == 7).all()
    dw = m.nvfp4_bf16_wgrad_grouped(a.cuda(), a.cuda(), off.cuda(), ws=ws).cpu()
    assert m.nvfp4_poll(ws) == 4
    for e in range(3):
        r = a[int(run[e]):int(run[e + 1])].double()
        _within(dw[e], r.t() @ r, r.abs().t() @ r.abs(), rows, f"wgrad {e}")


def test_no_rows():
    m = nv()
    w = torch.randn(2, 16, 8).bfloat16().cuda()
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert m.nvfp4_bf16_gemm_grouped(torch.empty(0, 8, dtype=torch.bfloat16, device="cuda"), w, off).shape == (0, 16)
    dw = m.nvfp4_bf16_wgrad_grouped(torch.empty(0, 16, dtype=torch.bfloat16, device="cuda"),
                                    torch.empty(0, 8, dtype=torch.bfloat16, device="cuda"), off)
    assert dw.shape == (2, 16, 8) and not dw.any()
    a = torch.full((300, 8), NAN, dtype=torch.bfloat16, device="cuda")
    out = torch.full((300, 16), 2.0, device="cuda")
    m.nvfp4_bf16_gemm_grouped(a, w, off, out=out)      # rows, but none that an expert owns
    assert (out == 2).all()


def test_most_experts():
    m = nv()
    g = torch.Generator().manual_seed(8)
    counts = torch.randint(0, 3, (1024,), generator=g).tolist()
    _check_gemm(counts, 16, 24, False, torch.float32, seed=1)
    _check_gemm(counts, 16, 24, True, torch.float32, seed=2)
    _check_gemm([0] * 1023 + [5], 16, 24, False, torch.float32, seed=3)
    _check_wgrad(counts, 16, 8, seed=4)


def test_far_offsets():
    # element offsets past 2^31: experts 2^30 elements apart, rows of a operand past 4 GiB
    m = nv()
    g = torch.Generator().manual_seed(6)
    K, N = 64, 72
    w = torch.randn(4, N, K, generator=g).bfloat16()
    store = torch.empty(3 * 2 ** 30 + N * K, dtype=torch.bfloat16, device="cuda")
    far = store.as_strided((4, N, K), (2 ** 30, K, 1))
    far.copy_(w)
    a = torch.randn(40, K, generator=g).bfloat16()
    off = _offsets([10, 0, 13, 17])
    got = m.nvfp4_bf16_gemm_grouped(a.cuda(), far, off.cuda(), out_dtype=torch.float32).cpu()
    ref, sabs = _reference(a, w, off, False)
    _within(got, ref, sabs, K, "far experts")
    del store, far
    rows, ld = 60000, 2 ** 16
    big = torch.zeros(rows, ld, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(100, K, generator=g).bfloat16()
    big[-100:, :K] = tail.cuda()
    off = torch.tensor([rows - 100, rows - 60, rows - 60, rows - 1, rows], dtype=torch.int32)
    out = torch.zeros(rows, N, device="cuda")
    m.nvfp4_bf16_gemm_grouped(big[:, :K], w.cuda(), off.cuda(), out=out)
    ref, sabs = _reference(tail, w, off - (rows - 100), False)
    _within(out[-100:].cpu(), ref, sabs, K, "far rows")
    dw = m.nvfp4_bf16_wgrad_grouped(big[:, :K], big[:, :K], off.cuda()).cpu()
    for e, (lo, hi) in enumerate(((0, 40), (40, 40), (40, 99), (99, 100))):
        r = tail[lo:hi].double()
        _within(dw[e], r.t() @ r, r.abs().t() @ r.abs(), 100, f"far rows wgrad {e}")


def test_repeats_bit_for_bit():
    m = nv()
    for counts in ([3, 0, 9], [300, 5, 700]):
        a, w, off = (t.cuda() for t in _inputs(counts, 520, 264, seed=1))
        dy = torch.randn(sum(counts), 264, device="cuda").bfloat16()
        first = (m.nvfp4_bf16_gemm_grouped(a, w, off, out_dtype=torch.float32), m.nvfp4_bf16_gemm_grouped(dy, w, off, b_kn=True),
                 m.nvfp4_bf16_wgrad_grouped(dy, a, off))
        for _ in range(3):
            again = (m.nvfp4_bf16_gemm_grouped(a, w, off, out_dtype=torch.float32), m.nvfp4_bf16_gemm_grouped(dy, w, off, b_kn=True),
                     m.nvfp4_bf16_wgrad_grouped(dy, a, off))
            assert all(torch.equal(p, q) for p, q in zip(first, again))


def test_streams_graphs_and_two_at_once():
    # captured once, replayed with other rows, offsets and weights in the same buffers; two graphs and an
    # eager call at the same time on three streams
    m = nv()
    K, N = 136, 264

    def state(counts, seed):
        a, w, off = _inputs(counts, K, N, seed=seed)
        return a, w, off

    sets = [state([3, 9, 0, 2], 1), state([0, 1, 13, 0], 2)], [state([300, 0, 80, 20], 3), state([1, 2, 3, 394], 4)]
    graphs = []
    for first, _ in sets:
        a, w, off = (t.cuda() for t in first)
        dy = a.new_zeros(a.shape[0], N)
        y = torch.zeros(a.shape[0], N, device="cuda")
        dx = torch.zeros(a.shape[0], K, device="cuda")
        dw = torch.zeros(4, N, K, device="cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()

        spare = torch.zeros_like(y)
        side = torch.cuda.Stream()

        def body():   # behind another stream's work, a memset, a copy and kernels
            here = torch.cuda.current_stream()
            side.wait_stream(here)
            with torch.cuda.stream(side):
                spare.add_(1)
            y.zero_()
            here.wait_stream(side)
            m.nvfp4_bf16_gemm_grouped(a, w, off, out=y)
            spare.copy_(y)
            m.nvfp4_bf16_gemm_grouped(a, w, off, out=y)
            dy.copy_(y)
            m.nvfp4_bf16_gemm_grouped(dy, w, off, b_kn=True, out=dx)
            m.nvfp4_bf16_wgrad_grouped(dy, a, off, out=dw)

        with torch.cuda.stream(s):
            body()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            body()
        graphs.append((g, s, a, w, off, y, dy, dx, dw))
    for which in (1, 0):
        for (g, s, a, w, off, *_), pair in zip(graphs, sets):
            for dst, src in zip((a, w, off), pair[which]):
                dst.copy_(src)
        torch.cuda.synchronize()
        for g, s, *_ in graphs:
            with torch.cuda.stream(s):
                for _ in range(3):
                    g.replay()
        a, w, off = sets[1][which]
        other = torch.cuda.Stream()
        eager = m.nvfp4_bf16_gemm_grouped(a.cuda(), w.cuda(), off.cuda(), out_dtype=torch.float32)
        side = torch.zeros_like(eager)
        other.wait_stream(torch.cuda.current_stream())
        ag, wg, og = a.cuda(), w.cuda(), off.cuda()
        torch.cuda.synchronize()
        m.nvfp4_bf16_gemm_grouped(ag, wg, og, out=side, stream=other)
        torch.cuda.synchronize()
        assert torch.equal(side, eager)
        for (g, s, ga, gw, goff, y, dy, dx, dw), pair in zip(graphs, sets):
            a, w, off = pair[which]
            ref, sabs = _reference(a, w, off, False)
            _within(y.cpu(), ref, sabs, K, "replayed fwd")
            d = dy.cpu()
            ref, sabs = _reference(d, w, off, True)
            _within(dx.cpu(), ref, sabs, N, "replayed dgrad")
            for e in range(4):
                lo, hi = int(off[e]), int(off[e + 1])
                p, q = d[lo:hi].double(), a[lo:hi].double()
                _within(dw[e].cpu(), p.t() @ q, p.abs().t() @ q.abs(), max(hi - lo, 1), "replayed wgrad")


def test_layer_gradients_against_differences():
    # the layer is linear in x and in w, and on small integers every product and sum is exact:
    # <dy, y(x + u) - y(x)> = <dx, u> and <dy, y(w + u) - y(w)> = <dw, u>, bit for bit
    m = nv()
    g = torch.Generator().manual_seed(7)
    counts, d, n = [40, 0, 150, 3], 64, 72
    rows, E = sum(counts), len(counts)
    off = _offsets(counts).cuda()
    ints = lambda *s: torch.randint(-3, 4, s, generator=g).bfloat16().cuda()
    x, w, dy, ux, uw = ints(rows, d), ints(E, n, d), torch.randint(-1, 2, (rows, n), generator=g).bfloat16().cuda(), ints(rows, d), ints(E, n, d)
    lay = m.GroupedLinearBF16(E, d, n)
    dx, dw = lay.bwd(x, w, dy, off)        # |dx| <= 216 = an integer that bf16 holds
    assert m.nvfp4_poll(lay.ws) == 0
    fwd = lambda x, w: m.nvfp4_bf16_gemm_grouped(x, w, off, out_dtype=torch.float32).double()
    diff_x = (dy.double() * (fwd(x + ux, w) - fwd(x, w))).sum()
    diff_w = (dy.double() * (fwd(x, w + uw) - fwd(x, w))).sum()
    assert float(diff_x) == float((dx.double() * ux.double()).sum())
    assert float(diff_w) == float((dw.double() * uw.double()).sum())


def test_binding_refuses():
    m = nv()
    a = torch.zeros(4, 16, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(2, 8, 16, dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        m.nvfp4_bf16_gemm_grouped(a.float(), w, off)
    with pytest.raises(TypeError):
        m.nvfp4_bf16_gemm_grouped(a, w[0], off)
    with pytest.raises(TypeError):
        m.nvfp4_bf16_gemm_grouped(a, w, off, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        m.nvfp4_bf16_gemm_grouped(a, w, off, b_kn=True)           # K differs
    with pytest.raises(ValueError):
        m.nvfp4_bf16_gemm_grouped(a, w, off[:2])
    with pytest.raises(ValueError):
        m.nvfp4_bf16_gemm_grouped(a, w, off.long())
    with pytest.raises(ValueError):
        m.nvfp4_bf16_gemm_grouped(a, w, off.cpu())
    with pytest.raises(ValueError):
        m.nvfp4_bf16_gemm_grouped(a, w, off, out=torch.zeros(4, 16, device="cuda"))
    with pytest.raises(ValueError):
        m.nvfp4_bf16_gemm_grouped(a.t().contiguous().t(), w, off)
    with pytest.raises(m.NVFP4Error):                             # K % 8
        m.nvfp4_bf16_gemm_grouped(a[:, :12], w[:, :, :12], off)
    with pytest.raises(m.NVFP4Error):                             # 16-byte rule
        m.nvfp4_bf16_gemm_grouped(a[:, 4:12], w[:, :, 4:12], off)
    with pytest.raises(ValueError):
        m.nvfp4_bf16_wgrad_grouped(a, a[:3], off)
    with pytest.raises(ValueError):
        m.nvfp4_bf16_wgrad_grouped(a, a, off, accumulate=True)
    with pytest.raises(ValueError):
        m.nvfp4_bf16_wgrad_grouped(a, a, off, out=torch.zeros(3, 16, 16, device="cuda"))
    with pytest.raises(m.NVFP4Error):                             # gradients that overlap
        m.nvfp4_bf16_wgrad_grouped(a, a, off, out=torch.zeros(1, 16, 16, device="cuda").expand(2, 16, 16), accumulate=True)
    with pytest.raises(ValueError):
        m.GroupedLinearBF16(2, 16, 16).fwd(a, w, off)


def test_a_workspace_of_another_device_is_refused():
    m = nv()
    a = torch.zeros(4, 16, dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(2, dtype=torch.int32, device="cuda")
    other = types.SimpleNamespace(index=a.get_device() + 1, addr=0)
    with pytest.raises(ValueError):
        m.nvfp4_bf16_gemm_grouped(a, torch.zeros(1, 8, 16, dtype=torch.bfloat16, device="cuda"), off, ws=other)
    with pytest.raises(ValueError):
        m.nvfp4_bf16_wgrad_grouped(a, a, off, ws=other)


@pytest.mark.parametrize("kn", [False, True], ids=["nk", "kn"])
def test_budget_expiry_is_reported_and_the_next_call_is_right(kn):
    # A bf16 output's accumulator holds the whole reduction: with K = 2^19 it takes over a millisecond,
    # far longer than the epilogue's first polls, so that with a budget of 1 ns its wait runs out for
    # certain.  The call drains its copies and MMAs, reports NVFP4_ERR_TIMEOUT (8) and leaves the device
    # usable.
    m = nv()
    g = torch.Generator(device="cuda").manual_seed(1)
    K, N, rows = 1 << 19, 256, 256
    a = torch.randn(rows, K, generator=g, device="cuda").bfloat16()
    w = torch.randn(*((1, K, N) if kn else (1, N, K)), generator=g, device="cuda").bfloat16()
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    ws = m.Workspace()
    want = m.nvfp4_bf16_gemm_grouped(a, w, off, b_kn=kn, ws=ws)
    assert m.nvfp4_poll(ws) == 0
    m.nvfp4_set_wait_budget_ns(1)
    try:
        m.nvfp4_bf16_gemm_grouped(a, w, off, b_kn=kn, ws=ws)
        status = m.nvfp4_poll(ws)
    finally:
        m.nvfp4_set_wait_budget_ns(0)     # back to the default
    assert status == 8 and m.nvfp4_poll(ws) == 0
    assert torch.equal(m.nvfp4_bf16_gemm_grouped(a, w, off, b_kn=kn, ws=ws), want) and m.nvfp4_poll(ws) == 0
    del a, w, want
    _check_gemm([300, 0, 77], 520, 264, kn, torch.float32)
    _check_wgrad([300, 0, 77], 136, 264)
