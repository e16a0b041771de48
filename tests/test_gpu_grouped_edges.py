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
