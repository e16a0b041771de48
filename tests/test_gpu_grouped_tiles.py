"""Products grouped by expert at sizes whose launches take many tiles: wide ones, several waves,
experts of more than one band of tiles.  The plan takes the width whose waves of tiles cost least,
so small cases never get there; it is restated here, and every case says what it has to reach.

Integer operands: products and sums are exact, so results are equal to the reference's."""
import math

import numpy as np
import pytest
import torch

from gpu_helpers import nv

pytestmark = pytest.mark.gpu

PAIRS, BAND = 74, 8


def _plan(lens, features, most_tiles):
    """The tile's width and the tiles per expert that the kernel chooses."""
    pairs = max(1, min(most_tiles, PAIRS))
    best = None
    for width in (256, 224, 192, 160, 128):
        n = [-(-x // width) for x in lens]
        rows = sum(k * 32 * math.ceil(x / (32 * k)) for k, x in zip(n, lens) if k)
        cost = math.ceil(sum(n) * -(-features // 256) / pairs) * (256 + rows / max(1, sum(n)))
        if best is None or cost < best[0] * (1 - 1e-6):
            best = cost, width, n
    _, width, n = best
    tall = [min(width, 32 * math.ceil(x / (32 * k))) for k, x in zip(n, lens) if k]
    return max(tall), max(n), sum(n) * -(-features // 256)


def _gemm_plan(counts, features):
    rows = sum(counts)
    return _plan([c for c in counts if c], features, -(-features // 256) * (rows // 128 + min(rows, len(counts))))


def _ints(g, *shape):
    return torch.randint(-3, 4, shape, generator=g, device="cuda", dtype=torch.int8).bfloat16()


def _off(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)


RAGGED = [1500, 900, 0, 1111, 1337, 1024, 977, 1203]     # many wide tiles
LONG = [4100, 1, 2900, 33]                               # more than a band of them


@pytest.mark.parametrize("counts", [RAGGED, LONG], ids=["ragged", "long"])
@pytest.mark.parametrize("K", [584, 640, 1096, 1152])    # one or two runs; whole blocks of 64, or not
@pytest.mark.parametrize("kn", [False, True], ids=["nk", "kn"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_gemm_wide_tiles(counts, K, kn, dtype):
    m = nv()
    N = 2568
    tall, most, tiles = _gemm_plan(counts, N)
    assert tiles > 2 * PAIRS and tall > 128 and (counts is not LONG or most > BAND)
    g = torch.Generator(device="cuda").manual_seed(K)
    E, rows, off = len(counts), sum(counts), _off(counts)
    a, w = _ints(g, rows, K), _ints(g, E, *((K, N) if kn else (N, K)))
    out = torch.full((rows + 9, N), 5.0, dtype=dtype, device="cuda")
    ws = m.Workspace()
    m.nvfp4_bf16_gemm_grouped(torch.cat([a, torch.full((9, K), float("nan"), dtype=torch.bfloat16, device="cuda")]), w, off.cuda(), b_kn=kn,
                              out=out, ws=ws)
    assert m.nvfp4_poll(ws) == 0 and (out[rows:] == 5).all()
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        ref = a[lo:hi].double() @ (w[e].double() if kn else w[e].double().t())
        assert torch.equal(out[lo:hi], ref.float().to(dtype)), e


def test_gemm_widths_between():
    # every width that the plan knows, from the rows of one expert
    m = nv()
    g = torch.Generator(device="cuda").manual_seed(1)
    K, N, seen = 520, 4096, set()
    for rows in (1200, 1340, 1600, 1900, 2200, 2400, 2700, 4100):
        seen.add(_gemm_plan([rows], N)[0])
        a, w = _ints(g, rows, K), _ints(g, 1, N, K)
        out = m.nvfp4_bf16_gemm_grouped(a, w, _off([rows]).cuda(), out_dtype=torch.float32)
        assert torch.equal(out.double(), a.double() @ w[0].double().t()), rows
    assert {x for x in seen if x > 128} >= {160, 192, 224, 256}, seen


@pytest.mark.parametrize("add", [False, True], ids=["store", "add"])
@pytest.mark.parametrize("M,N", [(2312, 2312), (2304, 1288), (520, 5128)])
def test_wgrad_wide_tiles(M, N, add):
    m = nv()
    counts = [700, 1, 0, 333, 130, 1024, 47, 515]
    E, off = len(counts), _off(counts)
    lens = [M for c in counts if c or not add]
    tall, most, tiles = _plan(lens, N, -(-N // 256) * -(-M // 128) * E)
    assert tiles > 2 * PAIRS and tall > 128 and (M < 2304 or most > BAND)
    g = torch.Generator(device="cuda").manual_seed(M + N)
    dy, x = _ints(g, sum(counts) + 5, M), _ints(g, sum(counts) + 5, N)
    dy[sum(counts):] = float("nan")
    x[sum(counts):] = float("nan")
    start = torch.randint(-9, 10, (E, M, N), generator=g, device="cuda").float()
    out = start.clone()
    ws = m.Workspace()
    m.nvfp4_bf16_wgrad_grouped(dy, x, off.cuda(), out=out, accumulate=add, ws=ws)
    assert m.nvfp4_poll(ws) == 0
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        ref = dy[lo:hi].double().t() @ x[lo:hi].double()
        assert torch.equal(out[e].double(), ref + start[e].double() if add else ref), e
