"""Offsets out of order or range, over more experts than a warp reads at once: the rows that the
running maximum of the clamped offsets gives, nothing written elsewhere, and the flag.

Integer operands: results are equal to the reference's."""
import numpy as np
import pytest
import torch

from gpu_helpers import nv

pytestmark = pytest.mark.gpu

FAR = 2 ** 31 - 1


def _cases(E, rows, seed):
    """Offsets with a bad value at each place in turn where a warp's 32 of them end or begin."""
    r = np.random.default_rng(seed)
    good = np.sort(r.integers(0, rows + 1, E + 1))
    yield "good", good
    for at in (0, 1, 31, 32, 33, 63, 64, 65, 255, 256, 257, E - 1, E):
        for value in (-1, -FAR - 1, FAR, rows + 1, rows // 2, 0, rows):
            if at <= E:
                bad = good.copy()
                bad[at] = value
                yield f"{value} at {at}", bad
    yield "falling", good[::-1].copy()
    yield "random", r.integers(-5, rows + 6, E + 1)
    yield "far", r.integers(-FAR - 1, FAR, E + 1)


def _ints(g, *shape):
    return torch.randint(-3, 4, shape, generator=g).bfloat16().cuda()


@pytest.mark.parametrize("E", [33, 70, 300])
@pytest.mark.parametrize("op,rows", [("fprop", 40), ("fprop", 500), ("dgrad", 40), ("dgrad", 500), ("wgrad", 300)])
def test_offsets_out_of_order_over_many_experts(op, rows, E):
    m = nv()
    K, N = 64, 72
    g = torch.Generator().manual_seed(E + rows)
    x, dy, w = _ints(g, rows, K), _ints(g, rows, N), _ints(g, E, N, K)
    ws = m.Workspace()
    run = lambda off, out: {"fprop": lambda: m.nvfp4_bf16_gemm_grouped(x, w, off, out=out, ws=ws),
                            "dgrad": lambda: m.nvfp4_bf16_gemm_grouped(dy, w, off, b_kn=True, out=out, ws=ws),
                            "wgrad": lambda: m.nvfp4_bf16_wgrad_grouped(dy, x, off, out=out, ws=ws)}[op]()
    each = {"fprop": lambda: torch.einsum("tk,enk->ten", x.double(), w.double()),
            "dgrad": lambda: torch.einsum("tn,enk->tek", dy.double(), w.double()), "wgrad": lambda: None}[op]()
    for name, values in _cases(E, rows, E):
        owned = np.maximum.accumulate(np.clip(values, 0, rows))
        off = torch.tensor(values, dtype=torch.int32).cuda()
        if op == "wgrad":
            big = torch.full((E + 2, N, K), 7.0, device="cuda")
            run(off, big[1:-1])
            want = torch.zeros(E, N, K, dtype=torch.float64, device="cuda")
            for e in range(E):
                lo, hi = int(owned[e]), int(owned[e + 1])
                if hi > lo:
                    want[e] = dy[lo:hi].double().t() @ x[lo:hi].double()
        else:
            big = torch.full((rows + 80, N if op == "fprop" else K), 7.0, device="cuda")
            run(off, big[40:-40])
            t = np.arange(rows)
            expert = np.searchsorted(owned[1:], t, side="right")
            mine = torch.from_numpy((t >= owned[0]) & (t < owned[-1])).cuda()
            expert = torch.from_numpy(np.minimum(expert, E - 1)).cuda()
            want = torch.where(mine[:, None], each[torch.arange(rows, device="cuda"), expert], 7.0)
        status = m.nvfp4_poll(ws)
        assert status == (0 if np.array_equal(owned, values) else 4), name
        pad = 1 if op == "wgrad" else 40
        assert torch.equal(big[pad:-pad].double(), want), name
        assert (big[:pad] == 7).all() and (big[-pad:] == 7).all(), name
