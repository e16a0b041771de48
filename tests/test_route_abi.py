"""The C entry points of routing and of the movement of token rows refuse what their shape rules
exclude, before any device work, and so does the binding (no GPU needed)."""
import ctypes
import math
import os

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    import nvfp4_bit_quantized_02_b200 as nv
    if not os.path.exists(nv.LIB_PATH):
        from nvfp4_bit_quantized_02_b200.csrc import build as b
        b.build()
    return nv.lib()


P = ctypes.c_void_p(64)
BIG = (1 << 30) + 8


def _args(change):
    import nvfp4_bit_quantized_02_b200 as nv
    a = nv.CRouteArgs(4, 0, 1, 1, 1, 1, 1.0, 0)
    for k in [k for k in change if hasattr(a, k)]:
        setattr(a, k, change.pop(k))
    return ctypes.byref(a)


ROUTE_ARGS = [(4, dict(score=2)), (4, dict(renormalize=2)), (4, dict(scale=math.nan)), (4, dict(scale=math.inf)), (4, dict(dtype=2)),
              (3, dict(tokens=-1)), (3, dict(experts=0)), (3, dict(k=0)), (3, dict(ld=60)), (3, dict(groups=0)), (3, dict(top_groups=0)),
              (3, dict(top_groups=2)), (3, dict(groups=3)), (3, dict(groups=32, top_groups=1)), (3, dict(k=32, groups=8, top_groups=3)),
              (3, dict(group_top=0)), (3, dict(group_top=3)), (10, dict(experts=1025, ld=1025)), (10, dict(k=33)), (10, dict(tokens=BIG)),
              (10, dict(tokens=(1 << 28) + 1)), (10, dict(groups=64, top_groups=64)), (10, dict(ld=BIG)), (2, dict(logits=ctypes.c_void_p(72)))]


def test_route_refuses(L):
    ok = dict(logits=P, dtype=1, ld=64, tokens=8, experts=64, args=None, bias=P, valid=P, chosen=P, weights=P, rows=P, sources=P,
              offsets=P, scratch=P, ws=P, stream=None)

    def call(**change):
        args = _args(change)
        return L.nvfp4_route(*{**ok, "args": args, **change}.values())

    for want, change in ROUTE_ARGS + [(5, dict(ws=None)), (1, dict(offsets=None)), (1, dict(scratch=None)), (1, dict(logits=None)),
                                      (1, dict(chosen=None)), (1, dict(weights=None)), (1, dict(rows=None)), (1, dict(sources=None)),
                                      (2, dict(bias=ctypes.c_void_p(66))), (2, dict(chosen=ctypes.c_void_p(66))),
                                      (2, dict(weights=ctypes.c_void_p(66))), (2, dict(rows=ctypes.c_void_p(66))),
                                      (2, dict(sources=ctypes.c_void_p(66))), (2, dict(offsets=ctypes.c_void_p(66))),
                                      (2, dict(scratch=ctypes.c_void_p(72)))]:
        assert call(**dict(change)) == want, change
    # a group of one expert has no two largest
    assert call(groups=32, top_groups=32, experts=32, ld=32, group_top=2) == 3
    assert L.nvfp4_route(*{**ok, "args": None}.values()) == 1


def test_route_bwd_refuses(L):
    ok = dict(dweights=P, logits=P, dtype=1, ld=64, tokens=8, experts=64, args=None, chosen=P, dlogits=P, ldd=64, stream=None)

    def call(**change):
        args = _args(change)
        return L.nvfp4_route_bwd(*{**ok, "args": args, **change}.values())

    for want, change in ROUTE_ARGS + [(3, dict(ldd=60)), (10, dict(ldd=BIG)), (1, dict(dweights=None)), (1, dict(logits=None)),
                                      (1, dict(chosen=None)), (1, dict(dlogits=None)), (2, dict(dlogits=ctypes.c_void_p(72))),
                                      (2, dict(dweights=ctypes.c_void_p(66))), (2, dict(chosen=ctypes.c_void_p(66)))]:
        assert call(**dict(change)) == want, change


def test_scratch_bytes(L):
    assert L.nvfp4_route_scratch_bytes(256) >= 4 * 256 and L.nvfp4_route_scratch_bytes(1024) == 4 * L.nvfp4_route_scratch_bytes(256)
    assert L.nvfp4_route_scratch_bytes(0) == L.nvfp4_route_scratch_bytes(1025) == L.nvfp4_route_scratch_bytes(-1) == 0


COMMON = [(3, dict(tokens=-1)), (3, dict(d=0)), (3, dict(d=60)), (3, dict(k=0)), (3, dict(total=-1)), (3, dict(total=31)),
          (10, dict(tokens=BIG)), (10, dict(d=(1 << 24) + 8)), (10, dict(k=33)), (10, dict(total=BIG)), (1, dict(rows=None)),
          (2, dict(rows=ctypes.c_void_p(66)))]


def test_dispatch_refuses(L):
    ok = dict(x=P, ldx=64, tokens=8, d=64, rows=P, k=4, xs=P, ldxs=64, total=32, stream=None)
    for want, change in COMMON + [(3, dict(ldx=56)), (3, dict(ldxs=56)), (10, dict(ldx=BIG)), (1, dict(x=None)), (1, dict(xs=None)),
                                  (2, dict(x=ctypes.c_void_p(72))), (2, dict(xs=ctypes.c_void_p(72))), (2, dict(ldx=68)), (2, dict(ldxs=68))]:
        assert L.nvfp4_dispatch(*{**ok, **change}.values()) == want, change


def test_combine_refuses(L):
    ok = dict(ys=P, ldys=64, ys_dtype=0, total=32, rows=P, weights=P, k=4, residual=P, ldr=64, y=P, ldy=64, y_dtype=0, tokens=8, d=64,
              stream=None)
    for want, change in COMMON + [(4, dict(ys_dtype=2)), (4, dict(y_dtype=-1)), (3, dict(ldys=56)), (3, dict(ldy=56)), (3, dict(ldr=56)),
                                  (10, dict(ldys=BIG)), (1, dict(ys=None)), (1, dict(y=None)), (2, dict(ys=ctypes.c_void_p(72))),
                                  (2, dict(y=ctypes.c_void_p(72))), (2, dict(residual=ctypes.c_void_p(72))), (2, dict(ldys=68)),
                                  (2, dict(ldr=68)), (2, dict(ldy=66, y_dtype=1, ldr=64)), (2, dict(weights=ctypes.c_void_p(66)))]:
        assert L.nvfp4_combine(*{**ok, **change}.values()) == want, change


def test_combine_bwd_refuses(L):
    ok = dict(dy=P, lddy=64, ys=P, ldys=64, ys_dtype=0, total=32, rows=P, weights=P, k=4, dys=P, lddys=64, dweights=P, tokens=8, d=64,
              stream=None)
    for want, change in COMMON + [(4, dict(ys_dtype=2)), (3, dict(lddy=56)), (3, dict(ldys=56)), (3, dict(lddys=56)), (1, dict(dy=None)),
                                  (1, dict(ys=None)), (1, dict(dys=None)), (1, dict(weights=None)), (1, dict(dweights=None)),
                                  (2, dict(dy=ctypes.c_void_p(72))), (2, dict(dys=ctypes.c_void_p(72))), (2, dict(lddy=68)),
                                  (2, dict(ldys=66, ys_dtype=1)), (2, dict(dweights=ctypes.c_void_p(66)))]:
        assert L.nvfp4_combine_bwd(*{**ok, **change}.values()) == want, change


def _routes(tokens=6, count=8, k=2, **change):
    import nvfp4_bit_quantized_02_b200 as nv
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    parts = dict(experts=i(tokens, k), weights=torch.zeros(tokens, k), rows=i(tokens, k), sources=i(tokens * k), offsets=i(count + 1))
    return nv.Routes(**{**parts, **change})


def test_binding_refuses(L):
    import nvfp4_bit_quantized_02_b200 as nv
    for change in (dict(experts=torch.zeros(12, dtype=torch.int32)), dict(weights=torch.zeros(6, 2, dtype=torch.float64)),
                   dict(rows=torch.zeros(2, 6, dtype=torch.int32)), dict(rows=torch.zeros(2, 6, dtype=torch.int32).t()),
                   dict(sources=torch.zeros(11, dtype=torch.int32)), dict(offsets=torch.zeros(9)),
                   dict(offsets=torch.zeros(3, 3, dtype=torch.int32))):
        with pytest.raises(ValueError):
            _routes(**change)
    r = _routes()
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        nv.nvfp4_route(torch.zeros(6, 8, dtype=torch.float64), 2)
    for call in (lambda: nv.nvfp4_route(torch.zeros(6, 8), 3, out=r), lambda: nv.nvfp4_route(torch.zeros(7, 8), 2, out=r),
                 lambda: nv.nvfp4_route(torch.zeros(6, 9), 2, out=r), lambda: nv.nvfp4_route(torch.zeros(8, 6).t(), 2, out=r),
                 lambda: nv.nvfp4_route_bwd(torch.zeros(6, 3), torch.zeros(6, 8), r),
                 lambda: nv.nvfp4_route_bwd(torch.zeros(6, 2), torch.zeros(6, 9), r),
                 lambda: nv.nvfp4_route_bwd(torch.zeros(6, 2), torch.zeros(6, 8), r, out=bf(6, 8)),
                 lambda: nv.nvfp4_dispatch(bf(5, 16), r), lambda: nv.nvfp4_dispatch(bf(16, 6).t(), r),
                 lambda: nv.nvfp4_dispatch(bf(6, 16), r, out=bf(11, 16)), lambda: nv.nvfp4_dispatch(bf(6, 16), r, out=bf(12, 24)),
                 lambda: nv.nvfp4_combine(bf(11, 16), r), lambda: nv.nvfp4_combine(bf(12, 16), r, out=bf(5, 16)),
                 lambda: nv.nvfp4_combine(bf(12, 16), r, residual=torch.zeros(6, 16), out=bf(6, 16)),
                 lambda: nv.nvfp4_combine(bf(12, 16), r, residual=bf(6, 24)),
                 lambda: nv.nvfp4_combine_bwd(bf(5, 16), bf(12, 16), r), lambda: nv.nvfp4_combine_bwd(bf(6, 16), bf(12, 24), r),
                 lambda: nv.nvfp4_combine_bwd(bf(6, 16), bf(12, 16), r, dys=torch.zeros(12, 16)),
                 lambda: nv.nvfp4_combine_bwd(bf(6, 16), bf(12, 16), r, dweights=torch.zeros(12))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        nv.nvfp4_dispatch(torch.zeros(6, 16), r)
    with pytest.raises(TypeError):
        nv.nvfp4_combine(torch.zeros(12, 16, dtype=torch.float16), r)
