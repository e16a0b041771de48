"""The C entry points of the products grouped by expert and of the AdamW step refuse what their
shape rules exclude, before any device work (no GPU needed)."""
import ctypes
import math
import os

import pytest


@pytest.fixture(scope="module")
def L():
    import nvfp4_bit_quantized_02_b200 as nv
    if not os.path.exists(nv.LIB_PATH):
        from nvfp4_bit_quantized_02_b200.csrc import build as b
        b.build()
    return nv.lib()


P = ctypes.c_void_p(64)
OK = dict(a=P, lda=64, rows=32, offsets=P, experts=4, b=P, ldb=64, stride_b=8192, b_kn=0, N=128, K=64, d=P, ldd=128,
          out=0, ws=P, stream=None)


def test_gemm_grouped_refuses(L):
    def call(**change):
        return L.nvfp4_bf16_gemm_grouped(*{**OK, **change}.values())

    big = (1 << 30) + 8
    for want, change in [(4, dict(out=2)), (4, dict(b_kn=2)), (3, dict(experts=0)), (3, dict(rows=-1)), (3, dict(N=0)),
                         (3, dict(N=124)), (3, dict(K=0)), (3, dict(K=60)), (3, dict(lda=56)), (3, dict(ldb=56)),
                         (3, dict(b_kn=1, ldb=64)), (3, dict(stride_b=-8)), (3, dict(ldd=120)), (10, dict(experts=1025)),
                         (10, dict(rows=big)), (10, dict(N=big, ldd=big)), (10, dict(K=big, lda=big, ldb=big)),
                         (10, dict(lda=big)), (10, dict(stride_b=1 << 39)), (5, dict(ws=None)), (1, dict(offsets=None)),
                         (1, dict(b=None)), (1, dict(a=None)), (1, dict(d=None)), (2, dict(a=ctypes.c_void_p(72))),
                         (2, dict(b=ctypes.c_void_p(68))), (2, dict(d=ctypes.c_void_p(66))),
                         (2, dict(offsets=ctypes.c_void_p(66))), (2, dict(lda=68)), (2, dict(ldb=68)),
                         (2, dict(stride_b=8196)), (2, dict(ldd=132)), (2, dict(out=1, ldd=130))]:
        assert call(**change) == want, change


def test_wgrad_grouped_refuses(L):
    ok = dict(a=P, lda=64, b=P, ldb=128, rows=32, offsets=P, experts=4, M=64, N=128, d=P, ldd=128, stride_d=8192,
              accumulate=0, ws=P, stream=None)
    big = (1 << 30) + 8
    for want, change in [(4, dict(accumulate=2)), (3, dict(experts=0)), (3, dict(rows=-1)), (3, dict(M=60)), (3, dict(N=0)),
                         (3, dict(lda=56)), (3, dict(ldb=120)), (3, dict(ldd=120)), (3, dict(stride_d=-4)),
                         (3, dict(stride_d=8188)), (3, dict(stride_d=0)), (10, dict(experts=1025)), (10, dict(rows=big)),
                         (10, dict(M=big, lda=big)), (10, dict(stride_d=1 << 38)), (5, dict(ws=None)),
                         (1, dict(offsets=None)), (1, dict(d=None)), (1, dict(a=None)), (1, dict(b=None)),
                         (2, dict(a=ctypes.c_void_p(72))), (2, dict(d=ctypes.c_void_p(72))), (2, dict(lda=68)),
                         (2, dict(ldb=132)), (2, dict(ldd=130, stride_d=16384)), (2, dict(stride_d=8194))]:
        assert L.nvfp4_bf16_wgrad_grouped(*{**ok, **change}.values()) == want, change


def _adamw_args(nv, **change):
    a = nv.CAdamWArgs(1e-3, 0.9, 0.95, 1e-8, 0.1, 1.0, 1, 0, 0, 1, None)
    for k, v in change.items():
        setattr(a, k, v)
    return a


def test_adamw_refuses(L):
    import nvfp4_bit_quantized_02_b200 as nv

    def call(t=None, ws=P, count=1, **args):
        e = nv.CAdamWTensor(64, 64, 64, 64, 64, 64, 64, None, 10, 1, 0)
        for k, v in (t or {}).items():
            setattr(e, k, v)
        return L.nvfp4_adamw(ctypes.byref(e), count, ctypes.byref(_adamw_args(nv, **args)), ws, None)

    nan, inf = math.nan, math.inf
    for want, args in [(4, dict(state=2)), (4, dict(mode=2)), (4, dict(beta1=1.0)), (4, dict(beta1=-0.1)), (4, dict(beta2=nan)),
                       (4, dict(eps=-1e-8)), (4, dict(eps=inf)), (4, dict(lr=nan)), (4, dict(weight_decay=inf)),
                       (4, dict(grad_scale=nan)), (4, dict(step=0)), (2, dict(dynamic=72)), (4, dict(dynamic=64, beta1=1.0))]:
        assert call(**args) == want, args
    for want, t in [(3, dict(n=-1)), (10, dict(n=(1 << 40) + 1)), (4, dict(g_dtype=2)), (4, dict(amax_ws=64, w=None)),
                    (1, dict(p=None)), (1, dict(g=None)), (1, dict(m=None)), (1, dict(v=None)), (2, dict(p=72)), (2, dict(g=72)),
                    (2, dict(w=72)), (2, dict(m=66)), (2, dict(v=66)), (2, dict(amax_ws=72))]:
        assert call(t) == want, t
    assert call(dict(m_scale=None), state=1) == 1 and call(dict(v_scale=66), state=1) == 2
    assert call(ws=None) == 5 and call(count=-1) == 3
    assert L.nvfp4_adamw(None, 1, ctypes.byref(_adamw_args(nv)), P, None) == 1
    assert L.nvfp4_adamw(None, 0, None, P, None) == 1


def test_adamw_dynamic_values(L):
    import numpy as np
    import nvfp4_bit_quantized_02_b200 as nv
    out = nv.CAdamWDynamic()
    for step in (1, 2, 10, 1000, 10 ** 9):
        a = _adamw_args(nv, step=step, sr_seed=0xFFFFFFFFFFFFFFFF, grad_scale=0.3)
        assert L.nvfp4_adamw_dynamic_values(ctypes.byref(a), ctypes.byref(out)) == 0
        assert out.keep == np.float32(1 - 1e-3 * 0.1) and out.grad_scale == np.float32(0.3)
        assert out.step_size == np.float32(1e-3 / (1 - 0.9 ** step))
        assert out.v_fix == np.float32(1 / math.sqrt(1 - 0.95 ** step)) and out.sr_seed == 0xFFFFFFFFFFFFFFFF
    assert L.nvfp4_adamw_dynamic_values(None, ctypes.byref(out)) == 1


def test_offsets_rule():
    # the rule by which the kernels read offsets, restated: whatever they hold, expert e's rows
    # [run[e], run[e + 1]) lie within [0, rows], ascend and never overlap
    import numpy as np
    rng = np.random.default_rng(0)
    for _ in range(200):
        rows, E = int(rng.integers(0, 50)), int(rng.integers(1, 9))
        off = rng.integers(-(2 ** 31), 2 ** 31, E + 1) if rng.random() < 0.3 else rng.integers(-5, rows + 6, E + 1)
        run = np.maximum.accumulate(np.clip(off, 0, rows))
        assert run[0] >= 0 and run[-1] <= rows and (np.diff(run) >= 0).all()
        good = off[0] >= 0 and off[-1] <= rows and (np.diff(off) >= 0).all()
        assert not good or np.array_equal(run, off)


def test_adamw_refuses_a_misplaced_amax_of_an_empty_tensor(L):
    import nvfp4_bit_quantized_02_b200 as nv
    e = nv.CAdamWTensor(None, None, None, None, None, None, None, 72, 0, 1, 0)
    assert L.nvfp4_adamw(ctypes.byref(e), 1, ctypes.byref(_adamw_args(nv)), P, None) == 2
    e.n, e.amax_ws = 10, 64
    e.p = e.g = e.m = e.v = 64
    assert L.nvfp4_adamw(ctypes.byref(e), 1, ctypes.byref(_adamw_args(nv)), P, None) == 4     # an amax without a weight


def test_a_weight_whose_amax_is_ready_needs_its_workspace(L):
    # the default workspace holds what some other call left there
    import torch
    import nvfp4_bit_quantized_02_b200 as nv
    with pytest.raises(ValueError):
        nv.nvfp4_quantize_weight(torch.zeros(16, 16, dtype=torch.bfloat16), amax_ready=True)
