"""The C entry points of the product with bias, activation and residual, and of its gradient, refuse what their shape
rules exclude, before any device work, and so does the binding (no GPU needed)."""
import ctypes
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


def test_gemm_act_refuses(L):
    ok = dict(a=P, lda=64, b=P, ldb=64, M=32, N=128, K=64, bias=P, act=3, residual=P, ldr=128, res=0, pre=P, ldpre=128, d=P, ldd=128,
              out=0, ws=P, stream=None)
    for want, change in [(4, dict(out=2)), (4, dict(act=5)), (4, dict(act=-1)), (4, dict(res=2)), (3, dict(M=-1)), (3, dict(N=0)),
                         (3, dict(K=0)), (3, dict(K=60)), (3, dict(lda=56)), (3, dict(ldb=56)), (3, dict(ldd=127)), (3, dict(ldr=127)),
                         (3, dict(ldpre=127)), (10, dict(M=BIG)), (10, dict(N=BIG, ldd=BIG, ldr=BIG, ldpre=BIG)),
                         (10, dict(K=BIG, lda=BIG, ldb=BIG)), (10, dict(lda=BIG)), (10, dict(ldr=BIG)), (10, dict(ldpre=BIG)),
                         (10, dict(M=1 << 30, N=1 << 12, ldd=1 << 12, ldr=1 << 12, ldpre=1 << 12)), (5, dict(ws=None)), (1, dict(a=None)),
                         (1, dict(b=None)), (1, dict(d=None)), (2, dict(a=ctypes.c_void_p(72))), (2, dict(b=ctypes.c_void_p(72))),
                         (2, dict(d=ctypes.c_void_p(72))), (2, dict(residual=ctypes.c_void_p(72))), (2, dict(pre=ctypes.c_void_p(72))),
                         (2, dict(bias=ctypes.c_void_p(66))), (2, dict(lda=68)), (2, dict(ldb=68))]:
        assert L.nvfp4_bf16_gemm_act(*{**ok, **change}.values()) == want, change


def test_act_bwd_refuses(L):
    ok = dict(dy=P, lddy=64, pre=P, ldpre=64, rows=8, n=64, act=3, dh=P, lddh=64, dbias=P, accumulate=0, scratch=P, stream=None)
    for want, change in [(4, dict(act=5)), (4, dict(accumulate=2)), (3, dict(rows=-1)), (3, dict(n=0)), (3, dict(n=60)), (3, dict(lddy=56)),
                         (3, dict(ldpre=56)), (3, dict(lddh=56)), (10, dict(rows=BIG)), (10, dict(lddy=BIG)), (1, dict(dh=None, dbias=None)),
                         (1, dict(scratch=None)), (1, dict(dy=None)), (1, dict(pre=None)), (2, dict(dy=ctypes.c_void_p(72))),
                         (2, dict(pre=ctypes.c_void_p(72))), (2, dict(dh=ctypes.c_void_p(72))), (2, dict(dbias=ctypes.c_void_p(66))),
                         (2, dict(scratch=ctypes.c_void_p(72))), (2, dict(lddy=68)), (2, dict(ldpre=68)), (2, dict(lddh=68))]:
        assert L.nvfp4_act_bwd(*{**ok, **change}.values()) == want, change
    assert L.nvfp4_act_bwd_scratch_bytes(64) >= 256 and L.nvfp4_act_bwd_scratch_bytes(0) == L.nvfp4_act_bwd_scratch_bytes(BIG) == 0


def test_binding_refuses(L):
    import nvfp4_bit_quantized_02_b200 as nv
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    a, b = bf(6, 16), bf(24, 16)
    for call in (lambda: nv.nvfp4_bf16_gemm_act(a, bf(24, 8)), lambda: nv.nvfp4_bf16_gemm_act(bf(16, 6).t(), b),
                 lambda: nv.nvfp4_bf16_gemm_act(a, b, torch.zeros(23)), lambda: nv.nvfp4_bf16_gemm_act(a, b, bf(24)),
                 lambda: nv.nvfp4_bf16_gemm_act(a, b, torch.zeros(48)[::2]), lambda: nv.nvfp4_bf16_gemm_act(a, b, out=bf(6, 23)),
                 lambda: nv.nvfp4_bf16_gemm_act(a, b, out=bf(24, 6).t()), lambda: nv.nvfp4_bf16_gemm_act(a, b, residual=bf(6, 23)),
                 lambda: nv.nvfp4_bf16_gemm_act(a, b, residual=torch.zeros(6, 24, dtype=torch.float16)),
                 lambda: nv.nvfp4_bf16_gemm_act(a, b, pre=torch.zeros(6, 24)), lambda: nv.nvfp4_bf16_gemm_act(a, b, pre=bf(5, 24)),
                 lambda: nv.nvfp4_act_bwd(a, None, nv.ACT_GELU), lambda: nv.nvfp4_act_bwd(a, bf(6, 24), nv.ACT_GELU),
                 lambda: nv.nvfp4_act_bwd(a, a, nv.ACT_GELU, out=bf(5, 16)), lambda: nv.nvfp4_act_bwd(a, a, nv.ACT_GELU, dbias=torch.zeros(15)),
                 lambda: nv.nvfp4_act_bwd(a, a, nv.ACT_GELU, dbias=torch.zeros(16), scratch=torch.zeros(16, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: nv.nvfp4_bf16_gemm_act(a.float(), b), lambda: nv.nvfp4_bf16_gemm_act(a, b, out=torch.zeros(6, 24, dtype=torch.float16)),
                 lambda: nv.nvfp4_act_bwd(a.float(), a, nv.ACT_GELU)):
        with pytest.raises(TypeError):
            call()


def test_gemm_act_kn_refuses(L):
    ok = dict(a=P, lda=64, b=P, ldb=128, M=32, N=128, K=64, bias=P, act=3, residual=P, ldr=128, res=0, pre=P, ldpre=128, d=P, ldd=128,
              out=0, ws=P, stream=None)
    for want, change in [(4, dict(out=2)), (4, dict(act=5)), (3, dict(M=-1)), (3, dict(N=0)), (3, dict(K=60)), (3, dict(lda=56)),
                         (3, dict(ldb=120)), (3, dict(ldd=127)), (10, dict(ldb=BIG)), (5, dict(ws=None)), (1, dict(b=None)),
                         (2, dict(b=ctypes.c_void_p(72))), (2, dict(ldb=132))]:
        assert L.nvfp4_bf16_gemm_act_kn(*{**ok, **change}.values()) == want, change
    import nvfp4_bit_quantized_02_b200 as nv
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    for call in (lambda: nv.nvfp4_bf16_gemm_act(bf(6, 16), bf(24, 16), b_kn=True), lambda: nv.nvfp4_bf16_gemm_act(bf(6, 16), bf(24, 16).t(), b_kn=True)):
        with pytest.raises(ValueError):
            call()


def test_wgrad_refuses(L):
    ok = dict(dy=P, lddy=64, x=P, ldx=128, rows=32, n=64, d=128, out=P, ldo=128, accumulate=0, ws=P, stream=None)
    for want, change in [(4, dict(accumulate=2)), (3, dict(rows=-1)), (3, dict(n=0)), (3, dict(d=0)), (3, dict(lddy=56)), (3, dict(ldx=120)),
                         (3, dict(ldo=127)), (10, dict(rows=BIG)), (10, dict(n=BIG, lddy=BIG)), (10, dict(ldo=BIG)), (10, dict(ldx=BIG)),
                         (5, dict(ws=None)), (1, dict(dy=None)), (1, dict(x=None)), (1, dict(out=None)), (2, dict(dy=ctypes.c_void_p(72))),
                         (2, dict(x=ctypes.c_void_p(72))), (2, dict(out=ctypes.c_void_p(72))), (2, dict(lddy=68)), (2, dict(ldx=132))]:
        assert L.nvfp4_bf16_wgrad(*{**ok, **change}.values()) == want, change
    import nvfp4_bit_quantized_02_b200 as nv
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    for call in (lambda: nv.nvfp4_bf16_wgrad(bf(6, 16), bf(5, 16)), lambda: nv.nvfp4_bf16_wgrad(bf(6, 16), bf(6, 24), accumulate=True),
                 lambda: nv.nvfp4_bf16_wgrad(bf(6, 16), bf(6, 24), out=torch.zeros(24, 16)), lambda: nv.nvfp4_bf16_wgrad(bf(16, 6).t(), bf(6, 24)),
                 lambda: nv.nvfp4_bf16_wgrad(bf(6, 16), bf(6, 24), out=bf(16, 24))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        nv.nvfp4_bf16_wgrad(torch.zeros(6, 16), bf(6, 24))
