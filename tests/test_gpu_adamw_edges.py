"""The AdamW step where its 8-bit moments, its amax and its checks of arguments have edges."""
import math

import numpy as np
import pytest
import torch

from gpu_helpers import nv

pytestmark = pytest.mark.gpu

f32 = np.float32


def test_a_root_held_as_zero_beside_a_moment_that_is_not():
    """One step from given codes, bit for bit: where sqrt(v) comes out as zero, the smallest code of the
    block's scale divides in its place; everywhere else the formula is the header's."""
    m = nv()
    n = 600                              # two whole blocks and a part of one
    r = np.random.default_rng(1)
    p = (0.02 * r.standard_normal(n)).astype(f32)
    g = np.where(r.random(n) < 0.5, 0, 1e-6 * r.standard_normal(n)).astype(f32)
    mc = r.integers(0, 0x60, n).astype(np.uint8) | (r.integers(0, 2, n) << 7).astype(np.uint8)
    vc = np.where(r.random(n) < 0.5, 0, r.integers(0, 0x60, n)).astype(np.uint8)
    ms, vs = (np.array(x, f32) for x in ([3e-6, 1e-4, 2e-3], [2e-6, 0.0, 1e-3]))
    vc[256:512] = 0                      # a block whose scale is zero: there only eps is left to divide by
    values = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    M, R = values[mc] * ms.repeat(256)[:n], values[vc] * vs.repeat(256)[:n]
    h = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
    step = 40
    codes = lambda c: torch.from_numpy(c).cuda().view(torch.float8_e4m3fn)
    ctx = m.AdamWContext([torch.from_numpy(p).cuda()], [torch.from_numpy(g).cuda()], m=[codes(mc)], v=[codes(vc)], state=m.STATE_FP8,
                         m_scale=[torch.from_numpy(ms).cuda()], v_scale=[torch.from_numpy(vs).cuda()])
    m.nvfp4_adamw_step(ctx, step=step, sr_seed=3, **h)
    M = M * f32(0.9) + g * f32(1 - 0.9)
    R = np.sqrt(R * R * f32(0.95) + (g * f32(1 - 0.95)) * g)
    lost = R == 0
    assert 100 < lost.sum() < n and (lost & (M != 0)).sum() > 100
    R = np.where(lost, vs.repeat(256)[:n] * f32(2.0 ** -9), R)
    fix, size = f32(1 / math.sqrt(1 - 0.95 ** step)), f32(1e-3 / (1 - 0.9 ** step))
    want = p * f32(1 - 1e-3 * 0.1) - (M / (R * fix + f32(1e-8))) * size
    assert np.array_equal(ctx.params[0].cpu().numpy(), want)
    # the codes are those of the root itself: zero stays zero
    assert not ctx.moment(0, "v").cpu().numpy()[lost].any()


@pytest.mark.parametrize("scale", [1.0, 1e-2])
def test_small_elements_of_a_wide_block_take_bounded_steps(scale):
    """Gradients of +-G = 1e-5 of the block's largest, zero in half of the steps.  With the block's largest
    gradient A in every step, a code of m is at most A / 229376 = 0.436 G and a code of the root times the
    correction at least 0.6 of that (0.716 from the correction of the step before, the rest its
    rounding).  Each step rounds |m| up by at most a code: |m| <= (1 - beta1^t) / 0.1 * (0.9 * 0.436 G + 0.1 G)
    = 4.9 G (1 - beta1^t).  The root is at least a code, or as a zero divides as one, or at least
    sqrt(0.05) G: the update is at most 4.9 / min(0.6 * 0.436, 0.95 * 0.6 * 0.436, 0.22) = 23 lr."""
    m = nv()
    n, lr = 4096, 1e-3
    gen = torch.Generator(device="cuda").manual_seed(int(1 / scale))
    small = torch.arange(n, device="cuda") % 4 != 0
    p, g = torch.zeros(n, device="cuda"), torch.empty(n, device="cuda")
    ctx = m.AdamWContext([p], [g], state=m.STATE_FP8)
    sign = lambda: torch.randint(0, 2, (n,), generator=gen, device="cuda").float() * 2 - 1
    worst = 0.0
    for step in range(1, 301):
        some = torch.randint(0, 2, (n,), generator=gen, device="cuda").float()
        g.copy_(scale * torch.where(small, 1e-5 * some, 1.0) * sign())
        before = p.clone()
        m.nvfp4_adamw_step(ctx, lr=lr, step=step, weight_decay=0.0, sr_seed=step)
        worst = max(worst, float((p - before)[small].abs().max()) / lr)
    assert worst <= 23, worst


@pytest.mark.parametrize("state", ["fp32", "fp8"])
def test_an_empty_weight_with_an_amax(state):
    # an empty tensor has no address, and the amax zero
    m = nv()
    p = [torch.randn(300, device="cuda"), torch.empty(0, device="cuda"), torch.randn(7, device="cuda")]
    g = [torch.randn_like(t) for t in p]
    w = [torch.zeros_like(t, dtype=torch.bfloat16) for t in p]
    ws = [m.Workspace() for _ in p]
    for x in ws:
        x.amax_words()[0] = 0x7F000000       # what an earlier call left
    ctx = m.AdamWContext(p, g, w, state=m.STATE_FP8 if state == "fp8" else m.STATE_FP32, amax_ws=ws)
    before = [t.clone() for t in p]
    m.nvfp4_adamw_step(ctx, lr=1e-2, step=1)
    assert int(ws[1].amax_words()[0]) == 0
    for i in (0, 2):
        assert (p[i] != before[i]).all() and torch.equal(w[i], p[i].bfloat16())
        assert int(ws[i].amax_words()[0]) == int(w[i].abs().max().float().view(torch.int32))


def test_gradients_that_overlap_what_a_step_writes_are_refused():
    m = nv()
    flat = torch.zeros(2048, device="cuda")
    p, g = flat[:512], torch.ones(512, device="cuda")
    w, v = flat[1024:1280].view(torch.bfloat16), flat[1536:2048]
    mk = lambda grad, **k: m.AdamWContext([p], [grad], [w], m=[torch.zeros(512, device="cuda")], v=[v], **k)
    bad = [flat[256:768], flat[511:1023], p, flat[1028:1284].view(torch.bfloat16), flat[800:1312], flat[1100:1612], v, flat[1400:1912]]
    for grad in bad:
        with pytest.raises(ValueError):
            mk(grad)
    ctx = mk(g)
    for grad in bad:
        with pytest.raises(ValueError):
            ctx.set_grads([grad])
    assert ctx.grads[0] is g
    ctx.set_grads([flat[512:1024]])      # between two of them
    m.nvfp4_adamw_step(ctx, lr=1e-3)
    assert not flat.any()                # the gradient is zero there
    q = [torch.zeros(512, device="cuda") for _ in range(2)]
    both = m.AdamWContext(q, [g, g])     # one gradient for two tensors
    m.nvfp4_adamw_step(both, lr=1e-3)
    assert torch.equal(q[0], q[1]) and q[0].all()
    one = torch.zeros(512, device="cuda")
    m.nvfp4_adamw_step(m.AdamWContext([one], [g], v=[torch.zeros(512, device="cuda")]), lr=1e-3)
    assert torch.equal(one, q[0])
    codes = torch.zeros(512, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):      # 8-bit moments and their scales
        m.AdamWContext([torch.zeros(128, device="cuda")], [codes[64:320].view(torch.bfloat16)], m=[codes[:128].view(torch.float8_e4m3fn)], state=m.STATE_FP8)


@pytest.mark.parametrize("mode", [0, 1], ids=["rne", "sr"])
def test_codes_of_blocks_held_as_zero_or_not_finite(mode):
    # a block below 2^-100: scale 0, codes 0x00 or, where m is negative, 0x80; one with a NaN: codes 0x00
    m = nv()
    g = torch.zeros(768)
    g[:256] = torch.where(torch.arange(256) % 3 == 0, -1e-31, 1e-31)
    g[256:512] = -1.0
    g[300] = float("nan")
    g[512:] = -1.0
    ctx = m.AdamWContext([torch.zeros(768, device="cuda")], [g.cuda()], state=m.STATE_FP8)
    m.nvfp4_adamw_step(ctx, lr=1e-3, mode=mode)
    mc, vc = (t[0].view(torch.uint8).cpu() for t in (ctx.m, ctx.v))
    assert torch.equal(mc[:256], torch.where(g[:256] < 0, 0x80, 0).to(torch.uint8)) and not vc[:256].any()
    assert not mc[256:512].any() and not vc[256:512].any()
    assert (mc[512:] == 0xFE).all() and (vc[512:] == 0x7E).all()
    for s in (ctx.m_scale[0].cpu(), ctx.v_scale[0].cpu()):
        assert s[0] == 0 and torch.isnan(s[1]) and s[2] > 0
