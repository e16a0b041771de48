"""The AdamW step (nvfp4_adamw_step) against a numpy restatement of its fp32 operations (bit for bit:
numpy's float32 +, *, / and sqrt are single IEEE operations) and against the update's formula in
fp64."""
import math
import types

import numpy as np
import pytest
import torch

from gpu_helpers import nv

pytestmark = pytest.mark.gpu

f32 = np.float32
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, grad_scale=0.75)


# ---------------------------------------------------------------------------------------
# numpy restatement
# ---------------------------------------------------------------------------------------
def philox_fields(n, seed, stream, tensor):
    """16-bit fields of elements 0..n-1: Philox4x32-10 (Salmon et al., SC'11) per eight elements."""
    g = np.arange(-(-n // 8), dtype=np.uint64)
    M = np.uint64(0xFFFFFFFF)
    c = [g & M, g >> np.uint64(32), np.full_like(g, stream), np.full_like(g, tensor)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), p1 & M, (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), p0 & M]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    words = np.stack(c, 1).reshape(-1)
    return np.stack([words & np.uint64(0xFFFF), words >> np.uint64(16)], 1).reshape(-1)[:n].astype(np.int64)


E4M3 = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()


def encode(x, mode, r16):
    """codes, scales of an fp32 vector in blocks of 256."""
    n = x.size
    nb = -(-n // 256)
    codes, scales = np.zeros(n, np.uint8), np.zeros(nb, f32)
    for b in range(nb):
        s = slice(256 * b, min(n, 256 * b + 256))
        v = x[s]
        if not np.isfinite(v).all():
            scales[b] = np.nan
            continue
        top = np.abs(v).max()
        if top >= f32(2.0 ** -100):
            scales[b] = top * f32(1 / 448)
            u = np.abs(v) * (f32(448) * (f32(1) / top))
        else:
            u = np.zeros_like(v)
        low = u < f32(2.0 ** -6)
        bits = np.where(low, u + f32(2.0 ** -6), u).astype(f32).view(np.uint32).astype(np.int64)
        cut = 0xFFFFF - (r16[s] << 4) if mode == 1 else 0x7FFFF + ((bits >> 20) & 1)
        c = np.minimum(((bits + cut) >> 20) - np.where(low, 968, 960), 0x7E)
        codes[s] = c | np.where(np.signbit(v), 128, 0)
    return codes, scales


def numpy_step(p, g, m, v, root, h, step, mode=1, seed=0, tensor=0):
    """One step; m and v as fp32 values (v itself, or with root its square root); returns what the kernel writes."""
    with np.errstate(all="ignore"):
        keep = f32(1 - h["lr"] * h["weight_decay"])
        size = f32(h["lr"] / (1 - h["beta1"] ** step))
        fix = f32(1 / math.sqrt(1 - h["beta2"] ** step))
        b1, c1, b2, c2 = f32(h["beta1"]), f32(1 - h["beta1"]), f32(h["beta2"]), f32(1 - h["beta2"])
        g = g * f32(h["grad_scale"])
        if root:
            v = v * v
        m = m * b1 + g * c1
        v = v * b2 + (g * c2) * g
        r = np.sqrt(v)
        p = p * keep - (m / (r * fix + f32(h["eps"]))) * size
        w = torch.from_numpy(p).bfloat16()
        if not root:
            return p, w, m, v
        return (p, w) + encode(m, mode, philox_fields(m.size, seed, 4, tensor)) + encode(r, mode, philox_fields(m.size, seed, 5, tensor))


def inputs(n, seed, bf16=False):
    r = np.random.default_rng(seed)
    p = (0.02 * r.standard_normal(n)).astype(f32)
    g = torch.from_numpy((1e-3 * r.standard_normal(n) * 10 ** r.uniform(-3, 1, n)).astype(f32))
    return p, (g.bfloat16() if bf16 else g)


def same(a, b):
    return np.array_equal(np.ascontiguousarray(a), np.ascontiguousarray(b), equal_nan=a.dtype.kind == "f")


def guarded(t, device="cuda"):
    """t on the device with a margin behind it that must stay as it is"""
    n = t.numel()
    big = torch.zeros(n + 64, dtype=t.dtype, device=device)
    big.view(torch.uint8).fill_(0x5A)
    big[:n] = t.to(device)
    return big[:n], big


def margins_kept(bigs, ns):
    for b, n in zip(bigs, ns):
        assert (b[n:].view(torch.uint8) == 0x5A).all(), "written past the end of a tensor"


SIZES = [1, 3, 4, 5, 127, 255, 256, 257, 1000, 2047, 2048, 2049, 4096, 6145, 20001]


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32grad", "bf16grad"])
@pytest.mark.parametrize("state", ["fp32", "fp8-sr", "fp8-rne"])
def test_steps_bit_for_bit(state, bf16):
    m = nv()
    fp8, mode = state != "fp32", 0 if state == "fp8-rne" else 1
    host, dev, bigs, ns = [], [], [], []
    for i, n in enumerate(SIZES):
        p, g = inputs(n, i, bf16)
        host.append([p, g])
        parts = [torch.from_numpy(p), g, torch.zeros(n, dtype=torch.bfloat16),
                 torch.zeros(n, dtype=torch.float8_e4m3fn if fp8 else torch.float32)]
        parts.append(parts[3])
        row = []
        for t in parts:
            d, b = guarded(t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t)
            row.append(d.view(torch.float8_e4m3fn) if t.dtype == torch.float8_e4m3fn else d)
            bigs.append(b)
            ns.append(n)
        dev.append(row)
    cols = list(zip(*dev))
    amax = [m.Workspace() if i % 2 else None for i in range(len(SIZES))]
    ws = m.Workspace()
    ctx = m.AdamWContext(cols[0], cols[1], cols[2], m=cols[3], v=cols[4], state=m.STATE_FP8 if fp8 else m.STATE_FP32,
                         amax_ws=amax, ws=ws)
    ref = [[p, np.zeros(p.size, f32), np.zeros(p.size, f32)] for p, _ in host]
    for step in range(1, 5):
        seed = 0x123456789ABCDEF0 + step
        if step == 3:
            for i in range(len(SIZES)):
                host[i][1] = inputs(SIZES[i], 100 + i, bf16)[1]
                dev[i][1].copy_(host[i][1])
        m.nvfp4_adamw_step(ctx, step=step, mode=mode, sr_seed=seed, **HYPER)
        assert m.nvfp4_poll(ws) == 0
        for i, n in enumerate(SIZES):
            out = numpy_step(ref[i][0], host[i][1].float().numpy(), ref[i][1], ref[i][2], fp8, HYPER, step, mode, seed, i)
            what = f"{state} size {n} step {step}"
            assert same(dev[i][0].cpu().numpy(), out[0]), what + ": p"
            assert torch.equal(dev[i][2].cpu().view(torch.int16), out[1].view(torch.int16)), what + ": w"
            if fp8:
                assert same(dev[i][3].view(torch.uint8).cpu().numpy(), out[2]), what + ": m codes"
                assert same(ctx.m_scale[i].cpu().numpy(), out[3]), what + ": m scales"
                assert same(dev[i][4].view(torch.uint8).cpu().numpy(), out[4]), what + ": v codes"
                assert same(ctx.v_scale[i].cpu().numpy(), out[5]), what + ": v scales"
                ref[i] = [out[0]] + [E4M3[c] * s.repeat(256)[:n] for c, s in ((out[2], out[3]), (out[4], out[5]))]
                assert same(ctx.moment(i, "m").cpu().numpy(), ref[i][1])
                assert same(ctx.moment(i, "v").cpu().numpy(), ref[i][2] * ref[i][2])
            else:
                assert same(dev[i][3].cpu().numpy(), out[2]) and same(dev[i][4].cpu().numpy(), out[3]), what + ": moments"
                ref[i] = [out[0], out[2], out[3]]
            if amax[i] is not None:
                word = int(amax[i].amax_words()[0])
                assert word == int(out[1].abs().max().float().view(torch.int32)), what + ": amax"
    margins_kept(bigs, ns)


@pytest.mark.parametrize("state", ["fp32", "fp8"])
def test_more_tensors_than_a_launch_holds(state):
    # 800 tensors, empty ones among them, against one context per tensor (whose index in the call is 0:
    # RNE codes, which do not depend on it)
    m = nv()
    st = m.STATE_FP8 if state == "fp8" else m.STATE_FP32
    ns = [(37 * i) % 701 for i in range(800)]
    mk = lambda: [torch.from_numpy(inputs(n, i)[0]).cuda() for i, n in enumerate(ns)]
    gs = [inputs(n, i)[1].cuda() for i, n in enumerate(ns)]
    a, b = mk(), mk()
    wa, wb = ([torch.zeros(n, dtype=torch.bfloat16, device="cuda") for n in ns] for _ in range(2))
    ca = m.AdamWContext(a, gs, wa, state=st)
    cb = [m.AdamWContext([b[i]], [gs[i]], [wb[i]], state=st) for i in range(0, 800, 9)]
    for step in (1, 2):
        m.nvfp4_adamw_step(ca, step=step, mode=m.RNE, **HYPER)
        for c in cb:
            m.nvfp4_adamw_step(c, step=step, mode=m.RNE, **HYPER)
    for c, i in zip(cb, range(0, 800, 9)):
        assert torch.equal(a[i], b[i]) and torch.equal(wa[i], wb[i]) and torch.equal(ca.moment(i, "v"), c.moment(0, "v"))
    assert all(bool((x != torch.from_numpy(inputs(n, i)[0]).cuda()).any()) for i, (x, n) in enumerate(zip(a, ns)) if n > 8)


def test_against_the_formula_in_64_bits():
    # p: its own rounding (2^-24 |p|, twice: the product and the difference) and the update's, whose
    # relative error is below 16 half steps (the products, sums, root and quotient that enter it)
    m = nv()
    n = 100003
    p, g = inputs(n, 5)
    dev = torch.from_numpy(p).cuda()
    w = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    ctx = m.AdamWContext([dev], [g.cuda()], [w])
    P, M, V = p.astype(np.float64), np.zeros(n), np.zeros(n)
    h, G = HYPER, g.double().numpy() * HYPER["grad_scale"]
    slack = np.zeros(n)
    for step in range(1, 21):
        m.nvfp4_adamw_step(ctx, step=step, **h)
        M = h["beta1"] * M + (1 - h["beta1"]) * G
        V = h["beta2"] * V + (1 - h["beta2"]) * G * G
        up = h["lr"] * (M / (1 - h["beta1"] ** step)) / (np.sqrt(V / (1 - h["beta2"] ** step)) + h["eps"])
        P = P * (1 - h["lr"] * h["weight_decay"]) - up
        # moments are running sums of terms of one sign: their relative error grows by at most 3 half steps a step
        slack += 2.0 ** -24 * (3 * np.abs(P) + (16 + 6 * step) * np.abs(up))
    assert (np.abs(dev.cpu().numpy() - P) <= slack).all()
    assert (np.abs(ctx.moment(0, "m").cpu().numpy() - M) <= 2.0 ** -24 * 4 * 20 * np.abs(M) + 1e-37).all()
    assert (np.abs(ctx.moment(0, "v").cpu().numpy() - V) <= 2.0 ** -24 * 5 * 20 * V + 1e-37).all()


def test_a_tensor_past_2_to_the_31_elements():
    # its last elements against a small tensor of the same values (RNE codes do not depend on the index)
    m = nv()
    n, k = 2 ** 31 + 300, 300 + 512
    p, g = inputs(k, 11, True)
    big = [torch.zeros(n, dtype=t, device="cuda") for t in (torch.float32, torch.bfloat16, torch.bfloat16)]
    big[0][-k:] = torch.from_numpy(p).cuda()
    big[1][-k:] = g.cuda()
    a = m.AdamWContext([big[0]], [big[1]], [big[2]], state=m.STATE_FP8)
    b = m.AdamWContext([torch.from_numpy(p).cuda()], [g.cuda()], [torch.zeros(k, dtype=torch.bfloat16, device="cuda")], state=m.STATE_FP8)
    for c in (a, b):
        for step in (1, 2):
            m.nvfp4_adamw_step(c, step=step, mode=m.RNE, **HYPER)
    assert torch.equal(big[0][-k:], b.params[0]) and torch.equal(big[2][-k:], b.weights[0])
    assert not big[0][:n - k].any() and not big[2][:n - k].any()
    for x, y in ((a.m, b.m), (a.v, b.v)):
        assert torch.equal(x[0].view(torch.uint8)[-k:], y[0].view(torch.uint8))
    assert torch.equal(a.m_scale[0][-4:], b.m_scale[0]) and torch.equal(a.v_scale[0][-4:], b.v_scale[0])


def test_gradients_of_zero_infinity_and_nan():
    m = nv()
    n = 1024
    for st in (m.STATE_FP32, m.STATE_FP8):
        p, g = inputs(n, 1)
        g[:256] = 0            # a block that stays at zero moments: only the decay moves it
        g[256:512] = 1e-38     # moments below 2^-100 (and squares below the fp32 range)
        g[600] = float("nan")  # a block of 8-bit moments becomes NaN as a whole, an fp32 moment alone
        g[800] = float("inf")
        w = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
        ws, aw = m.Workspace(), m.Workspace()
        ctx = m.AdamWContext([torch.from_numpy(p).cuda()], [g.cuda()], [w], state=st, amax_ws=[aw], ws=ws)
        m.nvfp4_adamw_step(ctx, step=1, **HYPER)
        assert m.nvfp4_poll(ws) == 7 and m.nvfp4_poll(ws) == 0     # the amax of w says so
        z = np.zeros(n, f32)
        out = numpy_step(p, g.numpy(), z, z, st == m.STATE_FP8, HYPER, 1, 1, 0)
        got = ctx.params[0].cpu().numpy()
        assert np.array_equal(got, out[0], equal_nan=True)
        assert np.isfinite(got[np.r_[:600, 601:800, 801:1024]]).all() and not np.isfinite(got[600])
        mm = ctx.moment(0, "m").cpu()
        assert not mm[:256].any()
        if st == m.STATE_FP8:
            assert not mm[256:512].any() and torch.isnan(mm[512:768]).all() and torch.isnan(mm[768:]).all()
            assert np.array_equal(ctx.m_scale[0].cpu().numpy(), out[3], equal_nan=True)
        else:
            assert torch.isnan(mm[600]) and torch.isinf(mm[800]) and torch.isfinite(mm).sum() == n - 2


def test_stochastic_codes_are_unbiased():
    # the mean of the decoded moments over 400 seeds lies within 5 standard deviations of the fp32
    # moment (the spread of one draw is at most half a step: f (1 - f) <= 1/4), block by block of 4096
    # elements at once; RNE's own error does not shrink
    m = nv()
    n = 4096
    p, g = inputs(n, 3)
    z = np.zeros(n, f32)
    exact_m, exact_v = numpy_step(p, g.numpy(), z, z, False, HYPER, 1)[2:]
    total = torch.zeros(2, n, dtype=torch.float64, device="cuda")
    draws = 400
    for s in range(draws):
        ctx = m.AdamWContext([torch.from_numpy(p).cuda()], [g.cuda()], state=m.STATE_FP8)
        m.nvfp4_adamw_step(ctx, step=1, sr_seed=s * 7919 + 1, **HYPER)
        total[0] += ctx.moment(0, "m").double()
        total[1] += ctx.moment(0, "v").double().sqrt()
    mean = (total / draws).cpu().numpy()
    for got, want in ((mean[0], exact_m.astype(np.float64)), (mean[1], np.sqrt(exact_v.astype(np.float64)))):
        top = np.abs(want).reshape(-1, 256).max(1).repeat(256) / 448
        u = np.abs(want) / top
        step = np.ldexp(1.0, np.maximum(np.frexp(u)[1] - 1, -6) - 3) * top
        z = np.abs(got - want) / (0.5 * step / math.sqrt(draws))
        assert z.max() < 5.5 and abs(float(np.mean((got - want) / step))) < 5 * 0.5 / math.sqrt(draws * n)


def test_amax_feeds_the_weight_quantizer():
    m = nv()
    rows, cols = 272, 320
    p = torch.randn(rows, cols, device="cuda") * 0.02
    w = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    aw = m.Workspace()
    aw.buf.fill_(0)
    aw.amax_words()[0] = 0x7F000000         # what an earlier call left is reset
    ctx = m.AdamWContext([p], [torch.randn_like(p)], [w], state=m.STATE_FP8, amax_ws=[aw])
    m.nvfp4_adamw_step(ctx, step=1, **HYPER)
    q, qt = m.nvfp4_quantize_weight(w, ws=aw, amax_ready=True)
    r, rt = m.nvfp4_quantize_weight(w)
    for a, b in ((q, r), (qt, rt)):
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales) and torch.equal(a.tensor_scale, b.tensor_scale)
    assert torch.equal(q.tile_scales, r.tile_scales)


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_amax_of_a_nonfinite_weight(value):
    """The flag, and the same quantized weight as with the quantizer's own amax pass."""
    m = nv()
    torch.manual_seed(6)
    p = torch.randn(128, 128, device="cuda")
    p[77, 5] = value
    w = torch.empty(128, 128, dtype=torch.bfloat16, device="cuda")
    aws, ws = m.Workspace(), m.Workspace()
    ctx = m.AdamWContext([p], [torch.zeros_like(p)], weights=[w], amax_ws=[aws], ws=ws)
    m.nvfp4_adamw_step(ctx, lr=1e-2)
    assert m.STATUS[m.nvfp4_poll(ws)] == "ERR_NONFINITE"
    got = m.nvfp4_quantize_weight(w, ws=aws, amax_ready=True)
    own = m.nvfp4_quantize_weight(w, ws=ws)
    assert m.STATUS[m.nvfp4_poll(ws)] == "ERR_NONFINITE"
    for a, b in zip(got, own):
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
        assert torch.equal(a.tensor_scale.view(torch.int32), b.tensor_scale.view(torch.int32)) or (a.tensor_scale.isnan() & b.tensor_scale.isnan()).all()


@pytest.mark.parametrize("state", ["fp32", "fp8"])
def test_captured_step_reads_its_values_when_replayed(state):
    m = nv()
    st = m.STATE_FP8 if state == "fp8" else m.STATE_FP32
    ns = [5, 3000, 257]
    mk = lambda: m.AdamWContext([torch.from_numpy(inputs(n, i)[0]).cuda() for i, n in enumerate(ns)],
                                [inputs(n, i)[1].cuda() for i, n in enumerate(ns)],
                                [torch.zeros(n, dtype=torch.bfloat16, device="cuda") for n in ns], state=st)
    a, b = mk(), mk()
    dyn = torch.zeros(32, dtype=torch.uint8, device="cuda")
    m.nvfp4_poll(a.ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.nvfp4_adamw_step(a, dynamic=dyn)
    for step in range(1, 5):
        h = dict(lr=1e-3 / step, step=step, weight_decay=0.01 * step, grad_scale=1.0 / step, sr_seed=(step << 40) + 5)
        dyn.copy_(a.dynamic(**h))
        g.replay()
        m.nvfp4_adamw_step(b, **h)
    torch.cuda.synchronize()
    for x, y in zip(a.params + a.weights, b.params + b.weights):
        assert torch.equal(x, y)
    for i in range(len(ns)):
        assert torch.equal(a.moment(i, "m"), b.moment(i, "m")) and torch.equal(a.moment(i, "v"), b.moment(i, "v"))


def test_other_stream_and_new_gradients():
    m = nv()
    n = 70000
    p, g = inputs(n, 1)
    mk = lambda: m.AdamWContext([torch.from_numpy(p).cuda()], [torch.zeros(n, device="cuda")], state=m.STATE_FP8)
    a, b = mk(), mk()
    s = torch.cuda.Stream()
    ga = g.cuda()
    torch.cuda.synchronize()
    a.set_grads([ga])
    m.nvfp4_adamw_step(a, lr=1e-3, step=3, sr_seed=9, stream=s)
    b.grads[0].copy_(ga)
    m.nvfp4_adamw_step(b, lr=1e-3, step=3, sr_seed=9)
    torch.cuda.synchronize()
    assert torch.equal(a.params[0], b.params[0]) and torch.equal(a.moment(0, "m"), b.moment(0, "m"))
    assert a.weights == [None]


def test_context_refuses():
    m = nv()
    p = torch.zeros(8, device="cuda")
    g = torch.zeros(8, device="cuda")
    for bad in (dict(params=[p.bfloat16()], grads=[g]), dict(params=[p], grads=[g.half()]), dict(params=[p], grads=[g[:7]]),
                dict(params=[p], grads=[g, g]), dict(params=[p], grads=[g.cpu()]), dict(params=[p], grads=[g], weights=[p]),
                dict(params=[p], grads=[g], state=2), dict(params=[p], grads=[torch.zeros(16, device="cuda")[::2]]),
                dict(params=[p], grads=[g], m=[p.view(torch.uint8)[:8]], state=m.STATE_FP8),
                dict(params=[p], grads=[g], m_scale=[torch.zeros(2, device="cuda")], state=m.STATE_FP8),
                dict(params=[p.cpu()], grads=[g.cpu()]),
                dict(params=[p, g], grads=[g, g], weights=[p.bfloat16(), g.bfloat16()], amax_ws=[m.default_workspace()] * 2)):
        with pytest.raises(ValueError):
            m.AdamWContext(**bad)
    ctx = m.AdamWContext([p], [g])
    for bad in (dict(step=0), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=float("nan")), dict(lr=float("inf")), dict(mode=2)):
        with pytest.raises(m.NVFP4Error):
            m.nvfp4_adamw_step(ctx, **{"lr": 1e-3, "step": 1, **bad})
    with pytest.raises(ValueError):
        m.nvfp4_adamw_step(ctx, dynamic=torch.zeros(31, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        ctx.set_grads([g[:4]])
    with pytest.raises(m.NVFP4Error):            # 16-byte rule
        m.nvfp4_adamw_step(m.AdamWContext([torch.zeros(9, device="cuda")[1:]], [g]), lr=1e-3)
    assert not p.any()
    m.nvfp4_adamw_step(m.AdamWContext([], []), lr=1e-3)


def test_context_refuses_tensors_twice_and_foreign_workspaces():
    m = nv()
    p, g = torch.zeros(512, device="cuda"), torch.zeros(512, device="cuda")
    other = types.SimpleNamespace(index=p.get_device() + 1, addr=0)     # a workspace of another device
    for bad in (dict(params=[p, p], grads=[g, g]),                       # the same tensor twice
                dict(params=[p[:300], p[256:]], grads=[g[:300], g[256:]]),
                dict(params=[p], grads=[g], m=[p]),
                dict(params=[p, g], grads=[g, p], v=[torch.zeros(512, device="cuda")] * 2),
                dict(params=[p], grads=[g], weights=[p.view(torch.bfloat16)[:512]]),
                dict(params=[p], grads=[g], weights=[p.bfloat16()], amax_ws=[other])):
        with pytest.raises(ValueError):
            m.AdamWContext(**bad)
    with pytest.raises(ValueError):
        m.nvfp4_adamw_step(m.AdamWContext([p], [g], ws=other), lr=1e-3)
    # neighbours in one buffer, and empty tensors wherever they lie, do not overlap
    m.nvfp4_adamw_step(m.AdamWContext([p[:256], p[256:], p[100:100]], [g[:256], g[256:], g[:0]]), lr=1e-3)
    assert not p.any()


@pytest.mark.parametrize("state", ["fp32", "fp8"])
def test_an_expert_layer_is_trained(state):
    # the operators as a training step uses them: forward, both gradients, the update of every expert's
    # weight, the next forward with the new weights; each stage against the values it was given
    m = nv()
    g = torch.Generator().manual_seed(2)
    E, d, n, rows = 4, 136, 72, 300
    counts = [120, 0, 175, 5]
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32).cuda()
    lay = m.GroupedLinearBF16(E, d, n)
    master = torch.randn(E, n, d, generator=g).cuda() * 0.02
    w = master.bfloat16()
    dw = torch.zeros(E, n, d, device="cuda")
    ctx = m.AdamWContext(list(master), list(dw), list(w), state=m.STATE_FP8 if state == "fp8" else m.STATE_FP32, ws=lay.ws)
    ref = [[master[e].cpu().numpy().reshape(-1), np.zeros(n * d, f32), np.zeros(n * d, f32)] for e in range(E)]
    for step in (1, 2):
        x = torch.randn(rows, d, generator=g).bfloat16().cuda()
        target = torch.randn(rows, n, generator=g).bfloat16().cuda()
        y = lay.fwd(x, w, off)
        dy = (y.float() - target.float()).bfloat16()
        dw.zero_()
        for lo, hi in ((0, 150), (150, rows)):      # two micro-batches, added
            part = off.clamp(lo, hi) - lo
            dx, _ = lay.bwd(x[lo:hi], w, dy[lo:hi], part, dw=dw, accumulate=True)
        grad = dw.cpu().numpy().copy()
        for e in range(E):
            lo, hi = int(off[e]), int(off[e + 1])
            a, b = dy[lo:hi].double().cpu(), x[lo:hi].double().cpu()
            bound = 2.0 ** -23 * (hi - lo + 4) * (a.abs().t() @ b.abs()) + 1e-30
            assert ((torch.from_numpy(grad[e]).double() - a.t() @ b).abs() <= bound).all()
            yy, ww = y[lo:hi].double().cpu(), w[e].double().cpu()
            full = b @ ww.t()
            assert ((yy - full).abs() <= 2.0 ** -8 * full.abs() + 2.0 ** -23 * d * (b.abs() @ ww.abs().t()) + 1e-30).all()
        m.nvfp4_adamw_step(ctx, step=step, sr_seed=step, **HYPER)
        assert m.nvfp4_poll(lay.ws) == 0
        for e in range(E):
            out = numpy_step(ref[e][0], grad[e].reshape(-1), ref[e][1], ref[e][2], state == "fp8", HYPER, step, 1, step, e)
            assert same(master[e].cpu().numpy().reshape(-1), out[0]) and torch.equal(w[e].cpu().reshape(-1), out[1])
            ref[e] = [out[0]] + ([E4M3[c] * s.repeat(256)[:n * d] for c, s in ((out[2], out[3]), (out[4], out[5]))]
                                 if state == "fp8" else [out[2], out[3]])


def test_the_quantized_layer_takes_the_updated_weight():
    # NVFP4 layer -> its fp32 dw -> AdamW (bf16 weight and its amax) -> the weight's forms without an
    # amax pass -> a forward pass on the cached forms, equal to one that quantizes the weight itself
    m = nv()
    T, d, n = 128, 192, 256
    g = torch.Generator().manual_seed(3)
    master = torch.randn(n, d, generator=g).cuda() * 0.02
    w = master.bfloat16()
    x, dy = torch.randn(T, d, generator=g).bfloat16().cuda(), (torch.randn(T, n, generator=g) * 1e-2).bfloat16().cuda()
    lay, check, aw = m.LinearContext(T, d, n), m.LinearContext(T, d, n), m.Workspace()
    dw = torch.empty(n, d, device="cuda")
    ctx = m.AdamWContext([master], [dw], [w], state=m.STATE_FP8, amax_ws=[aw])
    for step in (1, 2):
        m.nvfp4_linear_fwd(lay, x, w)
        m.nvfp4_linear_bwd(lay, dy, step, dw=dw)
        m.nvfp4_adamw_step(ctx, lr=1e-2, step=step, sr_seed=step)
        m.nvfp4_quantize_weight(w, out=lay.wq, out_t=lay.wqt, ws=aw, amax_ready=True)
        lay.w_cached = True
        y = m.nvfp4_linear_fwd(lay, x, None)
        lay.w_cached = False
        assert torch.equal(y, m.nvfp4_linear_fwd(check, x, w))
