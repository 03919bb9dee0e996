"""AdamW on the GPU against the oracle.

Tolerances. 32-bit states: m and v carry three roundings of 2^-24 relative to their larger term. p
is p (1 - lr wd) minus a step of about lr: two roundings of p plus a few of the step, and the step's
square root and division are good to a few ulp: |error| <= 2^-23 |p| + 2^-20 |step|. 8-bit states: the
bytes are equal, as the oracle carries out the same fp32 operations.
"""
import numpy as np
import pytest
import torch

import tile_level_copy_gb300 as tlc
from oracle import block_ref as ref

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16
HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1)


def f64(t):
    return t.double().cpu().numpy()


def tensors(sizes, pt, gt, bits, seed=0, shift=0):
    g = torch.Generator().manual_seed(seed)

    def place(v):  # `shift` values off an aligned start
        buf = torch.zeros(v.numel() + shift, dtype=v.dtype, device="cuda")
        buf[shift:] = v.cuda()
        return buf[shift:]

    p = [place((torch.randn(n, generator=g) * 0.02).to(pt)) for n in sizes]
    gr = [place((torch.randn(n, generator=g) * 1e-3 * torch.exp(torch.randn(n, generator=g) * 2)).to(gt)) for n in sizes]
    if bits == 32:
        m = [place(torch.randn(n, generator=g) * 3e-4) for n in sizes]
        v = [place((torch.randn(n, generator=g) * 1e-3) ** 2) for n in sizes]
        return p, gr, m, v, None, None
    code = lambda n, hi: place(torch.randint(0, hi, (n,), generator=g, dtype=torch.uint8))  # noqa: E731
    m = [code(n, 256) for n in sizes]
    for t in m:  # no code above 0x77: larger ones do not occur (a block's largest is below 2^8)
        t[:] = torch.where((t & 0x7F) > 0x77, t & 0x77, t)
    v = [code(n, 0xF0) for n in sizes]
    blocks = [-(-n // 128) for n in sizes]
    ms = [torch.randint(95, 110, (k,), generator=g, dtype=torch.uint8).cuda() for k in blocks]
    vs = [torch.randint(80, 90, (k,), generator=g, dtype=torch.uint8).cuda() for k in blocks]
    return p, gr, m, v, ms, vs


BIG = [1 << 20]  # one last bit of m or v that differs shows in a code once in some 50,000 values
SIZES = [[1], [127, 128, 129], [3, 0, 5000, 4096, 4097, 1, 12289], [100] * 40, [17 + i for i in range(400)]]


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("pt,gt,copy", [(F32, F32, False), (F32, BF, True), (BF, BF, False), (BF, F32, True)])
@pytest.mark.parametrize("sizes", SIZES)
def test_32_bits(sizes, pt, gt, copy, shift):
    p, g, m, v, _, _ = tensors(sizes, pt, gt, 32, len(sizes), shift)
    c = [torch.zeros_like(t, dtype=BF) for t in p] if copy else None
    cfg = tlc.AdamWConfig(**HYPER)
    before = [[f64(t) for t in l] for l in (p, g, m, v)]
    scale = torch.full((1,), 0.37, device="cuda") if copy else None
    tlc.adamw_step(cfg, tlc.AdamWList(cfg, p, g, m, v, copy=c), 7, scale)
    for i in range(len(sizes)):
        p0, g0, m0, v0 = (b[i] for b in before)
        g0 = g0 * (float(np.float32(0.37)) if copy else 1.0)
        wp, wm, wv = ref.adamw_step(p0, g0, m0, v0, step=7, **HYPER)
        assert (np.abs(f64(m[i]) - wm) <= 4 * 2.0 ** -24 * (np.abs(m0) + np.abs(g0))).all()
        assert (np.abs(f64(v[i]) - wv) <= 6 * 2.0 ** -24 * (v0 + g0 * g0) + 2.0 ** -140).all()
        far = 2.0 ** -23 * np.abs(p0) + 2.0 ** -20 * (np.abs(wp - p0) + 1e-3 * 0.1 * np.abs(p0)) + \
            1e-3 * 8 * 2.0 ** -24 * (np.abs(m0) + np.abs(g0)) / (np.sqrt(wv / (1 - 0.999 ** 7)) + 1e-8) * 3
        assert (np.abs(f64(p[i]) - wp) <= far + (2.0 ** -8 * np.abs(wp) if pt == BF else 0)).all()
        if copy:
            assert (np.abs(f64(c[i]) - wp) <= far + 2.0 ** -8 * np.abs(wp)).all()


@pytest.mark.parametrize("shift", [0, 3])
@pytest.mark.parametrize("pt,gt", [(F32, BF), (F32, F32), (BF, BF)])
@pytest.mark.parametrize("sizes", SIZES[:4] + [BIG])
def test_8_bits_equal_the_oracle(sizes, pt, gt, shift):
    p, g, m, v, ms, vs = tensors(sizes, pt, gt, 8, len(sizes), shift)
    base = [5 + (1 << 33) * i for i in range(len(sizes))]
    seed, step = 0x123456789ABCDEF, 4321
    cfg = tlc.AdamWConfig(**HYPER, bits=8, seed=seed)
    before = [[t.cpu().numpy().copy() for t in l] for l in (m, v, ms, vs)]
    p0, g0 = [f64(t) for t in p], [f64(t) for t in g]
    lst = tlc.AdamWList(cfg, p, g, m, v, ms, vs, rng_base=base)
    tlc.adamw_step(cfg, lst, step)
    out = [[torch.full((n,), 9.0, device="cuda") for n in sizes] for _ in range(2)]
    tlc.adamw_read_state(cfg, lst, tlc.AdamWValues(lst, *out))
    for i, n in enumerate(sizes):
        if n == 0:
            continue
        dm = ref.decode(before[0][i], before[2][i], "m").astype(np.float32)
        dv = ref.decode(before[1][i], before[3][i], "v").astype(np.float32)
        nm, nv = ref.moments_f32(g0[i].astype(np.float32), dm, dv, 0.9, 0.999)
        r = ref.noise(n, seed, step, base[i])
        for x, name, codes, scales, read, bits in ((nm, "m", m, ms, out[0], r & 0xFFFF), (nv, "v", v, vs, out[1], r >> 16)):
            wc, wsc = ref.encode(x, bits, name)
            np.testing.assert_array_equal(scales[i].cpu().numpy(), wsc)
            np.testing.assert_array_equal(codes[i].cpu().numpy(), wc)
            assert np.array_equal(read[i].cpu().numpy(), ref.decode(wc, wsc, name).astype(np.float32))
        wp, _, wv = ref.adamw_step(p0[i], g0[i], dm.astype(np.float64), dv.astype(np.float64), step=step, **HYPER)
        den = np.sqrt(wv / (1 - 0.999 ** step)) + 1e-8
        far = 2.0 ** -23 * np.abs(p0[i]) + 2.0 ** -20 * (np.abs(wp - p0[i]) + 1e-4 * np.abs(p0[i])) + \
            1e-3 * 24 * 2.0 ** -24 * (np.abs(dm) + np.abs(g0[i])) / den
        assert (np.abs(f64(p[i]) - wp) <= far + (2.0 ** -8 * np.abs(wp) if pt == BF else 0)).all()


@pytest.mark.parametrize("gt", [F32, BF])
def test_8_bits_long_list(gt):
    """More chunks than a launch has under way, in tensors of whole and of odd chunks, one with scales off an
    aligned start: the states are those of the same tensors one by one, off an aligned start."""
    sizes = [4096 * 700 + 5, 3, 4096 * 300, 130, 4096 * 250 + 4095, 77, 4096 * 40]
    one, two = ([list(l) for l in tensors(sizes, F32, gt, 8, 1, shift)] for shift in (0, 3))
    odd = torch.zeros(one[4][2].numel() + 1, dtype=torch.uint8, device="cuda")
    odd[1:] = one[4][2]
    one[4][2] = odd[1:]
    base = [7 * i for i in range(len(sizes))]
    cfg = tlc.AdamWConfig(**HYPER, bits=8, seed=9)
    tlc.adamw_step(cfg, tlc.AdamWList(cfg, *one, rng_base=base), 3)
    for i in range(len(sizes)):
        tlc.adamw_step(cfg, tlc.AdamWList(cfg, *([l[i]] for l in two), rng_base=base[i:i + 1]), 3)
    for a, b in zip(one[2:], two[2:]):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
    for x, y in zip(one[0], two[0]):  # one rounding more or less of the sum, and of its smaller term
        assert ((x - y).abs() <= 2.0 ** -22 * x.abs() + 1e-3 * 2.0 ** -18).all()


def test_small_changes_are_not_lost():
    """v decays by 0.1 % a step with no gradient: after 1000 steps its mean has fallen by 1/e, although
    one step is far below half a rounding step. Rounding adds variance but no drift: the mean over
    2^16 values of a walk of 1000 steps with relative deviation at most 1/16 * sqrt(step share)."""
    n = 1 << 16
    p, g = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    m, v = torch.zeros(n, dtype=torch.uint8, device="cuda"), torch.full((n,), 0x60, dtype=torch.uint8, device="cuda")
    ms, vs = torch.zeros(n // 128, dtype=torch.uint8, device="cuda"), torch.full((n // 128,), 100, dtype=torch.uint8, device="cuda")
    cfg = tlc.AdamWConfig(lr=0.0, bits=8, seed=1)
    lst = tlc.AdamWList(cfg, [p], [g], [m], [v], [ms], [vs])
    out = tlc.AdamWValues(lst, [torch.empty(n, device="cuda")], [torch.empty(n, device="cuda")])
    tlc.adamw_read_state(cfg, lst, out)
    start = out.keep[1][0].mean().item()
    for t in range(1, 1001):
        tlc.adamw_step(cfg, lst, t)
    tlc.adamw_read_state(cfg, lst, out)
    # a rounding's variance is at most (1/8)^2 / 4 of the value's square times the share of a step that
    # one decay is (0.001 / (1/8)): after 1000 steps at most 1000 * 0.008 / 256 = 0.03 relative
    # variance a value, 0.18 / 256 = 7e-4 for the mean; five deviations
    assert abs(out.keep[1][0].mean().item() / start - 0.999 ** 1000) <= 5 * 7e-4 * 1.0


def test_non_finite_gradients_are_seen():
    n = 300
    for bits in (32, 8):
        p, g, m, v, ms, vs = tensors([n], F32, F32, bits)
        g[0][200] = float("inf")
        cfg = tlc.AdamWConfig(**HYPER, bits=bits)
        lst = tlc.AdamWList(cfg, p, g, m, v, ms, vs)
        tlc.adamw_step(cfg, lst, 1)
        tlc.adamw_step(cfg, lst, 2)
        bad = ~torch.isfinite(p[0])
        assert bad[200] and torch.isfinite(p[0][:128]).all() and torch.isfinite(p[0][256:]).all()
        if bits == 8:  # the state's block reads as NaN
            assert bad[128:256].all()


def test_zero_state_zero_gradient_and_graph():
    n = 1000
    p = torch.randn(n, device="cuda")
    g, m, v = (torch.zeros(n, device="cuda") for _ in range(3))
    cfg = tlc.AdamWConfig(lr=0.5, weight_decay=0.25)
    want = p * (1 - 0.125)
    lst = tlc.AdamWList(cfg, [p], [g], [m], [v])
    tlc.adamw_step(cfg, lst, 1)
    assert torch.equal(p, want) and not m.any() and not v.any()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tlc.adamw_step(cfg, lst, 1)
    graph.replay()
    assert torch.equal(p, want * (1 - 0.125))


def test_refusals():
    p, g, m, v, _, _ = tensors([64], F32, F32, 32)
    for kw in (dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1.0), dict(lr=float("nan"))):
        cfg = tlc.AdamWConfig(**{**HYPER, **kw})
        with pytest.raises(tlc.MoEError) as e:
            tlc.adamw_step(cfg, tlc.AdamWList(cfg, p, g, m, v), 1)
        assert e.value.code == tlc.MOE_ERR_ARG
    cfg = tlc.AdamWConfig(**HYPER)
    with pytest.raises(tlc.MoEError):
        tlc.adamw_step(cfg, tlc.AdamWList(cfg, p, g, m, v), 0)
    with pytest.raises(ValueError):
        tlc.AdamWList(tlc.AdamWConfig(**HYPER, bits=8), p, g, m, v)
    with pytest.raises(ValueError):
        tlc.AdamWList(cfg, p, [g[0][:5]], m, v)
    with pytest.raises(ValueError):
        tlc.AdamWList(cfg, p, g, [m[0].to(BF)], v)
    with pytest.raises(ValueError):
        tlc.adamw_step(tlc.AdamWConfig(**HYPER, bits=8), tlc.AdamWList(cfg, p, g, m, v), 1)
    bad = tlc.AdamWConfig(**HYPER, bits=16)
    lst = tlc.AdamWList(cfg, p, g, m, v)
    lst.bits = 16
    with pytest.raises(tlc.MoEError):
        tlc.adamw_step(bad, lst, 1)
    tlc.adamw_step(cfg, tlc.AdamWList(cfg, [], [], [], []), 1)  # no tensors: nothing to do
