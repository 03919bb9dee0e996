"""Layer norm on the GPU against the 64-bit oracle.

Tolerances (relative 2-norm). fp32 outputs: a row's sums are trees over at most 32 sequential values a
thread, so mean, variance and the outputs carry a few roundings of 2^-24 each: 16 * 2^-24 = 1e-6.
bf16 and fp16 outputs are the rounding to nearest of such a value: each lies between the roundings of
the oracle's value minus and plus the fp32 error. dw and db are sums over the rows, one after another
in a CTA: errors of random sign grow with the square root of the number of terms.
"""
import numpy as np
import pytest
import torch

import tile_level_copy_gb300 as tlc
from oracle import block_ref as ref

pytestmark = pytest.mark.gpu
F32, BF, F16 = torch.float32, torch.bfloat16, torch.float16


def f64(t):
    return t.double().cpu().numpy()


def close(got, want, rel):
    got = f64(got)
    assert np.isfinite(got).all()
    err, n = np.linalg.norm(got - want), np.linalg.norm(want)
    assert err <= rel * n, (err / n, rel)


def near(got, want, err):
    """Every value is a rounding to got's type of some number within err of want."""
    lo, hi = (torch.from_numpy(np.asarray(want + e)).to(got.dtype).double().numpy() for e in (-err, err))
    g = f64(got)
    assert ((lo <= g) & (g <= hi)).all()


def make(rows, d, dt, wt, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return ((r(rows, d) * 1.5 + 0.25).to(dt).cuda(), (r(d) * 0.1 + 1).to(wt).cuda(), (r(d) * 0.1).to(wt).cuda(),
            (r(rows, d) * 0.1).to(dt).cuda())


SHAPES = [(1, 1), (3, 2), (1, 4096), (5, 7), (2, 64), (33, 100), (700, 128), (513, 257), (40, 511), (41, 512), (42, 513),
          (300, 1000), (129, 1003), (7, 2048), (1003, 2050), (64, 4099), (31, 8192), (5, 8193), (9, 16384), (6, 16383),
          (5000, 96), (2000, 768)]
TYPES = [(BF, BF), (BF, F32), (F16, F16), (F16, F32), (F32, F32)]


@pytest.mark.parametrize("dt,wt", TYPES)
@pytest.mark.parametrize("rows,d", SHAPES)
def test_forward_and_backward(rows, d, dt, wt):
    x, w, b, dy = make(rows, d, dt, wt, rows + d)
    cfg = tlc.LayerNormConfig(rows, d, dt, wt, 1e-5)
    y = torch.full_like(x, float("nan"))
    mean, rstd = (torch.full((rows,), float("nan"), device="cuda") for _ in range(2))
    tlc.layernorm_forward(cfg, x, w, b, y, mean, rstd)
    wy, wm, wr = ref.layernorm_forward(f64(x), f64(w), f64(b), float(np.float32(1e-5)))
    np.testing.assert_allclose(f64(mean), wm, rtol=0, atol=16 * 2.0 ** -24 * np.abs(f64(x)).max())
    # with few values the variance may be small beside the values' own size: its error is 2^-24 of
    # their square, relative to var + eps
    amp = (np.abs(f64(x)).max(1) * wr) ** 2
    assert (np.abs(f64(rstd) / wr - 1) <= 16 * 2.0 ** -24 * (1 + amp)).all()
    far = 16 * 2.0 ** -24 * (1 + amp.max() if d < 64 else 4)
    if dt == F32:
        close(y, wy, far)
    near(y, wy, 32 * 2.0 ** -24 * (1 + amp[:, None]) * (1 + np.abs(wy)))
    # backward, from the kept statistics
    ws = tlc.LayerNormWorkspace(cfg)
    dx = torch.full_like(x, float("nan"))
    dw, db = torch.full_like(w, float("nan")), torch.full_like(w, float("nan"))
    tlc.layernorm_backward(cfg, dy, x, w, mean, rstd, dx, dw, db, ws)
    gx, gw, gb = ref.layernorm_backward(f64(dy), f64(x), f64(w), f64(mean), f64(rstd))
    # dx is a difference of terms of the size of rstd dy w: the error is relative to them
    parts = f64(rstd)[:, None] * f64(dy) * f64(w)
    if dt == F32:
        assert np.linalg.norm(f64(dx) - gx) <= 32 * 2.0 ** -24 * np.linalg.norm(parts)
    xh = (f64(x) - f64(mean)[:, None]) * f64(rstd)[:, None]
    near(dx, gx, 32 * 2.0 ** -24 * np.abs(parts).max(1, keepdims=True) * (1 + np.abs(xh)))
    for got, want, terms in ((dw, gw, f64(dy) * xh), (db, gb, f64(dy))):
        size = np.linalg.norm(np.sqrt((terms ** 2).sum(0)))  # 2-norm over all terms
        if wt == F32:
            assert np.linalg.norm(f64(got) - want) <= 2.0 ** -24 * 4 * np.sqrt(rows) * size
        near(got, want, 2.0 ** -24 * 4 * np.sqrt(rows) * np.abs(terms).max() * np.sqrt(rows))
    dx2, dw2, db2 = torch.empty_like(dx), torch.empty_like(dw), torch.empty_like(db)
    tlc.layernorm_backward(cfg, dy, x, w, mean, rstd, dx2, dw2, db2, ws)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(db, db2)


def test_optional_arguments_and_in_place():
    rows, d = 37, 1000
    x, w, b, dy = make(rows, d, BF, F32)
    cfg = tlc.LayerNormConfig(rows, d, BF, F32)
    y = torch.empty_like(x)
    tlc.layernorm_forward(cfg, x, None, None, y)
    eps = float(np.float32(1e-5))
    want, m, r = ref.layernorm_forward(f64(x), 1.0, 0.0, eps)
    near(y, want, 1e-4 * 2.0 ** -8 * (1 + np.abs(want)))
    z = x.clone()
    tlc.layernorm_forward(cfg, z, None, None, z)
    assert torch.equal(z, y)
    mean, rstd = torch.from_numpy(m).float().cuda(), torch.from_numpy(r).float().cuda()
    dx = torch.empty_like(x)
    tlc.layernorm_backward(cfg, dy, x, None, mean, rstd, dx)
    near(dx, ref.layernorm_backward(f64(dy), f64(x), 1.0, f64(mean), f64(rstd))[0], 1e-6)
    g = dy.clone()
    tlc.layernorm_backward(cfg, g, x, None, mean, rstd, g)
    assert torch.equal(g, dx)
    ws, db = tlc.LayerNormWorkspace(cfg), torch.empty(d, device="cuda")
    tlc.layernorm_backward(cfg, dy, x, w, mean, rstd, dx, None, db, ws)
    close(db, f64(dy).sum(0), 1e-6)


def test_no_rows():
    cfg = tlc.LayerNormConfig(0, 64, F32, F32)
    x, w, b, dy = make(0, 64, F32, F32)
    s = torch.empty(0, device="cuda")
    tlc.layernorm_forward(cfg, x, w, b, x, s, s)
    dw, db = torch.full_like(w, 5), torch.full_like(w, 5)
    tlc.layernorm_backward(cfg, dy, x, w, s, s, x, dw, db, tlc.LayerNormWorkspace(cfg))
    assert (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("d", [64, 777, 4096])
def test_hard_rows(d):
    """Constant rows (variance 0), values far from zero, and a row with NaN or infinity among others."""
    x = torch.randn(6, d, device="cuda")
    x[0] = 3.0
    x[1] += 4096.0  # the variance is a 2^-24 part of the mean square
    x[2, d // 2] = float("nan")
    x[3, d // 3] = float("inf")
    cfg = tlc.LayerNormConfig(6, d, F32, F32, 1e-5)
    y, mean, rstd = torch.empty_like(x), torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
    tlc.layernorm_forward(cfg, x, None, None, y, mean, rstd)
    # a constant row: what is left is the mean's rounding (2^-24 of 3) times rstd (1 / sqrt(1e-5))
    assert (y[0].abs() <= 3 * 4 * 2.0 ** -24 * 317).all() and abs(rstd[0].item() * 1e-5 ** 0.5 - 1) < 1e-5
    want = ref.layernorm_forward(f64(x[1:2]), 1.0, 0.0, 1e-5)[0]
    assert np.abs(f64(y[1:2]) - want).max() <= 4096 * 8 * 2.0 ** -24  # the mean's rounding
    assert torch.isnan(y[2]).all() and torch.isnan(y[3]).all()
    want = ref.layernorm_forward(f64(x[4:]), 1.0, 0.0, 1e-5)[0]
    close(y[4:], want, 4e-6)


@pytest.mark.parametrize("dt", [BF, F32])
def test_unaligned_tensors_and_stream(dt):
    rows, d = 21, 1024
    x, w, b, dy = make(rows, d, dt, F32)
    cfg = tlc.LayerNormConfig(rows, d, dt, F32)
    shift = lambda t: torch.cat([t.flatten()[:1], t.flatten()])[1:].view(t.shape)  # noqa: E731
    y0, y1 = torch.empty_like(x), shift(x)
    m, r = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    tlc.layernorm_forward(cfg, x, w, b, y0, m, r)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    xs = shift(x)
    assert xs.data_ptr() % 16
    st.wait_stream(torch.cuda.current_stream())
    tlc.layernorm_forward(cfg, xs, shift(w), shift(b), y1, stream=st)
    st.synchronize()
    # other pieces, other order of the sums: equal up to the last bit
    close(y1, f64(y0), (2.0 ** -8 if dt == BF else 0) + 2e-6)


def test_refusals():
    x, w, b, dy = make(4, 64, BF, F32)
    s = torch.empty(4, device="cuda")
    for kw in (dict(rows=-1), dict(d=0), dict(d=16385), dict(eps=-1.0), dict(dtype=F32, wdtype=BF)):
        cfg = tlc.LayerNormConfig(**{**dict(rows=4, d=64), **kw})
        with pytest.raises(tlc.MoEError) as e:
            tlc.LayerNormWorkspace(cfg)
        assert e.value.code == tlc.MOE_ERR_ARG
    cfg = tlc.LayerNormConfig(4, 64)
    for a in ((x.float(), w, b, x), (x[:3], w, b, x), (x, w.to(BF), b, x), (x, w[:5], b, x), (x.cpu(), w, b, x),
              (x.t().contiguous().t(), w, b, x)):
        with pytest.raises(ValueError):
            tlc.layernorm_forward(cfg, *a)
    with pytest.raises(tlc.MoEError) as e:
        tlc.layernorm_backward(cfg, dy, x, w, s, s, x.clone(), w.clone(), b.clone(), None)
    assert e.value.code == tlc.MOE_ERR_ARG
