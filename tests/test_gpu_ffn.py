"""Gated feed-forward block on the GPU against the 64-bit oracle.

Tolerances. y, dx and the weight gradients are rounded to bf16 at the end and are sums of products of
which one factor was rounded to bf16 before. A rounding to nearest is off by at most 2^-8 relative, by
2^-8 / sqrt(3) times 1 to 1/2 over a binade in the mean square: at most 2.3e-3, 1.7e-3 for values
spread over binades. Two such errors of independent signs add up to less than 4.3e-3 in the
relative 2-norm, 2.4e-3 as a rule.
"""
import numpy as np
import pytest
import torch

import tile_level_copy_gb300 as tlc
from oracle import block_ref as ref

pytestmark = pytest.mark.gpu
REL = 4.3e-3
BF = torch.bfloat16


def make(T, d, f, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(BF).cuda()  # noqa: E731
    return r(T, d), r(f, d, std=d ** -0.5), r(f, d, std=d ** -0.5), r(d, f, std=f ** -0.5), r(T, d, std=0.01)


def f64(t):
    return t.double().cpu().numpy()


def close(got, want, rel=REL):
    got = f64(got)
    assert np.isfinite(got).all()
    n = np.linalg.norm(want)
    assert np.linalg.norm(got - want) <= rel * n, (np.linalg.norm(got - want) / n, got.shape)


def forward(cfg, x, W1, W3, W2, save, ws=None):
    ws = ws or tlc.FFNWorkspace(cfg)
    y = torch.full_like(x, float("nan"))
    saved = tlc.ffn_saved(cfg).fill_(0xFF) if save else None
    tlc.ffn_forward(cfg, x, W1, W3, W2, y, ws, saved=saved)
    assert tlc.ffn_status(cfg, ws) == (tlc.MOE_OK, 0)
    return y, saved, ws


SHAPES = [(1, 8, 8), (1, 128, 256), (2, 2048, 1408), (3, 136, 264), (5, 4096, 520), (16, 1000, 2744), (17, 72, 3000),
          (37, 200, 1000), (63, 512, 4096), (64, 520, 136), (65, 256, 384), (128, 128, 256), (129, 264, 136),
          (255, 8, 520), (256, 256, 256), (257, 512, 1408), (300, 1000, 2744), (1003, 136, 264)]


@pytest.mark.parametrize("T,d,f", SHAPES)
@pytest.mark.parametrize("save", [False, True])
def test_forward(T, d, f, save):
    x, W1, W3, W2, _ = make(T, d, f, T + d)
    y, _, _ = forward(tlc.FFNConfig(T, d, f), x, W1, W3, W2, save)
    close(y, ref.ffn_forward(f64(x), f64(W1), f64(W3), f64(W2)))


# Input and weight gradients in one launch, of more tiles than go at once: the input gradients' tiles
# longer than the others (cut into parts or not), and shorter.
LONG = [(300, 1032, 4104), (1100, 1032, 2056), (2500, 520, 2056), (4000, 136, 264)]


@pytest.mark.parametrize("T,d,f", SHAPES + LONG)
def test_backward(T, d, f):
    cfg = tlc.FFNConfig(T, d, f)
    x, W1, W3, W2, dy = make(T, d, f, T + f)
    y, saved, ws = forward(cfg, x, W1, W3, W2, True)
    outs = [torch.full_like(t, float("nan")) for t in (x, W1, W3, W2)]
    kept = saved.clone()
    tlc.ffn_backward(cfg, x, W1, W3, W2, dy, saved, *outs, ws)
    assert tlc.ffn_status(cfg, ws) == (tlc.MOE_OK, 0)
    for got, want in zip(outs, ref.ffn_backward(*(f64(t) for t in (x, W1, W3, W2, dy)))):
        close(got, want)
    assert torch.equal(saved, kept)  # read only
    again = [torch.empty_like(t) for t in outs]
    tlc.ffn_backward(cfg, x, W1, W3, W2, dy, saved, *again, ws)
    torch.cuda.synchronize()
    for a, b in zip(outs, again):
        assert torch.equal(a, b)


def test_no_write_outside_the_outputs():
    T, d, f = 131, 136, 264
    cfg = tlc.FFNConfig(T, d, f)
    x, W1, W3, W2, dy = make(T, d, f)
    ws = tlc.FFNWorkspace(cfg)
    guard = 4096

    def fenced(t):
        buf = torch.full((t.numel() + 2 * guard,), 7.0, dtype=BF, device="cuda")
        return buf, buf[guard:guard + t.numel()].view(t.shape)

    n = tlc.ffn_saved(cfg).numel()
    sbuf = torch.full((n + 2 * guard,), 77, dtype=torch.uint8, device="cuda")
    saved = sbuf[guard:guard + n]
    by, y = fenced(x)
    tlc.ffn_forward(cfg, x, W1, W3, W2, y, ws, saved=saved)
    pairs = [fenced(t) for t in (x, W1, W3, W2)]
    tlc.ffn_backward(cfg, x, W1, W3, W2, dy, saved, *(p[1] for p in pairs), ws)
    assert tlc.ffn_status(cfg, ws) == (tlc.MOE_OK, 0)
    for buf in [by] + [p[0] for p in pairs]:
        assert (buf[:guard] == 7).all() and (buf[-guard:] == 7).all()
    assert (sbuf[:guard] == 77).all() and (sbuf[-guard:] == 77).all()


def test_no_tokens():
    cfg = tlc.FFNConfig(0, 128, 256)
    x, W1, W3, W2, _ = make(0, 128, 256)
    y, saved, ws = forward(cfg, x, W1, W3, W2, True)
    outs = [torch.full_like(t, 3.0) for t in (x, W1, W3, W2)]
    tlc.ffn_backward(cfg, x, W1, W3, W2, x, saved, *outs, ws)
    assert all((t == 0).all() for t in outs[1:])


@pytest.mark.parametrize("T", [1, 9, 40, 300])
def test_rows_are_independent_and_nan_stays_in_its_row(T):
    cfg = tlc.FFNConfig(T, 264, 520)
    x, W1, W3, W2, _ = make(T, 264, 520)
    y, _, ws = forward(cfg, x, W1, W3, W2, False)
    bad = T // 2
    x2 = x.clone()
    x2[bad, 3] = float("nan")
    y2, _, _ = forward(cfg, x2, W1, W3, W2, False, ws)
    assert torch.isnan(y2[bad]).all()
    keep = [i for i in range(T) if i != bad]
    assert torch.equal(y2[keep], y[keep])


@pytest.mark.parametrize("T", [1, 7, 300])
def test_large_gates_saturate(T):
    """silu(g) is g above and 0 below the range of exp: no overflow turns into NaN."""
    d, f = 128, 256
    x = torch.ones(T, d, dtype=BF, device="cuda")
    W1 = torch.ones(f, d, dtype=BF, device="cuda")
    W1[::2] = -1.0  # g = -128, 128
    W3 = torch.full((f, d), 2.0 ** -7, dtype=BF, device="cuda")  # u = 1
    W2 = torch.full((d, f), 2.0 ** -7, dtype=BF, device="cuda")
    cfg = tlc.FFNConfig(T, d, f)
    y, saved, ws = forward(cfg, x, W1, W3, W2, True)
    assert torch.equal(y, torch.full_like(y, 128.0))
    y, _, _ = forward(cfg, x, W1, W3, W2, False, ws)
    assert torch.equal(y, torch.full_like(y, 128.0))
    dy = torch.ones_like(x)
    outs = [torch.empty_like(t) for t in (x, W1, W3, W2)]
    tlc.ffn_backward(cfg, x, W1, W3, W2, dy, saved, *outs, ws)
    for got, want in zip(outs, ref.ffn_backward(*(f64(t) for t in (x, W1, W3, W2, dy)))):
        close(got, want)


def test_stream_and_graph():
    """On a stream of its own, and captured into a graph that is replayed on new inputs."""
    for T in (2, 200):
        cfg = tlc.FFNConfig(T, 256, 512)
        x, W1, W3, W2, dy = make(T, 256, 512)
        ws, saved = tlc.FFNWorkspace(cfg), tlc.ffn_saved(cfg)
        y, y0 = torch.empty_like(x), torch.empty_like(x)
        outs = [torch.empty_like(t) for t in (x, W1, W3, W2)]
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())

        def step():
            tlc.ffn_forward(cfg, x, W1, W3, W2, y0, ws, stream=st)
            tlc.ffn_forward(cfg, x, W1, W3, W2, y, ws, saved=saved, stream=st)
            tlc.ffn_backward(cfg, x, W1, W3, W2, dy, saved, *outs, ws, stream=st)

        with torch.cuda.stream(st):
            step()
        st.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            step()
        x.copy_(torch.randn(T, 256).to(BF))
        dy.copy_(torch.randn(T, 256).to(BF))
        graph.replay()
        torch.cuda.synchronize()
        a = [f64(t) for t in (x, W1, W3, W2, dy)]
        close(y, ref.ffn_forward(*a[:4]))
        close(y0, ref.ffn_forward(*a[:4]))
        for got, want in zip(outs, ref.ffn_backward(*a)):
            close(got, want)


def test_large_offsets():
    """Tensors whose byte offsets pass 2^32: the last rows of a long batch and of its kept values."""
    T, d, f = 270000, 128, 4096  # kept values: 8.8 GB
    cfg = tlc.FFNConfig(T, d, f)
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(BF)  # noqa: E731
    x, dy = r(T, d), r(T, d, std=0.01)
    W1, W3, W2 = r(f, d, std=d ** -0.5), r(f, d, std=d ** -0.5), r(d, f, std=f ** -0.5)
    y, saved, ws = forward(cfg, x, W1, W3, W2, True)
    outs = [torch.empty_like(t) for t in (x, W1, W3, W2)]
    tlc.ffn_backward(cfg, x, W1, W3, W2, dy, saved, *outs, ws)
    assert tlc.ffn_status(cfg, ws) == (tlc.MOE_OK, 0)
    for rows in (slice(0, 200), slice(T - 200, T)):
        a = [f64(t) for t in (x[rows], W1, W3, W2, dy[rows])]
        close(y[rows], ref.ffn_forward(*a[:4]))
        close(outs[0][rows], ref.ffn_backward(*a)[0])


def test_refusals():
    for kw in (dict(d=100), dict(ffn=12), dict(T=-1), dict(d=0), dict(ffn=1 << 20), dict(T=1 << 24)):
        cfg = tlc.FFNConfig(**{**dict(T=4, d=128, ffn=256), **kw})
        with pytest.raises(tlc.MoEError) as e:
            tlc.FFNWorkspace(cfg)
        assert e.value.code == tlc.MOE_ERR_ARG
    cfg = tlc.FFNConfig(4, 128, 256)
    x, W1, W3, W2, dy = make(4, 128, 256)
    ws, y = tlc.FFNWorkspace(cfg), torch.empty_like(x)
    for args in ((x.float(), W1, W3, W2, y), (x.cpu(), W1, W3, W2, y), (x[:3], W1, W3, W2, y), (x, W2, W3, W2, y),
                 (x, W1.t().contiguous().t(), W3, W2, y), (x, W1, W3, W2, y.T.contiguous().T)):
        with pytest.raises(ValueError):
            tlc.ffn_forward(cfg, *args, ws)
    with pytest.raises(ValueError):
        tlc.ffn_forward(cfg, x, W1, W3, W2, y, ws, saved=torch.empty(16, dtype=torch.uint8, device="cuda"))
    buf = torch.empty(4 * 128 + 1, dtype=BF, device="cuda")[1:].view(4, 128)
    with pytest.raises(tlc.MoEError) as e:
        tlc.ffn_forward(cfg, x, W1, W3, W2, buf, ws)
    assert e.value.code == tlc.MOE_ERR_ARG
    small = tlc.FFNWorkspace(tlc.FFNConfig(1, 128, 8))
    with pytest.raises(tlc.MoEError) as e:
        tlc.ffn_forward(cfg, x, W1, W3, W2, y, small)
    assert e.value.code == tlc.MOE_ERR_WORKSPACE


@pytest.mark.parametrize("T,d,f", [(5, 512, 1024), (90, 2048, 1408), (700, 264, 2744), (1500, 1024, 1024)])
def test_back_to_back_passes_equal_their_own_results(T, d, f):
    """Passes over two inputs in turn, nothing waited for in between (each launch may start while the one
    before it ends, the weight gradients beside the input gradients): every result is bit for bit the
    one that a pass by itself gave."""
    cfg = tlc.FFNConfig(T, d, f)
    sets, ws, saved = [make(T, d, f, seed) for seed in (1, 2)], tlc.FFNWorkspace(cfg), tlc.ffn_saved(cfg)

    def one(x, W1, W3, W2, dy):
        y, outs = torch.empty_like(x), [torch.empty_like(t) for t in (x, W1, W3, W2)]
        tlc.ffn_forward(cfg, x, W1, W3, W2, y, ws, saved=saved)
        tlc.ffn_backward(cfg, x, W1, W3, W2, dy, saved, *outs, ws)
        return [y, *outs]

    alone = []
    for s in sets:
        alone.append(one(*s))
        torch.cuda.synchronize()
    runs = [one(*sets[i % 2]) for i in range(12)]
    torch.cuda.synchronize()
    for i, got in enumerate(runs):
        for a, b in zip(got, alone[i % 2]):
            assert torch.equal(a, b)
    assert tlc.ffn_status(cfg, ws) == (tlc.MOE_OK, 0)


@pytest.mark.parametrize("T", [3, 2000])
def test_a_wait_that_runs_out_is_reported(T):
    """With a limit of 1 us some waits may run out (the limit is looked at between the hardware's own
    suspended tries, so a short wait can also succeed): the calls end either way, the status says which,
    the values are right if it says so, and the workspace is usable again once its status words are zero."""
    d, f = 4096, 2048
    x, W1, W3, W2, dy = make(T, d, f)
    short, cfg = tlc.FFNConfig(T, d, f, timeout_us=1), tlc.FFNConfig(T, d, f)
    ws, y, saved = tlc.FFNWorkspace(cfg), torch.empty_like(x), tlc.ffn_saved(cfg)
    want = ref.ffn_forward(f64(x), f64(W1), f64(W3), f64(W2))
    for _ in range(5):
        tlc.ffn_forward(short, x, W1, W3, W2, y, ws, saved=saved)
        tlc.ffn_backward(short, x, W1, W3, W2, dy, saved, *(torch.empty_like(t) for t in (x, W1, W3, W2)), ws)
        rc, detail = tlc.ffn_status(short, ws)
        assert rc in (tlc.MOE_OK, tlc.MOE_ERR_TIMEOUT)
        if rc == tlc.MOE_OK:
            close(y, want)
        else:
            assert detail > 0
            ws.buf[:tlc.MOE_FFN_STATUS_BYTES].zero_()
    y, _, _ = forward(cfg, x, W1, W3, W2, False, ws)
    close(y, want)
