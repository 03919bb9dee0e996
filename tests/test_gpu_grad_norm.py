"""Global gradient norm and clipping on the GPU against the 64-bit oracle.

Tolerances. A thread's 16 or 32 squares are added in fp32 in chains of at most 8 pairs, with errors of at most 2^-24
each: relative to the sum of these positive terms at most 10 * 2^-24, and half of that after the root. All later sums
keep at least 48 bits. norm and scale are then rounded to fp32: 6 * 2^-24 in all, 4e-7.
"""
import numpy as np
import pytest
import torch

import tile_level_copy_gb300 as tlc
from oracle import train_ref as ref
from tests.test_gpu_layernorm import f64, near

pytestmark = pytest.mark.gpu
F32, BF, F16 = torch.float32, torch.bfloat16, torch.float16
REL = 4e-7


def grads(sizes, types, seed=0, std=1e-2, shift=0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n + shift, generator=g) * std).to(types[i % len(types)]).cuda()[shift:] for i, n in enumerate(sizes)]


def run(gs, max_norm=1.0, eps=1e-6, ws=None, **kw):
    out, lst = torch.full((2,), float("nan"), device="cuda"), tlc.GradList(gs)
    tlc.grad_norm(tlc.GradNormConfig(max_norm, eps), lst, out, ws or tlc.GradNormWorkspace(), **kw)
    return out, lst


def check(gs, out, max_norm=1.0, eps=1e-6):
    norm, scale = ref.grad_norm([f64(g) for g in gs], max_norm, eps)
    np.testing.assert_allclose(f64(out), [norm, scale], rtol=REL, atol=0)


SIZES = [[1], [0, 5, 0], [8], [7, 9, 4097], [4096 * 4, 16384 * 3 + 5, 3], list(range(1, 120)), [1 << 20, 77] * 3, [333] * 2700]


@pytest.mark.parametrize("types", [(F32,), (BF,), (F16,), (BF, F32, F16)])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_norm_and_clipping(sizes, types, shift):
    gs = grads(sizes, types, len(sizes), shift=shift)
    ws = tlc.GradNormWorkspace()
    max_norm = 0.37 * ref.grad_norm([f64(g) for g in gs], 1.0, 0.0)[0]
    out, lst = run(gs, max_norm, ws=ws)
    check(gs, out, max_norm)
    assert torch.equal(run(gs, max_norm, ws=ws)[0], out)  # the workspace is ready again, sums repeat
    before = [g.clone() for g in gs]
    around = [g.storage_offset() and g._base[:shift].clone() for g in gs]
    tlc.grad_clip(lst, out[1:])
    s = f64(out)[1]
    for g, b in zip(gs, before):
        near(g, f64(b) * s, 2.0 ** -24 * np.abs(f64(b)))
    for g, a in zip(gs, around):  # what lies beside a tensor stays
        if shift:
            assert torch.equal(g._base[:shift], a)


def test_below_the_limit_the_gradients_stay():
    gs = grads([1000, 7], (BF,), 1)
    out, lst = run(gs, 1e3)
    assert out[1] == 1
    before = [g.clone() for g in gs]
    tlc.grad_clip(lst, out[1:])
    assert all(torch.equal(a, b) for a, b in zip(gs, before))
    check(gs, run(gs, float("inf"))[0], np.inf)


@pytest.mark.parametrize("size", [1e-30, 1e-22, 1e-15, 1.0, 1e15, 1e22, 1e30])
@pytest.mark.parametrize("dt", [F32, BF])
def test_every_size_that_fp32_holds(size, dt):
    """Squares beyond fp32's range at either end, alone and beside values of ordinary size."""
    gs = [(torch.randn(5000, generator=torch.Generator().manual_seed(1)) * size).to(dt).cuda()]
    check(gs, run(gs)[0])
    gs += [torch.randn(40000, generator=torch.Generator().manual_seed(2)).to(dt).cuda(), torch.zeros(9000, device="cuda")]
    check(gs, run(gs)[0])


def test_zeros_infinities_and_nan():
    z = [torch.zeros(10000, device="cuda"), torch.zeros(3, dtype=BF, device="cuda")]
    assert run(z)[0].tolist() == [0.0, 1.0]
    assert run([])[0].tolist() == [0.0, 1.0]
    z[0][777] = float("inf")
    out, lst = run(z)
    assert out.tolist() == [float("inf"), 0.0]
    tlc.grad_clip(lst, out[1:])
    assert torch.isnan(z[0][777]) and z[0].nan_to_num().eq(0).all()
    z[0][777] = float("nan")
    out, lst = run(z)
    assert torch.isnan(out).all()
    tlc.grad_clip(lst, out[1:])
    assert torch.isnan(z[0]).all() and torch.isnan(z[1]).all()


def test_long_list_of_equal_values():
    """2^27 values of 2^-10: the norm is sqrt(2^27 2^-20), which a plain fp32 sum of so many terms would miss."""
    g = torch.full((1 << 27,), 2.0 ** -10, dtype=BF, device="cuda")
    out, _ = run([g])
    assert abs(out[0].item() / 2.0 ** 3.5 - 1) <= REL


def test_more_values_than_32_bits_count():
    """A tensor of more than 2^32 values among short ones: 2^-10 each but for large ones at its ends."""
    n = 2 ** 32 + 12345
    g = [torch.ones(7, device="cuda"), torch.full((n + 1,), 2.0 ** -10, dtype=BF, device="cuda")[1:], torch.ones(9, dtype=F16, device="cuda")]
    g[1][0] = g[1][-1] = 64.0
    out, lst = run(g, max_norm=2.0)
    norm = np.sqrt(16 + (n - 2) * 2.0 ** -20 + 2 * 64.0 ** 2)
    assert abs(out[0].item() / norm - 1) <= REL and abs(out[1].item() / (2 / (norm + 1e-6)) - 1) <= REL
    tlc.grad_clip(lst, torch.full((1,), 0.5, device="cuda"))
    assert (g[0] == 0.5).all() and (g[2] == 0.5).all() and g[1][0] == 32 and g[1][-1] == 32
    lo, hi = g[1][1:-1].aminmax()
    assert lo == hi == 2.0 ** -11


def test_nothing_is_left_with_a_limit_of_zero():
    g = grads([100, 7], (F32, BF))
    out, lst = run(g, 0.0)
    assert out[0] > 0 and out[1] == 0
    tlc.grad_clip(lst, out[1:])
    assert not any(t.any() for t in g)


def test_stream_capture_and_adamw():
    """Norm, clipped step: captured together on a stream; adamw_step with grad_scale takes the step that clipped
    gradients give, up to the rounding of the clipped values (none in fp32 with a scale that is a power of two)."""
    gs = grads([5000, 300], (F32,), 3)
    norm = ref.grad_norm([f64(g) for g in gs], 1.0, 0.0)[0]
    cfg = tlc.AdamWConfig(lr=1e-3)
    p = [[torch.ones_like(g) for g in gs] for _ in range(2)]
    state = lambda: [torch.zeros_like(g) for g in gs]  # noqa: E731
    copies = [g.clone() for g in gs]
    lists = [tlc.AdamWList(cfg, p[0], gs, state(), state()), tlc.AdamWList(cfg, p[1], copies, state(), state())]
    out, gl, cl = torch.zeros(2, device="cuda"), tlc.GradList(gs), tlc.GradList(copies)
    ws, quarter = tlc.GradNormWorkspace(), torch.full((1,), 0.25, device="cuda")
    nc = tlc.GradNormConfig(norm / 3, 0.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tlc.grad_norm(nc, gl, out, ws)
        tlc.adamw_step(cfg, lists[0], 1, grad_scale=quarter)
        tlc.grad_clip(cl, quarter)
        tlc.adamw_step(cfg, lists[1], 1)
    graph.replay()
    torch.cuda.synchronize()
    check(gs, out, norm / 3, 0.0)
    assert all(torch.equal(a, b) for a, b in zip(*p))


def test_refusals():
    g = grads([100, 100], (F32,))
    for bad in ([g[0], g[0]], [g[0], g[0][50:]], [g[0].double()], [g[0].cpu()], [g[0][::2]], [g[0], g[1].to(torch.int32)]):
        with pytest.raises(ValueError):
            tlc.GradList(bad)
    lst, ws, out = tlc.GradList(g), tlc.GradNormWorkspace(), torch.empty(2, device="cuda")
    for cfg in (tlc.GradNormConfig(-0.5), tlc.GradNormConfig(float("nan")), tlc.GradNormConfig(1.0, -1.0), tlc.GradNormConfig(1.0, float("inf"))):
        with pytest.raises(tlc.MoEError) as e:
            tlc.grad_norm(cfg, lst, out, ws)
        assert e.value.code == tlc.MOE_ERR_ARG
    for o in (out.double(), out[:1], out.cpu()):
        with pytest.raises(ValueError):
            tlc.grad_norm(tlc.GradNormConfig(1.0), lst, o, ws)
    with pytest.raises(ValueError):
        tlc.grad_clip(lst, out)
    for call in (lambda: tlc.grad_clip(lst, g[1][99:]), lambda: tlc.grad_norm(tlc.GradNormConfig(1.0), lst, g[0][:2], ws)):
        with pytest.raises(tlc.MoEError) as e:  # the factor or the norm in a gradient
            call()
        assert e.value.code == tlc.MOE_ERR_ARG
