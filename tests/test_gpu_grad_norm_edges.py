"""Gradient norm and clipping where the formula ends: limits of zero and infinity, a factor of 1, sums that round one way."""
import pytest
import torch

import tile_level_copy_gb300 as tlc
from tests.test_gpu_grad_norm import REL, run

pytestmark = pytest.mark.gpu
F32, BF, F16 = torch.float32, torch.bfloat16, torch.float16
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("dt", [F32, BF, F16])
def test_an_infinite_limit_never_clips(dt):
    g = [torch.ones(1000, dtype=dt, device="cuda"), torch.ones(33, device="cuda")]
    g[0][123] = INF
    out, lst = run(g, INF)
    assert out.tolist() == [INF, 1.0]
    before = [t.clone() for t in g]
    tlc.grad_clip(lst, out[1:])
    assert all(torch.equal(a, b) for a, b in zip(g, before))
    out, _ = run(g, 1.0)
    assert out.tolist() == [INF, 0.0]
    g[1][5] = NAN
    assert torch.isnan(run(g, INF)[0]).all() and torch.isnan(run(g, 1.0)[0]).all()


@pytest.mark.parametrize("max_norm", [0.0, 1.0, INF])
def test_nothing_to_clip_without_eps(max_norm):
    """Norm and eps 0: there is nothing to scale, and the factor leaves it so."""
    z = [torch.zeros(5000, device="cuda"), torch.zeros(3, dtype=BF, device="cuda")]
    for gs in (z, [], [z[0][:0]]):
        out, lst = run(gs, max_norm, eps=0.0)
        assert out.tolist() == [0.0, 1.0]
        tlc.grad_clip(lst, out[1:])
    assert not any(t.any() for t in z)
    z[0][7] = 2.0
    out, lst = run(z, 0.0, eps=0.0)
    assert out.tolist() == [2.0, 0.0]


@pytest.mark.parametrize("dt", [F32, BF, F16])
@pytest.mark.parametrize("shift", [0, 1])
def test_a_factor_of_one_writes_nothing(dt, shift):
    """Every bit stays, those of a NaN among them (arithmetic would leave its own NaN)."""
    bits = torch.int32 if dt == F32 else torch.int16
    g = torch.randn(40001 + shift, device="cuda").to(dt)[shift:]
    quiet = torch.full((1,), NAN, dtype=dt).view(bits).item()
    g.view(bits)[::1000] = quiet | 0x5
    want, lst = g.view(bits).clone(), tlc.GradList([g])
    tlc.grad_clip(lst, torch.ones(1, device="cuda"))
    assert torch.equal(g.view(bits), want)
    tlc.grad_clip(lst, torch.full((1,), 0.5, device="cuda"))
    assert not torch.equal(g.view(bits), want)


@pytest.mark.parametrize("dt", [BF, F16])
@pytest.mark.parametrize("first", [1, 2, 4, 8])
def test_sums_that_round_one_way(dt, first):
    """Squares that are each just too small to change a sum that began with 1: what a chain of n additions loses is (n - 1)
    times 2^-24 of it. With the 64 squares of a thread's 128 bytes added in chains of 8 on each of 8 sums, 3 steps to add
    these up and one more rounding of each, the sum is off by at most 11 * 2^-24, the norm by half of that and its
    own rounding: 6.5 * 2^-24 < REL, whichever value of a piece is large."""
    n = 16384 * 5
    g = torch.full((n,), 2.0 ** -12 * (1 - 2.0 ** -7), dtype=dt, device="cuda").view(-1, 8)
    g.view(5, 8, 256, 8)[:, 0, :, :first] = 1.0           # the first piece of every thread
    g = g.view(-1)
    out, _ = run([g])
    norm = g.double().square().sum().sqrt().item()
    assert abs(out[0].item() / norm - 1) <= REL
