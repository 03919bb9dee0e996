"""Balance loss at logits of every size that fp32 holds, and log-sum-exps next to zero, on the GPU against the 64-bit oracle.

Tolerances, with u = 2^-24. Rows whose largest logit m is at most 1024 in magnitude have exponents (l - m) log2(e) off by one
rounding of them and one of the constant, and by what the row's m log2(e) is rounded by, which p does not see; beyond, l - m
is rounded once and its product once: with d = |l - m|, exp is off by less than 3 d u of itself. exp2 adds 4 u (2 units in the
last place), a sum of E <= 256 terms 13 u (a chain of 8 pairs and 5 steps), the inverse 4 u (as exp2), the product u: p is off by
(3 d + 24) u of itself. sum p a is off by the mean of that, with sum p d <= log 256, and by its own chain, 54 u in all; lse by
the rounding of m log2(e) and its own, 16 u; a and the last products by 10 u: a gradient's terms by (3 d + 104) u. Losses
are sums of positive terms: relative error 2e-5 allows 300 roundings of each.
"""
import numpy as np
import pytest
import torch

import tile_level_copy_gb300 as tlc
from tests.test_gpu_balance import make, oracle, run
from tests.test_gpu_layernorm import f64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def rows_at(v, E, g):
    """Rows whose largest logit has the size of v."""
    n = lambda: torch.randn(E, generator=g)  # noqa: E731
    ulp = float(np.spacing(np.float32(abs(v))))
    peak = n()
    peak[E // 2] = v                                        # one expert far above the others, or far below them
    some = torch.full((E,), 4.0 * v if v < 0 else -v)
    some[: (E + 1) // 2] = v                                # half of the experts masked by a finite value
    return torch.stack([torch.full((E,), v), v + n(), v + ulp * torch.arange(E).float(), peak, some])


SIZES = [1e2, 1023.0, 1025.0, 65504.0, 1e6, 1e9, 3e9, 1e10, 1e15, 1e20, 1e30, 4e37, 8.4e37]


@pytest.mark.parametrize("E", [1, 3, 16, 60, 64, 128, 200, 256])
@pytest.mark.parametrize("v", [s * x for x in SIZES for s in (1, -1)])
def test_rows_of_every_size(v, E):
    T, k = 64, min(E, 2)
    t = make(T, E, k, 1, drop=False, seed=E)
    rows = rows_at(v, E, torch.Generator().manual_seed(1)).cuda()
    t["logits"][:5], t["logits"][7:12], t["logits"][40:45] = rows, rows, rows
    t["mask"][:5], t["mask"][40:45] = 1, 0
    cfg = tlc.BalanceConfig(T, E, k, balance=0.3, z=0.02 if abs(v) < 1e16 else 0.0)  # (lse^2 has to stay in fp32)
    got = run(cfg, t)
    (loss, counts, lse, dl), _, mask, up, wb, wz = oracle(cfg, t)
    assert np.isfinite(lse).all()
    assert np.array_equal(got[1].cpu().numpy(), counts)
    n = 3 if wz else 2
    if wz:
        np.testing.assert_allclose(f64(got[0])[:n], loss[:n], rtol=2e-5, atol=0)
    else:
        np.testing.assert_allclose(f64(got[0])[:n], [wb * loss[1], loss[1]], rtol=2e-5, atol=0)
    l = f64(t["logits"])
    assert (np.abs(f64(got[2]) - lse) <= 16 * U * (1 + np.abs(lse) + np.abs(l.max(1)))).all()
    p, N = np.exp(l - lse[:, None]), (mask != 0).sum()
    slope = counts.max() * E / (k * N * N)
    size = up * p * (2 * wb * slope + 2 * wz * np.abs(lse)[:, None] / N)
    err = (3 * np.minimum(l.max(1, keepdims=True) - l, 100) + 110) * U * size + 16 * U * k * np.abs(f64(t["dgates"])).max(1, keepdims=True)
    g = f64(got[3])
    assert np.isfinite(g).all() and (np.abs(g - dl) <= err + 1e-20).all(), (np.abs(g - dl) / (err + 1e-20)).max()


def test_a_batch_of_masked_rows_alone():
    """Experts that are all filled with one finite value: every probability 1 / E, the loss E / k times a load's mean."""
    T, E, k = 300, 64, 6
    for v in (-1e9, -1e10, -1e30, torch.finfo(torch.float32).min, 1e30):
        t = make(T, E, k, 1, mask=False, drop=False, seed=2)
        t["logits"].fill_(v)
        t["dloss"] = None
        cfg = tlc.BalanceConfig(T, E, k, balance=1.0, z=0.0)
        loss, counts, lse, dl = run(cfg, t, gates=False)
        assert counts.sum().item() == T * k and abs(loss[0].item() - 1) <= 2e-5 and loss[0] == loss[1]
        assert (lse.double() - v).abs().max() <= np.log(E) + 2 * U * abs(v)
        a = counts.double() * E / (k * T ** 2)
        assert (dl.double() - (a - a.mean()) / E).abs().max() <= 128 * U * 2 * a.max() / E


@pytest.mark.parametrize("E", [2, 3, 64, 256])
def test_log_sum_exps_next_to_zero(E):
    """Largest logit 0, the others x below: lse = log(1 + q), q = sum of exp(-x). exp is off by (1.5 x + 4) u of itself (its
    argument by two roundings, of the constant and of the product, at most 1.5 x u together), the sum 1 + q by u for each of its
    n <= 13 additions, the logarithm by one unit in its last place, 2 u: u ((1.5 x + 4) q / (1 + q) + n + 2 lse) in all."""
    T, g = 4096, torch.Generator().manual_seed(E)
    x = 16 * torch.rand(T, 1, generator=g)
    logits = (-x).expand(T, E).clone()
    at = torch.randint(0, E, (T,), generator=g)
    logits[torch.arange(T), at] = 0
    t = {"logits": logits.cuda(), "idx": at[:, None].to(torch.int32).cuda(), "offsets": None, "mask": None, "dloss": None}
    got = f64(run(tlc.BalanceConfig(T, E, 1, balance=0.0, z=1.0), t, gates=False)[2])
    x = f64(x)[:, 0]
    q = (E - 1) * np.exp(-x)
    want = np.log1p(q)
    err = U * ((1.5 * x + 4) * q / (1 + q) + min(E - 1, 13) + 2 * want)
    assert (np.abs(got - want) <= err).all(), (np.abs(got - want) / err).max()


def test_the_z_loss_gradient_next_to_zero():
    """2 lse p / T, with lse as above and p off by (1.5 x + 10) u of itself: two experts, so one addition in the sum."""
    T, g = 4096, torch.Generator().manual_seed(1)
    x = 16 * torch.rand(T, 1, generator=g)
    logits = torch.cat([torch.zeros(T, 1), -x], 1).cuda()
    t = {"logits": logits, "idx": torch.zeros(T, 1, dtype=torch.int32, device="cuda"), "offsets": None, "mask": None, "dloss": None}
    got = f64(run(tlc.BalanceConfig(T, 2, 1, balance=0.0, z=1.0), t, gates=False)[3])
    x = f64(x)
    q = np.exp(-x)
    lse, p = np.log1p(q), np.concatenate([1 / (1 + q), q / (1 + q)], 1)
    err = U * p * ((1.5 * x + 4) * q / (1 + q) + 1 + 2 * lse + (1.5 * x + 12) * lse) * 2 / T
    want = 2 * lse * p / T
    assert (np.abs(got - want) <= err).all(), (np.abs(got - want) / err).max()
