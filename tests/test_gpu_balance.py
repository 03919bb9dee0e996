"""Balance loss, loads and the router's gradient on the GPU against the 64-bit oracle.

Tolerances. exp's argument is a difference rounded once (2^-24 of at most 40) and exp2f is off by 2 units in the last
place, so a probability is off by less than 48 * 2^-24 of itself; sums of n positive terms add at most 2^-24 each
for the longest chain of additions, which is short (a lane's tokens of a sequence, 8 warps, CTAs). The losses are
sums of positive terms: relative error 2e-5 allows 300 roundings. lse is off by 2^-24 of itself and of its parts.
A gradient's error is relative to its terms: p (a + sum p a), the z loss's and the gates' parts.
"""
import numpy as np
import pytest
import torch

import tile_level_copy_gb300 as tlc
from oracle import train_ref as ref
from tests.test_gpu_layernorm import f64

pytestmark = pytest.mark.gpu
F32, I32, U8 = torch.float32, torch.int32, torch.uint8
ULP = 2.0 ** -24


def make(T, E, k, S, mask=True, drop=True, seed=0, lean=1.0):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, E, generator=g) - lean * torch.log(torch.arange(1, E + 1.0))
    top, idx = torch.topk(logits, k, dim=1)
    if drop and T:
        idx = torch.where(torch.rand(T, k, generator=g) < 0.1, torch.randint(-3, 0, (T, k), generator=g), idx)
        idx[0, 0] = E  # beyond the last
    offsets = None
    if S > 1:
        cut = torch.randint(0, T + 1, (S,), generator=g).sort().values
        offsets = torch.cat([cut[:1] // 2, cut]).to(I32).cuda()
    m = (torch.rand(T, generator=g) > 0.2).to(U8).cuda() if mask else None
    return {"logits": logits.cuda(), "idx": idx.to(I32).cuda(), "gates": torch.softmax(top, 1).cuda(), "offsets": offsets, "mask": m,
            "dgates": (torch.randn(T, k, generator=g) * 1e-2).cuda(), "dloss": torch.full((1,), 0.5, device="cuda")}


def run(cfg, t, gates=True, dlogits=None, ws=None, **kw):
    loss, counts = torch.full((3,), float("nan"), device="cuda"), torch.full((cfg.seqs, cfg.E), -1, dtype=I32, device="cuda")
    lse, saved = torch.full((cfg.T,), float("nan"), device="cuda"), tlc.balance_saved(cfg)
    dl = torch.full_like(t["logits"], float("nan")) if dlogits is None else dlogits
    if kw:  # on another stream: what was filled here is ready
        torch.cuda.synchronize()
    tlc.balance_forward(cfg, t["logits"], t["idx"], loss, counts, lse, ws or tlc.BalanceWorkspace(cfg), offsets=t["offsets"],
                        mask=t["mask"], saved=saved, **kw)
    tlc.balance_backward(cfg, t["logits"], t["idx"], saved, dl, offsets=t["offsets"], mask=t["mask"],
                         gates=t["gates"] if gates else None, dgates=t["dgates"] if gates else None, dloss=t["dloss"], **kw)
    return loss, counts, lse, dl


def oracle(cfg, t, gates=True):
    off = np.array([0, cfg.T]) if t["offsets"] is None else t["offsets"].cpu().numpy()
    mask = np.ones(cfg.T) if t["mask"] is None else t["mask"].cpu().numpy()
    g = (f64(t["gates"]), f64(t["dgates"])) if gates else (None, None)
    wb, wz = float(np.float32(cfg.balance)), float(np.float32(cfg.z))
    up = 1.0 if t["dloss"] is None else t["dloss"].item()
    return ref.balance(f64(t["logits"]), t["idx"].cpu().numpy(), off, mask, wb, wz, up, *g), off, mask, up, wb, wz


def check(cfg, t, got, gates=True):
    (loss, counts, lse, dl), off, mask, up, wb, wz = oracle(cfg, t, gates)
    with np.errstate(over="ignore"):  # lse of logits at the type's lowest value squared is beyond fp32
        np.testing.assert_allclose(f64(got[0]), loss.astype(np.float32), rtol=2e-5, atol=0)
    assert np.array_equal(got[1].cpu().numpy(), counts)
    l = f64(t["logits"])
    fin = np.isfinite(lse)
    assert (np.abs(f64(got[2])[fin] - lse[fin]) <= 16 * ULP * (1 + np.abs(lse[fin]) + np.abs(l[fin]).max(1, initial=0))).all()
    # a row's terms: p times the slopes' and the z loss's parts; the gates' parts
    p = np.exp(l - np.where(fin, lse, 0)[:, None])
    n = np.array([max(1, (mask[a:b] != 0).sum()) for a, b in zip(off, off[1:])])
    slope = (counts.max(1, initial=0) * cfg.E / (cfg.topk * n * n)).max(initial=0)
    size = up * p * (2 * wb * slope + 2 * wz * np.abs(np.where(fin, lse, 0))[:, None] / max(1, n.sum() - (n == 1).sum()))
    err = 128 * ULP * size
    if gates:
        err = err + 16 * ULP * (np.abs(f64(t["dgates"])).max(1, initial=0, keepdims=True) * cfg.topk)
    g = f64(got[3])
    assert (np.abs(g - dl) <= err + 1e-30).all(), (np.abs(g - dl) / (err + 1e-30)).max()
    assert not g[dl.any(1) == 0].any()


SHAPES = [(1, 1, 1, 1), (1, 8, 2, 1), (3, 4, 4, 2), (37, 64, 6, 1), (256, 8, 2, 3), (509, 60, 6, 7), (1000, 16, 2, 1), (777, 13, 8, 5),
          (4096, 64, 8, 1), (3001, 256, 8, 11), (5000, 128, 3, 40), (20000, 255, 8, 1), (300, 33, 5, 100), (9000, 2, 1, 3)]


@pytest.mark.parametrize("mask", [False, True])
@pytest.mark.parametrize("T,E,k,S", SHAPES)
def test_losses_loads_and_gradient(T, E, k, S, mask):
    t = make(T, E, k, S, mask=mask, drop=mask, seed=T + E)
    cfg = tlc.BalanceConfig(T, E, k, S, balance=0.3, z=0.02)
    got = run(cfg, t)
    check(cfg, t, got)
    again = run(cfg, t)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    t["dloss"] = None
    check(cfg, t, run(cfg, t, gates=False), gates=False)


def test_no_tokens_and_only_padding():
    for T, S in ((0, 1), (0, 4), (50, 4)):
        t = make(T, 8, 2, S, seed=1)
        if S > 1:
            t["offsets"] = torch.zeros(S + 1, dtype=I32, device="cuda")
        else:
            t["mask"] = torch.zeros(T, dtype=U8, device="cuda")
        cfg = tlc.BalanceConfig(T, 8, 2, S, z=1.0)
        loss, counts, lse, dl = run(cfg, t)
        assert not loss.any() and not counts.any() and not dl.any() and torch.isfinite(lse).all()


def test_hard_logits():
    """Masked experts (-inf, the lowest fp32 value), rows that leave nothing, logits of equal and of far values."""
    T, E, k = 40, 16, 2
    t = make(T, E, k, 1, mask=False, drop=False, seed=3)
    l = t["logits"]
    low = torch.finfo(F32).min
    l[0, 3:] = -float("inf")
    l[1, 3:] = low
    l[2] = low
    l[3] = -float("inf")  # padding
    l[4] = 5.0
    l[5, 0] = 80.0
    l[6] -= 300.0
    l[7] += 300.0
    cfg = tlc.BalanceConfig(T, E, k, balance=0.3, z=0.0)
    got = run(cfg, t)
    check(cfg, t, got)
    assert got[2][3] == -float("inf") and not got[3][3].any()
    assert got[1].sum().item() == (T - 1) * k


def test_nan_stays_in_its_row_of_the_gradient():
    t = make(100, 16, 2, 1, mask=False, drop=False, seed=4)
    cfg = tlc.BalanceConfig(100, 16, 2, balance=0.3, z=0.1)
    want = run(cfg, t)[3]
    t["mask"] = torch.ones(100, dtype=U8, device="cuda")
    t["mask"][7] = 0
    clean = run(cfg, t)
    t["logits"][7] = float("nan")  # in padding: nowhere
    got = run(cfg, t)
    assert torch.equal(got[0], clean[0]) and torch.equal(got[3], clean[3]) and torch.equal(got[1], clean[1])
    t["mask"] = None
    loss, _, _, dl = run(cfg, t)
    assert torch.isnan(loss[0]) and torch.isnan(dl[7]).all() and want.shape == dl.shape


def test_an_expert_chosen_twice():
    t = make(64, 8, 3, 1, mask=False, drop=False, seed=5)
    t["idx"][:, 1] = t["idx"][:, 0]
    t["idx"][::2, 2] = t["idx"][::2, 0]
    cfg = tlc.BalanceConfig(64, 8, 3, balance=0.3, z=0.1)
    check(cfg, t, run(cfg, t))


def test_in_place_unaligned_stream_and_workspace_in_turn():
    t = make(333, 64, 6, 3, seed=6)
    cfg = tlc.BalanceConfig(333, 64, 6, 3, balance=0.3, z=0.1)
    ws = tlc.BalanceWorkspace(cfg)
    want = run(cfg, t, ws=ws)
    st = torch.cuda.Stream()
    shift = lambda v: torch.cat([v.flatten()[:1], v.flatten()])[1:].view(v.shape)  # noqa: E731
    s = {**t, "logits": shift(t["logits"]), "idx": shift(t["idx"]), "gates": shift(t["gates"]), "dgates": shift(t["dgates"])}
    assert s["logits"].data_ptr() % 16
    got = run(cfg, s, stream=st, dlogits=s["logits"].clone())
    st.synchronize()
    check(cfg, t, got)
    c = {**t, "logits": t["logits"].clone()}
    assert torch.equal(run(cfg, c, dlogits=c["logits"], ws=ws)[3], want[3])


def test_offsets_that_are_out_of_range_stay_inside():
    """Offsets beyond [0, T] are clamped, decreasing ones leave their sequence empty: the results are those of some
    sequences, and nothing outside of the buffers is touched."""
    T, E, k = 700, 32, 2
    t = make(T, E, k, 4, mask=False, drop=False, seed=7)
    cfg = tlc.BalanceConfig(T, E, k, 4)
    t["offsets"] = torch.tensor([-5, 100, 100, 600, 1 << 30], dtype=I32, device="cuda")
    a = run(cfg, t)
    t["offsets"] = torch.tensor([0, 100, 100, 600, T], dtype=I32, device="cuda")
    b = run(cfg, t)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_many_empty_sequences():
    """A few tokens' sequences among 200000 empty ones, in which a CTA's next sequence is found by a search."""
    T, E, k, S = 5000, 16, 2, 200000
    t = make(T, E, k, 1, seed=11)
    cut = torch.zeros(S + 1, dtype=I32)
    cut[50000:], cut[120000:], cut[120001:], cut[199999:] = 1000, 1003, 4000, T
    t["offsets"] = cut.cuda()
    cfg = tlc.BalanceConfig(T, E, k, S, balance=0.3, z=0.1)
    got = run(cfg, t)
    few = {**t, "offsets": torch.tensor([0, 1000, 1003, 4000, T], dtype=I32, device="cuda")}
    want = run(tlc.BalanceConfig(T, E, k, 4, balance=0.3, z=0.1), few)
    where = torch.tensor([49999, 119999, 120000, 199998], device="cuda")
    assert torch.equal(got[1][where], want[1]) and got[1].sum() == want[1].sum() and torch.equal(got[2], want[2])
    check(tlc.BalanceConfig(T, E, k, 4, balance=0.3, z=0.1), few, (got[0], got[1][where], *got[2:]))


def test_more_values_than_32_bits_count():
    """The last tokens' logits lie beyond value 2^31."""
    T, E, k = 2 ** 23 + 1001, 256, 2
    cfg, end = tlc.BalanceConfig(T, E, k, balance=0.3, z=0.1), slice(T - 2000, T)
    logits = torch.empty(T, E, device="cuda").normal_()
    idx = torch.randint(0, E, (T, k), device="cuda", dtype=I32)
    loss, counts = torch.empty(3, device="cuda"), torch.empty(1, E, dtype=I32, device="cuda")
    lse, saved = torch.empty(T, device="cuda"), tlc.balance_saved(cfg)
    tlc.balance_forward(cfg, logits, idx, loss, counts, lse, tlc.BalanceWorkspace(cfg), saved=saved)
    c = torch.bincount(idx.flatten(), minlength=E)
    assert torch.equal(counts[0].long(), c)
    l = logits[end].double()
    p, want = torch.softmax(l, 1), torch.logsumexp(l, 1)
    assert ((lse[end] - want).abs() <= 16 * ULP * (1 + want.abs() + l.abs().amax(1))).all()
    tlc.balance_backward(cfg, logits, idx, saved, logits)
    a = 0.3 * E / (k * T ** 2) * c.double()
    dl = p * (a - (p * a).sum(1, keepdim=True) + 0.2 / T * want[:, None])
    assert ((logits[end] - dl).abs() <= 128 * ULP * p * (2 * a.max() + 0.2 / T * want.abs()[:, None])).all()


def test_captured_and_replayed():
    t = make(2000, 64, 6, 5, seed=8)
    cfg = tlc.BalanceConfig(2000, 64, 6, 5, balance=0.3, z=0.1)
    want = run(cfg, t)
    ws, saved = tlc.BalanceWorkspace(cfg), tlc.balance_saved(cfg)
    out = [torch.zeros_like(v) for v in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tlc.balance_forward(cfg, t["logits"], t["idx"], out[0], out[1], out[2], ws, offsets=t["offsets"], mask=t["mask"], saved=saved)
        tlc.balance_backward(cfg, t["logits"], t["idx"], saved, out[3], offsets=t["offsets"], mask=t["mask"], gates=t["gates"],
                             dgates=t["dgates"], dloss=t["dloss"])
    for _ in range(3):
        for o in out:
            o.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_with_the_routers_plan():
    """idx and gates as moe_plan gives them: the loads are those that it lays its rows out by."""
    T, E, k, R = 256, 8, 2, 2
    logits = torch.randn(T, E, generator=torch.Generator().manual_seed(9)).cuda()
    cfg = tlc.Config(T=T, d=128, ffn=128, E=E, topk=k, R=R, tile_M=64, flags=tlc.MOE_PLAN_SKIP_PERMUTE)
    ws = tlc.Workspace(cfg)
    idx, gates = torch.empty(T, k, dtype=I32, device="cuda"), torch.empty(T, k, device="cuda")
    tlc.plan(cfg, logits, None, ws, idx, gates)
    t = {"logits": logits, "idx": idx, "gates": gates, "offsets": None, "mask": None, "dgates": torch.randn(T, k, device="cuda"),
         "dloss": None}
    bc = tlc.BalanceConfig(T, E, k, balance=0.01, z=0.001)
    got = run(bc, t)
    check(bc, t, got)
    assert torch.equal(got[1][0], ws.view("counts").sum(1).to(I32))


def test_refusals():
    t = make(100, 8, 2, 3, seed=10)
    cfg = tlc.BalanceConfig(100, 8, 2, 3)
    loss, counts, lse, ws = torch.empty(3, device="cuda"), torch.empty(3, 8, dtype=I32, device="cuda"), None, tlc.BalanceWorkspace(cfg)
    small = torch.empty(16, dtype=U8, device="cuda")
    with pytest.raises(ValueError, match="needs"):
        tlc.balance_forward(cfg, t["logits"], t["idx"], loss, counts, lse, ws, offsets=t["offsets"], saved=small)
    with pytest.raises(ValueError, match="needs"):
        tlc.balance_backward(cfg, t["logits"], t["idx"], small, t["logits"], offsets=t["offsets"])
    with pytest.raises(tlc.MoEError) as e:  # several sequences without offsets
        tlc.balance_forward(cfg, t["logits"], t["idx"], loss, counts, lse, ws)
    assert e.value.code == tlc.MOE_ERR_ARG
    with pytest.raises(tlc.MoEError) as e:  # gates without their gradients
        tlc.balance_backward(cfg, t["logits"], t["idx"], tlc.balance_saved(cfg), t["logits"], offsets=t["offsets"], gates=t["gates"])
    assert e.value.code == tlc.MOE_ERR_ARG
    wide = torch.empty(101, 8, device="cuda")
    with pytest.raises(tlc.MoEError) as e:  # dlogits a row beside logits
        tlc.balance_backward(cfg, wide[:100], t["idx"], tlc.balance_saved(cfg), wide[1:], offsets=t["offsets"])
    assert e.value.code == tlc.MOE_ERR_ARG
    ws.nbytes = 64
    with pytest.raises(tlc.MoEError) as e:
        tlc.balance_forward(cfg, t["logits"], t["idx"], loss, counts, lse, ws, offsets=t["offsets"])
    assert e.value.code == tlc.MOE_ERR_WORKSPACE
