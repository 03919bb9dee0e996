"""Norms around a block with its gate and the residual sum on the GPU against the 64-bit oracle.

Tolerances. Each value is computed in fp32 from the inputs by at most about ten roundings of 2^-24, the sums of a row by
trees over at most 64 sequential values a thread, 32 lanes and 16 warps: with errors of random sign a sum is off by less
than 16 * 2^-24 of its terms' size. The result, a rounding to the outputs' type, lies between the roundings of
the oracle's value minus and plus that. The sizes that the errors are relative to stand beside each check.
"""
import itertools

import numpy as np
import pytest
import torch

import tile_level_copy_gb300 as tlc
from oracle import train_ref as ref
from tests.test_gpu_layernorm import f64, near

pytestmark = pytest.mark.gpu
F32, BF, F16 = torch.float32, torch.bfloat16, torch.float16
KIND = {"none": tlc.MOE_NORM_NONE, "rms": tlc.MOE_NORM_RMS, "layer": tlc.MOE_NORM_LAYER}
ULP = 2.0 ** -24
EPS, RES, BRANCH = 1e-5, 0.75, 0.375
WEIGHTS = ("post_w", "post_b", "gate", "pre_w", "pre_b")


def make(rows, d, dt, wt, post, pre, gate_rows, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    t = {"x": (r(rows, d) * 1.5 + 0.25).to(dt), "u": (r(rows, d) * 0.7 + 0.1).to(dt), "dz": (r(rows, d) * 0.1).to(dt),
         "dh": (r(rows, d) * 0.1).to(dt), "post_w": (r(d) * 0.1 + 1).to(wt), "post_b": (r(d) * 0.1).to(wt),
         "pre_w": (r(d) * 0.1 + 1).to(wt), "pre_b": (r(d) * 0.1).to(wt),
         "gate": (r(-(-rows // max(gate_rows, 1)), d) * 0.3 + 0.8).to(wt)}
    t = {n: v.cuda() for n, v in t.items()}
    for n, there in (("post_w", post != "none"), ("post_b", post == "layer"), ("pre_w", pre != "none"),
                     ("pre_b", pre == "layer"), ("gate", gate_rows > 0), ("dz", pre != "none")):
        if not there:
            t[n] = None
    return t


def config(rows, d, dt, wt, post, pre, gate_rows, **kw):
    return tlc.ResidualNormConfig(rows, d, dt, wt, KIND[post], KIND[pre], gate_rows, **{**dict(eps=EPS, residual_scale=RES,
                                                                                              branch_scale=BRANCH), **kw})


def num(t, none):
    return none if t is None else f64(t)


def nan_like(t):
    return None if t is None else torch.full_like(t, float("nan"))


def forward(cfg, t, h=None, z=None, **kw):
    h = nan_like(t["x"]) if h is None else h
    z = (nan_like(t["x"]) if z is None else z) if cfg.pre else None
    stats = [torch.full((cfg.rows, 2), float("nan"), device="cuda") if k else None for k in (cfg.post, cfg.pre)]
    if kw:  # on another stream: what was filled here is ready
        torch.cuda.synchronize()
    tlc.residual_norm_forward(cfg, t["x"], t["u"], t["post_w"], t["post_b"], t["gate"], t["pre_w"], t["pre_b"], h, z, *stats, **kw)
    return h, z, stats


def check_stats(got, x, kind, want):
    got, amp = f64(got), (np.abs(x).max(1) * want[:, 1]) ** 2
    if kind == "layer":
        assert (np.abs(got[:, 0] - want[:, 0]) <= 16 * ULP * np.abs(x).max(1)).all()
    else:
        assert (got[:, 0] == 0).all()
        amp = 1
    # the variance is off by 2^-24 of the values' squares, relative to var + eps
    assert (np.abs(got[:, 1] / want[:, 1] - 1) <= 16 * ULP * (1 + amp)).all()
    return np.broadcast_to(amp, (len(x),))[:, None]


def check_forward(cfg, t, post, pre, h, z, stats):
    eps = float(np.float32(cfg.eps))
    x, u = f64(t["x"]), num(t["u"], None)
    w, b, gate = num(t["post_w"], 1.0), num(t["post_b"], 0.0), num(t["gate"], None)
    a, c = float(np.float32(cfg.residual_scale)), float(np.float32(cfg.branch_scale))
    want, st = ref.residual_norm_h(x, u, post, w, b, gate, cfg.gate_rows, a, c, eps)
    amp = 0 if st is None else check_stats(stats[0], u, post, st)
    v = 0 if u is None else np.abs(u) if st is None else np.abs(ref.normed(u, st) * w) + np.abs(b) + np.abs(st[:, 1:] * st[:, :1] * w)
    size = np.abs(a * x) + np.abs(c * ref.per_row(gate, len(x), cfg.gate_rows)) * v
    near(h, want, 32 * ULP * size * (1 + amp))
    if pre != "none":
        h64 = f64(h)  # the norm of h as it is stored
        st = ref.norm_stats(h64, pre, eps)
        amp = check_stats(stats[1], h64, pre, st)
        w, b = num(t["pre_w"], 1.0), num(t["pre_b"], 0.0)
        near(z, ref.normed(h64, st) * w + b,
             32 * ULP * (np.abs(ref.normed(h64, st) * w) + np.abs(b) + np.abs(st[:, 1:] * st[:, :1] * w)) * (1 + amp))


def backward(cfg, t, h, stats, dx=None, du=None, ws=True, want=WEIGHTS):
    dx, du = (nan_like(t["u"]) if o is None else o for o in (dx, du))
    grads = [nan_like(t[n]) if n in want else None for n in WEIGHTS]
    tlc.residual_norm_backward(cfg, t["dz"], t["dh"], t["u"], h, t["post_w"], t["post_b"], t["gate"], t["pre_w"], *stats, dx, du,
                               *grads, tlc.ResidualNormWorkspace(cfg) if ws else None)
    return dx, du, grads


def check_backward(cfg, t, post, pre, h, stats, dx, du, grads):
    rows, d = cfg.rows, cfg.d
    a, c = float(np.float32(cfg.residual_scale)), float(np.float32(cfg.branch_scale))
    ps, qs = (None if s is None else f64(s) for s in stats)
    w, b, gate, pw = num(t["post_w"], 1.0), num(t["post_b"], 0.0), num(t["gate"], None), num(t["pre_w"], 1.0)
    dz, dh, u, h = num(t["dz"], None), num(t["dh"], None), f64(t["u"]), f64(h)
    want = ref.residual_norm_backward(dz, dh, u, h, post, w, b, gate, cfg.gate_rows, pre, pw, ps, qs, a, c)
    # dt's terms: dh, rstd dz w2 and its projections, each at most the row's largest times |hn|
    top = lambda v: np.abs(v).max(1, keepdims=True)  # noqa: E731
    e, hn = (0.0 if dh is None else top(dh)), 0.0
    if pre != "none":
        hn = np.abs(ref.normed(h, qs)) + np.abs(qs[:, :1] * qs[:, 1:])
        e = e + qs[:, 1:] * top(dz * pw) * (1 + top(hn))
        e = e * (1 + hn)
    err = 64 * ULP * e                                     # of dt
    near(dx, want[0], np.abs(a) * err + ULP * np.abs(want[0]))
    k = c * ref.per_row(gate, rows, cfg.gate_rows) * (w if post != "none" else 1.0)
    un = np.abs(u)
    if post == "none":
        near(du, want[1], 2 * np.abs(k) * err + 4 * ULP * np.abs(want[1]))
    else:
        un = np.abs(ref.normed(u, ps)) + np.abs(ps[:, :1] * ps[:, 1:])
        near(du, want[1], 2 * ps[:, 1:] * top(k) * top(np.broadcast_to(err, u.shape)) * (1 + un) * (1 + top(un)))
    # sums over the rows: terms with the errors above, and the adding, whose errors of random sign grow with the root
    # of the number of terms; some 2 sqrt(rows) roundings of the terms' 2-norm
    terms = {"post_w": k / np.where(w == 0, 1, w) * e * un, "post_b": k / np.where(w == 0, 1, w) * e,
             "gate": c * e * (un * np.abs(w) + np.abs(b)), "pre_w": 0.0, "pre_b": 0.0}
    if pre != "none":
        terms.update(pre_w=dz * hn, pre_b=dz)
    for n, got, wt in zip(WEIGHTS, grads, want[2:]):
        if got is None:
            continue
        x = np.abs(np.broadcast_to(terms[n], (rows, d)))
        if n == "gate":
            g = cfg.gate_rows
            size = np.stack([np.sqrt((x[i:i + g] ** 2).sum(0)) for i in range(0, rows, g)])
        else:
            size = np.sqrt((x ** 2).sum(0))
        near(got, wt.reshape(got.shape), ULP * (64 + 4 * np.sqrt(rows)) * size.reshape(got.shape))


KINDS = list(itertools.product(["none", "rms", "layer"], repeat=2))
SHAPES = [(1, 1), (3, 8), (5, 7), (33, 104), (70, 128), (41, 513), (130, 1000), (129, 1003), (7, 2048), (300, 2056), (21, 4099),
          (31, 8192), (5, 8200), (9, 16384), (6, 16383), (700, 768)]
TYPES = [(BF, BF), (BF, F32), (F16, F16), (F32, F32)]


@pytest.mark.parametrize("dt,wt", TYPES)
@pytest.mark.parametrize("rows,d", SHAPES)
def test_forward_and_backward(rows, d, dt, wt):
    """Every pair of kinds, with a gate for all rows, for groups of them (a ragged last one) or none."""
    for i, (post, pre) in enumerate(KINDS):
        gate_rows = (0, rows, max(1, rows // 3), min(2, rows), 1)[(i + d) % 5]
        t = make(rows, d, dt, wt, post, pre, gate_rows, rows + d + i)
        if i % 3 == 2 and pre != "none":
            t["dh"] = None
        cfg = config(rows, d, dt, wt, post, pre, gate_rows)
        h, z, stats = forward(cfg, t)
        check_forward(cfg, t, post, pre, h, z, stats)
        out = backward(cfg, t, h, stats)
        check_backward(cfg, t, post, pre, h, stats, *out)
        again = backward(cfg, t, h, stats)
        assert all(a is None or torch.equal(a, b) for a, b in zip((*out[:2], *out[2]), (*again[:2], *again[2])))


@pytest.mark.parametrize("gate_rows", [1, 2, 3, 7, 64, 500, 999, 1000, 5000])
@pytest.mark.parametrize("d", [64, 1000, 1001])
@pytest.mark.parametrize("post", ["none", "layer"])
def test_gates_of_groups(post, d, gate_rows):
    """Groups that end inside a group of warps' rows, that span several, and a last one that is ragged."""
    rows = 1000 if gate_rows != 5000 else 2003
    t = make(rows, d, BF, F32, post, "rms", gate_rows, d + gate_rows)
    cfg = config(rows, d, BF, F32, post, "rms", gate_rows)
    h, z, stats = forward(cfg, t)
    check_forward(cfg, t, post, "rms", h, z, stats)
    check_backward(cfg, t, post, "rms", h, stats, *backward(cfg, t, h, stats))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("d", [1000, 777])
def test_in_place_and_optional(dt, d):
    rows = 37
    t = make(rows, d, dt, F32, "layer", "layer", rows, 3)
    cfg = config(rows, d, dt, F32, "layer", "layer", rows)
    h, z, stats = forward(cfg, t)
    dx, du, grads = backward(cfg, t, h, stats)
    for a, b in (("x", "u"), ("u", "x")):
        c = {**t, "x": t["x"].clone(), "u": t["u"].clone()}
        h2, z2, _ = forward(cfg, c, h=c[a], z=c[b])
        assert torch.equal(h2, h) and torch.equal(z2, z)
    for a, b in itertools.permutations(("dz", "dh", "u", "h"), 2):
        c = {n: None if v is None else v.clone() for n, v in {**t, "h": h}.items()}
        dx2, du2, g2 = backward(cfg, c, c["h"], stats, dx=c[a], du=c[b])
        assert torch.equal(dx2, dx) and torch.equal(du2, du) and all(torch.equal(x, y) for x, y in zip(grads, g2))
    # without the gradients that nobody wants
    dx2, du2, _ = backward(cfg, t, h, stats, ws=False, want=())
    assert torch.equal(dx2, dx) and torch.equal(du2, du)
    _, _, g2 = backward(cfg, t, h, stats, want=("gate", "pre_b"))
    assert torch.equal(g2[2], grads[2]) and torch.equal(g2[4], grads[4])
    dx2 = torch.empty_like(dx)
    tlc.residual_norm_backward(cfg, t["dz"], t["dh"], t["u"], h, t["post_w"], t["post_b"], t["gate"], t["pre_w"], *stats, dx2, None)
    assert torch.equal(dx2, dx)
    # statistics and h that nobody wants; weights of 1 and biases of 0
    z2 = nan_like(z)
    tlc.residual_norm_forward(cfg, t["x"], t["u"], t["post_w"], t["post_b"], t["gate"], t["pre_w"], t["pre_b"], None, z2)
    assert torch.equal(z2, z)
    one = {**t, "post_w": torch.ones(d, device="cuda"), "pre_w": torch.ones(d, device="cuda"),
           "post_b": torch.zeros(d, device="cuda"), "pre_b": torch.zeros(d, device="cuda")}
    none = {**t, "post_w": None, "pre_w": None, "post_b": None, "pre_b": None}
    (h1, z1, s1), (h0, z0, s0) = forward(cfg, one), forward(cfg, none)
    assert torch.equal(h1, h0) and torch.equal(z1, z0)
    for a, b in zip(backward(cfg, one, h1, s1)[:2], backward(cfg, none, h0, s0)[:2]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("d", [776, 777, 8191, 8200, 9001])
def test_in_place_beside_other_rows(d):
    """Rows whose 16-byte pieces hold values of their neighbours, which others write meanwhile; rows that are read twice."""
    rows = 3001
    t = make(rows, d, BF, F32, "layer", "layer", rows, 13)
    cfg = config(rows, d, BF, F32, "layer", "layer", rows)
    h, z, stats = forward(cfg, t)
    check_forward(cfg, t, "layer", "layer", h, z, stats)
    dx, du, grads = backward(cfg, t, h, stats)
    for a, b in (("x", "u"), ("u", "x")):
        c = {**t, "x": t["x"].clone(), "u": t["u"].clone()}
        h2, z2, _ = forward(cfg, c, h=c[a], z=c[b])
        assert torch.equal(h2, h) and torch.equal(z2, z)
    for a, b in (("dz", "dh"), ("dh", "dz"), ("u", "h"), ("h", "u")):
        c = {n: None if v is None else v.clone() for n, v in {**t, "h": h}.items()}
        dx2, du2, g2 = backward(cfg, c, c["h"], stats, dx=c[a], du=c[b])
        assert torch.equal(dx2, dx) and torch.equal(du2, du) and all(torch.equal(x, y) for x, y in zip(grads, g2))


@pytest.mark.parametrize("d", [4096, 4095])
def test_more_values_than_32_bits_count(d):
    """The last rows lie beyond value 2^31; in place, so that only the rows that are compared are kept."""
    rows = 2 ** 31 // d + 1000
    near_end = torch.cat([torch.arange(2), 2 ** 31 // d + torch.arange(-2, 2), rows - torch.arange(4, 0, -1)]).cuda()
    t = make(1, d, BF, F32, "rms", "rms", 0, 14)
    for n in ("x", "u", "dz", "dh"):
        t[n] = torch.empty(rows, d, dtype=BF, device="cuda").normal_()
    cfg, few = config(rows, d, BF, F32, "rms", "rms", 0), config(len(near_end), d, BF, F32, "rms", "rms", 0)
    part = {n: v[near_end] if n in ("x", "u", "dz", "dh") else v for n, v in t.items()}
    h, z, stats = forward(cfg, t, h=t["x"])
    some = [s[near_end] for s in stats]
    check_forward(few, part, "rms", "rms", h[near_end], z[near_end], some)
    want, size = torch.zeros(d, dtype=torch.float64, device="cuda"), torch.zeros(d, dtype=torch.float64, device="cuda")
    for i in range(0, rows, 4000):
        v = t["dz"][i:i + 4000].double() * h[i:i + 4000].double() * stats[1][i:i + 4000, 1:].double()
        want += v.sum(0)
        size += v.square().sum(0)
    dx, du, grads = backward(cfg, t, h, stats, dx=t["dz"], du=t["u"], want=("pre_w",))
    check_backward(few, part, "rms", "rms", h[near_end], some, dx[near_end], du[near_end], [None] * 5)
    near(grads[3], f64(want), ULP * (64 + 4 * np.sqrt(rows)) * f64(size.sqrt()))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("rows,d", [(5, 33), (4, 777), (3001, 777), (700, 1411), (6, 16383)])
def test_norms_without_weights_or_gate(rows, d, dt):
    """No factor takes what lies beyond a row of odd width to zero: a mean is taken off nothing there."""
    for post, pre in KINDS:
        t = make(rows, d, dt, F32, post, pre, 0, rows + d)
        t.update(post_w=None, post_b=None, pre_w=None, pre_b=None)
        cfg = config(rows, d, dt, F32, post, pre, 0)
        h, z, stats = forward(cfg, t)
        check_forward(cfg, t, post, pre, h, z, stats)
        check_backward(cfg, t, post, pre, h, stats, *backward(cfg, t, h, stats))
        t["post_b"] = torch.ones(d, device="cuda") if post == "layer" else None
        h, z, stats = forward(cfg, t)
        check_forward(cfg, t, post, pre, h, z, stats)


@pytest.mark.parametrize("groups", [0, 4])
def test_no_weight_gradients_with_gates_of_groups(groups):
    rows, d = 37, 256
    t = make(rows, d, BF, F32, "rms", "rms", groups, 4)
    cfg = config(rows, d, BF, F32, "rms", "rms", groups)
    h, z, stats = forward(cfg, t)
    dx, du, _ = backward(cfg, t, h, stats)
    dx2, du2, _ = backward(cfg, t, h, stats, ws=False, want=())
    assert torch.equal(dx, dx2) and torch.equal(du, du2)


@pytest.mark.parametrize("pre", ["rms", "layer"])
@pytest.mark.parametrize("d", [128, 1001])
def test_without_a_branch(pre, d):
    """The first norm of a stack: u NULL, h = residual_scale x; with scale 1 x serves as h."""
    rows = 65
    t = make(rows, d, BF, BF, "none", pre, 0, 5)
    t["u"] = None
    cfg = config(rows, d, BF, BF, "none", pre, 0, residual_scale=1.0)
    h, z, stats = forward(cfg, t)
    assert torch.equal(h, t["x"])
    check_forward(cfg, t, "none", pre, h, z, stats)
    dx, dw = torch.empty_like(h), torch.empty_like(t["pre_w"])
    tlc.residual_norm_backward(cfg, t["dz"], None, None, t["x"], None, None, None, t["pre_w"], None, stats[1], dx, None,
                               dpre_w=dw, ws=tlc.ResidualNormWorkspace(cfg))
    t2 = {**t, "u": t["x"], "dh": torch.zeros_like(t["x"])}
    dx2, _, grads = backward(cfg, t2, h, stats)
    assert torch.equal(dx, dx2) and torch.equal(dw, grads[3])


def test_no_rows():
    cfg = config(0, 64, F32, F32, "layer", "layer", 4)
    t = make(0, 64, F32, F32, "layer", "layer", 4)
    h, z, stats = forward(cfg, t)
    _, _, grads = backward(cfg, t, h, stats)
    assert all((g == 0).all() for g in grads)
    assert grads[2].numel() == 0


@pytest.mark.parametrize("d", [64, 777, 4096])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_hard_rows(kind, d):
    """Rows of zeros and constants, a row with NaN or infinity among others, values near fp32's ends."""
    t = make(8, d, F32, F32, kind, kind, 0, 6)
    for n in ("x", "u"):
        t[n][0] = 0
    t["u"][1] = 3.0
    t["u"][2, d // 2] = float("nan")
    t["x"][3, d // 3] = float("inf")
    t["u"][4] *= 1e15
    t["u"][5] *= 1e-18
    cfg = config(8, d, F32, F32, kind, kind, 0)
    h, z, stats = forward(cfg, t)
    for r in (2, 3):
        assert torch.isnan(z[r]).any()
    fine = [0, 1, 4, 5, 6, 7]
    part = {n: v[fine] if n in ("x", "u", "dz", "dh") else v for n, v in t.items()}
    check_forward(config(6, d, F32, F32, kind, kind, 0), part, kind, kind, h[fine], z[fine], [s[fine] for s in stats])
    dx, du, _ = backward(cfg, t, h, stats)
    assert torch.isfinite(dx[fine]).all() and torch.isfinite(du[fine]).all()


@pytest.mark.parametrize("dt", [BF, F32])
def test_unaligned_tensors_and_stream(dt):
    """Other pieces, other order of the sums: equal up to a few last bits of fp32, rounded."""
    rows, d = 21, 1024
    t = make(rows, d, dt, F32, "layer", "rms", 5, 7)
    cfg = config(rows, d, dt, F32, "layer", "rms", 5)
    h, z, stats = forward(cfg, t)
    shift = lambda v: None if v is None else torch.cat([v.flatten()[:1], v.flatten()])[1:].view(v.shape)  # noqa: E731
    s = {n: shift(v) for n, v in t.items()}
    assert s["x"].data_ptr() % 16
    h1, z1, st = shift(h), shift(z), torch.cuda.Stream()
    torch.cuda.synchronize()
    h1, z1, stats1 = forward(cfg, s, h=h1, z=z1, stream=st)
    st.synchronize()
    check_forward(cfg, t, "layer", "rms", h1, z1, stats1)
    check_backward(cfg, t, "layer", "rms", h1, stats1, *backward(cfg, s, shift(h1), stats1, dx=shift(h), du=shift(h)))
    # rows aligned, weights not: pieces of one value in the forward pass
    w = {n: shift(v) if n in WEIGHTS else v for n, v in t.items()}
    check_forward(cfg, t, "layer", "rms", *forward(cfg, w))
    a, b = backward(cfg, t, h, stats), backward(cfg, w, h, stats)
    assert all(x is None or torch.equal(x, y) for x, y in zip((*a[:2], *a[2]), (*b[:2], *b[2])))


def test_captured_and_replayed():
    rows, d = 300, 512
    t = make(rows, d, BF, F32, "rms", "layer", rows, 8)
    cfg = config(rows, d, BF, F32, "rms", "layer", rows)
    h, z, stats = forward(cfg, t)
    dx, du, grads = backward(cfg, t, h, stats)
    outs = [torch.zeros_like(v) for v in (h, z, dx, du, *(g for g in grads if g is not None))]
    ws = tlc.ResidualNormWorkspace(cfg)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tlc.residual_norm_forward(cfg, t["x"], t["u"], t["post_w"], None, t["gate"], t["pre_w"], t["pre_b"], outs[0], outs[1], *stats)
        tlc.residual_norm_backward(cfg, t["dz"], t["dh"], t["u"], outs[0], t["post_w"], None, t["gate"], t["pre_w"], *stats,
                                   outs[2], outs[3], outs[4], None, *outs[5:], ws)
    for _ in range(3):
        for o in outs:
            o.zero_()
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, (h, z, dx, du, *(g for g in grads if g is not None))):
        assert torch.equal(a, b)


def test_refusals():
    t = make(5, 64, BF, F32, "layer", "rms", 5, 9)
    cfg = config(5, 64, BF, F32, "layer", "rms", 5)
    h, z, stats = forward(cfg, t)
    for bad in (dict(x=t["x"].float()), dict(x=t["x"][:3]), dict(post_w=t["post_w"].to(BF)), dict(gate=t["post_w"].repeat(2)),
                dict(u=t["u"].cpu()), dict(pre_w=t["pre_w"][:5]), dict(x=t["x"].t().contiguous().t())):
        with pytest.raises(ValueError):
            forward(cfg, {**t, **bad})
    for bad in (dict(z=None), dict(h=z, z=z), dict(pre_b=t["post_b"]), dict(gate=None), dict(u=None)):
        a = {**t, "h": h, "z": z, **bad}
        with pytest.raises(tlc.MoEError) as e:
            tlc.residual_norm_forward(cfg, *(a[n] for n in ("x", "u", "post_w", "post_b", "gate", "pre_w", "pre_b", "h", "z")))
        assert e.value.code == tlc.MOE_ERR_ARG
    ws = tlc.ResidualNormWorkspace(cfg)
    ws.nbytes = 64
    for w, code in ((None, tlc.MOE_ERR_ARG), (ws, tlc.MOE_ERR_WORKSPACE)):
        with pytest.raises(tlc.MoEError) as e:
            tlc.residual_norm_backward(cfg, t["dz"], t["dh"], t["u"], h, t["post_w"], t["post_b"], t["gate"], t["pre_w"], *stats,
                                       torch.empty_like(h), torch.empty_like(h), torch.empty_like(t["post_w"]), ws=w)
        assert e.value.code == code
