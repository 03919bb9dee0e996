"""Host-only checks of a training step's C entry points: sizes, and refusals before any CUDA call."""
import ctypes

import pytest

import tile_level_copy_gb300 as tlc

OK, ODD = ctypes.c_void_p(1 << 30), ctypes.c_void_p((1 << 30) + 1)
ARG = tlc.MOE_ERR_ARG


def at(k):
    """Pointers far enough apart for the small rows below."""
    return ctypes.c_void_p((1 << 30) + (k << 20))


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(d=0), dict(d=16385), dict(eps=-1e-9), dict(eps=float("nan")), dict(gate_rows=-1),
                                 dict(post=3), dict(pre=-1), dict(residual_scale=float("inf")), dict(branch_scale=float("nan")),
                                 dict(rows=1 << 62)])
def test_residual_norm_configs_are_refused(built_library, bad):
    c = tlc.ResidualNormConfig(**{**dict(rows=4, d=64), **bad}).to_c()
    n = ctypes.c_size_t()
    assert built_library.moe_residual_norm_workspace_size(ctypes.byref(c), ctypes.byref(n)) == ARG
    assert len(built_library.moe_last_error()) > 10
    c = tlc.ResidualNormConfig(4, 64).to_c()
    c.reserved[1] = 1
    assert built_library.moe_residual_norm_workspace_size(ctypes.byref(c), ctypes.byref(n)) == ARG
    c.reserved[1], c.wdtype, c.dtype = 0, tlc.MOE_DTYPE_BF16, tlc.MOE_DTYPE_F16
    assert built_library.moe_residual_norm_workspace_size(ctypes.byref(c), ctypes.byref(n)) == ARG
    assert built_library.moe_residual_norm_workspace_size(None, ctypes.byref(n)) == ARG


def test_residual_norm_workspaces_hold_their_sums(built_library):
    for rows, d, gate_rows, kind in ((1, 1, 0, 1), (16384, 4096, 0, 1), (16384, 4096, 250, 2), (100, 16384, 1, 2), (0, 8, 3, 2)):
        c = tlc.ResidualNormConfig(rows, d, post=kind, pre=kind, gate_rows=gate_rows).to_c()
        n = ctypes.c_size_t()
        assert built_library.moe_residual_norm_workspace_size(ctypes.byref(c), ctypes.byref(n)) == tlc.MOE_OK
        assert n.value >= min(rows, 1) * 2 * kind * d * 4


def test_residual_norm_arguments_are_refused(built_library):
    """x u pw pb gate qw qb h z ps qs stream / dz dh u h pw pb gate qw ps qs dx du g... ws"""
    f, b = built_library.moe_residual_norm_forward, built_library.moe_residual_norm_backward
    make = lambda **kw: ctypes.byref(tlc.ResidualNormConfig(**{**dict(rows=4, d=64, post=1, pre=1, gate_rows=4), **kw}).to_c())  # noqa: E731
    good = [at(i) for i in range(11)]

    def forward(cfg=None, **kw):
        a = dict(zip("x u pw pb gate qw qb h z ps qs".split(), good), pb=None, qb=None)
        a.update(kw)
        return f(cfg or make(), *a.values(), None)

    for bad in (dict(x=None), dict(u=None), dict(gate=None), dict(z=None), dict(h=None, z=None), dict(pb=OK), dict(qb=OK), dict(x=ODD),
                dict(pw=ODD), dict(z=ODD), dict(ps=ctypes.c_void_p(4)), dict(h=at(8)),
                dict(h=ctypes.c_void_p(at(0).value + 8)), dict(z=ctypes.c_void_p(at(1).value - 8))):
        assert forward(**bad) == ARG, bad
    assert forward(make(gate_rows=0)) == ARG             # a gate without gate_rows
    assert forward(make(post=0)) == ARG                  # a weight without its norm
    assert forward(make(pre=0), qw=None) == ARG          # z without a pre norm
    assert forward(make(rows=0)) == tlc.MOE_OK           # nothing to do, no CUDA call

    def backward(cfg=None, bytes=1 << 40, **kw):
        a = dict(zip("dz dh u h pw pb gate qw ps qs dx du gpw gpb gg gqw gqb ws".split(), [at(i) for i in range(18)]), pb=None,
                 gpb=None, gqb=None)
        a.update(kw)
        return b(cfg or make(), *a.values(), bytes, None)

    for bad in (dict(dz=None), dict(u=None), dict(h=None), dict(dx=None), dict(ps=None), dict(qs=None), dict(gate=None), dict(pb=OK),
                dict(gpb=OK), dict(gqb=OK), dict(dz=ODD), dict(gg=ODD), dict(qs=ctypes.c_void_p(4)), dict(du=at(10)),
                dict(dx=ctypes.c_void_p(at(1).value + 4)), dict(du=ctypes.c_void_p(at(3).value - 16))):
        assert backward(**bad) == ARG, bad
    assert backward(make(pre=0), qw=None, gqw=None) == ARG                       # dz without a pre norm
    assert backward(make(pre=0), qw=None, gqw=None, dz=None, dh=None) == ARG     # no gradient at all
    assert backward(make(post=0), pw=None) == ARG                                # a gradient of a weight that is not there
    assert backward(make(rows=0), gpw=None, gg=None, gqw=None) == tlc.MOE_OK


@pytest.mark.parametrize("bad", [dict(T=-1), dict(T=1 << 24), dict(E=0), dict(E=257), dict(topk=0), dict(topk=9), dict(seqs=0),
                                 dict(balance=float("nan")), dict(z=float("inf"))])
def test_balance_configs_are_refused(built_library, bad):
    c = tlc.BalanceConfig(**{**dict(T=4, E=8, topk=2), **bad}).to_c()
    n = ctypes.c_size_t()
    assert built_library.moe_balance_workspace_size(ctypes.byref(c), ctypes.byref(n)) == ARG
    assert built_library.moe_balance_saved_size(ctypes.byref(c), ctypes.byref(n)) == ARG
    assert len(built_library.moe_last_error()) > 10


def test_balance_arguments_are_refused(built_library):
    f, b = built_library.moe_balance_forward, built_library.moe_balance_backward
    make = lambda **kw: ctypes.byref(tlc.BalanceConfig(**{**dict(T=4, E=8, topk=2, seqs=3), **kw}).to_c())  # noqa: E731

    def forward(cfg=None, **kw):
        a = dict.fromkeys("logits idx offsets mask loss counts lse saved ws".split(), OK)
        a.update(kw)
        return f(cfg or make(), *a.values(), 1 << 40, None)

    for n in ("logits", "idx", "offsets", "loss", "counts", "ws"):
        assert forward(**{n: None}) == ARG, n
    for n in ("logits", "idx", "offsets", "loss", "counts", "lse", "saved", "ws"):
        assert forward(**{n: ODD}) == ARG, n
    assert f(None, *[OK] * 9, 1 << 40, None) == ARG

    def backward(cfg=None, **kw):
        a = dict.fromkeys("logits idx offsets mask saved gates dgates dloss dlogits".split(), OK)
        a.update(kw)
        return b(cfg or make(), *a.values(), None)

    for n in ("logits", "idx", "offsets", "saved", "gates", "dgates", "dlogits"):
        assert backward(**{n: None}) == ARG, n
    for n in ("logits", "idx", "offsets", "saved", "gates", "dgates", "dloss", "dlogits"):
        assert backward(**{n: ODD}) == ARG, n
    assert backward(make(T=0)) == tlc.MOE_OK


def test_grad_norm_arguments_are_refused(built_library):
    f, clip = built_library.moe_grad_norm, built_library.moe_grad_clip
    cfg = lambda m=1.0, e=1e-6: ctypes.byref(tlc.GradNormConfig(m, e).to_c())  # noqa: E731
    t = (tlc._GradTensor * 2)()
    t[0].g, t[0].n = 1 << 31, 10
    call = lambda c=cfg(), ts=t, n=2, out=OK, ws=OK, size=1 << 20: f(c, ts, n, out, ws, size, None)  # noqa: E731
    for bad in (dict(c=cfg(-0.5)), dict(c=cfg(-1.0)), dict(c=cfg(float("nan"))), dict(c=cfg(1.0, -1.0)), dict(c=cfg(1.0, float("inf"))),
                dict(ts=None), dict(n=-1), dict(out=None), dict(out=ODD), dict(ws=None), dict(ws=ctypes.c_void_p(8))):
        assert call(**bad) == ARG, bad
    assert call(size=100) == tlc.MOE_ERR_WORKSPACE
    assert clip(t, 2, None, None) == ARG and clip(t, 2, ODD, None) == ARG and clip(t, -1, OK, None) == ARG
    for field, value in (("n", -1), ("dtype", 7), ("g", (1 << 30) + 2), ("g", None), ("reserved", 1)):
        old = getattr(t[0], field)
        setattr(t[0], field, value)
        assert call() == ARG and clip(t, 2, OK, None) == ARG, field
        setattr(t[0], field, old)
    t[0].n = 0
    assert clip(t, 2, OK, None) == tlc.MOE_OK  # nothing to do, no CUDA call
