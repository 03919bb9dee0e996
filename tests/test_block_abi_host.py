"""Host-only checks of the block operators' C entry points: sizes, refusals before any CUDA call."""
import ctypes

import pytest

import tile_level_copy_gb300 as tlc


def ffn_sizes(lib, **kw):
    c = tlc.FFNConfig(**{**dict(T=5, d=128, ffn=256), **kw}).to_c()
    ws, saved = ctypes.c_size_t(), ctypes.c_size_t()
    rc = lib.moe_ffn_workspace_size(ctypes.byref(c), ctypes.byref(ws))
    assert rc == lib.moe_ffn_saved_size(ctypes.byref(c), ctypes.byref(saved))
    return rc, ws.value, saved.value


def test_ffn_sizes_hold_their_regions(built_library):
    for T, d, f in ((0, 8, 8), (1, 2048, 1408), (1003, 1000, 2744), (4096, 4096, 14336)):
        rc, ws, saved = ffn_sizes(built_library, T=T, d=d, ffn=f)
        assert rc == tlc.MOE_OK
        assert ws >= tlc.MOE_FFN_STATUS_BYTES + 2 * T * f * 2  # two hidden matrices in bf16
        assert saved >= T * f * (2 + 8)                        # h in bf16, g and u in fp32


@pytest.mark.parametrize("bad", [dict(T=-1), dict(T=1 << 24), dict(d=0), dict(d=12), dict(ffn=1 << 20), dict(ffn=-8)])
def test_ffn_configs_are_refused(built_library, bad):
    assert ffn_sizes(built_library, **bad)[0] == tlc.MOE_ERR_ARG
    assert len(built_library.moe_last_error()) > 10


def test_ffn_null_and_small_workspaces_are_refused(built_library):
    c = tlc.FFNConfig(5, 128, 256).to_c()
    ref, one = ctypes.byref(c), ctypes.c_void_p(1 << 20)
    assert built_library.moe_ffn_forward(ref, *[one] * 6, None, 0, None) == tlc.MOE_ERR_ARG
    assert built_library.moe_ffn_forward(ref, *[one] * 6, ctypes.c_void_p(100), 1 << 40, None) == tlc.MOE_ERR_ARG
    assert built_library.moe_ffn_forward(ref, *[one] * 7, 100, None) == tlc.MOE_ERR_WORKSPACE
    assert built_library.moe_ffn_forward(None, *[one] * 7, 1 << 40, None) == tlc.MOE_ERR_ARG
    c.reserved[2] = 1
    assert built_library.moe_ffn_forward(ref, *[one] * 7, 1 << 40, None) == tlc.MOE_ERR_ARG


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(d=0), dict(d=16385), dict(eps=-1e-9), dict(eps=float("nan"))])
def test_layernorm_configs_are_refused(built_library, bad):
    c = tlc.LayerNormConfig(**{**dict(rows=4, d=64), **bad}).to_c()
    n = ctypes.c_size_t()
    assert built_library.moe_layernorm_workspace_size(ctypes.byref(c), ctypes.byref(n)) == tlc.MOE_ERR_ARG


def test_layernorm_pointers_are_refused(built_library):
    c = tlc.LayerNormConfig(4, 64).to_c()
    ref, ok, odd = ctypes.byref(c), ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 1)
    f = built_library.moe_layernorm_forward
    assert f(ref, None, ok, ok, ok, ok, ok, None) == tlc.MOE_ERR_ARG
    assert f(ref, odd, ok, ok, ok, ok, ok, None) == tlc.MOE_ERR_ARG
    assert f(ref, ok, odd, ok, ok, ok, ok, None) == tlc.MOE_ERR_ARG
    assert built_library.moe_layernorm_backward(ref, ok, None, ok, ok, ok, ok, ok, ok, ok, 1 << 40, None) == tlc.MOE_ERR_ARG


def test_adamw_arguments_are_refused(built_library):
    step = built_library.moe_adamw_step

    def cfg(**kw):
        return ctypes.byref(tlc.AdamWConfig(**{**dict(lr=1e-3), **kw}).to_c(kw.pop("step", 1)))

    t = (tlc._AdamWTensor * 1)()
    p = 1 << 20
    for n in ("p", "g", "m", "v"):
        setattr(t[0], n, p)
    t[0].n = 10
    assert step(cfg(beta1=1.0), t, 1, None, None) == tlc.MOE_ERR_ARG
    assert step(cfg(beta2=-0.5), t, 1, None, None) == tlc.MOE_ERR_ARG
    assert step(cfg(eps=float("inf")), t, 1, None, None) == tlc.MOE_ERR_ARG
    assert step(cfg(bits=4), t, 1, None, None) == tlc.MOE_ERR_ARG
    assert step(cfg(), t, -1, None, None) == tlc.MOE_ERR_ARG
    assert step(cfg(), None, 1, None, None) == tlc.MOE_ERR_ARG
    assert step(cfg(bits=8), t, 1, None, None) == tlc.MOE_ERR_ARG  # no scales
    assert step(cfg(), t, 1, ctypes.c_void_p(p + 2), None) == tlc.MOE_ERR_ARG
    c = tlc.AdamWConfig(lr=1e-3).to_c(0)
    assert step(ctypes.byref(c), t, 1, None, None) == tlc.MOE_ERR_ARG
    t[0].m = p + 1
    assert step(cfg(), t, 1, None, None) == tlc.MOE_ERR_ARG
    t[0].m, t[0].p_dtype = p, tlc.MOE_DTYPE_F16
    assert step(cfg(), t, 1, None, None) == tlc.MOE_ERR_ARG
    t[0].p_dtype, t[0].n = tlc.MOE_DTYPE_F32, -1
    assert step(cfg(), t, 1, None, None) == tlc.MOE_ERR_ARG
    t[0].n = 0
    assert step(cfg(), t, 1, None, None) == tlc.MOE_OK  # nothing to do, no CUDA call
    t[0].n = 10
    t[0].g = None
    assert step(cfg(), t, 1, None, None) == tlc.MOE_ERR_ARG


def test_a_config_that_changes_is_marshalled_again():
    c = tlc.FFNConfig(4, 128, 256)
    assert c.ref()[1].T == 4 and c.ref() is c.ref()
    c.T = 9
    assert c.ref()[1].T == 9
    a = tlc.AdamWConfig(lr=1e-3)
    a.ref()
    a.lr = 5e-4
    assert a.ref()[1].lr == 5e-4
