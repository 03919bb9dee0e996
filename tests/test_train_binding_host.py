"""Host-only checks of the binding of a training step's operators: what it hands to the library, and what it refuses."""
import copy
import gc
import pickle
import weakref

import pytest
import torch

import tile_level_copy_gb300 as tlc
from tests.test_block_binding_host import BF, F32, U8, Device, device_0, launches, workspace  # noqa: F401

I32 = torch.int32


def residual_call(backward):
    cfg = tlc.ResidualNormConfig(4, 64, post=tlc.MOE_NORM_LAYER, pre=tlc.MOE_NORM_LAYER, gate_rows=3)
    rows, vec, gate, stats = (4, 64), (64,), (2, 64), (4, 2)
    t = {n: Device(F32, *s) for n, s in (("post_w", vec), ("post_b", vec), ("gate", gate), ("pre_w", vec), ("post_stats", stats),
                                         ("pre_stats", stats))}
    if not backward:
        t.update(pre_b=Device(F32, *vec), **{n: Device(BF, *rows) for n in ("x", "u", "h", "z")})
        return t, lambda **a: tlc.residual_norm_forward(cfg, **a)
    t.update({n: Device(BF, *rows) for n in ("dz", "dh", "u", "h", "dx", "du")})
    t.update({n: Device(F32, *s) for n, s in (("dpost_w", vec), ("dpost_b", vec), ("dgate", gate), ("dpre_w", vec), ("dpre_b", vec))})
    t["ws"] = workspace(tlc.ResidualNormWorkspace)
    return t, lambda **a: tlc.residual_norm_backward(cfg, **a)


def balance_call(backward):
    cfg = tlc.BalanceConfig(10, 8, 2, 3)
    t = {"logits": Device(F32, 10, 8), "idx": Device(I32, 10, 2), "offsets": Device(I32, 4), "mask": Device(U8, 10),
         "saved": Device(U8, 1 << 20)}
    if not backward:
        t.update(loss=Device(F32, 3), counts=Device(I32, 3, 8), lse=Device(F32, 10), ws=workspace(tlc.BalanceWorkspace))
        return t, lambda **a: tlc.balance_forward(cfg, **a)
    t.update(dlogits=Device(F32, 10, 8), gates=Device(F32, 10, 2), dgates=Device(F32, 10, 2), dloss=Device(F32, 1))
    return t, lambda **a: tlc.balance_backward(cfg, **a)


class Apart(Device):
    """A tensor with an address of its own."""
    at = 0

    def __init__(self, *a, **kw):
        super().__init__(*a, **kw)
        Apart.at += 1 << 16
        self.address = Apart.at

    def data_ptr(self):
        return self.address


def grad_call(clip):
    t = {"a": Apart(F32, 100), "b": Apart(BF, 7, 3)}
    if clip:
        t["scale"] = Device(F32, 1)
        return t, lambda **a: tlc.grad_clip(tlc.GradList([a["a"], a["b"]]), a["scale"])
    t.update(out=Device(F32, 2), ws=workspace(tlc.GradNormWorkspace))
    return t, lambda **a: tlc.grad_norm(tlc.GradNormConfig(1.0), tlc.GradList([a["a"], a["b"]]), a["out"], a["ws"])


CALLS = [(f, second) for f in (residual_call, balance_call, grad_call) for second in (False, True)]


@pytest.mark.parametrize("make,second", CALLS)
def test_tensors_of_the_current_device_are_handed_over(device_0, make, second):  # noqa: F811
    tensors, call = make(second)
    call(**tensors)
    assert len(launches(device_0)) == 1 and device_0.calls[-1][1][-1] == 1000  # on its current stream
    call(**tensors, **({} if make is grad_call else {"stream": 77}))
    if make is not grad_call:
        assert device_0.calls[-1][1][-1].value == 77


@pytest.mark.parametrize("make,second", CALLS)
def test_a_tensor_elsewhere_or_of_another_type_or_size_is_refused(device_0, make, second):  # noqa: F811
    names, _ = make(second)
    for name in names:
        for change in (dict(index=1), dict(index=-1), dict(dtype=torch.float64), dict(shape=torch.Size([999]))):
            if name == "ws" and change != dict(index=1):
                continue
            if "shape" in change and (make is grad_call and name in "ab" or name == "saved"):
                continue  # any size serves
            if name == "saved" and "dtype" in change:
                continue
            tensors, call = make(second)
            t = tensors[name].buf if name == "ws" else tensors[name]
            for k, v in change.items():
                setattr(t, k, v)
            with pytest.raises(ValueError):
                call(**tensors)
    assert launches(device_0) == []


@pytest.mark.parametrize("cfg", [tlc.ResidualNormConfig(4, 64), tlc.BalanceConfig(4, 8, 2), tlc.GradNormConfig(1.0)],
                         ids=lambda c: type(c).__name__)
def test_a_used_config_is_copied_pickled_and_marshalled_again(built_library, cfg):
    cfg.ref()
    for other in (copy.deepcopy(cfg), pickle.loads(pickle.dumps(cfg))):
        assert other == cfg and other.ref()[1] is not cfg.ref()[1] and bytes(other.ref()[1]) == bytes(cfg.ref()[1])
    old = bytes(cfg.ref()[1])
    for name, value in (("eps", 0.25), ("z", 0.25)):
        if hasattr(cfg, name):
            setattr(cfg, name, value)
    assert bytes(cfg.ref()[1]) != old


def test_a_list_of_gradients_keeps_them_and_refuses_shared_memory(device_0):  # noqa: F811
    a, b = Apart(F32, 100), Apart(F32, 100)
    mine = [a, b]
    lst = tlc.GradList(mine)
    alive = weakref.ref(a)
    mine.clear()
    del a
    gc.collect()
    assert alive() is not None and lst.count == 2
    c = Apart(F32, 50)
    c.address = b.address + 399
    with pytest.raises(ValueError, match="share memory"):
        tlc.GradList([b, c])
    c.address = b.address + 400
    tlc.GradList([b, c])
    tlc.GradList([b, Apart(F32, 0)])
    with pytest.raises(ValueError, match="share memory"):
        tlc.GradList([c, b, c])
