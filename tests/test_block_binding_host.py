"""Host-only checks of the block operators' binding: what it hands to the library, and what it refuses."""
import copy
import ctypes
import dataclasses
import gc
import pickle
import weakref

import pytest
import torch

import tile_level_copy_gb300 as tlc


class Library:
    """Stands for the loaded library: `on` maps an entry point to a function, the others return MOE_OK."""

    def __init__(self, **on):
        self.on, self.calls = on, []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return self.on[name](*args) if name in self.on else tlc.MOE_OK
        return call


def test_adamw_step_hands_over_its_own_step(monkeypatch):
    """Another thread steps with the same config while the call of this one is under way (the call releases
    the interpreter's lock): made here by a step from within the call."""
    cfg, seen = tlc.AdamWConfig(lr=1e-3), []
    lst = tlc.AdamWList(cfg, [], [], [], [])

    def step(ref, *_):
        if not seen:
            seen.append(None)
            tlc.adamw_step(cfg, lst, 9, stream=0)
        seen.append(ref._obj.step)
        return tlc.MOE_OK

    monkeypatch.setattr(tlc, "lib", lambda: Library(moe_adamw_step=step))
    monkeypatch.setattr(tlc, "_device", lambda: 0)
    tlc.adamw_step(cfg, lst, 5, stream=0)
    assert seen == [None, 9, 5]
    assert cfg.ref()[1].step == 1  # the config's own struct stays as it was made


@pytest.mark.parametrize("cfg", [tlc.FFNConfig(4, 128, 256), tlc.LayerNormConfig(4, 64), tlc.AdamWConfig(lr=1e-3, seed=7)],
                         ids=lambda c: type(c).__name__)
def test_a_used_config_is_copied_and_pickled(built_library, cfg):
    cfg.ref()
    for other in (copy.copy(cfg), copy.deepcopy(cfg), pickle.loads(pickle.dumps(cfg)), dataclasses.replace(cfg)):
        assert other == cfg and type(other) is type(cfg)
        assert other.ref()[1] is not cfg.ref()[1]  # a C form of its own
        assert bytes(other.ref()[1]) == bytes(cfg.ref()[1])


class Device:
    """Stands for a tensor on device `index` (-1: in host memory)."""

    def __init__(self, dtype, *shape, index=0):
        self.dtype, self.shape, self.index = dtype, torch.Size(shape), index

    is_cuda = property(lambda self: self.index >= 0)
    device = property(lambda self: torch.device("cuda", self.index))

    def get_device(self):
        return self.index

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return (self.index + 2) << 20


BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


def workspace(cls):
    ws = object.__new__(cls)
    ws.buf = Device(U8, 1 << 20)
    ws.ptr, ws.nbytes = ws.buf.data_ptr(), 1 << 20
    return ws


def ffn_call(backward):
    cfg, rows, up, down = tlc.FFNConfig(4, 128, 256), (4, 128), (256, 128), (128, 256)
    t = {n: Device(BF, *s) for n, s in (("x", rows), ("W1", up), ("W3", up), ("W2", down))}
    t["saved"], t["ws"] = Device(U8, 1 << 20), workspace(tlc.FFNWorkspace)
    if not backward:
        t["y"] = Device(BF, *rows)
        return t, lambda **a: tlc.ffn_forward(cfg, **a)
    t.update({n: Device(BF, *s) for n, s in (("dy", rows), ("dx", rows), ("dW1", up), ("dW3", up), ("dW2", down))})
    return t, lambda **a: tlc.ffn_backward(cfg, **a)


def layernorm_call(backward):
    cfg = tlc.LayerNormConfig(4, 64)
    t = {"x": Device(BF, 4, 64), "w": Device(F32, 64), "mean": Device(F32, 4), "rstd": Device(F32, 4)}
    if not backward:
        t["b"], t["y"] = Device(F32, 64), Device(BF, 4, 64)
        return t, lambda **a: tlc.layernorm_forward(cfg, **a)
    t.update(dy=Device(BF, 4, 64), dx=Device(BF, 4, 64), dw=Device(F32, 64), db=Device(F32, 64),
             ws=workspace(tlc.LayerNormWorkspace))
    return t, lambda **a: tlc.layernorm_backward(cfg, **a)


def adamw_call(read):
    cfg = tlc.AdamWConfig(lr=1e-3, bits=8)
    t = {n: Device(d, k) for n, d, k in (("p", F32, 200), ("g", BF, 200), ("m", U8, 200), ("v", U8, 200),
                                         ("m_scale", U8, 2), ("v_scale", U8, 2), ("copy", BF, 200))}
    names = list(t)
    make = lambda a: tlc.AdamWList(cfg, **{n: [Device(F32, 7), a[n]] if n in "p" else  # noqa: E731
                                           [Device(a[n].dtype, 1 if "scale" in n else 7), a[n]] for n in names})
    if not read:
        t["grad_scale"] = Device(F32, 1)
        return t, lambda **a: tlc.adamw_step(cfg, make(a), 1, a["grad_scale"])
    t["m_out"], t["v_out"] = Device(F32, 200), Device(F32, 200)

    def run(**a):
        lst = make(a)
        tlc.adamw_read_state(cfg, lst, tlc.AdamWValues(lst, *([Device(F32, 7), a[n]] for n in ("m_out", "v_out"))))
    return t, run


CALLS = [(ffn_call, False), (ffn_call, True), (layernorm_call, False), (layernorm_call, True), (adamw_call, False),
         (adamw_call, True)]


@pytest.fixture
def device_0(monkeypatch):
    """A current device 0, and a library that notes its calls."""
    fake = Library()
    monkeypatch.setattr(tlc, "lib", lambda: fake)
    monkeypatch.setattr(tlc, "_device", lambda: 0)
    monkeypatch.setattr(tlc, "_current_stream", lambda i: 1000 + i)
    return fake


def launches(fake):
    return [n for n, _ in fake.calls if not n.endswith("_size")]


@pytest.mark.parametrize("make,second", CALLS)
def test_tensors_of_the_current_device_are_handed_over(device_0, make, second):
    tensors, call = make(second)
    call(**tensors)
    assert len(launches(device_0)) == 1 and device_0.calls[-1][1][-1] == 1000  # on its current stream


@pytest.mark.parametrize("make,second", CALLS)
def test_a_tensor_elsewhere_is_refused(device_0, make, second):
    """The kernels are launched on the current device: a tensor of another one, or of the host, is refused,
    whichever it is, and so are tensors that are all of another device."""
    tensors, call = make(second)
    for index in (1, -1):
        for name in tensors:
            if name == "ws" and index < 0:
                continue
            tensors, call = make(second)
            (tensors[name].buf if name == "ws" else tensors[name]).index = index
            with pytest.raises(ValueError):
                call(**tensors)
    tensors, call = make(second)
    for t in tensors.values():
        getattr(t, "buf", t).index = 1
    with pytest.raises(ValueError):
        call(**tensors)
    assert launches(device_0) == []


def test_a_list_made_on_another_device_is_refused(device_0, monkeypatch):
    """Every tensor on device 1, the list made while device 1 was current, the step called on device 0."""
    cfg = tlc.AdamWConfig(lr=1e-3)
    one = lambda: [Device(F32, 100, index=1)]  # noqa: E731
    lst = tlc.AdamWList(cfg, one(), one(), one(), one())
    with pytest.raises(ValueError, match="cuda:1"):
        tlc.adamw_step(cfg, lst, 1)
    monkeypatch.setattr(tlc, "_device", lambda: 1)
    tlc.adamw_step(cfg, lst, 1)
    assert device_0.calls[-1][1][-1] == 1001


def test_a_status_of_another_device_is_refused(device_0, monkeypatch):
    ws = workspace(tlc.FFNWorkspace)
    ws.buf.index = 1
    with pytest.raises(ValueError, match="cuda:1"):
        tlc.ffn_status(tlc.FFNConfig(4, 128, 256), ws, stream=0)


def test_a_list_keeps_its_tensors_whatever_becomes_of_the_callers(device_0):
    """The library reads the pointers at every step: the tensors live as long as the list, although the
    caller empties or refills the lists that it made it from."""
    cfg = tlc.AdamWConfig(lr=1e-3, bits=8)
    names = {"p": F32, "g": BF, "m": U8, "v": U8, "m_scale": U8, "v_scale": U8, "copy": BF}
    mine = {n: [Device(d, 1 if "scale" in n else 100)] for n, d in names.items()}
    lst = tlc.AdamWList(cfg, **mine)
    m, v = [Device(F32, 100)], [Device(F32, 100)]
    values = tlc.AdamWValues(lst, m, v)
    alive = [weakref.ref(l[0]) for l in (*mine.values(), m, v)]
    for l in (*mine.values(), m, v):
        l.clear()
    gc.collect()
    assert all(r() is not None for r in alive)
    del lst, values
    gc.collect()
    assert all(r() is None for r in alive)


def test_unknown_ffn_flags_are_refused(built_library):
    n = ctypes.c_size_t()
    for flags, rc in ((0, tlc.MOE_OK), (tlc.MOE_FFN_TEST_STALL0 | tlc.MOE_FFN_TEST_STALL1, tlc.MOE_OK), (4, tlc.MOE_ERR_ARG),
                      (1 << 31, tlc.MOE_ERR_ARG)):
        c = tlc.FFNConfig(4, 128, 256, flags=flags).to_c()
        assert built_library.moe_ffn_workspace_size(ctypes.byref(c), ctypes.byref(n)) == rc
