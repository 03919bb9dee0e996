"""GB300 (sm_103a) MoE expert layer with tile-level overlapped return copy.

Thin ctypes binding of libmoe (C ABI in include/moe.h): argument marshalling only. Every step of
the layer runs in the library's CUDA kernels; there is no CPU or PyTorch fallback, and every call
raises if the library cannot be loaded. PyTorch supplies device memory and streams.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libmoe.so")

MOE_OK = 0
MOE_ERR_ARG = -1
MOE_ERR_WORKSPACE = -2
MOE_ERR_CUDA = -3
MOE_ERR_TIMEOUT = -4
MOE_ERR_DEVICE = -5
MOE_ERR_PLAN = -6

MOE_PLAN_SKIP_PERMUTE = 0x1
MOE_TAIL_ASSIST = 0x2
MOE_COPY_WARPS = 0x4
MOE_PAIR_UMMA = 0x8
MOE_DIRECT_TAIL = 0x10
MOE_FUSED_DISPATCH = 0x20
MOE_FUSED_GEMMS = 0x40
MOE_PDL = 0x80
MOE_TEST_STALL_CONSUMER = 0x100
MOE_TEST_PLAN_FAIL = 0x200
MOE_ADAPTIVE_CONSUMERS = 0x1000
MOE_TEST_STALL_LAYOUT = 0x2000
MOE_TEST_STALL_PIPE0 = 0x400
MOE_TEST_STALL_PIPE1 = 0x800

TRACE_GEMM2_START, TRACE_GEMM2_END, TRACE_COPY_START, TRACE_COPY_END = 0, 1, 2, 3
TRACE_BAND_DONE, TRACE_LAST_ACQUIRE, TRACE_LAST_LOAD, TRACE_LAST_DRAIN = 4, 5, 6, 7
TRACE_UP_CYCLES, TRACE_UP_NS, TRACE_DOWN_CYCLES, TRACE_DOWN_NS = 8, 9, 10, 11

# types of values, block of the 8-bit optimiser states, status bytes of a feed-forward workspace
MOE_DTYPE_F32, MOE_DTYPE_BF16, MOE_DTYPE_F16 = 0, 1, 2
MOE_ADAMW_BLOCK = 128
MOE_FFN_STATUS_BYTES = 8192
MOE_FFN_TEST_STALL0, MOE_FFN_TEST_STALL1 = 0x1, 0x2
_DTYPES = {torch.float32: MOE_DTYPE_F32, torch.bfloat16: MOE_DTYPE_BF16, torch.float16: MOE_DTYPE_F16}

# names of the C entry points (each declared in include/moe.h)
EXPORTS = ("moe_workspace_size", "moe_workspace_layout", "moe_plan", "moe_forward", "moe_forward_sequential",
           "moe_forward_ex", "moe_forward_host", "moe_forward_host_pipelined", "moe_copy_only", "moe_dma_host_bytes",
           "moe_forward_dma", "moe_status", "moe_device_info", "moe_route_static", "moe_ffn_workspace_size",
           "moe_ffn_saved_size", "moe_ffn_forward", "moe_ffn_backward", "moe_ffn_status", "moe_layernorm_forward",
           "moe_layernorm_workspace_size", "moe_layernorm_backward", "moe_adamw_step", "moe_adamw_read_state",
           "moe_last_error")

# stage events of moe_forward_ex
EV_BEGIN, EV_PLANNED, EV_UP, EV_DOWN, EV_COPIED, EV_END, EV_COUNT = range(7)


class MoEError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"libmoe error {code}: {message}")
        self.code = code


class _Config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "d", "ffn", "E", "topk", "R", "tile_M", "consumer_ctas", "mgb")] + [
        ("flags", ctypes.c_uint32), ("timeout_us", ctypes.c_uint32), ("tail_window", ctypes.c_int32),
        ("reserved", ctypes.c_int32 * 4)]


_LAYOUT_INTS = ("P_max", "MT_max", "n_chunks", "chunk_tokens", "n_tiles_n2", "block_n2", "rows_per_unit",
                "units_per_band", "PC_max", "IU_max")
LAYOUT_REGIONS = ("idx", "gate", "rank", "chunk_cnt", "chunk_base", "counts", "offsets", "ret_off", "tiles",
                  "tile_ret", "sched", "order", "seg", "experts", "items_up", "items_down", "slot", "cslot", "ret_slot", "yrow",
                  "tile_crow", "band_item", "tok_of", "xrows", "xready", "meta", "flags", "bands", "trace", "Xc", "Hc", "Yp", "Ret", "in_logits", "in_x", "out")


class _Layout(ctypes.Structure):
    _fields_ = [("bytes", ctypes.c_size_t)] + [(n, ctypes.c_int32) for n in _LAYOUT_INTS] + [
        (n, ctypes.c_size_t) for n in LAYOUT_REGIONS]


@dataclasses.dataclass
class Config:
    """Problem and knobs of one MoE layer call (mirrors moe_config)."""

    T: int
    d: int
    ffn: int
    E: int
    topk: int
    R: int
    tile_M: int = 128
    consumer_ctas: int = 8
    mgb: int = 1
    flags: int = 0
    timeout_us: int = 0
    tail_window: int = 0

    def to_c(self) -> _Config:
        c = _Config()
        for f in dataclasses.fields(self):
            setattr(c, f.name, int(getattr(self, f.name)))
        return c

    @classmethod
    def from_workload(cls, w, **kw) -> "Config":
        return cls(T=w.T, d=w.d, ffn=w.ffn, E=w.E, topk=w.topk, R=w.R, tile_M=w.tile_M, **kw)


class _FFNConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "d", "ffn")] + [
        ("timeout_us", ctypes.c_uint32), ("flags", ctypes.c_uint32), ("reserved", ctypes.c_int32 * 3)]


class _LayerNormConfig(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("d", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("wdtype", ctypes.c_int32), ("eps", ctypes.c_float), ("reserved", ctypes.c_int32 * 4)]


class _AdamWConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps", "weight_decay")] + [
        ("step", ctypes.c_int64), ("seed", ctypes.c_uint64), ("bits", ctypes.c_int32), ("reserved", ctypes.c_int32 * 3)]


class _AdamWTensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("p", "g", "copy", "m", "v", "m_scale", "v_scale")] + [
        ("n", ctypes.c_int64), ("rng_base", ctypes.c_int64), ("p_dtype", ctypes.c_int32), ("g_dtype", ctypes.c_int32)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libmoe; raises if it has not been built for this machine."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libmoe is not built ({LIB_PATH} missing): run tile_level_copy_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        vp, sz, i32p = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(ctypes.c_int32)
        cfgp = ctypes.POINTER(_Config)
        L.moe_workspace_size.argtypes = [cfgp, ctypes.POINTER(sz)]
        L.moe_workspace_layout.argtypes = [cfgp, ctypes.POINTER(_Layout)]
        L.moe_plan.argtypes = [cfgp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_forward.argtypes = [cfgp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_forward_sequential.argtypes = [cfgp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_forward_ex.argtypes = [cfgp, vp, vp, vp, vp, vp, vp, vp, sz, ctypes.c_int, ctypes.POINTER(vp), vp]
        L.moe_forward_host.argtypes = [cfgp, vp, vp, vp, vp, vp, vp, vp, sz, ctypes.c_int, vp]
        L.moe_forward_host_pipelined.argtypes = [cfgp, ctypes.c_int, ctypes.POINTER(vp), ctypes.POINTER(vp), vp, vp,
                                                 vp, ctypes.POINTER(vp), vp, sz, ctypes.c_int, vp]
        L.moe_copy_only.argtypes = [cfgp, vp, sz, ctypes.c_int, vp]
        L.moe_dma_host_bytes.argtypes = [cfgp, ctypes.POINTER(sz)]
        L.moe_forward_dma.argtypes = [cfgp, vp, vp, vp, vp, vp, vp, vp, sz, vp, sz, ctypes.POINTER(vp), vp]
        L.moe_status.argtypes = [cfgp, vp, vp, i32p]
        L.moe_device_info.argtypes = [i32p, i32p]
        L.moe_route_static.argtypes = [cfgp, vp, vp, vp, vp, vp, vp, vp]
        fcfg, lcfg, acfg = (ctypes.POINTER(t) for t in (_FFNConfig, _LayerNormConfig, _AdamWConfig))
        szp, tens, vpp = ctypes.POINTER(sz), ctypes.POINTER(_AdamWTensor), ctypes.POINTER(vp)
        L.moe_ffn_workspace_size.argtypes = [fcfg, szp]
        L.moe_ffn_saved_size.argtypes = [fcfg, szp]
        L.moe_ffn_forward.argtypes = [fcfg] + [vp] * 7 + [sz, vp]
        L.moe_ffn_backward.argtypes = [fcfg] + [vp] * 11 + [sz, vp]
        L.moe_ffn_status.argtypes = [fcfg, vp, vp, i32p]
        L.moe_layernorm_forward.argtypes = [lcfg] + [vp] * 7
        L.moe_layernorm_workspace_size.argtypes = [lcfg, szp]
        L.moe_layernorm_backward.argtypes = [lcfg] + [vp] * 9 + [sz, vp]
        L.moe_adamw_step.argtypes = [acfg, tens, ctypes.c_int32, vp, vp]
        L.moe_adamw_read_state.argtypes = [tens, ctypes.c_int32, vpp, vpp, vp]
        L.moe_last_error.restype = ctypes.c_char_p
        for n in EXPORTS[:-1]:
            getattr(L, n).restype = ctypes.c_int
        _lib = L
    return _lib


def _check(rc: int) -> None:
    if rc != MOE_OK:
        raise MoEError(rc, lib().moe_last_error().decode())


def workspace_size(cfg: Config) -> int:
    n = ctypes.c_size_t()
    c = cfg.to_c()
    _check(lib().moe_workspace_size(ctypes.byref(c), ctypes.byref(n)))
    return n.value


def workspace_layout(cfg: Config) -> dict:
    L = _Layout()
    c = cfg.to_c()
    _check(lib().moe_workspace_layout(ctypes.byref(c), ctypes.byref(L)))
    return {name: getattr(L, name) for name, _ in _Layout._fields_}


def _ptr(t: Optional[torch.Tensor], dtype=None, device=None, name="tensor"):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if device == "cuda" and not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    if device == "cpu" and t.is_cuda:
        raise ValueError(f"{name} must be in host memory")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


class Workspace:
    """Device workspace of one config (a torch uint8 buffer) with typed views of its regions."""

    _DT = {"idx": (torch.int32, "TK"), "gate": (torch.float32, "TK"), "rank": (torch.int32, "TK"),
           "slot": (torch.int32, "TK"), "cslot": (torch.int32, "TK"), "ret_slot": (torch.int32, "TK"),
           "counts": (torch.int32, "ER"), "yrow": (torch.int32, "PC"), "tile_crow": (torch.int32, "MT"),
           "band_item": (torch.int32, "MT"), "tok_of": (torch.int32, "PC"), "xrows": (torch.int32, "E"),
           "xready": (torch.int32, "E"),
           "offsets": (torch.int32, "G1"), "ret_off": (torch.int32, "RE1"), "tiles": (torch.int32, "MT4"),
           "tile_ret": (torch.int32, "MT"), "sched": (torch.int32, "MT"), "order": (torch.int32, "MT"),
           "seg": (torch.int32, "MT2"),
           "experts": (torch.int32, "E8"), "items_up": (torch.int32, "IU2"),
           "items_down": (torch.int32, "MT2"), "meta": (torch.int32, "META"), "flags": (torch.int32, "FL"),
           "bands": (torch.int32, "MT"),
           "trace": (torch.int64, "TR"), "Xc": (torch.bfloat16, "PCd"), "Hc": (torch.bfloat16, "PCF"),
           "Yp": (torch.bfloat16, "Pd"), "Ret": (torch.bfloat16, "TKd")}

    def __init__(self, cfg: Config, device="cuda"):
        self.cfg = cfg
        self.layout = workspace_layout(cfg)
        self.nbytes = self.layout["bytes"]
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device)

    def view(self, name: str) -> torch.Tensor:
        c, L = self.cfg, self.layout
        dt, kind = self._DT[name]
        TK = c.T * c.topk
        shape = {"TK": (c.T, c.topk), "ER": (c.E, c.R), "G1": (c.E * c.R + 1,), "RE1": (c.R, c.E + 1),
                 "MT4": (L["MT_max"], 4), "MT": (L["MT_max"],), "MT2": (L["MT_max"], 2), "E8": (c.E, 8),
                 "META": (64,), "FL": (L["MT_max"], L["n_tiles_n2"]), "TR": (16,), "Pd": (L["P_max"], c.d),
                 "PCd": (L["PC_max"], c.d), "PC": (L["PC_max"],), "E": (c.E,), "PCF": (L["PC_max"], c.ffn), "IU2": (L["IU_max"], 2),
                 "TKd": (TK, c.d)}[kind]
        n = 1
        for s in shape:
            n *= s
        esz = torch.empty((), dtype=dt).element_size()
        off = L[name]
        return self.buf[off:off + n * esz].view(dt).view(shape)

    @property
    def ptr(self) -> ctypes.c_void_p:
        return ctypes.c_void_p(self.buf.data_ptr())


def plan(cfg: Config, logits: torch.Tensor, x: Optional[torch.Tensor], ws: Workspace,
         topk_idx: Optional[torch.Tensor] = None, topk_w: Optional[torch.Tensor] = None, stream=None) -> None:
    c = cfg.to_c()
    _check(lib().moe_plan(ctypes.byref(c), _ptr(logits, torch.float32, "cuda", "logits"),
                          _ptr(x, torch.bfloat16, "cuda", "x"), _ptr(topk_idx, torch.int32, "cuda", "topk_idx"),
                          _ptr(topk_w, torch.float32, "cuda", "topk_w"), ws.ptr, ws.nbytes, _stream(stream)))


def forward(cfg: Config, logits: torch.Tensor, x: torch.Tensor, W1: torch.Tensor, W3: torch.Tensor,
            W2: torch.Tensor, out: torch.Tensor, ws: Workspace, sequential: bool = False, stream=None,
            events=None) -> None:
    """moe_forward (tile-level overlapped return copy) or moe_forward_sequential.

    events: optional list of EV_COUNT recorded-once torch.cuda.Event (or None entries); the library
    records them between its launches (moe_forward_ex).
    """
    c = cfg.to_c()
    bf = torch.bfloat16
    args = (ctypes.byref(c), _ptr(logits, torch.float32, "cuda", "logits"), _ptr(x, bf, "cuda", "x"),
            _ptr(W1, bf, "cuda", "W1"), _ptr(W3, bf, "cuda", "W3"), _ptr(W2, bf, "cuda", "W2"),
            _ptr(out, torch.float32, "cuda", "out"), ws.ptr, ws.nbytes)
    if events is None:
        fn = lib().moe_forward_sequential if sequential else lib().moe_forward
        _check(fn(*args, _stream(stream)))
        return
    arr = (ctypes.c_void_p * EV_COUNT)(*[None if e is None else ctypes.c_void_p(e.cuda_event) for e in events])
    _check(lib().moe_forward_ex(*args, 1 if sequential else 0, arr, _stream(stream)))


def stage_events(n: int = EV_COUNT):
    """Timing events usable by forward(events=...): created and recorded once so they own a handle."""
    evs = [torch.cuda.Event(enable_timing=True) for _ in range(n)]
    for e in evs:
        e.record()
    return evs


def forward_host(cfg: Config, logits_h: torch.Tensor, x_h: torch.Tensor, W1: torch.Tensor, W3: torch.Tensor,
                 W2: torch.Tensor, out_h: torch.Tensor, ws: Workspace, sequential: bool = False, stream=None) -> None:
    """moe_forward_host: host logits / x in, host out; weights on the device."""
    c = cfg.to_c()
    bf = torch.bfloat16
    _check(lib().moe_forward_host(ctypes.byref(c), _ptr(logits_h, torch.float32, "cpu", "logits_h"),
                                  _ptr(x_h, bf, "cpu", "x_h"), _ptr(W1, bf, "cuda", "W1"),
                                  _ptr(W3, bf, "cuda", "W3"), _ptr(W2, bf, "cuda", "W2"),
                                  _ptr(out_h, torch.float32, "cpu", "out_h"), ws.ptr, ws.nbytes,
                                  1 if sequential else 0, _stream(stream)))


def forward_host_pipelined(cfg: Config, logits_h, x_h, W1: torch.Tensor, W3: torch.Tensor, W2: torch.Tensor,
                           out_h, ws: Workspace, sequential: bool = False, stream=None) -> None:
    """moe_forward_host_pipelined: len(out_h) batches, host inputs / outputs given as lists of pinned
    tensors (one per batch), transfers of neighbouring batches overlapped with the layer."""
    c = cfg.to_c()
    bf = torch.bfloat16
    n = len(out_h)
    if len(logits_h) != n or len(x_h) != n:
        raise ValueError("logits_h, x_h and out_h must have one entry per batch")
    arr = ctypes.c_void_p * max(n, 1)
    pl = arr(*[_ptr(t, torch.float32, "cpu", "logits_h") for t in logits_h])
    px = arr(*[_ptr(t, bf, "cpu", "x_h") for t in x_h])
    po = arr(*[_ptr(t, torch.float32, "cpu", "out_h") for t in out_h])
    _check(lib().moe_forward_host_pipelined(ctypes.byref(c), n, pl, px, _ptr(W1, bf, "cuda", "W1"),
                                            _ptr(W3, bf, "cuda", "W3"), _ptr(W2, bf, "cuda", "W2"), po, ws.ptr,
                                            ws.nbytes, 1 if sequential else 0, _stream(stream)))


def dma_host_bytes(cfg: Config) -> int:
    n = ctypes.c_size_t()
    c = cfg.to_c()
    _check(lib().moe_dma_host_bytes(ctypes.byref(c), ctypes.byref(n)))
    return n.value


def forward_dma(cfg: Config, logits: torch.Tensor, x: torch.Tensor, W1: torch.Tensor, W3: torch.Tensor,
                W2: torch.Tensor, out: torch.Tensor, ws: Workspace, host_rec: torch.Tensor, stream=None,
                events=None) -> None:
    """moe_forward_dma: the return copy on the copy engines. host_rec: a pinned host tensor of at least
    dma_host_bytes(cfg) bytes. Blocks until the down-projection has finished on the GPU."""
    c = cfg.to_c()
    bf = torch.bfloat16
    if not host_rec.is_pinned():
        raise ValueError("host_rec must be pinned host memory")
    arr = None if events is None else (ctypes.c_void_p * EV_COUNT)(
        *[None if e is None else ctypes.c_void_p(e.cuda_event) for e in events])
    _check(lib().moe_forward_dma(ctypes.byref(c), _ptr(logits, torch.float32, "cuda", "logits"), _ptr(x, bf, "cuda", "x"),
                                 _ptr(W1, bf, "cuda", "W1"), _ptr(W3, bf, "cuda", "W3"), _ptr(W2, bf, "cuda", "W2"),
                                 _ptr(out, torch.float32, "cuda", "out"), ws.ptr, ws.nbytes,
                                 _ptr(host_rec, None, "cpu", "host_rec"), host_rec.numel() * host_rec.element_size(),
                                 arr, _stream(stream)))


def copy_only(cfg: Config, ws: Workspace, ctas: int, stream=None) -> None:
    """moe_copy_only: the return copy of the last forward on ws, alone, on `ctas` SMs."""
    c = cfg.to_c()
    _check(lib().moe_copy_only(ctypes.byref(c), ws.ptr, ws.nbytes, int(ctas), _stream(stream)))


def status(cfg: Config, ws: Optional[Workspace], stream=None):
    """(return code, detail) of the last call on ws (ws None: of the last moe_route_static call on this
    device); synchronises the stream."""
    c = cfg.to_c()
    detail = ctypes.c_int32()
    rc = lib().moe_status(ctypes.byref(c), None if ws is None else ws.ptr, _stream(stream), ctypes.byref(detail))
    return rc, detail.value


def route_static(cfg: Config, logits: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor,
                 slot: torch.Tensor, ret_slot: torch.Tensor, offsets: torch.Tensor, stream=None) -> None:
    """moe_route_static: routing and row layout with the library's own static scratch (no workspace)."""
    c = cfg.to_c()
    i32 = torch.int32
    _check(lib().moe_route_static(ctypes.byref(c), _ptr(logits, torch.float32, "cuda", "logits"),
                                  _ptr(topk_idx, i32, "cuda", "topk_idx"), _ptr(topk_w, torch.float32, "cuda", "topk_w"),
                                  _ptr(slot, i32, "cuda", "slot"), _ptr(ret_slot, i32, "cuda", "ret_slot"),
                                  _ptr(offsets, i32, "cuda", "offsets"), _stream(stream)))


def device_info():
    sms, ok = ctypes.c_int32(), ctypes.c_int32()
    _check(lib().moe_device_info(ctypes.byref(sms), ctypes.byref(ok)))
    return sms.value, bool(ok.value)


# ---- operators of a training and serving block around the layer -----------------------------------


# The checks below are written for the calls of a decoding step, where a microsecond counts: one test of
# everything that is right, and the search for what is wrong only after it has failed.


# The current device: the kernels are launched there, so every tensor of a call has to be on it. The default
# stream is the current one of that device (as a raw handle).
_device = getattr(torch._C, "_cuda_getDevice", None)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _local(t: torch.Tensor, dtype, dev: int, name: str):
    """Device pointer of a contiguous tensor of this type (None: of any) on device dev."""
    p = _ptr(t, dtype, "cuda", name)
    if t.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the call is for cuda:{dev}")
    return p


def _dev(t: Optional[torch.Tensor], dtype, shape, dev: int, name: str):
    """Device pointer of a contiguous tensor of this type and shape on device dev (None: NULL)."""
    if t is None:
        return None
    if t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return _local(t, dtype, dev, name)


def _flat(t: Optional[torch.Tensor], dtype, n: int, dev: int, name: str):
    """The same for a tensor of n values of any shape."""
    if t is None:
        return None
    if t.dtype is dtype and t.get_device() == dev and t.numel() == n and t.is_contiguous():
        return t.data_ptr()
    if t.numel() != n:
        raise ValueError(f"{name} must hold {n} values, got {t.numel()}")
    return _local(t, dtype, dev, name)


def _space(ws, dev: int):
    """Pointer to a workspace on device dev."""
    if ws.buf.get_device() != dev:
        raise ValueError(f"the workspace is on {ws.buf.device}, the call is for cuda:{dev}")
    return ws.ptr


class _Marshalled:
    """A config that keeps its C form, and a pointer to it, until one of its fields is set."""

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        object.__setattr__(self, "_kept", None)

    def __getstate__(self):  # a copy, and a pickle, is made without the C form and its pointer
        return {**self.__dict__, "_kept": None}

    def ref(self):
        """Pointer to the C form (and whatever sizes the config's class keeps beside it)."""
        if self._kept is None:
            object.__setattr__(self, "_kept", self._make())
        return self._kept

    def _make(self):
        c = self.to_c()
        return (ctypes.byref(c), c)


@dataclasses.dataclass
class FFNConfig(_Marshalled):
    """Gated feed-forward block (mirrors moe_ffn_config): x, y [T, d]; W1, W3 [ffn, d]; W2 [d, ffn]."""

    T: int
    d: int
    ffn: int
    timeout_us: int = 0
    flags: int = 0

    def to_c(self) -> _FFNConfig:
        return _FFNConfig(int(self.T), int(self.d), int(self.ffn), int(self.timeout_us), int(self.flags))

    def _make(self):
        c, n = self.to_c(), ctypes.c_size_t()
        _check(lib().moe_ffn_saved_size(ctypes.byref(c), ctypes.byref(n)))
        return (ctypes.byref(c), c, (self.T, self.d), (self.ffn, self.d), (self.d, self.ffn), n.value)


class FFNWorkspace:
    """Device workspace of one feed-forward config; its status words start as zero, and are so for calls on
    any stream (the constructor waits for their clearing, unless the current stream is being captured)."""

    def __init__(self, cfg: FFNConfig, device="cuda"):
        n, c = ctypes.c_size_t(), cfg.to_c()
        _check(lib().moe_ffn_workspace_size(ctypes.byref(c), ctypes.byref(n)))
        self.nbytes = n.value
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        self.buf[:MOE_FFN_STATUS_BYTES].zero_()
        if self.buf.is_cuda and not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(self.buf.device).synchronize()
        self.ptr = self.buf.data_ptr()


def ffn_saved(cfg: FFNConfig, device="cuda") -> torch.Tensor:
    """Buffer in which ffn_forward keeps what ffn_backward needs (uint8, opaque)."""
    return torch.empty(cfg.ref()[5], dtype=torch.uint8, device=device)


def _saved(saved, need: int, dev: int):
    if saved is None:
        return None
    n = saved.numel() * saved.element_size()
    if n < need:
        raise ValueError(f"saved has {n} bytes, needs {need}")
    return _local(saved, None, dev, "saved")


def ffn_forward(cfg: FFNConfig, x: torch.Tensor, W1: torch.Tensor, W3: torch.Tensor, W2: torch.Tensor,
                y: torch.Tensor, ws: FFNWorkspace, saved: Optional[torch.Tensor] = None, stream=None) -> None:
    """moe_ffn_forward: y = (silu(x W1^T) * (x W3^T)) W2^T; saved (ffn_saved) for a backward pass."""
    bf, on = torch.bfloat16, _device()
    c, _, rows, up, down, need = cfg.ref()
    _check(lib().moe_ffn_forward(c, _dev(x, bf, rows, on, "x"), _dev(W1, bf, up, on, "W1"), _dev(W3, bf, up, on, "W3"),
                                 _dev(W2, bf, down, on, "W2"), _dev(y, bf, rows, on, "y"), _saved(saved, need, on),
                                 _space(ws, on), ws.nbytes,
                                 _current_stream(on) if stream is None else _stream(stream)))


def ffn_backward(cfg: FFNConfig, x: torch.Tensor, W1: torch.Tensor, W3: torch.Tensor, W2: torch.Tensor,
                 dy: torch.Tensor, saved: torch.Tensor, dx: torch.Tensor, dW1: torch.Tensor, dW3: torch.Tensor,
                 dW2: torch.Tensor, ws: FFNWorkspace, stream=None) -> None:
    """moe_ffn_backward: gradients of x and the weights from dy and the forward pass's saved buffer."""
    bf, on = torch.bfloat16, _device()
    c, _, rows, up, down, need = cfg.ref()
    _check(lib().moe_ffn_backward(c, _dev(x, bf, rows, on, "x"), _dev(W1, bf, up, on, "W1"),
                                  _dev(W3, bf, up, on, "W3"), _dev(W2, bf, down, on, "W2"),
                                  _dev(dy, bf, rows, on, "dy"), _saved(saved, need, on), _dev(dx, bf, rows, on, "dx"),
                                  _dev(dW1, bf, up, on, "dW1"), _dev(dW3, bf, up, on, "dW3"),
                                  _dev(dW2, bf, down, on, "dW2"), _space(ws, on), ws.nbytes,
                                  _current_stream(on) if stream is None else _stream(stream)))


def ffn_status(cfg: FFNConfig, ws: FFNWorkspace, stream=None):
    """(return code, detail) of the calls on ws; synchronises the stream."""
    detail = ctypes.c_int32()
    rc = lib().moe_ffn_status(cfg.ref()[0], _space(ws, _device()), _stream(stream), ctypes.byref(detail))
    return rc, detail.value


@dataclasses.dataclass
class LayerNormConfig(_Marshalled):
    """Layer norm over rows of d values (mirrors moe_layernorm_config)."""

    rows: int
    d: int
    dtype: torch.dtype = torch.bfloat16
    wdtype: torch.dtype = torch.float32
    eps: float = 1e-5

    def to_c(self) -> _LayerNormConfig:
        if self.dtype not in _DTYPES or self.wdtype not in _DTYPES:
            raise ValueError(f"layer norm takes float32, bfloat16 or float16, got {self.dtype}, {self.wdtype}")
        return _LayerNormConfig(int(self.rows), int(self.d), _DTYPES[self.dtype], _DTYPES[self.wdtype],
                                float(self.eps))


class LayerNormWorkspace:
    """Device workspace of layernorm_backward."""

    def __init__(self, cfg: LayerNormConfig, device="cuda"):
        n = ctypes.c_size_t()
        _check(lib().moe_layernorm_workspace_size(cfg.ref()[0], ctypes.byref(n)))
        self.nbytes = n.value
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        self.ptr = self.buf.data_ptr()


def layernorm_forward(cfg: LayerNormConfig, x: torch.Tensor, w: Optional[torch.Tensor], b: Optional[torch.Tensor],
                      y: torch.Tensor, mean: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
                      stream=None) -> None:
    """moe_layernorm_forward: y = (x - mean) * rstd * w + b; mean and rstd [rows] for a backward pass."""
    dt, wt, rows, d, on = cfg.dtype, cfg.wdtype, cfg.rows, cfg.d, _device()
    n, f32 = rows * d, torch.float32
    _check(lib().moe_layernorm_forward(
        cfg.ref()[0], _flat(x, dt, n, on, "x"), _flat(w, wt, d, on, "w"), _flat(b, wt, d, on, "b"),
        _flat(y, dt, n, on, "y"), _flat(mean, f32, rows, on, "mean"), _flat(rstd, f32, rows, on, "rstd"),
        _current_stream(on) if stream is None else _stream(stream)))


def layernorm_backward(cfg: LayerNormConfig, dy: torch.Tensor, x: torch.Tensor, w: Optional[torch.Tensor],
                       mean: torch.Tensor, rstd: torch.Tensor, dx: torch.Tensor, dw: Optional[torch.Tensor] = None,
                       db: Optional[torch.Tensor] = None, ws: Optional[LayerNormWorkspace] = None,
                       stream=None) -> None:
    """moe_layernorm_backward: dx, and dw, db summed over the rows (both may be None, then ws too)."""
    dt, wt, rows, d, on = cfg.dtype, cfg.wdtype, cfg.rows, cfg.d, _device()
    n, f32 = rows * d, torch.float32
    _check(lib().moe_layernorm_backward(
        cfg.ref()[0], _flat(dy, dt, n, on, "dy"), _flat(x, dt, n, on, "x"), _flat(w, wt, d, on, "w"),
        _flat(mean, f32, rows, on, "mean"), _flat(rstd, f32, rows, on, "rstd"), _flat(dx, dt, n, on, "dx"),
        _flat(dw, wt, d, on, "dw"), _flat(db, wt, d, on, "db"), None if ws is None else _space(ws, on),
        0 if ws is None else ws.nbytes, _current_stream(on) if stream is None else _stream(stream)))


@dataclasses.dataclass
class AdamWConfig(_Marshalled):
    """AdamW's numbers (mirrors moe_adamw_config; the step is an argument of adamw_step). bits: 32 or 8."""

    lr: float
    beta1: float = 0.9
    beta2: float = 0.999
    eps: float = 1e-8
    weight_decay: float = 0.01
    bits: int = 32
    seed: int = 0

    def to_c(self, step: int = 1) -> _AdamWConfig:
        return _AdamWConfig(self.lr, self.beta1, self.beta2, self.eps, self.weight_decay, int(step),
                            int(self.seed) & (2 ** 64 - 1), int(self.bits))


class AdamWList:
    """The tensors of an AdamW step, marshalled once: parameters p and gradients g (float32 or bfloat16),
    states m and v (float32; with bits = 8 uint8 codes with one uint8 scale per MOE_ADAMW_BLOCK values in
    m_scale, v_scale), and optional bfloat16 copies of the updated parameters. rng_base: index of each
    tensor's first value under the config's seed (default: one tensor after another, each rounded up
    to whole blocks). The list keeps its tensors alive; a tensor that moves needs a new list."""

    def __init__(self, cfg: AdamWConfig, p, g, m, v, m_scale=None, v_scale=None, copy=None, rng_base=None):
        n, f32, bf, u8 = len(p), torch.float32, torch.bfloat16, torch.uint8
        eight = cfg.bits == 8
        if eight != (m_scale is not None) or eight != (v_scale is not None):
            raise ValueError("m_scale and v_scale go with bits = 8")
        for name, l in (("g", g), ("m", m), ("v", v), ("m_scale", m_scale), ("v_scale", v_scale), ("copy", copy),
                        ("rng_base", rng_base)):
            if l is not None and len(l) != n:
                raise ValueError(f"{name} must have one entry per tensor")
        self.bits, self.count = cfg.bits, n
        self.device = p[0].get_device() if n else None
        self.c = (_AdamWTensor * max(n, 1))()
        self.keep = [list(l) for l in (p, g, m, v, m_scale, v_scale, copy) if l is not None]
        base = 0
        for i in range(n):
            k = p[i].numel()
            blocks = -(-k // MOE_ADAMW_BLOCK)
            for name, t, dt, want in (("p", p[i], (f32, bf), k), ("g", g[i], (f32, bf), k),
                                      ("m", m[i], (u8,) if eight else (f32,), k),
                                      ("v", v[i], (u8,) if eight else (f32,), k),
                                      ("m_scale", m_scale[i] if eight else None, (u8,), blocks),
                                      ("v_scale", v_scale[i] if eight else None, (u8,), blocks),
                                      ("copy", copy[i] if copy is not None else None, (bf,), k)):
                if t is None:
                    continue
                if t.dtype not in dt:
                    raise ValueError(f"{name}[{i}] must be {' or '.join(map(str, dt))}, got {t.dtype}")
                if t.numel() != want:
                    raise ValueError(f"{name}[{i}] must hold {want} values, got {t.numel()}")
                setattr(self.c[i], name, _local(t, None, self.device, f"{name}[{i}]"))
            e = self.c[i]
            e.n, e.rng_base = k, base if rng_base is None else int(rng_base[i])
            e.p_dtype, e.g_dtype = _DTYPES[p[i].dtype], _DTYPES[g[i].dtype]
            base += blocks * MOE_ADAMW_BLOCK


class AdamWValues:
    """Where adamw_read_state writes: float32 tensors, one m and one v for each tensor of the list."""

    def __init__(self, tensors: AdamWList, m, v):
        if len(m) != tensors.count or len(v) != tensors.count:
            raise ValueError("m and v must have one entry per tensor")
        arr = ctypes.c_void_p * max(tensors.count, 1)
        for name, l in (("m", m), ("v", v)):
            for i, t in enumerate(l):
                if t.numel() != tensors.c[i].n:
                    raise ValueError(f"{name}[{i}] must hold {tensors.c[i].n} values, got {t.numel()}")
        self.m = arr(*[_local(t, torch.float32, tensors.device, "m") for t in m])
        self.v = arr(*[_local(t, torch.float32, tensors.device, "v") for t in v])
        self.keep = [list(m), list(v)]


def _list_device(tensors: AdamWList, on: int) -> None:
    """Refuses a list whose tensors are not on the current device."""
    if tensors.count and tensors.device != on:
        raise ValueError(f"the list's tensors are on cuda:{tensors.device}, the call is for cuda:{on}")


def adamw_step(cfg: AdamWConfig, tensors: AdamWList, step: int, grad_scale: Optional[torch.Tensor] = None,
               stream=None) -> None:
    """moe_adamw_step: one step (counted from 1) over every tensor; grad_scale: a float32 value on the GPU.
    Captured into a graph, it is the same step, with the same random bits, at every replay."""
    if cfg.bits != tensors.bits:
        raise ValueError(f"the list was made for {tensors.bits}-bit states")
    on = _device()
    if tensors.device != on:
        _list_device(tensors, on)
    c = _AdamWConfig.from_buffer_copy(cfg.ref()[1])  # its own: threads may step at once with one config
    c.step = step
    _check(lib().moe_adamw_step(ctypes.byref(c), tensors.c, tensors.count,
                                None if grad_scale is None else _flat(grad_scale, torch.float32, 1, on, "grad_scale"),
                                _current_stream(on) if stream is None else _stream(stream)))


def adamw_read_state(cfg: AdamWConfig, tensors: AdamWList, out: AdamWValues, stream=None) -> None:
    """moe_adamw_read_state: the float32 values that the list's 8-bit states stand for."""
    if cfg.bits != 8 or tensors.bits != 8:
        raise ValueError("32-bit states are read as they are")
    on = _device()
    _list_device(tensors, on)
    _check(lib().moe_adamw_read_state(tensors.c, tensors.count, out.m, out.v,
                                      _current_stream(on) if stream is None else _stream(stream)))
