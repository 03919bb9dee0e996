"""Memory that the residual norm's outputs share with its inputs: refused before any CUDA call where a row's output could
change what another row reads, and tensors side by side in one buffer taken."""
import ctypes
import itertools

import pytest
import torch

import tile_level_copy_gb300 as tlc

ROWS, D, GROUP = 10, 24, 4
CFG = tlc.ResidualNormConfig(ROWS, D, torch.bfloat16, torch.float32, tlc.MOE_NORM_LAYER, tlc.MOE_NORM_LAYER, GROUP)
GATES = -(-ROWS // GROUP)
BYTES = {**dict.fromkeys("x u h z dz dh dx du".split(), ROWS * D * 2), **dict.fromkeys(("post_stats", "pre_stats"), ROWS * 8),
         **dict.fromkeys("post_w post_b pre_w pre_b dpost_w dpost_b dpre_w dpre_b".split(), D * 4), "gate": GATES * D * 4,
         "dgate": GATES * D * 4}
FORWARD = "x u post_w post_b gate pre_w pre_b h z post_stats pre_stats".split()
BACKWARD = "dz dh u h post_w post_b gate pre_w post_stats pre_stats dx du dpost_w dpost_b dgate dpre_w dpre_b ws".split()
WEIGHTS = ["post_w", "post_b", "gate", "pre_w", "pre_b"]
SUMS = ["dpost_w", "dpost_b", "dgate", "dpre_w", "dpre_b"]


def workspace_bytes(lib):
    n = ctypes.c_size_t()
    assert lib.moe_residual_norm_workspace_size(ctypes.byref(CFG.to_c()), ctypes.byref(n)) == tlc.MOE_OK
    return n.value


def refused(lib, names, a, b, where):
    """The call with a's memory over the end or the start of b's, or right at its start."""
    at = {n: (1 << 40) + (i << 24) for i, n in enumerate(names)}
    at[a] = at[b] + {"end": BYTES[b] - 16 + BYTES[b] % 16, "start": 16 - BYTES[a] - BYTES[a] % 16, "same": 0}[where]
    p = [ctypes.c_void_p(at[n]) for n in names]
    cfg = ctypes.byref(CFG.to_c())
    if names is FORWARD:
        return lib.moe_residual_norm_forward(cfg, *p, None)
    return lib.moe_residual_norm_backward(cfg, *p, workspace_bytes(lib), None)


@pytest.mark.parametrize("where", ["end", "start", "same"])
def test_forward_outputs_apart_from_weights_and_one_another(built_library, where):
    pairs = [*itertools.product(["h", "z", "post_stats", "pre_stats"], WEIGHTS), *itertools.product(["post_stats", "pre_stats"], "xuhz"),
             ("h", "z"), ("post_stats", "pre_stats")]
    for a, b in pairs:
        assert refused(built_library, FORWARD, a, b, where) == tlc.MOE_ERR_ARG, (a, b)
        assert b"share" in built_library.moe_last_error(), (a, b)


@pytest.mark.parametrize("where", ["end", "start", "same"])
def test_backward_outputs_apart_from_weights_and_one_another(built_library, where):
    rows, ins = ["dx", "du"], ["dz", "dh", "u", "h", *WEIGHTS[:4], "post_stats", "pre_stats"]
    pairs = [*itertools.product(rows, [*ins[4:], *SUMS]), *itertools.product(SUMS, ins), ("dx", "du"), *itertools.combinations(SUMS, 2)]
    for a, b in pairs:
        assert refused(built_library, BACKWARD, a, b, where) == tlc.MOE_ERR_ARG, (a, b)
        assert b"share" in built_library.moe_last_error(), (a, b)


KIND = {n: torch.bfloat16 if b == ROWS * D * 2 else torch.float32 for n, b in BYTES.items()}
SHAPE = {n: {ROWS * D * 2: (ROWS, D), D * 4: (D,), GATES * D * 4: (GATES, D), ROWS * 8: (ROWS, 2)}[b] for n, b in BYTES.items()}


@pytest.mark.gpu
@pytest.mark.parametrize("name", BACKWARD[:-1])
def test_workspace_apart_from_everything(name):
    """A workspace that begins or ends inside of a tensor, in a buffer that holds both."""
    ws = tlc.ResidualNormWorkspace(CFG)
    buf = torch.zeros(2 * ws.nbytes + 4096, dtype=torch.uint8, device="cuda")
    t = {n: torch.zeros(SHAPE[n], dtype=KIND[n], device="cuda") for n in BACKWARD[:-1]}
    t[name] = buf[ws.nbytes:ws.nbytes + BYTES[name]].view(KIND[name]).view(SHAPE[name])
    for at in (ws.nbytes, ws.nbytes + (BYTES[name] - 1) // 16 * 16):
        ws.buf, ws.ptr = buf, buf.data_ptr() + at
        with pytest.raises(tlc.MoEError, match="share") as e:
            tlc.residual_norm_backward(CFG, *(t[n] for n in BACKWARD[:-1]), ws)
        assert e.value.code == tlc.MOE_ERR_ARG


@pytest.mark.gpu
def test_tensors_side_by_side_in_one_buffer():
    """Every tensor of both calls next to the one before, no byte between them: what separate tensors give."""
    g = torch.Generator().manual_seed(1)

    def call(place):
        t = {n: place(n) for n in dict.fromkeys(FORWARD + BACKWARD) if n != "ws"}
        g.manual_seed(1)
        for n in ("x", "u", "dz", "dh", *WEIGHTS):
            t[n].copy_(torch.randn(t[n].shape, generator=g))
        tlc.residual_norm_forward(CFG, *(t[n] for n in FORWARD))
        tlc.residual_norm_backward(CFG, *(t[n] for n in BACKWARD[:-1]), tlc.ResidualNormWorkspace(CFG))
        return {n: t[n].clone() for n in ("h", "z", "dx", "du", *SUMS, "post_stats", "pre_stats")}

    arena, used = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda"), [0]

    def inside(n):
        used[0] += BYTES[n]
        return arena[used[0] - BYTES[n]:used[0]].view(KIND[n]).view(SHAPE[n])

    want = call(lambda n: torch.zeros(SHAPE[n], dtype=KIND[n], device="cuda"))
    got = call(inside)
    assert all(torch.equal(got[n], want[n]) for n in want)
