"""Calls of the block operators beside one another: threads, streams, graphs."""
import sys
import threading

import pytest
import torch

import tile_level_copy_gb300 as tlc

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16


def norm(rows, d, seed):
    g = torch.Generator().manual_seed(seed)
    x, dy = (torch.randn(rows, d, generator=g).to(BF).cuda() for _ in range(2))
    w = torch.randn(d, generator=g).cuda()
    cfg = tlc.LayerNormConfig(rows, d, BF, F32)
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    tlc.layernorm_forward(cfg, x, w, w, y, mean, rstd)
    ws, dx, dw, db = tlc.LayerNormWorkspace(cfg), torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    torch.cuda.synchronize()
    return lambda: tlc.layernorm_backward(cfg, dy, x, w, mean, rstd, dx, dw, db, ws), (dx, dw, db)


def test_layernorm_backward_of_two_widths_in_threads():
    """Widths that share a kernel and differ in its shared memory, each from a thread of its own, with streams
    and buffers of their own: every call is launched and gives what it gives alone."""
    errors = []

    def work(d):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                call, out = norm(8, d, d)
                call()
                torch.cuda.current_stream().synchronize()
                alone = [t.clone() for t in out]
                for _ in range(4000):
                    call()
                torch.cuda.current_stream().synchronize()
                for a, b in zip(out, alone):
                    assert torch.equal(a, b)
        except Exception as e:
            errors.append(f"d={d}: {e!r}")

    old = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        threads = [threading.Thread(target=work, args=(d,)) for d in (1280, 2048, 3080, 4096)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(old)
    assert not errors


def test_layernorm_backward_of_two_widths_in_a_graph():
    """The wider call's launch is captured before the narrower one's: the graph is made and gives what the
    calls give by themselves."""
    (wide, a), (narrow, b) = norm(8, 4096, 1), norm(8, 2048, 2)
    wide()
    narrow()
    torch.cuda.synchronize()
    alone = [t.clone() for t in (*a, *b)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wide()
        narrow()
    for t in (*a, *b):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for t, want in zip((*a, *b), alone):
        assert torch.equal(t, want)


def test_a_new_ffn_workspace_is_ready_on_every_stream():
    """The workspace's status words and counts have to be zero before a call on any stream reads them: nothing
    of their clearing is left on the stream that was current when the workspace was made."""
    cfg = tlc.FFNConfig(4, 128, 256)
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)  # about 10 ms on the current stream
    ws = tlc.FFNWorkspace(cfg)
    assert torch.cuda.current_stream().query()
    assert not ws.buf[:tlc.MOE_FFN_STATUS_BYTES].any()
