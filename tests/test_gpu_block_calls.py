"""Calls of the block operators beside one another: threads, streams, graphs."""
import sys
import threading

import pytest
import torch

import tile_level_copy_gb300 as tlc
from oracle import block_ref as ref
from tests.test_gpu_adamw import HYPER, tensors
from tests.test_gpu_ffn import close, f64, forward, make

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


@pytest.mark.parametrize("T", [5, 700])
def test_backward_outputs_over_inputs_are_refused(T):
    """dx is written while dy is still read for the weight gradients (and the weights and x beside it): an
    output that shares memory with an input or with another output is refused."""
    d, f = 264, 264  # so that every matrix has the shape of every other
    cfg = tlc.FFNConfig(T, d, f)
    x, W1, W3, W2, dy = make(T, d, f)
    _, saved, ws = forward(cfg, x, W1, W3, W2, True)
    outs = [torch.empty_like(t) for t in (x, W1, W3, W2)]
    for i, others in ((0, (dy, x)), (1, (W1, W3, W2, outs[2], outs[3])), (2, (W1, W2, outs[3])), (3, (W3,))):
        for o in others:
            bad = list(outs)
            bad[i] = o
            with pytest.raises(tlc.MoEError) as e:
                tlc.ffn_backward(cfg, x, W1, W3, W2, dy, saved, *bad, ws)
            assert e.value.code == tlc.MOE_ERR_ARG
    tlc.ffn_backward(cfg, x, W1, W3, W2, dy, saved, *outs, ws)
    for got, want in zip(outs, ref.ffn_backward(*(f64(t) for t in (x, W1, W3, W2, dy)))):
        close(got, want)


def test_forward_in_place_and_over_its_inputs():
    """y may be x, which the second product no longer needs; over W2, which it reads, it is refused."""
    T, d, f = 264, 264, 264
    cfg = tlc.FFNConfig(T, d, f)
    x, W1, W3, W2, _ = make(T, d, f)
    y, saved, ws = forward(cfg, x, W1, W3, W2, True)
    with pytest.raises(tlc.MoEError) as e:
        tlc.ffn_forward(cfg, x, W1, W3, W2, W2, ws)
    assert e.value.code == tlc.MOE_ERR_ARG
    tlc.ffn_forward(cfg, x, W1, W3, W2, x, ws, saved=saved)
    assert torch.equal(x, y)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_captured_step_is_the_same_step_at_every_replay(bits):
    """The step is an argument of the launch: three replays give what three calls with its number give, bias
    correction and random bits among it, and not what steps that count on give."""
    def state():
        p, g, m, v, ms, vs = tensors([5000, 77], F32, BF, bits, 4)
        cfg = tlc.AdamWConfig(**HYPER, bits=bits, seed=11)
        return cfg, tlc.AdamWList(cfg, p, g, m, v, ms, vs), (*p, *m, *v, *(ms or []), *(vs or []))

    (cfg, lst, a), (_, calls, b), (_, counted, c) = state(), state(), state()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tlc.adamw_step(cfg, lst, 2)
    for i in range(3):
        graph.replay()
        tlc.adamw_step(cfg, calls, 2)
        tlc.adamw_step(cfg, counted, 2 + i)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert not torch.equal(a[0], c[0])


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-8, 1e-12])
@pytest.mark.parametrize("pt,gt", [(F32, F32), (F32, BF), (BF, BF)])
def test_a_step_does_not_depend_on_place_or_alignment(pt, gt, eps, bits):
    """Whole aligned chunks take a path of their own: p, copy and states have the same bits as those of the
    same values off an aligned start, and in a tensor's last chunk."""
    n = 3 * 4096 + 77
    out = []
    for shift in (0, 1):
        p, g, m, v, ms, vs = tensors([n], pt, gt, bits, 5, shift)
        c = [torch.zeros(n + shift, dtype=BF, device="cuda")[shift:]]
        cfg = tlc.AdamWConfig(**{**HYPER, "eps": eps}, bits=bits, seed=3)
        tlc.adamw_step(cfg, tlc.AdamWList(cfg, p, g, m, v, ms, vs, copy=c), 5)
        out.append((p[0], c[0], m[0], v[0]))
    for a, b in zip(*out):
        assert torch.equal(a, b)
