"""Bounded waits of the feed-forward block made to run out: by a load that never comes."""
import pytest
import torch

import tile_level_copy_gb300 as tlc
from oracle import block_ref as ref
from tests.test_gpu_ffn import close, f64, forward, make

pytestmark = pytest.mark.gpu
STALL0, STALL1 = tlc.MOE_FFN_TEST_STALL0, tlc.MOE_FFN_TEST_STALL1
# First launches on single CTAs (their k-blocks split over clusters of 4, of 8): status details from 20 on; on CTA
# pairs (whole tiles; tiles of the last wave in three parts): details below 20.
FEW, MANY = [(3, 264, 520), (2, 2048, 1408)], [(2304, 1032, 2048), (721, 2880, 3728)]
CASES = [(s, STALL0, 2) for s in FEW] + [(s, h, 1) for s in MANY for h in (STALL0, STALL1)]


@pytest.mark.parametrize("shape,hook,kernel", CASES)
def test_a_load_that_never_comes_is_reported_and_settled(shape, hook, kernel):
    """The TMA threads stop halfway through their first tile (of a pair one does: rank 1 then runs a ring of
    stages ahead of rank 0, or rank 0 waits for bytes that never come). Every call's waits run out and it ends,
    the status says so, and once the status words are zero the same workspace gives what it gave before."""
    T, d, f = shape
    x, W1, W3, W2, dy = make(T, d, f)
    cfg, stuck = tlc.FFNConfig(T, d, f), tlc.FFNConfig(T, d, f, timeout_us=20000, flags=hook)
    y, saved, ws = forward(cfg, x, W1, W3, W2, True)
    once = forward(cfg, x, W1, W3, W2, False, ws)[0]
    outs = [torch.empty_like(t) for t in (x, W1, W3, W2)]
    tlc.ffn_backward(cfg, x, W1, W3, W2, dy, saved, *outs, ws)
    assert tlc.ffn_status(cfg, ws) == (tlc.MOE_OK, 0)
    close(y, ref.ffn_forward(*(f64(t) for t in (x, W1, W3, W2))))
    spare, junk = torch.empty_like(saved), [torch.empty_like(t) for t in (x, W1, W3, W2)]
    calls = [lambda: tlc.ffn_forward(stuck, x, W1, W3, W2, junk[0], ws),
             lambda: tlc.ffn_forward(stuck, x, W1, W3, W2, junk[0], ws, saved=spare),
             lambda: tlc.ffn_backward(stuck, x, W1, W3, W2, dy, saved, *junk, ws)]
    for call in calls:
        call()
        rc, detail = tlc.ffn_status(stuck, ws)
        assert rc == tlc.MOE_ERR_TIMEOUT and detail // 10 == kernel, detail
        assert "ran out" in tlc.lib().moe_last_error().decode()
        # what has gone wrong stays on record, through a call that does not stall, until the words are zeroed
        tlc.ffn_forward(cfg, x, W1, W3, W2, junk[0], ws)
        assert tlc.ffn_status(cfg, ws) == (tlc.MOE_ERR_TIMEOUT, detail)
        ws.buf[:tlc.MOE_FFN_STATUS_BYTES].zero_()
        again = [torch.empty_like(t) for t in (x, x, *outs)]
        tlc.ffn_forward(cfg, x, W1, W3, W2, again[0], ws)
        tlc.ffn_forward(cfg, x, W1, W3, W2, again[1], ws, saved=spare)
        tlc.ffn_backward(cfg, x, W1, W3, W2, dy, spare, *again[2:], ws)
        assert tlc.ffn_status(cfg, ws) == (tlc.MOE_OK, 0)
        for a, b in zip(again, (once, y, *outs)):
            assert torch.equal(a, b)
