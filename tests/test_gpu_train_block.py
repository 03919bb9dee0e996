"""The operators together: a pre-norm gated block's training step and its single-token form."""
import pytest
import torch

import tile_level_copy_gb300 as tlc
from tile_level_copy_gb300 import train_block

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def reference(block, x, dy):
    """y, dx and the parameters' gradients by autograd in 64 bits, from the block's current weights."""
    D = torch.float64
    p = {n: (block.weights.get(n, block.p[n])).to(D).requires_grad_() for n in block.p}
    xd = x.to(D).requires_grad_()
    z = torch.nn.functional.layer_norm(xd, (x.shape[1],), p["w"], p["b"], 1e-5)
    g = z @ p["W1"].T
    y = xd + (g * torch.sigmoid(g) * (z @ p["W3"].T)) @ p["W2"].T
    y.backward(dy.to(D))
    return y.detach(), xd.grad, {n: t.grad for n, t in p.items()}


def rel(a, b):
    return ((a.double() - b).norm() / b.norm()).item()


@pytest.mark.parametrize("tokens,d,ffn", [(1, 64, 128), (77, 136, 264), (512, 256, 1000)])
def test_gradients_are_autograds(tokens, d, ffn):
    """The norm's output is rounded to bf16 before the products, which adds an error like that of the
    operands h, dg and du (each at most 2^-8 / sqrt(3) of the norm): up to four such errors of
    independent signs, and the result's own rounding: 2^-8 / sqrt(3) * sqrt(5) = 5.1e-3, twice that
    where a sum has few terms."""
    block = train_block.PreNormBlock(tokens, d, ffn, seed=3)
    block.p["w"].add_(0.1 * torch.randn(d, device="cuda"))
    block.p["b"].add_(0.1 * torch.randn(d, device="cuda"))
    x, dy = torch.randn(tokens, d, device="cuda").to(BF), (torch.randn(tokens, d, device="cuda") * 0.01).to(BF)
    y = block.forward(x)
    dx = block.backward(dy)
    wy, wdx, wg = reference(block, x, dy)
    assert rel(y, wy) <= 1.1e-2 and rel(dx, wdx) <= 1.1e-2
    for n, g in block.grads.items():
        assert rel(g, wg[n]) <= 1.1e-2, n
    assert tlc.ffn_status(block.ffn_cfg, block.ffn_ws) == (tlc.MOE_OK, 0)


@pytest.mark.parametrize("bits", [8, 32])
def test_training_lowers_the_loss(bits):
    """80 steps of AdamW on a block of 64 by 128 towards a fixed one, learning rate 3e-3: a weight moves by
    up to 0.24 in all, three times the matrices' deviation of 1 / sqrt(64), so most of the distance to
    the teacher can be covered."""
    losses = train_block.main(["--tokens", "2048", "--d", "64", "--ffn", "128", "--bits", str(bits), "--steps", "80",
                               "--lr", "3e-3"])
    assert losses[-1] < 0.7 * losses[0]


def test_copies_follow_the_parameters_and_decoding_agrees():
    block = train_block.PreNormBlock(300, 128, 256, seed=5)
    x = torch.randn(300, 128, device="cuda").to(BF)
    block.backward(block.forward(x))
    before = block.weights["W1"].clone()
    block.step()
    for n, w in block.weights.items():
        assert torch.equal(w, block.p[n].to(BF)), n
    assert not torch.equal(before, block.weights["W1"])
    y = block.forward(x)
    for batch in (1, 5):
        one = block.decoder(batch)(x[:batch].contiguous())
        # h and the result rounded twice in another order of sums: one unit in the last place of each
        assert rel(one, y[:batch].double()) <= 2.0 ** -7
