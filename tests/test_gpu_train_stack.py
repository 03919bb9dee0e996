"""A training step's operators together: a stack of blocks with norms on both sides, a router beside it, clipping and AdamW."""
import pytest
import torch

import tile_level_copy_gb300 as tlc
from tile_level_copy_gb300 import train_block

pytestmark = pytest.mark.gpu
BF, D = torch.bfloat16, torch.float64


def rms(x, w):
    return x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-5) * w


def reference(stack, x, dy):
    """y, dx and the parameters' gradients by autograd in 64 bits, from the stack's current weights."""
    p = {n: stack.weights.get(n, stack.p[n]).to(D).requires_grad_() for n in stack.p}
    h = xd = x.to(D).requires_grad_()
    z = rms(h, p["pre0"])
    for i in range(stack.layers):
        g = z @ p[f"W1_{i}"].T
        u = (g * torch.sigmoid(g) * (z @ p[f"W3_{i}"].T)) @ p[f"W2_{i}"].T
        h = h + p[f"gate{i}"] * rms(u, p[f"post{i}"])
        z = rms(h, p[f"pre{i + 1}"])
    z.backward(dy.to(D))
    return z.detach(), xd.grad, {n: t.grad for n, t in p.items()}


def rel(a, b):
    return ((a.double() - b).norm() / b.norm()).item()


@pytest.mark.parametrize("tokens,d,ffn,layers", [(77, 136, 264, 1), (512, 256, 1000, 2), (130, 1024, 512, 3)])
def test_gradients_are_autograds(tokens, d, ffn, layers):
    """A block rounds z, its hidden values, u and h on the way up, and dh, du, dz and two hidden gradients on the way
    down, to bf16. A rounding is off by at most 2^-8 of the value, evenly spread over half a step: for significands m spread
    over [1, 2) the relative error's root mean square is 2^-8 / sqrt(3) sqrt(mean of 1 / m^2) = 2^-8 / sqrt(6) = 1.6e-3.
    Nine of independent signs, which every norm passes on at about their size: 4.8e-3 sqrt(layers); twice that where a
    sum has few terms, less than the 1.02e-2 sqrt(layers) here."""
    stack = train_block.NormedStack(tokens, d, ffn, layers, seed=3)
    for n, t in stack.p.items():
        if t.dim() == 1:
            t.add_(0.1 * torch.randn(d, device="cuda"))
    x, dy = torch.randn(tokens, d, device="cuda").to(BF), (torch.randn(tokens, d, device="cuda") * 0.01).to(BF)
    y = stack.forward(x).clone()
    dx = stack.backward(dy)
    wy, wdx, wg = reference(stack, x, dy)
    most = 3 * 3.4e-3 * layers ** 0.5
    assert rel(y, wy) <= most and rel(dx, wdx) <= most
    for n, g in stack.grads.items():
        assert rel(g, wg[n]) <= most, n
    assert tlc.ffn_status(stack.ffn_cfg, stack.ffn_ws) == (tlc.MOE_OK, 0)


@pytest.mark.parametrize("bits", [8, 32])
def test_the_command_trains_a_stack(bits):
    losses = train_block.main(["--tokens", "300", "--d", "64", "--ffn", "128", "--bits", str(bits), "--steps", "6", "--layers", "2"])
    assert len(losses) == 6 and all(torch.isfinite(torch.tensor(losses)))


def test_a_step_is_clipped_by_the_norm_of_all_gradients():
    stack = train_block.NormedStack(200, 64, 128, 2, bits=32, max_norm=1e-3, seed=4)
    stack.forward(torch.randn(200, 64, device="cuda").to(BF))
    stack.backward(torch.randn(200, 64, device="cuda").to(BF))
    norm = torch.stack([g.double().square().sum() for g in stack.grads.values()]).sum().sqrt().item()
    before = {n: t.clone() for n, t in stack.p.items()}
    stack.step()
    n, scale = stack.clip.tolist()
    assert abs(n / norm - 1) <= 1e-6 and abs(scale * norm / 1e-3 - 1) <= 1e-6
    want = {k: t.clone() for k, t in before.items()}
    lst = tlc.AdamWList(stack.opt, list(want.values()), [stack.grads[k] for k in want],
                        *([torch.zeros_like(t) for t in want.values()] for _ in range(2)))
    tlc.adamw_step(stack.opt, lst, 1, grad_scale=torch.full((1,), scale, device="cuda"))
    for k in want:
        assert torch.equal(stack.p[k], want[k]), k


@pytest.mark.parametrize("tokens,d", [(37, 64), (300, 1032)])
def test_steps_behind_one_another_read_what_the_step_before_wrote(tokens, d):
    """Dependent launches start early: steps without a wait give bit for bit what steps with a wait between all calls give."""
    x, dy = (torch.randn(tokens, d, device="cuda").to(BF) for _ in range(2))
    a, b = (train_block.NormedStack(tokens, d, 128, 2, bits=32, lr=0.1, seed=6) for _ in range(2))
    torch.cuda.synchronize()
    for wait, stack in ((False, a), (True, b)):
        for _ in range(6):
            for call in (lambda: stack.forward(x), lambda: stack.backward(dy), stack.step):
                call()
                if wait:
                    torch.cuda.synchronize()
    assert all(torch.equal(a.p[n], b.p[n]) for n in a.p)


def test_a_routers_step_beside_a_stack():
    """Tokens normed by the stack, routed by the library; the router's loss = balance and z losses + <gates, r>: its
    weight's gradient through balance_backward against autograd in 64 bits, then both trained under one norm. logits in
    fp32 products of bf16 tokens: errors of 2^-24 in sums of 64 terms, and choices that are the library's."""
    T, d, E, k = 256, 64, 8, 2
    stack = train_block.NormedStack(T, d, 128, 1, bits=32, seed=5)
    z = stack.forward(torch.randn(T, d, device="cuda").to(BF))
    Wr = torch.randn(E, d, device="cuda") * d ** -0.5
    mask = (torch.rand(T, device="cuda") > 0.1).to(torch.uint8)
    logits = (z.double() @ Wr.double().T).float()
    cfg = tlc.Config(T=T, d=128, ffn=128, E=E, topk=k, R=2, tile_M=64, flags=tlc.MOE_PLAN_SKIP_PERMUTE)
    idx, gates = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    tlc.plan(cfg, logits, None, tlc.Workspace(cfg), idx, gates)
    r = torch.randn(T, k, device="cuda")
    bc = tlc.BalanceConfig(T, E, k, balance=0.5, z=0.1)
    loss, counts, saved = torch.empty(3, device="cuda"), torch.empty(1, E, dtype=torch.int32, device="cuda"), tlc.balance_saved(bc)
    tlc.balance_forward(bc, logits, idx, loss, counts, None, tlc.BalanceWorkspace(bc), mask=mask, saved=saved)
    dlogits = torch.empty_like(logits)
    tlc.balance_backward(bc, logits, idx, saved, dlogits, mask=mask, gates=gates, dgates=r)
    live = mask.bool()
    l = logits.double().requires_grad_()
    p, n = torch.softmax(l, 1)[live], live.sum()
    c = torch.zeros(E, dtype=D, device="cuda").index_add_(0, idx[live].long().flatten(), torch.ones(int(n) * k, dtype=D, device="cuda"))
    want = 0.5 * (E / (k * n) * c * p.sum(0) / n).sum() + 0.1 * torch.logsumexp(l, 1)[live].square().mean()
    assert abs(loss[0].item() / want.item() - 1) <= 2e-6 and torch.equal(counts[0], c.to(torch.int32))
    (want + (torch.softmax(l.gather(1, idx.long()), 1) * r)[live].sum()).backward()
    assert rel(dlogits, l.grad) <= 2e-6
    dWr = (dlogits.double().T @ z.double()).float()
    stack.backward((dlogits @ Wr).to(BF))
    params, grads = [*stack.p.values(), Wr], [*stack.grads.values(), dWr]
    gl, out = tlc.GradList(grads), torch.empty(2, device="cuda")
    tlc.grad_norm(tlc.GradNormConfig(0.1), gl, out, tlc.GradNormWorkspace())
    norm = torch.stack([g.double().square().sum() for g in grads]).sum().sqrt().item()
    assert abs(out[0].item() / norm - 1) <= 1e-6
    tlc.grad_clip(gl, out[1:])
    opt = tlc.AdamWConfig(lr=1e-3)
    lst = tlc.AdamWList(opt, params, grads, *([torch.zeros_like(t) for t in params] for _ in range(2)))
    tlc.adamw_step(opt, lst, 1)
    assert all(torch.isfinite(t).all() for t in params)
