"""A pre-norm gated block trained with the library's operators: y = x + FFN(LN(x)).

PreNormBlock keeps what a training program keeps: fp32 parameters and the optimiser's states, bf16 copies
of the matrices for the products, gradients, workspaces and the kept activations. Each part runs in the
library: layer norm and feed-forward block in both directions, and one AdamW step over all
tensors (states in 8 or 32 bits, gradients scaled on the GPU to a largest norm). The residual sum and the
loss are torch operations.

    python -m tile_level_copy_gb300.train_block [--tokens 4096 --d 1024 --ffn 2816 --bits 8 --steps 50]

trains a block towards a fixed random one and prints the loss and the time of a step; with --decode it
then runs the trained block on single tokens.
"""
from __future__ import annotations

import argparse
import math

import torch

import tile_level_copy_gb300 as tlc

BF = torch.bfloat16


class PreNormBlock:
    def __init__(self, tokens: int, d: int, ffn: int, bits: int = 8, lr: float = 1e-3, weight_decay: float = 0.0,
                 max_norm: float = 1.0, seed: int = 0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        shapes = {"w": (d,), "b": (d,), "W1": (ffn, d), "W3": (ffn, d), "W2": (d, ffn)}
        self.p = {n: torch.randn(s, generator=g, device=device) * s[-1] ** -0.5 for n, s in shapes.items()}
        self.p["w"].fill_(1.0)
        self.p["b"].zero_()
        self.weights = {n: self.p[n].to(BF) for n in ("W1", "W3", "W2")}
        self.grads = {n: torch.empty(s, device=device, dtype=BF if n in self.weights else torch.float32)
                      for n, s in shapes.items()}
        self.ffn_cfg = tlc.FFNConfig(T=tokens, d=d, ffn=ffn)
        self.ffn_ws, self.saved = tlc.FFNWorkspace(self.ffn_cfg, device), tlc.ffn_saved(self.ffn_cfg, device)
        self.ln_cfg = tlc.LayerNormConfig(rows=tokens, d=d, dtype=BF, wdtype=torch.float32)
        self.ln_ws = tlc.LayerNormWorkspace(self.ln_cfg, device)
        rows = lambda: torch.empty(tokens, d, dtype=BF, device=device)  # noqa: E731
        self.normed, self.out, self.dnormed, self.dx = rows(), rows(), rows(), rows()
        self.mean, self.rstd = (torch.empty(tokens, device=device) for _ in range(2))
        self.max_norm, self.steps = max_norm, 0

        self.opt = tlc.AdamWConfig(lr=lr, weight_decay=weight_decay, bits=bits, seed=seed)
        names = list(shapes)
        state = torch.uint8 if bits == 8 else torch.float32
        zeros = lambda: [torch.zeros(s, dtype=state, device=device) for s in shapes.values()]  # noqa: E731
        scales = lambda: [torch.zeros(-(-math.prod(s) // tlc.MOE_ADAMW_BLOCK), dtype=torch.uint8, device=device)  # noqa: E731
                          for s in shapes.values()] if bits == 8 else None
        self.list = tlc.AdamWList(self.opt, [self.p[n] for n in names], [self.grads[n] for n in names], zeros(),
                                  zeros(), scales(), scales(), copy=[self.weights.get(n) for n in names])

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        """y = x + FFN(LN(x)) for x [tokens, d] bf16; keeps what backward needs."""
        self.x = x
        tlc.layernorm_forward(self.ln_cfg, x, self.p["w"], self.p["b"], self.normed, self.mean, self.rstd)
        W = self.weights
        tlc.ffn_forward(self.ffn_cfg, self.normed, W["W1"], W["W3"], W["W2"], self.out, self.ffn_ws, saved=self.saved)
        return x + self.out

    def backward(self, dy: torch.Tensor) -> torch.Tensor:
        """The loss's gradient at x; the parameters' gradients are left in self.grads."""
        W, g = self.weights, self.grads
        tlc.ffn_backward(self.ffn_cfg, self.normed, W["W1"], W["W3"], W["W2"], dy, self.saved, self.dnormed, g["W1"],
                         g["W3"], g["W2"], self.ffn_ws)
        tlc.layernorm_backward(self.ln_cfg, self.dnormed, self.x, self.p["w"], self.mean, self.rstd, self.dx, g["w"],
                               g["b"], self.ln_ws)
        return dy + self.dx

    def step(self) -> None:
        """AdamW, the gradients scaled so that their norm is at most max_norm (decided on the GPU)."""
        norm = torch.stack([t.float().square().sum() for t in self.grads.values()]).sum().sqrt()
        scale = (self.max_norm / (norm + 1e-12)).clamp(max=1.0).reshape(1)
        self.steps += 1
        tlc.adamw_step(self.opt, self.list, self.steps, grad_scale=scale)

    def decoder(self, batch: int):
        """A function x [batch, d] -> y with the trained weights: the form of single-token decoding."""
        d, ffn = self.ffn_cfg.d, self.ffn_cfg.ffn
        fc, lc = tlc.FFNConfig(T=batch, d=d, ffn=ffn), tlc.LayerNormConfig(rows=batch, d=d, dtype=BF)
        W, device = self.weights, self.dx.device
        ws = tlc.FFNWorkspace(fc, device)
        normed, out = (torch.empty(batch, d, dtype=BF, device=device) for _ in range(2))

        def run(x: torch.Tensor) -> torch.Tensor:
            tlc.layernorm_forward(lc, x, self.p["w"], self.p["b"], normed)
            tlc.ffn_forward(fc, normed, W["W1"], W["W3"], W["W2"], out, ws)
            return x + out

        return run


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--d", type=int, default=1024)
    ap.add_argument("--ffn", type=int, default=2816)
    ap.add_argument("--bits", type=int, default=8, choices=(8, 32))
    ap.add_argument("--steps", type=int, default=50)
    ap.add_argument("--lr", type=float, default=1e-3)
    ap.add_argument("--decode", action="store_true")
    a = ap.parse_args(argv)
    teacher = PreNormBlock(a.tokens, a.d, a.ffn, seed=1)
    block = PreNormBlock(a.tokens, a.d, a.ffn, bits=a.bits, lr=a.lr, seed=2)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    losses = []
    for i in range(a.steps):
        if i == min(3, a.steps - 1):
            start.record()
        x = torch.randn(a.tokens, a.d, device="cuda").to(BF)
        target = teacher.forward(x)
        err = block.forward(x).float() - target.float()
        losses.append(err.square().mean())
        block.backward((err * (2.0 / err.numel())).to(BF))
        block.step()
    end.record()
    torch.cuda.synchronize()
    rc, detail = tlc.ffn_status(block.ffn_cfg, block.ffn_ws)
    if rc != tlc.MOE_OK:
        raise RuntimeError(f"feed-forward block: status {rc}, detail {detail}")
    timed = a.steps - min(3, a.steps - 1)
    print(f"loss {losses[0].item():.4f} -> {losses[-1].item():.4f} in {a.steps} steps, "
          f"{start.elapsed_time(end) / timed:.3f} ms a step")
    if a.decode:
        run, x = block.decoder(1), torch.randn(1, a.d, device="cuda").to(BF)
        full = block.forward(x.expand(a.tokens, a.d).contiguous())[:1]
        print(f"one token: largest difference from the batched pass {(run(x) - full).abs().max().item():.4f}")
    return [v.item() for v in losses]


if __name__ == "__main__":
    main()
