"""Every plan of the feed-forward block against the formulas in 64 bits.

How a product runs (on single CTAs: tokens a tile and CTAs its k-blocks are split over; on CTA pairs: parts that the
last wave's tiles are cut into, with or without whole waves before them) follows from its sizes. The shapes below
were searched so that each plan that occurs for 1 to 8192 tokens and widths of 8 to 4096 and 8 to 14336 is
taken by one of them: for h with and without kept projections, the hidden gradients, the down-projection,
and the last launch (dx alone with the weight gradients beside it, or all in one with dx's tiles first or last, in
one to eight parts, with and without a second round for the clusters that got less).

Tolerance: as in test_gpu_ffn.py, two bf16 roundings.
"""
import pytest
import torch

import tile_level_copy_gb300 as tlc

pytestmark = pytest.mark.gpu
REL = 4.3e-3
BF, D = torch.bfloat16, torch.float64

SHAPES = [
    (7356, 8, 8), (4293, 8, 16), (1, 288, 13040), (1, 584, 7064), (1, 960, 5632), (6464, 64, 64), (33, 656, 1760),
    (41, 1456, 664), (287, 160, 912), (5077, 144, 72), (653, 88, 1112), (55, 1232, 1040), (1334, 1000, 64),
    (7669, 168, 80), (79, 1416, 984), (35, 1944, 1752), (74, 528, 4456), (2197, 64, 1280), (586, 144, 2224),
    (179, 1144, 1032), (49, 1208, 3768), (6143, 8, 4576), (2188, 64, 1784), (1138, 72, 3264), (914, 264, 1232),
    (8107, 8, 4800), (3044, 64, 1720), (6805, 64, 800), (6536, 8, 8560), (1911, 3544, 72), (7368, 80, 1016),
    (1917, 184, 1792), (150, 1856, 2392), (8036, 1704, 64), (7577, 88, 1360), (52, 1888, 11144), (4553, 3112, 80),
    (2847, 2856, 144), (65, 2416, 8736), (3900, 64, 5600), (4433, 88, 4296), (3921, 3344, 136), (6707, 72, 4112),
    (5579, 2848, 160), (3487, 176, 4536), (2817, 88, 12096), (79, 2952, 13000), (371, 2528, 3368), (3639, 3416, 280),
    (6670, 64, 8256), (6485, 288, 2240), (2368, 144, 13440), (8066, 80, 7520), (105, 3704, 13496), (401, 3160, 5784),
    (721, 2880, 3728), (677, 1488, 8288), (234, 3072, 12384), (254, 3424, 12944), (2781, 1672, 2856),
    (4893, 968, 3016), (443, 2960, 11144), (3529, 1288, 4624), (1982, 3448, 3280), (726, 2848, 13416),
    (1679, 2728, 8416), (3892, 1192, 8896), (6859, 640, 11736)]


def reference(x, W1, W3, W2, dy):
    """y, dx, dW1, dW3, dW2 in 64 bits."""
    x, W1, W3, W2, dy = (t.to(D) for t in (x, W1, W3, W2, dy))
    g, u, dh = x @ W1.T, x @ W3.T, dy @ W2
    s = 1 / (1 + torch.exp(-g))
    h, dg, du = g * s * u, dh * u * s * (1 + g * (1 - s)), dh * g * s
    return h @ W2.T, dg @ W1 + du @ W3, dg.T @ x, du.T @ x, dy.T @ h


@pytest.mark.parametrize("T,d,f", SHAPES)
def test_forward_and_backward(T, d, f):
    gen = torch.Generator(device="cuda").manual_seed(T + d + f)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=gen, device="cuda") * std).to(BF)  # noqa: E731
    x, W1, W3, W2 = r(T, d), r(f, d, std=d ** -0.5), r(f, d, std=d ** -0.5), r(d, f, std=f ** -0.5)
    dy = r(T, d, std=0.01)
    cfg = tlc.FFNConfig(T, d, f)
    ws, saved = tlc.FFNWorkspace(cfg), tlc.ffn_saved(cfg).fill_(0xFF)
    nan = lambda t: torch.full_like(t, float("nan"))  # noqa: E731
    y0, y, outs = nan(x), nan(x), [nan(t) for t in (x, W1, W3, W2)]
    tlc.ffn_forward(cfg, x, W1, W3, W2, y0, ws)
    tlc.ffn_forward(cfg, x, W1, W3, W2, y, ws, saved=saved)
    tlc.ffn_backward(cfg, x, W1, W3, W2, dy, saved, *outs, ws)
    again = [nan(t) for t in outs]
    tlc.ffn_backward(cfg, x, W1, W3, W2, dy, saved, *again, ws)
    assert tlc.ffn_status(cfg, ws) == (tlc.MOE_OK, 0)
    wy, *want = reference(x, W1, W3, W2, dy)
    for got, w in zip((y0, y, *outs), (wy, wy, *want)):
        assert ((got.to(D) - w).norm() <= REL * w.norm()).item(), tuple(got.shape)
    for a, b in zip(outs, again):
        assert torch.equal(a, b)
