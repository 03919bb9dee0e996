"""Range of AdamW's 8-bit states: how large steps get where a block's gradients differ widely in size.

A block keeps v down to 2^-33 of its largest value, m down to 2^-17: gradients down to 2^-16.5 = 1e-5 of the
block's largest. Ten times above that a step is at most twice the largest that 64-bit states take (each average
carries roundings of at most 1/8, of which a few add up). Below it v is mostly held as zero beside an m that is not,
and a step is many times lr.
"""
import numpy as np
import pytest

from oracle import block_ref as ref


def largest_steps(ratio, steps=150, blocks=8):
    """Largest |step| / lr of 8-bit and of 64-bit states for the values whose gradients are `ratio` of their
    block's largest (which is of size 1), after a start of 20 steps."""
    rng, n, f = np.random.default_rng(0), 128 * blocks, np.float32
    codes = {k: (np.zeros(n, np.uint8), np.zeros(blocks, np.uint8)) for k in "mv"}
    m64, v64, most = np.zeros(n), np.zeros(n), [0.0, 0.0]
    small = np.arange(n) % 128 != 0
    for t in range(1, steps + 1):
        g = rng.standard_normal(n) * np.where(small, ratio, 1.0)
        m, v = ref.moments_f32(g.astype(f), *(ref.decode(*codes[k], k).astype(f) for k in "mv"), 0.9, 0.999)
        m64, v64 = 0.9 * m64 + 0.1 * g, 0.999 * v64 + 0.001 * g * g
        if t > 20:
            for i, (a, b) in enumerate(((m.astype(float), v.astype(float)), (m64, v64))):
                step = a / (1 - 0.9 ** t) / (np.sqrt(b / (1 - 0.999 ** t)) + 1e-8)
                most[i] = max(most[i], np.abs(step[small]).max())
        r = ref.noise(n, 5, t)
        codes = {"m": ref.encode(m, r & 0xFFFF, "m"), "v": ref.encode(v, r >> 16, "v")}
    return most


@pytest.mark.parametrize("ratio", [1.0, 1e-2, 1e-3, 1e-4])
def test_within_the_range_steps_are_those_of_adamw(ratio):
    eight, exact = largest_steps(ratio)
    assert eight <= 2 * exact


@pytest.mark.parametrize("ratio", [1e-5, 1e-6])
def test_below_the_range_steps_are_not(ratio):
    eight, exact = largest_steps(ratio)
    assert eight > 10 * exact
