"""The block operators' oracle: gradients against central differences, 8-bit states' encoding."""
import numpy as np
import pytest

from oracle import block_ref as ref


def differences(f, a, grad_out, h=1e-5):
    """Central differences of sum(f() * grad_out) over the entries of a (changed in place). Their error is
    h^2 f''' / 6 plus 2^-52 |f| / h: about 1e-10 here for values around 1."""
    out = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        keep = a[i]
        a[i] = keep + h
        hi = (f() * grad_out).sum()
        a[i] = keep - h
        lo = (f() * grad_out).sum()
        a[i] = keep
        out[i] = (hi - lo) / (2 * h)
    return out


def test_ffn_gradients_are_the_differences():
    rng = np.random.default_rng(0)
    x, W1, W3, W2 = (rng.standard_normal(s) for s in ((3, 5), (7, 5), (7, 5), (5, 7)))
    dy = rng.standard_normal((3, 5))
    got = ref.ffn_backward(x, W1, W3, W2, dy)
    for a, g in zip((x, W1, W3, W2), got):
        np.testing.assert_allclose(g, differences(lambda: ref.ffn_forward(x, W1, W3, W2), a, dy), rtol=0, atol=1e-7)


def test_layernorm_gradients_are_the_differences():
    rng = np.random.default_rng(1)
    x, w, b, dy = (rng.standard_normal(s) for s in ((4, 9), 9, 9, (4, 9)))
    _, mean, rstd = ref.layernorm_forward(x, w, b, 1e-5)
    got = ref.layernorm_backward(dy, x, w, mean, rstd)
    for a, g in zip((x, w, b), got):
        d = differences(lambda: ref.layernorm_forward(x, w, b, 1e-5)[0], a, dy)
        np.testing.assert_allclose(g, d, rtol=0, atol=1e-7)


@pytest.mark.parametrize("name,step", [("m", 2 ** -3), ("v", 2 ** -3)])
def test_rounding_is_to_a_neighbour_and_unbiased(name, step):
    """Every value goes to one of its two neighbours (relative distance up to 1/8), and the mean over
    all 16 random bits of a value is the value to 2^-17 of the distance."""
    x = np.float32([1.0, 0.3, 0.0071, -0.9 if name == "m" else 0.9, 1e-4, 0.0])
    top, bias, _, _ = ref._formats(name)
    for v in x:
        block = np.float32([1.5, v])
        r = np.arange(0, 65536, 257)
        vals = []
        for q in r[:64]:
            c, s = ref.encode(block, np.array([0, q]), name)
            vals.append(ref.decode(c, s, name)[1])
        assert all(abs(a - v) <= max(step * abs(v), 2.0 ** (1 - bias - 3 - top + 1)) for a in vals)
        allv = []
        for q in r:
            c, s = ref.encode(block, np.array([0, q]), name)
            allv.append(ref.decode(c, s, name)[1])
        gap = max(allv) - min(allv)
        assert abs(np.mean(allv) - v) <= gap / 256 + 1e-12


def test_codes_round_trip():
    for name, codes in (("m", [c for c in range(256) if c & 0x7F < 0x70]), ("v", list(range(0xF8)))):
        codes = np.array(codes, np.uint8)
        block = np.concatenate([codes[i:i + 1] for i in range(len(codes))])
        scales = np.full(-(-len(block) // ref.BLOCK), 130, np.uint8)
        v = ref.decode(block, scales, name).astype(np.float32)
        for i in range(0, len(block), ref.BLOCK):  # each block with its own largest value
            c, s = ref.encode(v[i:i + ref.BLOCK], np.zeros(min(ref.BLOCK, len(block) - i), np.int64), name)
            w = ref.decode(c, s, name)
            # codes whose subnormal steps the block's own scale still holds come back as they were
            np.testing.assert_allclose(w, v[i:i + ref.BLOCK], rtol=1 / 8, atol=2.0 ** 3 * 2.0 ** (1 - 15 - 3))


def test_non_finite_block_reads_as_nan_and_zero_buffer_as_zero():
    for bad in (np.nan, np.inf):
        c, s = ref.encode(np.float32([1, bad, 2]), np.zeros(3, np.int64), "v")
        assert s[0] == 255 and np.isnan(ref.decode(c, s, "v")).all()
    z = np.zeros(3, np.uint8)
    assert (ref.decode(z, np.zeros(1, np.uint8), "m") == 0).all()
