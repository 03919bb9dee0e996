"""The oracle of a training step's operators against differences of its own forward passes, and by hand."""
import numpy as np
import pytest

from oracle import train_ref as ref


def slopes(f, x, at, step=1e-6):
    """Central differences of f() in x[i] for the places in `at`."""
    out = []
    for i in at:
        old = x[i]
        x[i] = old + step
        up = f()
        x[i] = old - step
        out.append((up - f()) / (2 * step))
        x[i] = old
    return np.array(out)


def some(r, x, n=6):
    return [tuple(int(r.integers(k)) for k in x.shape) for _ in range(n)]


@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
@pytest.mark.parametrize("gate_rows", [0, 2, 5])
def test_residual_norm_gradients_are_differences(post, pre, gate_rows):
    """Central differences with step 1e-6 are off by the third derivative times 1e-12 and by 2^-53 / 1e-6 times the
    loss's size (about 10): 1e-8 is five times what the two come to."""
    r = np.random.default_rng(1)
    rows, d, a, c, eps = 5, 7, 0.7, 0.4, 1e-5
    p = {n: r.normal(size=s) for n, s in (("x", (rows, d)), ("u", (rows, d)), ("w", (d,)), ("b", (d,)), ("pw", (d,)), ("pb", (d,)))}
    if post != "layer":
        p["b"][:] = 0
    if pre != "layer":
        p["pb"][:] = 0
    if gate_rows:
        p["gate"] = r.normal(size=(-(-rows // gate_rows), d))
    dz, dh = r.normal(size=(rows, d)), r.normal(size=(rows, d))

    def forward():
        h, ps = ref.residual_norm_h(p["x"], p["u"], post, p["w"], p["b"], p.get("gate"), gate_rows, a, c, eps)
        loss, st = (h * dh).sum(), None
        if pre != "none":
            st = ref.norm_stats(h, pre, eps)
            loss += (dz * (ref.normed(h, st) * p["pw"] + p["pb"])).sum()
        return loss, h, ps, st

    _, h, ps, st = forward()
    got = ref.residual_norm_backward(dz, dh, p["u"], h, post, p["w"], p["b"], p.get("gate"), gate_rows, pre, p["pw"], ps, st, a, c)
    for name, g in zip(("x", "u", "w", "b", "gate", "pw", "pb"), got):
        if g is None or (name == "b" and post != "layer") or (name == "pb" and pre != "layer"):
            continue
        at = some(r, p[name])
        np.testing.assert_allclose([g[i] for i in at], slopes(lambda: forward()[0], p[name], at), rtol=0, atol=1e-8, err_msg=name)


def test_balance_gradient_is_the_differences():
    """The loss with fixed choices and gates = softmax over the chosen logits: the gradient that the oracle gives, the
    gates' part among it. Same error as above."""
    r = np.random.default_rng(2)
    T, E, k = 9, 6, 3
    l = r.normal(size=(T, E))
    idx = np.argsort(-l, 1)[:, :k]
    offsets, mask = np.array([0, 3, 3, 8]), np.array([1, 1, 0, 1, 1, 1, 1, 1, 1])
    dg = r.normal(size=(T, k))
    live = mask.astype(bool) & (np.arange(T) < 8)

    def gates():
        c = np.exp(np.take_along_axis(l, idx, 1))
        return c / c.sum(1, keepdims=True)

    def f():
        loss = ref.balance(l, idx, offsets, mask, 0.3, 0.2)[0]
        return 1.7 * loss[0] + (gates() * dg)[live].sum()

    d = ref.balance(l, idx, offsets, mask, 0.3, 0.2, 1.7, gates(), dg)[3]
    at = [(t, e) for t in range(T) for e in range(E)]
    np.testing.assert_allclose([d[i] for i in at], slopes(f, l, at), rtol=0, atol=1e-8)
    assert not d[2].any() and not d[8].any()


def test_balance_by_hand():
    """Two tokens on two experts, top 1: equal logits give p = 1/2 and lse = log 2. Both on expert 0: f = (2, 0), P =
    (1/2, 1/2), balance = 1; a dropped pair takes its part away."""
    l = np.zeros((2, 2))
    loss, counts, lse, _ = ref.balance(l, np.array([[0], [0]]), np.array([0, 2]), np.ones(2), 1.0, 1.0)
    np.testing.assert_allclose(loss, [1 + np.log(2) ** 2, 1, np.log(2) ** 2])
    assert counts.tolist() == [[2, 0]]
    loss, counts, _, _ = ref.balance(l, np.array([[0], [-1]]), np.array([0, 2]), np.ones(2), 1.0, 0.0)
    assert loss[1] == 0.5 and counts.tolist() == [[1, 0]]


def test_grad_norm_by_hand():
    norm, scale = ref.grad_norm([np.array([3.0, 0.0]), np.array([4.0])], 1.0, 0.0)
    assert norm == 5 and scale == 0.2
    assert ref.grad_norm([np.array([1e200]), np.zeros(0)], 1.0, 0.0)[0] == 1e200
    assert ref.grad_norm([np.zeros(3)], 1.0, 1e-6) == (0.0, 1.0)
    assert np.isnan(ref.grad_norm([np.array([np.nan, 1.0])], 1.0, 1e-6)[0])
