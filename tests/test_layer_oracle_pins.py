"""The layer operators' float64 oracle against independent statements of the
same definitions: central differences of a scalar loss for every gradient,
closed forms, and hand-worked 8-bit groups."""

import numpy as np
import pytest

from oracle import layer_oracle as lo


def _num_grad(f, x, h):
    """Central differences of a scalar f at every element of x."""
    g = np.zeros_like(x)
    it = np.nditer(x, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        old = x[i]
        x[i] = old + h
        a = f()
        x[i] = old - h
        b = f()
        x[i] = old
        g[i] = (a - b) / (2 * h)
    return g


# central differences with step h are off by h^2/6 f''' + eps |f| / h: with
# h = 1e-5 and |f|, f''' of order 10 about 1e-9
H, TOL = 1e-5, 1e-7


def test_layernorm_gradient_by_differences():
    rng = np.random.default_rng(1)
    x, g, b = rng.standard_normal((3, 7)), 1 + rng.standard_normal(7) * 0.1, rng.standard_normal(7)
    c = rng.standard_normal((3, 7))
    loss = lambda: float((lo.layernorm(x, g, b)[0] * c).sum())  # noqa: E731
    _, mean, rstd = lo.layernorm(x, g, b)
    dx, dg, db = lo.layernorm_grad(c, x, g, mean, rstd)
    for t, d in ((x, dx), (g, dg), (b, db)):
        assert np.abs(_num_grad(loss, t, H) - d).max() <= TOL
    assert np.allclose(lo.layernorm_grad(c, x, g, mean, rstd, add=c)[0], dx + c, rtol=0, atol=1e-15)


def test_layernorm_normalises():
    x = np.random.default_rng(2).standard_normal((4, 33)) * 5 + 3
    y, mean, rstd = lo.layernorm(x, np.ones(33), eps=0.0)
    assert np.abs(y.mean(1)).max() < 1e-14 and np.abs((y ** 2).mean(1) - 1).max() < 1e-13
    assert np.allclose(mean, x.mean(1)) and np.allclose(rstd, 1 / x.std(1))


@pytest.mark.parametrize("act", ["none", "gelu", "relu_sq"])
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
def test_linear_gradients_by_differences(act, layout):
    """Two layers: u = act(x W1 + b1), y = u W2 + res; the chain of the operators
    gives every parameter's gradient."""
    rng = np.random.default_rng(3)
    x, b1 = rng.standard_normal((4, 5)), rng.standard_normal(6)
    w1 = rng.standard_normal((6, 5) if layout == "out_in" else (5, 6))
    w2 = rng.standard_normal((3, 6) if layout == "out_in" else (6, 3))
    res, c = rng.standard_normal((4, 3)), rng.standard_normal((4, 3))

    def loss():
        u, _ = lo.linear(x, w1, b1, act, w_layout=layout)
        return float((lo.linear(u, w2, None, "none", res, layout)[0] * c).sum())

    u, z = lo.linear(x, w1, b1, act, w_layout=layout)
    dz, u2 = lo.linear_grad_input(c, w2, act, z, w_layout=layout)
    assert np.array_equal(u, u2)
    dw2, _ = lo.linear_grad_weight(u, c, layout)
    dw1, db1 = lo.linear_grad_weight(x, dz, layout)
    dx, _ = lo.linear_grad_input(dz, w1, w_layout=layout)
    for t, d in ((x, dx), (w1, dw1), (b1, db1), (w2, dw2), (res, c)):
        assert np.abs(_num_grad(loss, t, H) - d).max() <= TOL * max(1.0, np.abs(d).max())


def test_gelu_known_values():
    v, d = lo.activation(np.array([0.0, 1.0, -1.0, 20.0, -20.0]), "gelu")
    assert np.allclose(v, [0.0, 0.8411919906082768, -0.15880800939172324, 20.0, 0.0], atol=1e-12)
    assert np.allclose(d[[0, 3, 4]], [0.5, 1.0, 0.0], atol=1e-12)


def test_act8_hand_worked_groups():
    # amax 127 takes step 1; just above it step 2; 63.5 takes step 1/2
    x = np.zeros((4, 40))
    x[0, 0], x[0, 1], x[0, 33] = 127.0, 0.5, -63.5
    x[1, 0], x[1, 2] = 127.0 * (1 + 2.0 ** -23), 3.0
    x[2, 0] = 2.0 ** -149
    x[3, 35] = np.inf
    q, e = lo.act8_encode(x)
    assert e.tolist() == [[127, 126], [128, 1], [1, 1], [1, 255]]
    assert q[0, 0] == 127 and q[0, 1] == 0 and q[0, 33] == -127          # 0.5 ties to even
    assert q[1, 0] == 64 and q[1, 2] == 2                                # 1.5 ties to even
    assert q[2, 0] == 0 and not q[3].any()
    y = lo.act8_decode(q, e)
    assert y[0, 0] == 127 and y[0, 33] == -63.5 and np.isnan(y[3, 32:]).all() and not y[3, :32].any()


def test_act8_error_is_half_a_step():
    x = np.random.default_rng(4).standard_normal((50, 100)) * np.exp(np.random.default_rng(5).uniform(-20, 20, (50, 1)))
    q, e = lo.act8_encode(x)
    step = np.exp2(np.repeat(e.astype(np.float64) - 127, 32, axis=1)[:, :100])
    assert np.all(np.abs(lo.act8_decode(q, e) - x) <= step / 2)
    top = np.stack([np.abs(x[:, j:j + 32]).max(1) for j in range(0, 100, 32)], axis=1)
    s = np.exp2(e.astype(np.float64) - 127)
    assert np.all(top <= 127 * s) and np.all(top > 63.5 * s)
