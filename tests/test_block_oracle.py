"""The fp64 definitions of oracle/block.py: gradients against central differences, reductions and
hand-checkable cases."""
import numpy as np
import pytest

from oracle import block


def _fd(f, x, h=1e-6):
    g = np.zeros_like(x)
    it = np.nditer(x, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        old = x[i]
        x[i] = old + h
        up = f()
        x[i] = old - h
        dn = f()
        x[i] = old
        g[i] = (up - dn) / (2 * h)
    return g


def _close(a, b):
    # central differences with h = 1e-6 in fp64: truncation h^2, cancellation 1e-16 / h = 1e-10 of f
    assert np.abs(a - b).max() <= 1e-7 * max(1.0, np.abs(b).max())


def test_layer_norm_gradients_and_constant_row():
    rng = np.random.default_rng(0)
    x, w, b, dy = rng.normal(size=(3, 8)), rng.normal(size=8), rng.normal(size=8), rng.normal(size=(3, 8))
    f = lambda: float((block.layer_norm_forward(x, w, b, 1e-3)[0] * dy).sum())  # noqa: E731
    g = block.layer_norm_backward(x, w, 1e-3, dy)
    _close(g["dx"], _fd(f, x))
    _close(g["dweight"], _fd(f, w))
    _close(g["dbias"], _fd(f, b))
    y, mu, rstd = block.layer_norm_forward(np.full((1, 8), 5.0), w, b, 1e-4)
    assert np.allclose(y, b) and mu[0] == 5.0 and np.isclose(rstd[0], 100.0)


def test_glr_gradients_and_running_sum():
    rng = np.random.default_rng(1)
    x, la = rng.normal(size=(2, 5, 3)), -np.abs(rng.normal(size=(2, 5, 3)))
    h0, dh, dhT = rng.normal(size=(2, 3)), rng.normal(size=(2, 5, 3)), rng.normal(size=(2, 3))

    def f():
        h, hT, _ = block.glr_forward(x, la, h0)
        return float((h * dh).sum() + (hT * dhT).sum())
    g = block.glr_backward(x, la, h0, dh, dhT)
    _close(g["dx"], _fd(f, x))
    _close(g["dlog_a"], _fd(f, la))
    _close(g["dh0"], _fd(f, h0))
    h, _, _ = block.glr_forward(x, np.zeros_like(la), None)
    assert np.allclose(h, x.cumsum(1))


@pytest.mark.parametrize("window,sinks,lengths", [(3, 0, None), (2, 1, [5, 3]), (9, 2, [4, 0])])
def test_swa_gradients(window, sinks, lengths):
    rng = np.random.default_rng(2)
    q, dO = rng.normal(size=(2, 5, 4, 3)), rng.normal(size=(2, 5, 4, 3))
    k, v = rng.normal(size=(2, 5, 2, 3)), rng.normal(size=(2, 5, 2, 3))
    if lengths is not None:
        for b, L in enumerate(lengths):
            dO[b, L:] = 0.0
    f = lambda: float((block.swa(q, k, v, window, sinks, 0.7, lengths)["o"] * dO).sum())  # noqa: E731
    r = block.swa(q, k, v, window, sinks, 0.7, lengths, dO)
    for n, x in (("dq", q), ("dk", k), ("dv", v)):
        _close(r[n], _fd(f, x))


def test_swa_window_of_one_returns_own_value_and_sinks_join():
    rng = np.random.default_rng(3)
    q, k, v = (rng.normal(size=(1, 4, 1, 2)) for _ in range(3))
    assert np.allclose(block.swa(q, k, v, 1, 0, 1.0)["o"], v)
    o = block.swa(q, k, v, 1, 1, 1.0)["o"][0, 3, 0]
    e = np.exp([q[0, 3, 0] @ k[0, 0, 0], q[0, 3, 0] @ k[0, 3, 0]])
    assert np.allclose(o, (e[0] * v[0, 0, 0] + e[1] * v[0, 3, 0]) / e.sum())


def test_swa_cache_keeps_sinks_and_the_last_window():
    k = np.arange(1.0, 8.0).reshape(1, 7, 1, 1)
    kc, _ = block.swa_cache(k, k, np.zeros((1, 5, 1, 1)), np.zeros((1, 5, 1, 1)), 3, 2)
    assert kc[0, :, 0, 0].tolist() == [1.0, 2.0, 6.0, 7.0, 5.0]   # positions 0, 1 | 5, 6, 4
