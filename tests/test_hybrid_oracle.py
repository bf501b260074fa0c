"""The fp64 definitions of oracle/hybrid.py against differences, the mixer's own oracle and each other."""
import numpy as np
import pytest

from oracle import block, hybrid
from oracle import oracle as orc


def _dla(seed, B=2, T=9, H=3, dk=4, dv=5, lengths=None):
    r = np.random.default_rng(seed)
    n = r.standard_normal
    g = -np.abs(n(H)) * np.array([0.1, 1.0, 3.0])[:H]
    return dict(q=n((B, T, H, dk)), k=n((B, T, H, dk)), v=n((B, T, H, dv)), g=g, S0=n((B, H, dk, dv)), dO=n((B, T, H, dv)),
                dS_T=n((B, H, dk, dv)), lengths=lengths)


def _forward(x):
    return hybrid.dla_forward(x["q"], x["k"], x["v"], x["g"], x["S0"], x["lengths"])


@pytest.mark.parametrize("lengths", [None, [9, 4], [0, 12]])
def test_dla_backward_against_differences(lengths):
    x = _dla(1, lengths=lengths)
    if lengths:
        for b, L in enumerate(lengths):
            x["dO"][b, L:] = 0.0
    r = hybrid.dla_backward(x["q"], x["k"], x["v"], x["g"], x["dO"], x["S0"], x["dS_T"], lengths)
    rng = np.random.default_rng(2)

    def loss(y):
        o, S = _forward(y)
        return (o * x["dO"]).sum() + (S * x["dS_T"]).sum()
    for n in ("q", "k", "v", "S0"):
        u = rng.standard_normal(x[n].shape)
        e = 1e-5
        d = (loss(dict(x, **{n: x[n] + e * u})) - loss(dict(x, **{n: x[n] - e * u}))) / (2 * e)
        want = (r["d" + n] * u).sum()
        assert abs(d - want) <= 1e-7 * (1 + abs(want)), n


def test_dla_is_the_mixer_without_its_erase_product():
    x = _dla(3, T=20, dk=8, dv=8)
    la = np.broadcast_to(x["g"][None, None, :, None], x["q"].shape).copy()
    o, S = orc.forward(x["q"], x["k"], x["v"], la, np.zeros_like(x["q"]), np.ones_like(x["v"]), x["S0"])
    ro, rS = _forward(x)
    assert np.allclose(o, ro, rtol=1e-12, atol=1e-12) and np.allclose(S, rS, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("reverse", [False, True])
def test_sizes_bound_the_passes(reverse):
    """With values of one sign nothing cancels: the double sum's size is the output itself."""
    x = _dla(4, T=150)
    x = {n: np.abs(v) if n not in ("g", "lengths") else v for n, v in x.items()}
    g = hybrid.dla_backward(x["q"], x["k"], x["v"], x["g"], x["dO"], x["S0"], x["dS_T"])
    if reverse:
        r = hybrid.dla_sizes(x["k"], x["q"], x["dO"], x["g"], x["dS_T"], reverse=True)
        ref, fin = g["dv"], g["dS0"] / np.exp(x["g"])[:, None, None]
    else:
        r = hybrid.dla_sizes(x["q"], x["k"], x["v"], x["g"], x["S0"])
        ref, fin = _forward(x)
    assert np.allclose(r["all"], ref, rtol=1e-10) and np.allclose(r["score"] + r["read"], ref, rtol=1e-10)
    assert np.allclose(r["state"], fin, rtol=1e-10)


def test_rms_backward_against_differences():
    r = np.random.default_rng(5)
    h, w, dy, dh = r.standard_normal((3, 16)), r.standard_normal(16), r.standard_normal((3, 16)), r.standard_normal((3, 16))
    g = hybrid.rms_backward(h, w, 1e-3, dy, dh)
    loss = lambda a, b: (hybrid.rms_forward(a, b, 1e-3)[0] * dy).sum() + (a * dh).sum()  # noqa: E731
    u, s, e = r.standard_normal(h.shape), r.standard_normal(16), 1e-5
    assert abs((loss(h + e * u, w) - loss(h - e * u, w)) / (2 * e) - (g["dx"] * u).sum()) < 1e-7
    assert abs((loss(h, w + e * s) - loss(h, w - e * s)) / (2 * e) - (g["dweight"] * s).sum()) < 1e-7


def test_paged_decode_is_attention_over_the_sequence():
    r = np.random.default_rng(6)
    H, Hkv, d, page, T = 4, 2, 8, 4, 11
    q, k, v = r.standard_normal((1, T, H, d)), r.standard_normal((1, T, Hkv, d)), r.standard_normal((1, T, Hkv, d))
    kp = np.full((7, page, Hkv, d), np.nan)
    table = np.array([[5, 0, 3]])
    kp, vp = hybrid.paged_fill(k[:, :-1], v[:, :-1], kp, kp.copy(), table)
    p = hybrid.paged_decode(q[:, -1], k[:, -1], v[:, -1], kp, vp, table, [T - 1], d ** -0.5)
    ref = block.swa(q, k, v, T, 0, d ** -0.5)
    assert np.allclose(p["o"], ref["o"][:, -1], rtol=1e-12)
    assert np.array_equal(p["k_pages"][3, 2], k[0, 10]) and np.isnan(p["k_pages"][[1, 2, 4, 6]]).all()
    # pages that name nothing are not seen
    bad = hybrid.paged_decode(q[:, -1], k[:, -1], v[:, -1], kp, vp, np.array([[5, 7, 3]]), [T - 1], d ** -0.5)
    keep = [0, 1, 2, 3, 8, 9, 10]
    s = np.einsum("hd,jhd->hj", q[0, -1], np.repeat(k[0, keep], 2, axis=1)) * d ** -0.5
    w = np.exp(s - s.max(1, keepdims=True))
    assert np.allclose(bad["o"][0], np.einsum("hj,jhd->hd", w / w.sum(1, keepdims=True), np.repeat(v[0, keep], 2, axis=1)))
