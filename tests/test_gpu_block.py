"""GPU parity of the operators around the mixer (layer norm, gated linear recurrence,
sliding-window attention with sinks, its bounded cache and decode) against the fp64 definitions of
oracle/block.py, element by element within the bounds of tests/_block.py."""
import numpy as np
import pytest
import torch

import gated_delta_rule_gdr_amd as g2
from oracle import block
from tests._block import DT, U, U32, f64, randn, swa_bounds, within
from tests._util import announce

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


# ------------------------------------------------------------------ layer norm
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,D,bias", [(1, 8, True), (37, 64, False), (5, 72, True), (130, 128, True), (9, 256, True),
                                         (70, 504, False), (33, 1000, True), (600, 2048, True), (3, 4096, True),
                                         (5, 5000, False), (11, 8192, True), (2, 16384, True), (4099, 24, True)])
def test_layer_norm(dtype, rows, D, bias):
    announce(f"layer norm {dtype} rows={rows} D={D}")
    gen = torch.Generator().manual_seed(rows * 7 + D)
    x = (3.0 * randn(gen, (rows, 1)) + randn(gen, (rows, D))).to(DT[dtype])
    w, b, dy = 1.0 + 0.1 * randn(gen, (D,)), randn(gen, (D,)) if bias else None, randn(gen, (rows, D), dtype)
    xd, wd, bd, dyd = dev(x, w, b, dy)
    y, mean, rstd = g2.gdr2_layer_norm_fwd(xd, wd, bd)
    g = g2.gdr2_layer_norm_bwd(xd, wd, mean, rstd, dyd, want_dbias=bias)
    torch.cuda.synchronize()
    X, W, B, DY = f64(x), f64(w), f64(b), f64(dy)
    ry, rm, rr = block.layer_norm_forward(X, W, B, 1e-5)
    rg = block.layer_norm_backward(X, W, 1e-5, DY)
    # sums pass at most 64 roundings; n is formed from x - mean with its terms' errors
    s, uo = 64 * U32, U[dtype]
    ax = np.abs(X).mean(-1)
    em, n = s * ax, np.abs((X - rm[:, None]) * rr[:, None])
    er = 2 * s * rr + 2 * rr * rr * em       # rstd: half the variance's relative error, and the mean's
    en = rr[:, None] * (em[:, None] + 2 * U32 * (np.abs(X) + np.abs(rm)[:, None])) + n * (er / rr)[:, None]
    within("mean", mean, rm, em + 2 * U32 * np.abs(rm))
    within("rstd", rstd, rr, er)
    within("y", y, ry, en * np.abs(W) + uo * np.abs(ry) + 4 * U32 * (n * np.abs(W) + (0 if B is None else np.abs(B))))
    a = np.abs(DY * W)
    ea = (a.mean(-1, keepdims=True) + n * (a * n).mean(-1, keepdims=True) + a)
    edx = rr[:, None] * (2 * s * ea + en * (a * n).mean(-1, keepdims=True) + n * (a * en).mean(-1, keepdims=True)) + (er / rr)[:, None] * rr[:, None] * ea
    within("dx", g["dx"], rg["dx"], edx + uo * np.abs(rg["dx"]))
    sr = (rows / 512 + 64) * U32
    within("dweight", g["dweight"], rg["dweight"], sr * (np.abs(DY) * n).sum(0) + (np.abs(DY) * en).sum(0) + 1e-30)
    if bias:
        within("dbias", g["dbias"], rg["dbias"], sr * np.abs(DY).sum(0))
    else:
        assert g["dbias"] is None


def test_layer_norm_no_rows():
    x, w = torch.zeros(0, 64, device=DEV), torch.ones(64, device=DEV)
    y, mean, rstd = g2.gdr2_layer_norm_fwd(x, w)
    g = g2.gdr2_layer_norm_bwd(x, w, mean, rstd, x)
    assert y.shape == x.shape and not g["dweight"].any() and not g["dbias"].any()


# ------------------------------------------------------------------ gated linear recurrence
def _glr_inputs(B, T, D, dtype, seed, decays="mixed"):
    gen = torch.Generator().manual_seed(seed)
    x, dh = randn(gen, (B, T, D), dtype), randn(gen, (B, T, D), dtype)
    la = -0.1 * torch.nn.functional.softplus(randn(gen, (B, T, D)))
    if decays == "mixed":
        la[..., : D // 4] = 0.0
        la[..., D // 4: D // 2] *= 300.0
        if T > 3:
            la[:, T // 2, : D // 2] = float("-inf")
    return x, la, randn(gen, (B, D)), dh, randn(gen, (B, D))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,D", [(1, 1, 8), (2, 5, 72), (1, 128, 64), (3, 129, 64), (2, 300, 136), (1, 2047, 64),
                                   (1, 2049, 200), (2, 4500, 16)])
def test_glr(dtype, B, T, D):
    announce(f"glr {dtype} B={B} T={T} D={D}")
    x, la, h0, dh, dhT = _glr_inputs(B, T, D, dtype, B * 100 + T + D)
    xd, lad, h0d, dhd, dhTd = dev(x, la, h0, dh, dhT)
    h, hT, ws = g2.gdr2_glr_fwd(xd, lad, h0d)
    g = g2.gdr2_glr_bwd(xd, lad, dhd, ws, dhTd)
    torch.cuda.synchronize()
    X, LA, H0, DH, DHT = (f64(t) for t in (x, la, h0, dh, dhT))
    rh, rhT, err = block.glr_forward(X, LA, H0)
    rg = block.glr_backward(X, LA, H0, DH, DHT)
    u = 2 * U32
    # a decay below the smallest normal fp32 number, 2^-126 = 1.2e-38, may be flushed to zero: it
    # multiplies states and gradients below 1e4 here, so a product loses at most 1.2e-38 (1e4)^2
    flush = 1e-29
    within("h", h, rh, u * err + U[dtype] * np.abs(rh) + flush)
    within("h_T", hT, rhT, u * err[:, -1] + flush)
    within("dx", g["dx"], rg["dx"], u * rg["dx_err"] + U[dtype] * np.abs(rg["dx"]) + flush)
    within("dlog_a", g["dlog_a"], rg["dlog_a"], u * rg["dlog_a_err"] + flush)
    within("dh0", g["dh0"], rg["dh0"], u * rg["dh0_err"] + flush)


def test_glr_defaults_empty_and_deterministic():
    x, la, _, dh, _ = _glr_inputs(2, 1000, 128, "bf16", 5)
    xd, lad, dhd = dev(x, la, dh)
    h, hT, ws = g2.gdr2_glr_fwd(xd, lad)
    a = g2.gdr2_glr_bwd(xd, lad, dhd, ws)
    h2, hT2, ws2 = g2.gdr2_glr_fwd(xd, lad, h0=torch.zeros(2, 128, device=DEV))
    b = g2.gdr2_glr_bwd(xd, lad, dhd, ws2, dh_T=torch.zeros(2, 128, device=DEV))
    assert torch.equal(h, h2) and torch.equal(hT, hT2)
    for n in ("dx", "dlog_a", "dh0"):
        assert torch.equal(a[n], b[n]), n
    h, hT, _ = g2.gdr2_glr_fwd(xd, lad, want_final_state=False)
    assert hT is None
    assert g2.gdr2_glr_bwd(xd, lad, dhd, ws, want_dh0=False)["dh0"] is None
    e, le, h0 = xd[:, :0].contiguous(), lad[:, :0].contiguous(), torch.randn(2, 128, device=DEV)
    h, hT, ws = g2.gdr2_glr_fwd(e, le, h0)
    g = g2.gdr2_glr_bwd(e, le, e, ws, h0)
    assert h.shape == e.shape and torch.equal(hT, h0) and torch.equal(g["dh0"], h0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_glr_steps_continue_a_prefill(dtype):
    x, la, h0, _, _ = _glr_inputs(3, 140, 72, dtype, 11)
    xd, lad, h0d = dev(x, la, h0)
    full, fT, _ = g2.gdr2_glr_fwd(xd, lad, h0d)
    _, st, _ = g2.gdr2_glr_fwd(xd[:, :130].contiguous(), lad[:, :130].contiguous(), h0d)
    for t in range(130, 140):
        h, st = g2.gdr2_glr_step(xd[:, t].contiguous(), lad[:, t].contiguous(), st)
    rh, rhT, err = block.glr_forward(f64(x), f64(la), f64(h0))
    within("h", h, rh[:, -1], 2 * U32 * err[:, -1] + U[dtype] * np.abs(rh[:, -1]))
    within("state", st, rhT, 2 * U32 * err[:, -1])
    h, st = g2.gdr2_glr_step(xd[:, 0].contiguous(), lad[:, 0].contiguous())
    assert torch.equal(h, xd[:, 0]) and torch.equal(st, xd[:, 0].float())


# ------------------------------------------------------------------ sliding-window attention
def _swa_inputs(B, T, H, Hkv, d, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    return (randn(gen, (B, T, H, d), dtype), randn(gen, (B, T, Hkv, d), dtype), randn(gen, (B, T, Hkv, d), dtype),
            randn(gen, (B, T, H, d), dtype))


def _swa_check(B, T, H, Hkv, d, dtype, window, sinks, lengths, seed, scale=None, garbage=float("nan")):
    announce(f"swa {dtype} B={B} T={T} H={H}/{Hkv} d={d} window={window} sinks={sinks} lengths={lengths}")
    q, k, v, dO = _swa_inputs(B, T, H, Hkv, d, dtype, seed)
    Ld = None
    if lengths is not None:
        Ld = torch.tensor(lengths, dtype=torch.int32, device=DEV)
        for b, L in enumerate(lengths):   # padding rows hold what they like
            for t in (q, k, v, dO):
                t[b, max(L, 0):] = garbage
    qd, kd, vd, dOd = dev(q, k, v, dO)
    o, lse = g2.gdr2_swa_fwd(qd, kd, vd, window, sinks=sinks, scale=scale, lengths=Ld)
    g = g2.gdr2_swa_bwd(qd, kd, vd, o, lse, dOd, window, sinks=sinks, scale=scale, lengths=Ld)
    torch.cuda.synchronize()
    r = block.swa(f64(q), f64(k), f64(v), window, sinks, d ** -0.5 if scale is None else scale, lengths, f64(dO))
    n = min(T, window + sinks) + (T * (H // Hkv) if sinks else (window + 128) * (H // Hkv))
    bd = swa_bounds(r, dtype, d, n)
    within("o", o, r["o"], bd["o"])
    within("lse", lse, r["lse"], bd["lse"])
    for name in ("dq", "dk", "dv"):
        within(name, g[name], r[name], bd[name])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,T,H,Hkv,window,sinks,lengths", [
    (1, 1, 1, 1, 1, 0, None), (2, 33, 2, 1, 7, 2, None), (1, 64, 1, 1, 64, 0, None), (1, 127, 3, 3, 1000, 64, None),
    (2, 129, 4, 2, 1, 1, [129, 60]), (3, 200, 2, 2, 50, 0, [200, 0, 1]), (1, 449, 4, 1, 100, 5, None),
    (1, 513, 2, 1, 130, 64, [500]), (2, 260, 6, 2, 64, 33, [-5, 300])])
def test_swa(dtype, d, B, T, H, Hkv, window, sinks, lengths):
    _swa_check(B, T, H, Hkv, d, dtype, window, sinks, lengths, seed=T + window + sinks)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_swa_many_workgroups(dtype, d):
    """Enough heads for 128 queries and whole query ranges per workgroup, with and without shared heads."""
    _swa_check(8, 520, 8, 8, d, dtype, 100, 5, [520, 519, 129, 128, 1, 0, 400, 33], seed=13)
    _swa_check(4, 600, 32, 16, d, dtype, 333, 0, None, seed=14)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H", [8, 9])
def test_swa_padded_grids(dtype, d, H):
    """320 and 360 workgroups of 128 queries, the two sides of the forward's and dq's split, over a padded batch."""
    _swa_check(8, 513, H, H, d, dtype, 70, 20, [513, 512, 129, 128, 1, 0, 400, 65], seed=16)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_swa_nonfinite_values_stay_in_their_sequence(dtype):
    """A NaN in one sequence's key/value head reaches neither another sequence nor another head."""
    q, k, v, dO = _swa_inputs(2, 200, 4, 2, 64, dtype, 15)
    ref = None
    for bad in (False, True):
        if bad:
            k[0, 50, 1] = float("nan")
            v[0, 60, 1] = float("inf")
            dO[0, 70, 2:] = float("nan")
        qd, kd, vd, gd = dev(q, k, v, dO)
        o, lse = g2.gdr2_swa_fwd(qd, kd, vd, 64, sinks=1)
        g = g2.gdr2_swa_bwd(qd, kd, vd, o, lse, gd, 64, sinks=1)
        out = [o[1], o[0, :, :2], lse[1], lse[0, :2], g["dq"][1], g["dq"][0, :, :2], g["dk"][1], g["dk"][0, :, 0], g["dv"][1],
               g["dv"][0, :, 0]]
        if ref is None:
            ref = out
        else:
            assert torch.isnan(o[0, 60:, 2:]).any()
            for a, b in zip(out, ref):
                assert torch.equal(a, b)


def test_rows_and_channels_are_isolated():
    x = torch.randn(40, 200, device=DEV)
    x[7, 3] = float("nan")
    w = torch.ones(200, device=DEV)
    y, mean, rstd = g2.gdr2_layer_norm_fwd(x, w)
    dx = g2.gdr2_layer_norm_bwd(x, w, mean, rstd, torch.ones_like(x))["dx"]
    for t in (y, dx):
        assert torch.isnan(t[7]).all() and torch.isfinite(t[torch.arange(40) != 7]).all()
    x, la = torch.randn(1, 5000, 64, device=DEV), -torch.rand(1, 5000, 64, device=DEV)
    x[0, 700, 9] = float("nan")
    h, hT, ws = g2.gdr2_glr_fwd(x, la)
    g = g2.gdr2_glr_bwd(x, la, torch.ones_like(x), ws)
    others = torch.arange(64) != 9
    assert torch.isnan(h[0, 700:, 9]).all() and torch.isfinite(h[0, :700, 9]).all() and torch.isfinite(h[..., others]).all()
    assert torch.isfinite(g["dx"]).all() and torch.isfinite(g["dlog_a"][..., others]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_swa_many_sink_pieces(dtype):
    """Queries far behind the window: several pieces of the sinks' gradients, the last one ragged."""
    _swa_check(1, 3000, 2, 1, 64, dtype, 33, 40, None, seed=3)
    _swa_check(2, 2500, 2, 2, 64, dtype, 100, 3, [2500, 700], seed=4, garbage=float("inf"))


def test_swa_large_scores_and_scale():
    """Scores whose exponentials leave fp32 without the running reference."""
    _swa_check(1, 200, 2, 2, 64, "bf16", 90, 2, None, seed=8, scale=4.0)
    _swa_check(1, 200, 2, 2, 64, "f32", 90, 2, None, seed=9, scale=4.0)


def test_swa_deterministic_and_empty():
    q, k, v, dO = dev(*_swa_inputs(2, 700, 4, 2, 128, "bf16", 12))
    a = g2.gdr2_swa_fwd(q, k, v, 200, sinks=4)
    b = g2.gdr2_swa_fwd(q, k, v, 200, sinks=4)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga = g2.gdr2_swa_bwd(q, k, v, *a, dO, 200, sinks=4)
    gb = g2.gdr2_swa_bwd(q, k, v, *b, dO, 200, sinks=4)
    for n in ga:
        assert torch.equal(ga[n], gb[n]), n
    e = [t[:, :0].contiguous() for t in (q, k, v, dO)]
    o, lse = g2.gdr2_swa_fwd(*e[:3], 5)
    assert o.shape == e[0].shape and g2.gdr2_swa_bwd(*e[:3], o, lse, e[3], 5)["dk"].shape == e[1].shape


# ------------------------------------------------------------------ the cache and decode
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv,window,sinks", [(1, 1, 1, 0), (4, 2, 7, 3), (8, 1, 200, 0), (20, 1, 150, 64), (6, 3, 700, 4)])
def test_decode(dtype, d, H, Hkv, window, sinks):
    """Positions from the first token to several turns of the ring, and a sequence without a token;
    unwritten slots hold NaN."""
    announce(f"decode {dtype} H={H}/{Hkv} d={d} window={window} sinks={sinks}")
    cap = window + sinks
    pos = [0, 1, max(sinks - 1, 0), sinks, cap - 1, cap, cap + 1, 3 * cap + 5, -1]
    N = len(pos)
    gen = torch.Generator().manual_seed(window + sinks)
    T = max(pos) + 1
    ks, vs = randn(gen, (N, T, Hkv, d), dtype), randn(gen, (N, T, Hkv, d), dtype)
    q = randn(gen, (N, H, d), dtype)
    kc = torch.full((N, cap, Hkv, d), float("nan"), dtype=DT[dtype], device=DEV)
    vc = kc.clone()
    ksd, vsd, qd = dev(ks, vs, q)
    L = torch.tensor([max(p, 0) for p in pos], dtype=torch.int32, device=DEV)
    g2.gdr2_swa_cache_fill(ksd, vsd, kc, vc, sinks=sinks, lengths=L)
    blank = np.full((N, cap, Hkv, d), np.nan)
    rk, rv = block.swa_cache(f64(ks), f64(vs), blank, blank, window, sinks, L.tolist())
    assert np.array_equal(f64(kc), rk, equal_nan=True) and np.array_equal(f64(vc), rv, equal_nan=True)
    at = [max(p, 0) for p in pos]
    kn = torch.stack([ksd[n, at[n]] for n in range(N)])
    vn = torch.stack([vsd[n, at[n]] for n in range(N)])
    P = torch.tensor(pos, dtype=torch.int32, device=DEV)
    o = g2.gdr2_swa_decode_step(qd, kn, vn, kc, vc, P, sinks=sinks)
    torch.cuda.synchronize()
    L2 = [p + 1 for p in pos]
    rk, rv = block.swa_cache(f64(ks), f64(vs), blank, blank, window, sinks, L2)
    assert np.array_equal(f64(kc), rk, equal_nan=True) and np.array_equal(f64(vc), rv, equal_nan=True)
    for n, p in enumerate(pos):
        if p < 0:
            assert not o[n].any()
            continue
        Q = np.zeros((1, p + 1, H, d))
        Q[0, p] = f64(q)[n]
        r = block.swa(Q, f64(ks)[n:n + 1, : p + 1], f64(vs)[n:n + 1, : p + 1], window, sinks, d ** -0.5)
        b = swa_bounds(r, dtype, d, cap)
        within(f"o[{n}]", o[n], r["o"][0, p], b["o"][0, p])


def test_decode_steps_continue_a_prefill():
    """A prefill, its cache, and tokens one by one equal the whole sequence's attention."""
    B, T, H, Hkv, d, window, sinks, T0 = 2, 150, 4, 2, 64, 40, 3, 100
    q, k, v, _ = _swa_inputs(B, T, H, Hkv, d, "bf16", 21)
    qd, kd, vd = dev(q, k, v)
    kc = torch.zeros(B, window + sinks, Hkv, d, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    lengths = [T0, T0 - 30]
    g2.gdr2_swa_cache_fill(kd[:, :T0].contiguous(), vd[:, :T0].contiguous(), kc, vc, sinks=sinks,
                           lengths=torch.tensor(lengths, dtype=torch.int32, device=DEV))
    r = block.swa(f64(q), f64(k), f64(v), window, sinks, d ** -0.5)
    b = swa_bounds(r, "bf16", d, window + sinks)
    pos = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    for _ in range(45):
        i = pos.tolist()
        tok = lambda t: torch.stack([t[n, i[n]] for n in range(B)])  # noqa: E731
        o = g2.gdr2_swa_decode_step(tok(qd), tok(kd), tok(vd), kc, vc, pos, sinks=sinks)
        for n in range(B):
            within(f"o at {i[n]}", o[n], r["o"][n, i[n]], b["o"][n, i[n]])
        pos += 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,H,Hkv,window,sinks", [(43, 6, 3, 500, 4), (64, 3, 3, 500, 0), (5, 2, 2, 4000, 10)])
def test_decode_parts_and_large_positions(dtype, N, H, Hkv, window, sinks):
    """Caches of which each part of the slots, none, or only the first parts hold anything; positions up to
    the last int32.  A full cache's slots are all visible, in any order."""
    d, cap = 64, window + sinks
    announce(f"decode parts {dtype} N={N} H={H}/{Hkv} window={window} sinks={sinks}")
    gen = torch.Generator().manual_seed(N)
    kc, vc = randn(gen, (N, cap, Hkv, d), dtype), randn(gen, (N, cap, Hkv, d), dtype)
    q, k, v = randn(gen, (N, H, d), dtype), randn(gen, (N, Hkv, d), dtype), randn(gen, (N, Hkv, d), dtype)
    pos = torch.randint(0, 3 * cap, (N,), generator=gen, dtype=torch.int32)
    pos[0], pos[1], pos[2], pos[3] = 2 ** 31 - 1, 130, cap - 1, -(2 ** 31)
    kd, vd, kn, vn, qd, pd = dev(kc, vc, k, v, q, pos)
    o = g2.gdr2_swa_decode_step(qd, kn, vn, kd, vd, pd, sinks=sinks)
    torch.cuda.synchronize()
    for n, p in enumerate(pos.tolist()):
        if p >= 0:
            slot = p if p < sinks else sinks + (p - sinks) % window
            kc[n, slot], vc[n, slot] = k[n], v[n]
    assert torch.equal(kd.cpu(), kc) and torch.equal(vd.cpu(), vc)
    for n in (0, 1, 2, 3, N - 1):
        held = min(int(pos[n]) + 1, cap)
        if held <= 0:
            assert not o[n].any()
            continue
        K, V, Q = f64(kc[n, :held]), f64(vc[n, :held]), f64(q[n])
        for h in range(H):
            Kh, Vh = K[:, h // (H // Hkv)], V[:, h // (H // Hkv)]
            s = Kh @ Q[h] * d ** -0.5
            w = np.exp(s - s.max())
            w /= w.sum()
            r = dict(smax=float((np.abs(Kh) @ np.abs(Q[h])).max()) * d ** -0.5, o=w @ Vh, o_abs=w @ np.abs(Vh), lse=np.zeros(()))
            within(f"o[{n}, {h}]", o[n, h], r["o"], swa_bounds(r, dtype, d, cap)["o"])
