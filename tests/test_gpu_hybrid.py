"""GPU parity of the residual stream's RMS norm, linear attention with a decay per head and the paged cache
against the fp64 definitions of oracle/hybrid.py, element by element within the bounds of tests/_hybrid.py."""
import numpy as np
import pytest
import torch

import gated_delta_rule_gdr_amd as g2
from oracle import hybrid
from tests._block import DT, U, U32, f64, randn, swa_bounds, within
from tests._hybrid import dla_bounds, dla_c32, dla_state_bounds, norm_close
from tests._util import announce

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
I32 = torch.int32


def dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def i32(x):
    return None if x is None else torch.tensor(x, dtype=I32, device=DEV)


# ------------------------------------------------------------------ RMS norm
ROWS = [(1, 8), (37, 64), (5, 72), (130, 128), (9, 256), (70, 504), (33, 1000), (600, 2048), (3, 4096), (5, 5000),
        (11, 8192), (2, 16384), (4099, 24)]


def _rms_inputs(rows, D, dtype, residual, seed):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.exp(randn(gen, (rows, 1))) * randn(gen, (rows, D))).to(DT[dtype])
    r = (2.0 * randn(gen, (rows, D))).to(DT[dtype]) if residual else None
    return x, r, 1.0 + 0.1 * randn(gen, (D,)), randn(gen, (rows, D), dtype), randn(gen, (rows, D), dtype)


def _stream(x, r):
    return x if r is None else (x.float() + r.float()).to(x.dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("rows,D", ROWS)
def test_rms_norm(dtype, residual, rows, D):
    announce(f"rms norm {dtype} rows={rows} D={D} residual={residual}")
    x, r, w, dy, dh = _rms_inputs(rows, D, dtype, residual, rows * 7 + D)
    xd, rd, wd, dyd, dhd = dev(x, r, w, dy, dh)
    y, h, rstd = g2.gdr2_rms_norm_fwd(xd, wd, rd)
    use = dhd if residual else None
    g = g2.gdr2_rms_norm_bwd(h, wd, rstd, dyd, use)
    torch.cuda.synchronize()
    hs = _stream(x, r)
    assert torch.equal(h.cpu(), hs)
    H, W, DY, DH = f64(hs), f64(w), f64(dy), f64(dh) if residual else None
    ry, rr = hybrid.rms_forward(H, W, 1e-6)
    rg = hybrid.rms_backward(H, W, 1e-6, DY, DH)
    # sums of one sign pass at most 64 roundings, rstd half of that and four more, n two more
    within("rstd", rstd, rr, 40 * U32 * rr)
    within("y", y, ry, (44 * U32 + U[dtype] * (1 + 2.0 ** -7)) * np.abs(ry))
    n, a = np.abs(H) * rr[:, None], np.abs(DY * W)
    m = (a * n).mean(-1, keepdims=True)
    edx = rr[:, None] * (a * 48 + n * m * 200) * U32 + 4 * U32 * (0 if DH is None else np.abs(DH))
    within("dx", g["dx"], rg["dx"], edx + U[dtype] * (1 + 2.0 ** -7) * np.abs(rg["dx"]))
    within("dweight", g["dweight"], rg["dweight"], (rows / 512 + 64 + 48) * U32 * (np.abs(DY) * n).sum(0) + 1e-30)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("rows,D", ROWS)
def test_rms_norm_q8(dtype, group, rows, D):
    announce(f"rms norm q8 {dtype} rows={rows} D={D} group={group}")
    residual = (rows + D) % 3 != 0
    x, r, w, _, _ = _rms_inputs(rows, D, dtype, residual, rows * 5 + D)
    x[rows // 2, D // 2:] = 0.0     # whole groups of zeros
    if residual:
        r[rows // 2, D // 2:] = 0.0
    xd, rd, wd = dev(x, r, w)
    y8, scale, h = g2.gdr2_rms_norm_q8_fwd(xd, wd, rd, group=group)
    torch.cuda.synchronize()
    hs = _stream(x, r)
    assert torch.equal(h.cpu(), hs) and y8.dtype == torch.float8_e4m3fn
    ry, _ = hybrid.rms_forward(f64(hs), f64(w), 1e-6)
    G = group or D
    pad = np.pad(np.abs(ry), ((0, 0), (0, -D % G))).reshape(rows, -1, G).max(-1)
    got = f64(scale) if group else f64(scale)[:, None]
    assert scale.shape == ((rows, -(-D // G)) if group else (rows,))
    within("scale", got, pad / 448.0, 50 * U32 * pad / 448.0)
    s = np.repeat(got, G, axis=1)[:, :D]
    # half a step of e4m3: 2^-4 of a normal value, 2^-10 scales of a subnormal one; y itself 50 u32
    within("y8", f64(y8.float()) * s, ry, (2.0 ** -4 + 100 * U32) * np.abs(ry) + 2.0 ** -10 * s * (1 + 1e-5))
    top = np.abs(f64(y8.float()))
    assert top.max() == 448.0 and not top[rows // 2, D // 2 + (-(D // 2)) % G:].any()


def test_rms_norm_q8_nonfinite_values_stay_under_their_scale():
    x = torch.randn(6, 256, device=DEV)
    x[1, 3], x[2, 200] = float("nan"), float("inf")
    w = torch.ones(256, device=DEV)
    y8, scale, _ = g2.gdr2_rms_norm_q8_fwd(x, w, group=64)
    f, s = y8.float(), scale
    rest = [0, 3, 4, 5]
    assert torch.isfinite(f[rest]).all() and torch.isfinite(s[rest]).all()
    assert torch.isnan(s[1]).all() and torch.isnan(f[1]).all()        # the row's rstd is NaN
    assert torch.isnan(s[2, 3]) and torch.isnan(f[2, 192:]).all() and not f[2, :192].any() and not s[2, :3].any()
    y8, scale, _ = g2.gdr2_rms_norm_q8_fwd(x, w)
    assert torch.isnan(scale[[1, 2]]).all() and torch.isnan(y8.float()[[1, 2]]).all() and torch.isfinite(y8.float()[rest]).all()


def test_rms_norm_in_place_empty_and_deterministic():
    gen = torch.Generator().manual_seed(3)
    x, r, w, dy, dh = dev(*[randn(gen, s, "bf16") if len(s) > 1 else randn(gen, s) for s in ((700, 1000), (700, 1000), (1000,), (700, 1000), (700, 1000))])
    y, h, rstd = g2.gdr2_rms_norm_fwd(x, w, r)
    r2 = r.clone()
    y2, h2, rstd2 = g2.gdr2_rms_norm_fwd(x, w, r2, h_out=r2)
    assert h2 is r2 and torch.equal(h, r2) and torch.equal(y, y2) and torch.equal(rstd, rstd2)
    r2 = r.clone()
    a = g2.gdr2_rms_norm_q8_fwd(x, w, r, group=32)
    b = g2.gdr2_rms_norm_q8_fwd(x, w, r2, group=32, h_out=r2)
    assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[1], b[1]) and torch.equal(a[2], r2)
    g, f = [g2.gdr2_rms_norm_bwd(h, w, rstd, dy, dh) for _ in range(2)]
    assert torch.equal(g["dx"], f["dx"]) and torch.equal(g["dweight"], f["dweight"])
    e = x[:0]
    y, h, rstd = g2.gdr2_rms_norm_fwd(e, w, e)
    assert y.shape == e.shape and not g2.gdr2_rms_norm_bwd(h, w, rstd, y)["dweight"].any()
    assert g2.gdr2_rms_norm_q8_fwd(e, w, group=64)[1].shape == (0, 16)


# ------------------------------------------------------------------ linear attention with a decay per head
DECAYS = [0.0, -0.5, -0.01, float("-inf"), -3.0, -1e-4, -40.0, -0.1]


def _dla_inputs(B, T, H, dk, dv, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    q = (dk ** -0.5 * randn(gen, (B, T, H, dk))).to(DT[dtype])
    g = torch.tensor([DECAYS[(h + seed) % len(DECAYS)] for h in range(H)])
    return dict(q=q, k=randn(gen, (B, T, H, dk), dtype), v=randn(gen, (B, T, H, dv), dtype), g=g,
                dO=randn(gen, (B, T, H, dv), dtype), S0=randn(gen, (B, H, dk, dv)), dS_T=randn(gen, (B, H, dk, dv)))


def _dla_check(B, T, H, dk, dv, dtype, lengths=None, states=True, seed=0, garbage=float("nan")):
    announce(f"dla {dtype} B={B} T={T} H={H} dk={dk} dv={dv} lengths={lengths} states={states}")
    x = _dla_inputs(B, T, H, dk, dv, dtype, seed + T + dk)
    if lengths is not None:
        for b, L in enumerate(lengths):
            for n in ("q", "k", "v", "dO"):
                x[n][b, max(L, 0):] = garbage
    if not states:
        x["S0"] = x["dS_T"] = None
    d = {n: None if t is None else t.to(DEV) for n, t in x.items()}
    Ld = i32(lengths)
    o, ST = g2.gdr2_dla_fwd(d["q"], d["k"], d["v"], d["g"], d["S0"], Ld)
    gr = g2.gdr2_dla_bwd(d["q"], d["k"], d["v"], d["g"], d["dO"], d["S0"], d["dS_T"], Ld)
    torch.cuda.synchronize()
    f = {n: f64(t) for n, t in x.items()}
    if lengths is not None:
        for b, L in enumerate(lengths):
            for n in ("q", "k", "v", "dO"):
                f[n][b, max(L, 0):] = 0.0
    ro, rS = hybrid.dla_forward(f["q"], f["k"], f["v"], f["g"], f["S0"], lengths)
    rg = hybrid.dla_backward(f["q"], f["k"], f["v"], f["g"], f["dO"], f["S0"], f["dS_T"], lengths)
    flip = lambda t: None if t is None else np.swapaxes(t, -1, -2)  # noqa: E731
    passes = {"o": (o, ro, ("q", "k", "v"), f["S0"], False), "dq": (gr["dq"], rg["dq"], ("dO", "v", "k"), flip(f["S0"]), False),
              "dk": (gr["dk"], rg["dk"], ("v", "dO", "q"), flip(f["dS_T"]), True),
              "dv": (gr["dv"], rg["dv"], ("k", "q", "dO"), f["dS_T"], True)}
    for name, (got, ref, (a, b, c), init, rev) in passes.items():
        r = hybrid.dla_sizes(f[a], f[b], f[c], f["g"], init, lengths, rev)
        within(name, got, ref, dla_bounds(r, ref, dtype, f[a].shape[-1], T))
        norm_close(name, got, ref, dtype, f[a].shape[-1], T)
        if name == "o":
            within("S_T", ST, rS, dla_state_bounds(r, dtype, dk, T))
        if name == "dv":
            a = np.exp(f["g"])[:, None, None]
            one = np.array([[1.0 if lengths is not None and lengths[b] <= 0 else 0.0] for b in range(B)])[..., None, None]
            r["state"] = r["state"] * np.where(one > 0, 1.0, a)
            within("dS0", gr["dS0"], rg["dS0"], dla_state_bounds(r, dtype, dk, T))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("B,T,H,lengths", [(1, 1, 8, None), (2, 33, 3, None), (1, 64, 4, None), (3, 65, 2, [65, 0, 1]),
                                           (1, 127, 8, None), (4, 200, 3, [200, 64, -7, 300]), (2, 321, 4, [320, 129])])
def test_dla(dtype, dk, dv, B, T, H, lengths):
    _dla_check(B, T, H, dk, dv, dtype, lengths, states=T != 64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128)])
def test_dla_segments(dtype, dk, dv):
    """Few chains: the sequence is cut into segments, some behind a sequence's length."""
    assert g2.dla_fwd_workspace_bytes(3, 2500, 1, dk, dv, DT[dtype]) > 0
    _dla_check(3, 2500, 1, dk, dv, dtype, [2500, 1300, 1024], seed=2, garbage=float("inf"))
    _dla_check(1, 2048, 2, dk, dv, dtype, None, seed=6)


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64), (64, 128), (128, 128)])
@pytest.mark.parametrize("T", [1, 2, 3, 7, 40, 65, 128])
def test_dla_short_sequences_round_once(T, dk, dv):
    """bf16, few tokens: what the products take keeps 16 bits, 2^-15 of the terms at most for each of three operands (the
    scores, the state as read, the state's decayed operand), so the error is that of the result's own rounding, u16, and
    3 2^-15 `all`."""
    announce(f"dla short T={T} dk={dk} dv={dv}")
    x = _dla_inputs(1, T, 1, dk, dv, "bf16", 3 * T)
    x["g"] = torch.tensor([-0.05])
    d = {n: t.to(DEV) for n, t in x.items()}
    f = {n: f64(t) for n, t in x.items()}
    o, _ = g2.gdr2_dla_fwd(d["q"], d["k"], d["v"], d["g"], d["S0"])
    gr = g2.gdr2_dla_bwd(d["q"], d["k"], d["v"], d["g"], d["dO"], d["S0"], d["dS_T"])
    ro, _ = hybrid.dla_forward(f["q"], f["k"], f["v"], f["g"], f["S0"])
    rg = hybrid.dla_backward(f["q"], f["k"], f["v"], f["g"], f["dO"], f["S0"], f["dS_T"])
    flip = lambda t: np.swapaxes(t, -1, -2)  # noqa: E731
    for name, got, ref, (a, b, c), init, rev in (
            ("o", o, ro, ("q", "k", "v"), f["S0"], False), ("dq", gr["dq"], rg["dq"], ("dO", "v", "k"), flip(f["S0"]), False),
            ("dk", gr["dk"], rg["dk"], ("v", "dO", "q"), flip(f["dS_T"]), True), ("dv", gr["dv"], rg["dv"], ("k", "q", "dO"), f["dS_T"], True)):
        r = hybrid.dla_sizes(f[a], f[b], f[c], f["g"], init, None, rev)
        low = (3 * 2.0 ** -15 + dla_c32(f[a].shape[-1], T)) * r["all"]
        within(name, got, ref, low + U["bf16"] * (1 + 2.0 ** -7) * np.abs(ref) + 1e-30)


def test_dla_defaults_empty_and_deterministic():
    x = {n: t.to(DEV) for n, t in _dla_inputs(2, 300, 4, 128, 128, "bf16", 5).items()}
    args = (x["q"], x["k"], x["v"], x["g"])
    zero = torch.zeros_like(x["S0"])
    o, S = g2.gdr2_dla_fwd(*args)
    o2, S2 = g2.gdr2_dla_fwd(*args, S0=zero, lengths=i32([300, 1000]))
    assert torch.equal(o, o2) and torch.equal(S, S2)
    a = g2.gdr2_dla_bwd(*args, x["dO"])
    b = g2.gdr2_dla_bwd(*args, x["dO"], S0=zero, dS_T=zero, lengths=i32([300, 300]))
    for n in a:
        assert torch.equal(a[n], b[n]), n
    o3, none = g2.gdr2_dla_fwd(*args, want_final_state=False)
    assert none is None and torch.equal(o, o3)
    assert g2.gdr2_dla_bwd(*args, x["dO"], want_dS0=False)["dS0"] is None
    e = [t[:, :0].contiguous() for t in (x["q"], x["k"], x["v"], x["dO"])]
    o, S = g2.gdr2_dla_fwd(*e[:3], x["g"], S0=x["S0"])
    g = g2.gdr2_dla_bwd(*e[:3], x["g"], e[3], S0=x["S0"], dS_T=x["dS_T"])
    assert o.shape == e[2].shape and torch.equal(S, x["S0"]) and torch.equal(g["dS0"], x["dS_T"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dla_nonfinite_values_stay_in_their_chain(dtype):
    x = _dla_inputs(2, 200, 4, 64, 64, dtype, 1)
    out = []
    for bad in (False, True):
        if bad:
            x["k"][0, 70, 1] = float("nan")
            x["v"][0, 90, 1] = float("inf")
            x["dO"][0, 100, 1] = float("nan")
        d = {n: t.to(DEV) for n, t in x.items()}
        o, S = g2.gdr2_dla_fwd(d["q"], d["k"], d["v"], d["g"])
        g = g2.gdr2_dla_bwd(d["q"], d["k"], d["v"], d["g"], d["dO"])
        out.append([o, g["dq"], g["dk"], g["dv"], S.unsqueeze(1), g["dS0"].unsqueeze(1)])
    assert torch.isnan(out[1][0][0, 70:, 1]).any()
    for a, b in zip(*out):
        keep = [0, 2, 3]
        assert torch.equal(a[1], b[1]) and torch.equal(a[0][:, keep], b[0][:, keep])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
def test_dla_steps_continue_a_prefill(dtype, dk, dv):
    B, T, T0, H = 3, 80, 70, 8
    announce(f"dla steps {dtype} dk={dk} dv={dv}")
    x = _dla_inputs(B, T, H, dk, dv, dtype, 9)
    d = {n: t.to(DEV) for n, t in x.items()}
    at = lambda t, i: t[:, i].contiguous()  # noqa: E731
    _, S = g2.gdr2_dla_fwd(*(d[n][:, :T0].contiguous() for n in "qkv"), d["g"], d["S0"])
    f = {n: f64(t) for n, t in x.items()}
    ro, rS = hybrid.dla_forward(f["q"], f["k"], f["v"], f["g"], f["S0"])
    r = hybrid.dla_sizes(f["q"], f["k"], f["v"], f["g"], f["S0"])
    bound = dla_bounds(r, ro, dtype, dk, T)
    for t in range(T0, T):
        o, S2 = g2.gdr2_dla_step(*(at(d[n], t) for n in "qkv"), d["g"], S)
        assert S2 is S
        within(f"o[{t}]", o, ro[:, t], bound[:, t])
    within("S", S, rS, dla_state_bounds(r, dtype, dk, T))
    # no state yet; a state of its own
    o, S = g2.gdr2_dla_step(*(at(d[n], 0) for n in "qkv"), d["g"])
    ref = x["k"][:, 0].float()[..., None] * x["v"][:, 0].float()[..., None, :]
    assert torch.equal(S.cpu(), ref)
    keep = S.clone()
    out = torch.empty_like(S)
    a, Sa = g2.gdr2_dla_step(*(at(d[n], 1) for n in "qkv"), d["g"], S, out)
    b, Sb = g2.gdr2_dla_step(*(at(d[n], 1) for n in "qkv"), d["g"], S)
    assert Sa is out and not torch.equal(out, keep) and torch.equal(out, Sb) and torch.equal(a, b)


# ------------------------------------------------------------------ the paged cache
def _table(gen, need, pages, spare=0):
    """Tables that own `need[n]` pages each, in any order, none shared; -1 behind."""
    width = max(need) + spare
    perm = torch.randperm(pages, generator=gen).int()
    assert sum(need) <= pages
    t = torch.full((len(need), width), -1, dtype=I32)
    i = 0
    for n, m in enumerate(need):
        t[n, :m] = perm[i:i + m]
        i += m
    return t


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page,d,Hkv", [(1, 64, 3), (8, 128, 1), (16, 64, 2), (64, 128, 4), (256, 64, 1)])
def test_paged_fill(dtype, page, d, Hkv):
    announce(f"paged fill {dtype} page={page} d={d} Hkv={Hkv}")
    gen = torch.Generator().manual_seed(page + d)
    B, T = 6, 77
    start, lengths = [0, 5, 130, -3, 0, 2 ** 31 - 20], [77, 40, 100, 50, 0, 77]
    need = [-(-max(0, min(s, 1000) + min(n, T)) // page) for s, n in zip(start, lengths)]
    need[2] = max(need[2] - 1, 1)                  # its last tokens have no page
    pages = sum(need) + 2
    table = _table(gen, need, pages)
    table[1, 0] = pages                            # not a page
    table[0, 0], gone = -5, table[0, 0].item()
    k, v = randn(gen, (B, T, Hkv, d), dtype), randn(gen, (B, T, Hkv, d), dtype)
    kp, vp = randn(gen, (pages, page, Hkv, d), dtype), randn(gen, (pages, page, Hkv, d), dtype)
    kd, vd, kpd, vpd, td = dev(k, v, kp, vp, table)
    g2.gdr2_paged_cache_fill(kd, vd, kpd, vpd, td, i32(start), i32(lengths))
    torch.cuda.synchronize()
    rk, rv = hybrid.paged_fill(f64(k), f64(v), f64(kp), f64(vp), table.numpy(), start, lengths)
    assert np.array_equal(f64(kpd), rk) and np.array_equal(f64(vpd), rv)
    assert torch.equal(kpd[gone].cpu(), kp[gone])
    # without start and lengths
    g2.gdr2_paged_cache_fill(kd, vd, kpd, vpd, td)
    rk, rv = hybrid.paged_fill(f64(k), f64(v), rk, rv, table.numpy())
    assert np.array_equal(f64(kpd), rk) and np.array_equal(f64(vpd), rv)


def _decode_check(dtype, d, H, Hkv, page, pos, seed, spare=0, spoil=(), scale=None):
    N = len(pos)
    announce(f"paged decode {dtype} d={d} H={H}/{Hkv} page={page} N={N} longest={max(pos)}")
    gen = torch.Generator().manual_seed(seed)
    need = [max(0, p) // page + 1 for p in pos]
    pages = sum(need) + 1
    table = _table(gen, need, pages, spare)
    for n, i, e in spoil:
        table[n, i] = e if e < 0 else pages + e
    kp, vp = randn(gen, (pages, page, Hkv, d), dtype), randn(gen, (pages, page, Hkv, d), dtype)
    # rows that no token has been written to hold NaN
    held = torch.zeros(pages * page, dtype=torch.bool)
    for n, p in enumerate(pos):
        rows = hybrid.paged_rows(table[n].tolist(), page, pages, range(max(p, 0)))
        held[rows[rows >= 0]] = True
    for t in (kp, vp):
        t.view(-1, Hkv, d)[~held] = float("nan")
    q, k, v = randn(gen, (N, H, d), dtype), randn(gen, (N, Hkv, d), dtype), randn(gen, (N, Hkv, d), dtype)
    kpd, vpd, qd, kd, vd, td = dev(kp, vp, q, k, v, table)
    o = g2.gdr2_paged_decode_step(qd, kd, vd, kpd, vpd, td, i32(pos), scale=scale)
    torch.cuda.synchronize()
    r = hybrid.paged_decode(f64(q), f64(k), f64(v), f64(kp), f64(vp), table.tolist(), pos, d ** -0.5 if scale is None else scale)
    assert np.array_equal(f64(kpd), r["k_pages"], equal_nan=True) and np.array_equal(f64(vpd), r["v_pages"], equal_nan=True)
    b = swa_bounds(dict(smax=r["smax"], o=r["o"], o_abs=r["o_abs"], lse=np.zeros(())), dtype, d, max(pos) + 1)
    within("o", o, r["o"], b["o"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv,page", [(1, 1, 1), (4, 2, 8), (8, 1, 16), (20, 1, 64), (34, 2, 16), (6, 3, 256)])
def test_paged_decode(dtype, d, H, Hkv, page):
    """Positions from the first token on, on both sides of a page's and a step's end; an idle slot."""
    _decode_check(dtype, d, H, Hkv, page, [0, 1, page - 1, page, 31, 32, 127, 128, 129, 300, -1, 1000], seed=page + H)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_paged_decode_one_long_sequence(dtype):
    """Many parts; and few of them used, in a table for a much longer sequence."""
    _decode_check(dtype, 128, 8, 2, 64, [20000], seed=1)
    _decode_check(dtype, 64, 4, 1, 16, [700], seed=2, spare=3000)
    _decode_check(dtype, 64, 3, 3, 32, [5, 4000, -1, 333], seed=3, spare=40)


def test_paged_decode_pages_that_name_nothing():
    """Entries outside of the cache, also the new token's; positions behind the table; no pages at all."""
    _decode_check("bf16", 64, 4, 2, 16, [100, 200, 50, 600], seed=4,
                  spoil=[(0, 0, -1), (0, 3, 0), (1, 12, -7), (2, 3, 5)] + [(3, i, -1) for i in range(38)])
    N, H, Hkv, d, page = 3, 4, 2, 64, 8
    gen = torch.Generator().manual_seed(9)
    q, k, v = dev(randn(gen, (N, H, d)), randn(gen, (N, Hkv, d)), randn(gen, (N, Hkv, d)))
    kp, vp = dev(randn(gen, (6, page, Hkv, d)), randn(gen, (6, page, Hkv, d)))
    table = torch.tensor([[0, 1], [2, 3], [4, 5]], dtype=I32, device=DEV)
    keep = kp.clone(), vp.clone()
    pos = [16, 2 ** 31 - 1, 15]      # the table names 16 positions
    o = g2.gdr2_paged_decode_step(q, k, v, kp, vp, table, i32(pos))
    r = hybrid.paged_decode(f64(q), f64(k), f64(v), f64(keep[0]), f64(keep[1]), table.tolist(), pos, d ** -0.5)
    within("o", o, r["o"], swa_bounds(dict(r, lse=np.zeros(())), "f32", d, 17)["o"])
    assert np.array_equal(f64(kp), r["k_pages"]) and np.array_equal(f64(vp), r["v_pages"])
    own = v.repeat_interleave(2, dim=1)
    for pages, width in ((kp, 0), (kp[:0], 2)):
        t = table[:, :width].contiguous()
        o = g2.gdr2_paged_decode_step(q, k, v, pages, vp[:pages.shape[0]], t, i32([3, 4, 5]))
        assert torch.equal(o, own)   # only the new token itself
        g2.gdr2_paged_cache_fill(k[:, None].contiguous(), v[:, None].contiguous(), pages, vp[:pages.shape[0]], t)


def test_paged_decode_large_scores_and_shared_prefix():
    _decode_check("bf16", 64, 4, 1, 16, [300, 40], seed=6, scale=4.0)
    _decode_check("f32", 64, 4, 1, 16, [300, 40], seed=7, scale=4.0)
    # two sequences that read the same pages and write to their own
    gen = torch.Generator().manual_seed(8)
    H, Hkv, d, page = 4, 2, 128, 16
    kp, vp = randn(gen, (6, page, Hkv, d), "bf16"), randn(gen, (6, page, Hkv, d), "bf16")
    table = torch.tensor([[2, 4, 0], [2, 4, 5]], dtype=I32)
    q, k, v = randn(gen, (2, H, d), "bf16"), randn(gen, (2, Hkv, d), "bf16"), randn(gen, (2, Hkv, d), "bf16")
    kpd, vpd, qd, kd, vd, td = dev(kp, vp, q, k, v, table)
    o = g2.gdr2_paged_decode_step(qd, kd, vd, kpd, vpd, td, i32([32, 40]))
    r = hybrid.paged_decode(f64(q), f64(k), f64(v), f64(kp), f64(vp), table.tolist(), [32, 40], d ** -0.5)
    within("o", o, r["o"], swa_bounds(dict(r, lse=np.zeros(())), "bf16", d, 41)["o"])
    assert np.array_equal(f64(kpd), r["k_pages"])


@pytest.mark.parametrize("n", [1, 2, 3, 6, 20, 33])
def test_paged_decode_few_positions_round_once(n):
    """bf16: probabilities keep 16 bits (2^-16 of each, half a step), so the error is that of the result's own rounding and
    the fp32 bounds of the sums."""
    gen = torch.Generator().manual_seed(n)
    H, Hkv, d, page = 4, 2, 64, 16
    kp, vp = randn(gen, (3, page, Hkv, d), "bf16"), randn(gen, (3, page, Hkv, d), "bf16")
    q, k, v = randn(gen, (1, H, d), "bf16"), randn(gen, (1, Hkv, d), "bf16"), randn(gen, (1, Hkv, d), "bf16")
    table = torch.tensor([[2, 0, 1]], dtype=I32)
    kpd, vpd, qd, kd, vd, td = dev(kp, vp, q, k, v, table)
    o = g2.gdr2_paged_decode_step(qd, kd, vd, kpd, vpd, td, i32([n - 1]))
    r = hybrid.paged_decode(f64(q), f64(k), f64(v), f64(kp), f64(vp), table.tolist(), [n - 1], d ** -0.5)
    fine = swa_bounds(dict(r, lse=np.zeros(())), "f32", d, n)["o"] + 2.0 ** -16 * r["o_abs"]
    within("o", o, r["o"], fine + U["bf16"] * (1 + 2.0 ** -7) * np.abs(r["o"]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_paged_decode_infinite_values_stay_in_their_channel(dtype):
    gen = torch.Generator().manual_seed(3)
    H, Hkv, d, page = 4, 2, 64, 16
    kp, vp = randn(gen, (8, page, Hkv, d), dtype), randn(gen, (8, page, Hkv, d), dtype)
    q, k, v = randn(gen, (2, H, d), dtype), randn(gen, (2, Hkv, d), dtype), randn(gen, (2, Hkv, d), dtype)
    table = torch.tensor([[0, 1, 2, 3], [4, 5, 6, 7]], dtype=I32)
    out = []
    for bad in (False, True):
        if bad:
            vp[1, 3, 1, 7] = float("inf")       # sequence 0, position 19, heads 2 and 3, channel 7
            vp[6, 0, 0, 9] = float("nan")       # sequence 1, position 32, behind its token
            kp[6, 1, 0, 9] = float("inf")
        kpd, vpd, qd, kd, vd, td = dev(kp, vp, q, k, v, table)
        out.append(g2.gdr2_paged_decode_step(qd, kd, vd, kpd, vpd, td, i32([40, 31])).cpu())
    same = torch.ones_like(out[0], dtype=torch.bool)
    same[0, 2:, 7] = False
    assert torch.equal(out[0][same], out[1][same]) and not torch.isfinite(out[1][~same]).any()
