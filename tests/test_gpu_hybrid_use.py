"""The residual stream's RMS norm, linear attention with a decay and the paged cache as a program uses them: together,
beside the sliding-window attention, on streams of its own, inside captured graphs, on buffers at odd addresses, with
workspaces it keeps, and past 32-bit offsets.  Results must equal those of the plain calls bit for bit."""
import pytest
import torch

import gated_delta_rule_gdr_amd as g2
from oracle import block
from tests._block import f64, randn, swa_bounds, within
from tests._util import announce
from tests.test_gpu_hybrid import _dla_check

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
I32 = torch.int32


def _i32(x):
    return torch.tensor(x, dtype=I32, device=DEV)


def _heads(t, d):
    return t.reshape(*t.shape[:-1], t.shape[-1] // d, d).contiguous()


def _inputs(B=2, T=700, H=4, d=64, dtype="bf16", seed=1):
    gen = torch.Generator().manual_seed(seed)
    D = H * d
    x = dict(x=randn(gen, (B, T, D), dtype), r=randn(gen, (B, T, D), dtype), w=1.0 + 0.1 * randn(gen, (D,)),
             dy=randn(gen, (B, T, D), dtype), dh=randn(gen, (B, T, D), dtype), dO=randn(gen, (B, T, H, d), dtype),
             g=-0.1 * torch.rand(H, generator=gen), S0=randn(gen, (B, H, d, d)), dS=randn(gen, (B, H, d, d)),
             L=torch.tensor([T, T // 3], dtype=I32))
    return {n: t.to(DEV) for n, t in x.items()}


def _training(s, **ws):
    """Every forward and backward once; a list of tensors."""
    y, h, rstd = g2.gdr2_rms_norm_fwd(s["x"], s["w"], s["r"])
    n = g2.gdr2_rms_norm_bwd(h, s["w"], rstd, s["dy"], s["dh"], workspace=ws.get("rms"))
    y8, scale, h8 = g2.gdr2_rms_norm_q8_fwd(s["x"], s["w"], s["r"], group=64)
    z = _heads(y, s["S0"].shape[-1])
    o, S = g2.gdr2_dla_fwd(z, z, z, s["g"], s["S0"], s["L"], workspace=ws.get("fwd"))
    a = g2.gdr2_dla_bwd(z, z, z, s["g"], s["dO"], s["S0"], s["dS"], s["L"], workspace=ws.get("bwd"))
    return [y, h, rstd, *n.values(), y8.view(torch.uint8), scale, h8, o, S, *a.values()]


def _pages(s, width=300, page=16):
    B, _, H, d = s["dO"].shape
    gen = torch.Generator().manual_seed(77)
    table = torch.randperm(B * width, generator=gen).to(I32).reshape(B, width).to(DEV)
    return torch.zeros(B * width, page, H, d, dtype=s["x"].dtype, device=DEV), torch.zeros(
        B * width, page, H, d, dtype=s["x"].dtype, device=DEV), table


def _serving(s, kp, vp, table, pos, state, ws=None):
    """A prompt into pages, then one token per sequence through norm, linear attention and attention."""
    d = kp.shape[-1]
    z = _heads(s["x"], d)
    g2.gdr2_paged_cache_fill(z, z, kp, vp, table, lengths=s["L"])
    one = lambda t: t[:, 7].contiguous()  # noqa: E731
    y, h, _ = g2.gdr2_rms_norm_fwd(one(s["x"]), s["w"], one(s["r"]))
    t = _heads(y, d)
    m, state = g2.gdr2_dla_step(t, t, t, s["g"], state)
    o = g2.gdr2_paged_decode_step(m, t, m, kp, vp, table, pos, workspace=ws)
    return [y, h, m, o, state]


def _equal(a, b):
    assert len(a) == len(b)
    for i, (x, y) in enumerate(zip(a, b)):
        assert torch.equal(x, y), i


def _offset(t, nbytes):
    buf = torch.zeros(t.numel() + nbytes // t.element_size(), dtype=t.dtype, device=t.device)
    v = buf[nbytes // t.element_size():].view(t.shape)
    v.copy_(t)
    return v


def test_side_stream_and_offset_buffers():
    s = _inputs()
    ref = _training(s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    busy = torch.randn(2048, 2048, device=DEV)
    with torch.cuda.stream(side):
        got = _training(s)
    for _ in range(4):
        busy = busy @ busy.T.contiguous() * 1e-3
    torch.cuda.current_stream().wait_stream(side)
    _equal(got, ref)
    moved = {n: _offset(t, 4 if n in ("L", "g") else 16) for n, t in s.items()}  # (these two need 4 bytes only)
    _equal(_training(moved), ref)
    kp, vp, table = _pages(s)
    pos = _i32([700, 233])
    ref = _serving(s, kp, vp, table, pos, s["S0"].clone()) + [kp, vp]
    kp2, vp2 = (_offset(torch.zeros_like(kp), 16) for _ in range(2))
    got = _serving(moved, kp2, vp2, _offset(table, 4), _offset(pos, 4), s["S0"].clone()) + [kp2, vp2]
    _equal(got, ref)


def test_two_streams_at_once():
    """Calls that overlap in time share nothing: each allocates its own workspaces."""
    s, u = _inputs(seed=3), _inputs(seed=4)
    pages = [_pages(x) for x in (s, u)]
    pos = _i32([700, 233])
    run = lambda i, x: _training(x) + _serving(x, *pages[i], pos, x["S0"].clone())  # noqa: E731
    ref = [run(i, x) for i, x in enumerate((s, u))]
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = [[], []]
    for _ in range(5):
        for i, (x, st) in enumerate(zip((s, u), streams)):
            with torch.cuda.stream(st):
                got[i].append(run(i, x))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            _equal(g, ref[i])


def test_captured_graphs_replay():
    """Training and serving passes captured once and replayed with new inputs, eager work between."""
    s, other = _inputs(seed=5), _inputs(seed=6)
    kp, vp, table = _pages(s)
    pos, state = s["L"].clone(), torch.zeros_like(s["S0"])
    keep = [t.clone() for t in (kp, vp, state)]
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        _training(s)
        _serving(s, kp, vp, table, pos, state)
    torch.cuda.current_stream().wait_stream(warm)
    torch.cuda.synchronize()
    gt, gs = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(gt):
        out_t = _training(s)
    with torch.cuda.graph(gs):
        out_s = _serving(s, kp, vp, table, pos, state)
    for rnd in range(4):
        announce(f"graph replay {rnd}")
        if rnd % 2:
            for n in s:
                s[n].copy_(other[n] if rnd == 1 else s[n].flip(0))
        pos.copy_(s["L"] + rnd)
        eager_t = [t.clone() for t in _training(s)]
        for t, k in zip((kp, vp, state), keep):
            t.copy_(k)
        eager_s = [t.clone() for t in _serving(s, kp, vp, table, pos, state)] + [kp.clone(), vp.clone()]
        for t, k in zip((kp, vp, state), keep):
            t.copy_(k)
        gt.replay()
        gs.replay()
        torch.cuda.synchronize()
        _equal(out_t, eager_t)
        _equal(out_s + [kp, vp], eager_s)


def test_given_workspaces_keep_results():
    """Workspaces that hold anything, larger than needed, used again for a smaller problem."""
    s, t = _inputs(T=1500, seed=7), _inputs(T=300, seed=8)
    ws = {n: torch.full((1 << 24,), 0xA5, dtype=torch.uint8, device=DEV) for n in ("rms", "fwd", "bwd", "dec")}
    for x in (s, t, s):
        ref = _training(x)
        _equal(_training(x, **ws), ref)
        kp, vp, table = _pages(x)
        pos = _i32([1500, 233])
        ref = _serving(x, kp, vp, table, pos, x["S0"].clone())
        _equal(_serving(x, kp, vp, table, pos, x["S0"].clone(), ws["dec"]), ref)


def test_hybrid_block_prefill_and_decode():
    """A hybrid pair: norm of the stream, linear attention, norm of the stream, attention over everything; a padded
    prefill and tokens one by one equal the whole sequence (attention within its bounds, norms bit for bit)."""
    B, T, H, d, page, steps = 2, 220, 2, 64, 16, 20
    T0 = [200, 90]
    gen = torch.Generator().manual_seed(31)
    x, r = (randn(gen, (B, T, H * d), "bf16").to(DEV) for _ in range(2))
    w = (1.0 + 0.1 * randn(gen, (H * d,))).to(DEV)
    g = _i32([0] * H).float() - torch.tensor([0.02, 0.3], device=DEV)
    y, h, _ = g2.gdr2_rms_norm_fwd(x, w, r)
    qkv = _heads(y, d)
    m, _ = g2.gdr2_dla_fwd(qkv, qkv, qkv, g)
    z, h2, _ = g2.gdr2_rms_norm_fwd(m.reshape(B, T, H * d), w, h)
    zh = _heads(z, d)
    o, _ = g2.gdr2_swa_fwd(zh, zh, zh, T)
    full = block.swa(f64(zh), f64(zh), f64(zh), T, 0, d ** -0.5)
    bound = swa_bounds(full, "bf16", d, T)["o"]
    within("o", o, full["o"], bound)
    # serving: state and pages after each sequence's own prompt, what lies behind it never looked at
    L = _i32(T0)
    pad = [t.clone() for t in (qkv, zh)]
    for t in pad:
        for b in range(B):
            t[b, T0[b]:] = float("nan")
    m0, state = g2.gdr2_dla_fwd(pad[0], pad[0], pad[0], g, lengths=L)
    assert torch.equal(m0[0, :T0[0]], m[0, :T0[0]]) and not m0[1, T0[1]:].any()
    width = -(-T // page)
    kp = torch.full((B * width, page, H, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    vp = kp.clone()
    table = torch.randperm(B * width, generator=gen).to(I32).reshape(B, width).to(DEV)
    g2.gdr2_paged_cache_fill(pad[1], pad[1], kp, vp, table, lengths=L)
    rows = torch.arange(B, device=DEV)
    for i in range(steps):
        pos = L + i
        at = lambda t: t[rows, pos.long()].contiguous()  # noqa: E731
        yt, ht, _ = g2.gdr2_rms_norm_fwd(at(x), w, at(r))
        assert torch.equal(yt, at(y)) and torch.equal(ht, at(h))
        y8, scale, h8 = g2.gdr2_rms_norm_q8_fwd(at(x), w, at(r))
        # one rounding to e4m3 (2^-4, or half of its smallest step 2^-10 scales) and the rounding of y to bf16
        back = y8.float() * scale[:, None]
        assert torch.equal(h8, ht) and ((back - yt.float()).abs() <= (2 ** -4 + 2 ** -8) * back.abs() + 2 ** -10 * scale[:, None]
                                        + 2 ** -8 * yt.float().abs()).all()
        t = _heads(yt, d)
        mt, state = g2.gdr2_dla_step(t, t, t, g, state)
        assert (mt.float() - at(m).float()).abs().max() <= 2e-2 * m.float().abs().max()
        zt, _, _ = g2.gdr2_rms_norm_fwd(at(m).reshape(B, H * d), w, ht)
        assert torch.equal(zt, at(z))
        zt = _heads(zt, d)
        ot = g2.gdr2_paged_decode_step(zt, zt, zt, kp, vp, table, pos)
        for b in range(B):
            within(f"o[{b}, {T0[b] + i}]", ot[b], full["o"][b, T0[b] + i], bound[b, T0[b] + i])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_before_a_sequence_are_not_read(dtype):
    """One head: the rows next to a sequence's first are its neighbour's padding (NaN), one row's bytes away."""
    _dla_check(3, 1400, 1, 64, 128, dtype, [1300, 1301, 1399], seed=3)
    _dla_check(3, 130, 1, 128, 64, dtype, [65, 1, 129], seed=4)


def test_one_page_twice_in_a_table():
    """A table may name a page twice as long as nothing is written to it: the same rows count twice."""
    gen = torch.Generator().manual_seed(12)
    H, d, page = 2, 64, 16
    kp, vp = (randn(gen, (4, page, H, d), "bf16").to(DEV) for _ in range(2))
    q, k, v = (randn(gen, (1, H, d), "bf16").to(DEV) for _ in range(3))
    o = g2.gdr2_paged_decode_step(q, k, v, kp.clone(), vp.clone(), _i32([[3, 3, 0]]), _i32([40]))
    kk, vv = torch.cat([kp, kp[3:]]), torch.cat([vp, vp[3:]])
    assert torch.equal(o, g2.gdr2_paged_decode_step(q, k, v, kk, vv, _i32([[3, 4, 0]]), _i32([40])))
    # two tokens stored at one position: one or the other, in pieces of sixteen bytes
    t = torch.stack([torch.full((1, H, d), 1.0), torch.full((1, H, d), 2.0)]).bfloat16().to(DEV)
    g2.gdr2_paged_cache_fill(t, t, kk, vv, _i32([[1], [1]]), start=_i32([5, 5]))
    for x in (kk, vv):
        row = x[1, 5].reshape(-1, 8)
        assert ((row == 1).all(-1) | (row == 2).all(-1)).all()


@pytest.mark.parametrize("operator", ["rms_norm", "dla"])
def test_gradients_against_differences(operator):
    """Directional differences of the kernels' own fp32 forwards along each input."""
    gen = torch.Generator().manual_seed(51)
    if operator == "rms_norm":
        x, w = randn(gen, (37, 200)).to(DEV), (1.0 + 0.1 * randn(gen, (200,))).to(DEV)
        dy, dh = (randn(gen, (37, 200)).to(DEV) for _ in range(2))
        _, _, rstd = g2.gdr2_rms_norm_fwd(x, w)
        g = g2.gdr2_rms_norm_bwd(x, w, rstd, dy, dh)
        args, grads = [x, w], [g["dx"], g["dweight"]]
        loss = lambda x, w: ((g2.gdr2_rms_norm_fwd(x, w)[0].double() * dy.double()).sum()  # noqa: E731
                             + (x.double() * dh.double()).sum()).item()
    else:
        B, T, H, dk, dv = 2, 300, 3, 64, 128
        q, k = (randn(gen, (B, T, H, dk)).to(DEV) * dk ** -0.5 for _ in range(2))
        v, dO = (randn(gen, (B, T, H, dv)).to(DEV) for _ in range(2))
        S0, dS = (randn(gen, (B, H, dk, dv)).to(DEV) for _ in range(2))
        la, L = torch.tensor([0.0, -0.05, -1.0], device=DEV), _i32([300, 171])
        g = g2.gdr2_dla_bwd(q, k, v, la, dO, S0, dS, L)
        args, grads = [q, k, v, S0], [g["dq"], g["dk"], g["dv"], g["dS0"]]

        def loss(q, k, v, S0):
            o, S = g2.gdr2_dla_fwd(q, k, v, la, S0, L)
            return ((o.double() * dO.double()).sum() + (S.double() * dS.double()).sum()).item()
    for i, (a, g) in enumerate(zip(args, grads)):
        u = randn(gen, a.shape).to(DEV)
        eps = 2.0 ** -7
        up, dn = list(args), list(args)
        up[i], dn[i] = a + eps * u, a - eps * u
        diff = (loss(*up) - loss(*dn)) / (2 * eps)
        want = (g.double() * u.double()).sum().item()
        # truncation: the norm's third derivatives, eps^2 / 6 = 1e-5 of the terms (linear attention is linear in each
        # input); rounding: 2^-22 of every output, of either sign, over 2 eps = 2^-6
        scale = (g.double().norm() * u.double().norm()).item()
        assert abs(diff - want) <= 2e-3 * scale / (u.numel() ** 0.5) + 1e-2, i


def test_rows_past_31_bits():
    rows, D = 1100000, 2048
    announce(f"rms norm of {rows} rows of {D}")
    x = torch.empty(rows, D, dtype=torch.bfloat16, device=DEV).normal_()
    assert x.numel() > 1 << 31
    w = torch.rand(D, device=DEV) + 0.5
    y, h, rstd = g2.gdr2_rms_norm_fwd(x, w, x)
    tail = x[-1000:].contiguous()
    y2, h2, r2 = g2.gdr2_rms_norm_fwd(tail, w, tail)
    assert torch.equal(y[-1000:], y2) and torch.equal(h[-1000:], h2) and torch.equal(rstd[-1000:], r2)
    y8, s8, _ = g2.gdr2_rms_norm_q8_fwd(x, w, group=128)
    t8, ts, _ = g2.gdr2_rms_norm_q8_fwd(tail, w, group=128)
    assert torch.equal(y8[-1000:].view(torch.uint8), t8.view(torch.uint8)) and torch.equal(s8[-1000:], ts)
    dx = g2.gdr2_rms_norm_bwd(h, w, rstd, x, y)["dx"]
    d2 = g2.gdr2_rms_norm_bwd(h2, w, r2, tail, y2)["dx"]
    assert torch.equal(dx[-1000:], d2)


def test_linear_attention_past_31_bits():
    """The last rows and the first equal those of a short problem: at e^-1 a token nothing older is left."""
    T, H, d = 131200, 128, 128
    announce(f"linear attention T={T} H={H} d={d}")
    q = torch.empty(1, T, H, d, dtype=torch.bfloat16, device=DEV).normal_()
    assert q.numel() > 1 << 31
    k, v = torch.empty_like(q).normal_(), torch.empty_like(q).normal_()
    g = torch.full((H,), -1.0, device=DEV)
    n, keep = 640, 128         # whole chunks of 64
    end = lambda t: t[:, T - n:].contiguous()  # noqa: E731
    o, S = g2.gdr2_dla_fwd(q, k, v, g)
    o2, S2 = g2.gdr2_dla_fwd(end(q), end(k), end(v), g)
    assert torch.equal(o[:, -keep:], o2[:, -keep:])
    assert (S - S2).abs().max() <= 2 ** -20 * S2.abs().max()
    gr = g2.gdr2_dla_bwd(q, k, v, g, v)
    first = lambda t: t[:, :n].contiguous()  # noqa: E731
    ge = g2.gdr2_dla_bwd(end(q), end(k), end(v), g, end(v))
    gf = g2.gdr2_dla_bwd(first(q), first(k), first(v), g, first(v))
    for name in ("dq", "dk", "dv"):
        assert torch.equal(gr[name][:, -keep:], ge[name][:, -keep:]), name
        assert torch.equal(gr[name][:, :keep], gf[name][:, :keep]), name
    assert (gr["dS0"] - gf["dS0"]).abs().max() <= 2 ** -20 * gf["dS0"].abs().max()
    del o, gr
    N = 132000
    announce(f"states of {N} chains")
    S = torch.ones(N // 16, 16, d, d, device=DEV)
    assert S.numel() > 1 << 31
    a = q.reshape(-1, d)[:N].reshape(N // 16, 16, d).contiguous()
    o, S = g2.gdr2_dla_step(a, a, a, g[:16], S)
    o2, S2 = g2.gdr2_dla_step(a[-2:], a[-2:], a[-2:], g[:16], torch.ones(2, 16, d, d, device=DEV))
    assert torch.equal(o[-2:], o2) and torch.equal(S[-2:], S2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_attention_of_the_most_heads(dtype):
    """Rows 2^15 heads apart (a chunk of 64 spans a gigabyte in fp32): heads at both ends equal those heads alone."""
    T, H, dk, dv = 130, 32768, 64, 64
    announce(f"linear attention of {H} heads, {dtype}")
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    q, k, v = (torch.empty(1, T, H, dk, dtype=dt, device=DEV).normal_() for _ in range(3))
    g = -0.1 * torch.rand(H, device=DEV)
    L = _i32([129])
    pick = [0, 1, H // 2, H - 1]
    few = lambda t: t[:, :, pick].contiguous()  # noqa: E731
    o, S = g2.gdr2_dla_fwd(q, k, v, g, lengths=L)
    o2, S2 = g2.gdr2_dla_fwd(few(q), few(k), few(v), g[pick].contiguous(), lengths=L)
    assert torch.equal(o[:, :, pick], o2) and torch.equal(S[:, pick], S2)
    gr = g2.gdr2_dla_bwd(q, k, v, g, v, lengths=L)
    g2r = g2.gdr2_dla_bwd(few(q), few(k), few(v), g[pick].contiguous(), few(v), lengths=L)
    for n in ("dq", "dk", "dv"):
        assert torch.equal(gr[n][:, :, pick], g2r[n]), n
    assert torch.equal(gr["dS0"][:, pick], g2r["dS0"])


def test_pages_past_31_bits():
    pages, page, Hkv, d = 72000, 64, 4, 128
    announce(f"pages of {pages * page * Hkv * d} elements")
    kp = torch.zeros(pages, page, Hkv, d, dtype=torch.bfloat16, device=DEV)
    vp = torch.zeros_like(kp)
    assert kp.numel() > 1 << 31
    gen = torch.Generator().manual_seed(41)
    T, H = 1000, 8
    k, v = (randn(gen, (2, T, Hkv, d), "bf16").to(DEV) for _ in range(2))
    q, kn, vn = (randn(gen, (2, h, d), "bf16").to(DEV) for h in (H, Hkv, Hkv))
    few = torch.randperm(40, generator=gen).to(I32).reshape(2, 20).to(DEV)
    table = pages - 1 - few
    g2.gdr2_paged_cache_fill(k, v, kp, vp, table, lengths=_i32([T, 700]))
    o = g2.gdr2_paged_decode_step(q, kn, vn, kp, vp, table, _i32([T, 700]))
    ks, vs = (torch.zeros(40, page, Hkv, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    g2.gdr2_paged_cache_fill(k, v, ks, vs, few, lengths=_i32([T, 700]))
    o2 = g2.gdr2_paged_decode_step(q, kn, vn, ks, vs, few, _i32([T, 700]))
    assert torch.equal(o, o2) and torch.equal(kp[-40:].flip(0), ks) and torch.equal(vp[-40:].flip(0), vs)
    assert not kp[:-40].any() and not vp[:-40].any()
