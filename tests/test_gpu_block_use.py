"""The operators around the mixer as a program uses them: together, beside the mixer, on streams of its
own, inside captured graphs, on unaligned-to-a-line buffers, with workspaces it keeps, and past 32-bit
offsets.  Results must equal those of the plain calls bit for bit."""
import pytest
import torch

import gated_delta_rule_gdr_amd as g2
from oracle import block
from tests._block import DT, f64, randn, swa_bounds, within
from tests._util import announce

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _inputs(B=2, T=400, H=4, Hkv=2, d=64, dtype="bf16", seed=1):
    gen = torch.Generator().manual_seed(seed)
    D = H * d
    x = dict(x=randn(gen, (B, T, D), dtype), w=1.0 + 0.1 * randn(gen, (D,)), b=randn(gen, (D,)),
             dy=randn(gen, (B, T, D), dtype), q=randn(gen, (B, T, H, d), dtype), k=randn(gen, (B, T, Hkv, d), dtype),
             v=randn(gen, (B, T, Hkv, d), dtype), dO=randn(gen, (B, T, H, d), dtype),
             la=-0.1 * torch.nn.functional.softplus(randn(gen, (B, T, D))), h0=randn(gen, (B, D)), dhT=randn(gen, (B, D)),
             L=torch.tensor([T, T // 3], dtype=torch.int32))
    return {n: t.to(DEV) for n, t in x.items()}


def _training(s):
    """Every forward and backward once; a list of tensors."""
    y, mean, rstd = g2.gdr2_layer_norm_fwd(s["x"], s["w"], s["b"])
    n = g2.gdr2_layer_norm_bwd(s["x"], s["w"], mean, rstd, s["dy"])
    o, lse = g2.gdr2_swa_fwd(s["q"], s["k"], s["v"], 100, sinks=3, lengths=s["L"])
    a = g2.gdr2_swa_bwd(s["q"], s["k"], s["v"], o, lse, s["dO"], 100, sinks=3, lengths=s["L"])
    h, hT, ws = g2.gdr2_glr_fwd(y, s["la"], s["h0"])
    r = g2.gdr2_glr_bwd(y, s["la"], s["dy"], ws, s["dhT"])
    return [y, mean, rstd, *n.values(), o, lse, *a.values(), h, hT, *r.values()]


def _serving(s, kc, vc, pos, state):
    """One token per sequence through norm, attention on the cache and recurrence."""
    y, _, _ = g2.gdr2_layer_norm_fwd(s["x"][:, 7].contiguous(), s["w"], s["b"])
    o = g2.gdr2_swa_decode_step(s["q"][:, 7].contiguous(), s["k"][:, 7].contiguous(), s["v"][:, 7].contiguous(), kc, vc, pos,
                                sinks=3)
    h, state = g2.gdr2_glr_step(y, s["la"][:, 7].contiguous(), state)
    return [y, o, h, state]


def _equal(a, b):
    assert len(a) == len(b)
    for i, (x, y) in enumerate(zip(a, b)):
        assert torch.equal(x, y), i


def _offset(t, nbytes=16):
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
    moved = {n: _offset(t, 4 if n == "L" else 16) for n, t in s.items()}  # (int32 arrays need 4 bytes only)
    _equal(_training(moved), ref)


def test_two_streams_at_once():
    """Calls that overlap in time share nothing: each allocates its own workspaces."""
    s, u = _inputs(seed=3), _inputs(seed=4)
    ref = _training(s), _training(u)
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = [[], []]
    for _ in range(5):
        for i, (x, st) in enumerate(zip((s, u), streams)):
            with torch.cuda.stream(st):
                got[i].append(_training(x))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            _equal(g, ref[i])


def test_captured_graphs_replay():
    """Training and serving passes captured once and replayed with new inputs, eager work between."""
    s, other = _inputs(seed=5), _inputs(seed=6)
    B, T, Hkv, d = s["k"].shape
    kc = torch.zeros(B, 3 + 100, Hkv, d, dtype=s["k"].dtype, device=DEV)
    vc, pos = torch.zeros_like(kc), s["L"].clone()
    state = torch.zeros(B, s["x"].shape[-1], device=DEV)
    g2.gdr2_swa_cache_fill(s["k"], s["v"], kc, vc, sinks=3, lengths=s["L"])
    keep = [t.clone() for t in (kc, vc, state)]
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        _training(s)
        _serving(s, kc, vc, pos, state)
    torch.cuda.current_stream().wait_stream(warm)
    torch.cuda.synchronize()
    gt, gs = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(gt):
        out_t = _training(s)
    with torch.cuda.graph(gs):
        out_s = _serving(s, kc, vc, pos, state)
    for rnd in range(4):
        announce(f"graph replay {rnd}")
        if rnd % 2:
            for n in s:
                s[n].copy_(other[n] if rnd == 1 else s[n].flip(0))
        pos.copy_(s["L"] + rnd)
        eager_t = [t.clone() for t in _training(s)]
        for t, k in zip((kc, vc, state), keep):
            t.copy_(k)
        eager_s = [t.clone() for t in _serving(s, kc, vc, pos, state)] + [kc.clone(), vc.clone()]
        for t, k in zip((kc, vc, state), keep):
            t.copy_(k)
        gt.replay()
        gs.replay()
        torch.cuda.synchronize()
        _equal(out_t, eager_t)
        _equal(out_s + [kc, vc], eager_s)


def test_given_workspaces_keep_results():
    """Workspaces that hold anything, larger than needed, used again for a smaller problem."""
    s, t = _inputs(T=700, seed=7), _inputs(T=300, seed=8)
    ws = {n: torch.full((1 << 24,), 0xA5, dtype=torch.uint8, device=DEV) for n in ("ln", "swa", "gf", "gb")}
    for x in (s, t, s):
        ref = _training(x)
        y, mean, rstd = g2.gdr2_layer_norm_fwd(x["x"], x["w"], x["b"])
        n = g2.gdr2_layer_norm_bwd(x["x"], x["w"], mean, rstd, x["dy"], workspace=ws["ln"])
        o, lse = g2.gdr2_swa_fwd(x["q"], x["k"], x["v"], 100, sinks=3, lengths=x["L"])
        a = g2.gdr2_swa_bwd(x["q"], x["k"], x["v"], o, lse, x["dO"], 100, sinks=3, lengths=x["L"], workspace=ws["swa"])
        h, hT, _ = g2.gdr2_glr_fwd(y, x["la"], x["h0"], workspace=ws["gf"])
        r = g2.gdr2_glr_bwd(y, x["la"], x["dy"], ws["gf"], x["dhT"], workspace=ws["gb"])
        _equal([y, mean, rstd, *n.values(), o, lse, *a.values(), h, hT, *r.values()], ref)
    kc = torch.zeros(2, 103, 2, 64, dtype=torch.bfloat16, device=DEV)
    vc, pos = torch.zeros_like(kc), torch.tensor([0, 0], dtype=torch.int32, device=DEV)
    args = (s["q"][:, 0].contiguous(), s["k"][:, 0].contiguous(), s["v"][:, 0].contiguous())
    a = g2.gdr2_swa_decode_step(*args, kc, vc, pos, sinks=3)
    b = g2.gdr2_swa_decode_step(*args, kc, vc, pos, sinks=3, workspace=ws["swa"])
    assert torch.equal(a, b) and torch.equal(a, args[2].repeat_interleave(2, dim=1))  # the first token sees itself


def test_hybrid_block_prefill_and_decode():
    """A hybrid pair: norm, the recurrent mixer, norm, attention; prefill of T0 tokens and tokens one by
    one equal the whole sequence (attention within its bounds, the norm bit for bit)."""
    B, T, T0, H, d, W, S = 2, 220, 200, 2, 64, 64, 2
    gen = torch.Generator().manual_seed(31)
    x = randn(gen, (B, T, H * d), "bf16").to(DEV)
    w = torch.ones(H * d, device=DEV)
    y, _, _ = g2.gdr2_layer_norm_fwd(x, w)
    la = (-0.1 * torch.nn.functional.softplus(randn(gen, (B, T, H, d)))).to(DEV)
    gate = torch.sigmoid(randn(gen, (B, T, H))).bfloat16().to(DEV)
    heads = lambda t: t.reshape(*t.shape[:-1], H, d).contiguous()  # noqa: E731
    qk = torch.nn.functional.normalize(heads(y).float(), dim=-1).bfloat16()
    m, ST, _ = g2.gdr2_fwd_chunked(qk, qk, heads(y), la, gate, gate)
    z, _, _ = g2.gdr2_layer_norm_fwd(m.reshape(B, T, H * d).contiguous(), w)
    zh = heads(z)
    o, _ = g2.gdr2_swa_fwd(zh, zh, zh, W, sinks=S)
    full = block.swa(f64(zh), f64(zh), f64(zh), W, S, d ** -0.5)
    bound = swa_bounds(full, "bf16", d, W + S)["o"]
    within("o", o, full["o"], bound)
    # serving: state and cache after T0 tokens, then one token at a time
    cut = lambda t: t[:, :T0].contiguous()  # noqa: E731
    m0, st = g2.gdr2_fwd_infer(cut(qk), cut(qk), cut(heads(y)), cut(la), cut(gate), cut(gate))
    kc = torch.empty(B, W + S, H, d, dtype=torch.bfloat16, device=DEV)
    vc = torch.empty_like(kc)
    g2.gdr2_swa_cache_fill(cut(zh), cut(zh), kc, vc, sinks=S)
    for t in range(T0, T):
        at = lambda v: v[:, t].contiguous()  # noqa: E731
        yt, _, _ = g2.gdr2_layer_norm_fwd(at(x), w)
        assert torch.equal(yt, at(y))
        mt, st = g2.gdr2_decode_step(at(qk), at(qk), heads(yt), at(la), at(gate), at(gate), st)
        assert (mt.float() - at(m).float()).abs().max() <= 2e-2 * m.float().abs().max()
        pos = torch.full((B,), t, dtype=torch.int32, device=DEV)
        ot = g2.gdr2_swa_decode_step(at(zh), at(zh), at(zh), kc, vc, pos, sinks=S)
        within(f"o[{t}]", ot, full["o"][:, t], bound[:, t])


def test_long_sequence_offsets():
    """Tensors past 2^31 elements: the last rows equal the same rows of a short problem (their window
    lies inside it), bit for bit."""
    T, H, d, W = 140000, 128, 128, 64
    announce(f"attention T={T} H={H} d={d}")
    tail = 1024
    q = torch.empty(1, T, H, d, dtype=torch.bfloat16, device=DEV)
    assert q.numel() > 1 << 31
    q.normal_()
    k = torch.empty_like(q).normal_()
    v = torch.empty_like(q).normal_()
    cut = lambda t: t[:, T - tail:].contiguous()  # noqa: E731
    o, lse = g2.gdr2_swa_fwd(q, k, v, W)
    o2, lse2 = g2.gdr2_swa_fwd(cut(q), cut(k), cut(v), W)
    # (tiles start at multiples of 128 from the end of the sequence in both: 140000 and 1024 differ by 138976,
    # a multiple of 32 but not of 128, so sums may be cut differently: compare within bf16 steps)
    a, b = o[:, -tail + W:].float(), o2[:, W:].float()
    assert (a - b).abs().max() <= 2 ** -6 * b.abs().max()
    assert (lse[:, :, -tail + W:] - lse2[:, :, W:]).abs().max() <= 1e-4
    g = g2.gdr2_swa_bwd(q, k, v, o, lse, v, W)
    gs = g2.gdr2_swa_bwd(cut(q), cut(k), cut(v), o2, lse2, cut(v), W)
    for n in g:
        a, b = g[n][:, -tail + 2 * W:].float(), gs[n][:, 2 * W:].float()
        assert (a - b).abs().max() <= 2 ** -5 * b.abs().max(), n


def test_long_cache_and_recurrence_offsets():
    N, W, Hkv, d = 40, 65536, 8, 128
    announce(f"cache of {N * W * Hkv * d} elements")
    kc = torch.zeros(N, W, Hkv, d, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    assert kc.numel() > 1 << 31
    gen = torch.Generator().manual_seed(41)
    P = 37   # the last sequence's tokens, at slots that lie past 2^31 elements, around the ring's end
    k, v, q = (randn(gen, (P, h, d), "bf16").to(DEV) for h in (Hkv, Hkv, 2 * Hkv))
    pos0 = 3 * W - P // 2
    for t in range(P):
        one = lambda x: torch.cat([torch.zeros(N - 1, *x.shape[1:], dtype=x.dtype, device=DEV), x[t:t + 1]])  # noqa: E731
        pos = torch.full((N,), -1, dtype=torch.int32, device=DEV)
        pos[-1] = pos0 + t
        o = g2.gdr2_swa_decode_step(one(q), one(k), one(v), kc, vc, pos)
    slots = [(pos0 + t) % W for t in range(P)]
    assert torch.equal(kc[-1, slots], k) and torch.equal(vc[-1, slots], v) and not kc[:-1].any() and not o[:-1].any()
    # the other slots hold zeros: weight exp(0) each, value 0
    s = (f64(q[-1]).reshape(Hkv, 2, d) @ f64(k).transpose(1, 2, 0)) * d ** -0.5
    p = torch.tensor(s).exp()
    ref = (p @ torch.tensor(f64(v).transpose(1, 0, 2))) / (p.sum(-1, keepdim=True) + (W - P))
    got = o[-1].double().cpu().reshape(Hkv, 2, d)
    assert (got - ref).abs().max() <= 2 ** -7 * ref.abs().max() + 2 ** -7 * p.max() / (W - P)
    del kc, vc
    B, T, D = 2, 300000, 4096
    announce(f"recurrence of {B * T * D} elements")
    x = torch.ones(B, T, D, dtype=torch.bfloat16, device=DEV)
    la = torch.full((B, T, D), -0.5, device=DEV)
    h, hT, ws = g2.gdr2_glr_fwd(x, la)
    lim = 1.0 / (1.0 - float(torch.exp(torch.tensor(-0.5, dtype=torch.float64))))
    assert ((hT - lim).abs() <= 1e-5).all() and ((h[:, 100:].float().amin() - lim).abs() <= 2 ** -7 * lim) and (
        (h[:, 100:].float().amax() - lim).abs() <= 2 ** -7 * lim)
    g = g2.gdr2_glr_bwd(x, la, x, ws)
    assert ((g["dx"][:, :-100].float().amin() - lim).abs() <= 2 ** -7 * lim)
    assert ((g["dlog_a"][:, 100:-100].amin() - (lim - 1) * lim).abs() <= 1e-4)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_against_differences(dtype):
    """fp32 directional differences of the kernels' own forwards: the gradient along a direction equals
    the change of the loss along it (fp32; the bf16 backward against the fp32 one)."""
    gen = torch.Generator().manual_seed(51)
    B, T, H, Hkv, d, W, S = 1, 150, 2, 1, 64, 40, 2
    q, k, v, dO = (randn(gen, (B, T, h, d), "bf16") for h in (H, Hkv, Hkv, H))
    t32 = [t.float().to(DEV) for t in (q, k, v, dO)]
    o, lse = g2.gdr2_swa_fwd(*t32[:3], W, sinks=S)
    g32 = g2.gdr2_swa_bwd(*t32[:3], o, lse, t32[3], W, sinks=S)
    if dtype == "bf16":
        b = [t.to(DEV) for t in (q, k, v, dO)]
        ob, lb = g2.gdr2_swa_fwd(*b[:3], W, sinks=S)
        gb = g2.gdr2_swa_bwd(*b[:3], ob, lb, b[3], W, sinks=S)
        for n in gb:  # three roundings of half a bf16 step in every term, terms of either sign
            assert (gb[n].float() - g32[n]).norm() <= 3 * 2 ** -8 * g32[n].norm(), n
        return
    loss = lambda a: (g2.gdr2_swa_fwd(*a, W, sinks=S)[0].double() * t32[3].double()).sum().item()  # noqa: E731
    for i, n in enumerate(("dq", "dk", "dv")):
        u = randn(gen, t32[i].shape).to(DEV)
        eps = 2.0 ** -7
        up, dn = [list(t32[:3]) for _ in range(2)]
        up[i], dn[i] = t32[i] + eps * u, t32[i] - eps * u
        diff = (loss(up) - loss(dn)) / (2 * eps)
        want = (g32[n].double() * u.double()).sum().item()
        # truncation: third derivatives are of the order of the loss, times eps^2 / 6 = 1e-5; rounding:
        # 2^-24 of sums of ~ 2e4 terms of order one, over 2 eps = 2^-6
        scale = (g32[n].double().norm() * u.double().norm()).item()
        assert abs(diff - want) <= 2e-3 * scale / (u.numel() ** 0.5) + 1e-2, n
