"""Large problems.  Those that take more than one launch (HIP counts a launch in work items, below 2^32):
rows on both sides of a cut equal those of a small call bit for bit.  Long sums: the rounding of a scan
grows with its groups, not with its segments."""
import pytest
import torch

import gated_delta_rule_gdr_amd as g2
from tests._util import announce

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
MAX_ITEMS = (1 << 32) - 1


def _room(nbytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < nbytes:
        pytest.skip(f"needs {nbytes >> 30} GiB of device memory")


def test_layer_norm_rows_beyond_a_launch():
    """8 channels: 64 rows per workgroup of 512 threads, a launch takes (2^32 - 1) // 512 workgroups."""
    D, cut = 8, MAX_ITEMS // 512 * 64
    rows = cut + 4099
    announce(f"layer norm rows={rows} D={D}")
    _room(24 << 30)
    x = torch.randn(rows, D, device=DEV, dtype=torch.bfloat16)
    w, b = torch.randn(D, device=DEV), torch.randn(D, device=DEV)
    y, mean, rstd = g2.gdr2_layer_norm_fwd(x, w, b)
    for at in (0, cut - 2000, rows - 4000):
        s = slice(at, at + 4000)
        for got, want in zip((y[s], mean[s], rstd[s]), g2.gdr2_layer_norm_fwd(x[s].contiguous(), w, b)):
            assert torch.equal(got, want), at


@pytest.mark.parametrize("T", [1, 300])
def test_recurrence_batch_beyond_a_launch(T):
    """One channel strip per batch row: a forward launch takes (2^32 - 1) // 512 segments of 256 tokens,
    a backward launch (2^32 - 1) // 256 of 128."""
    D, nf, nb = 8, (T + 255) // 256, (T + 127) // 128
    cf, cb = MAX_ITEMS // 512 // nf, MAX_ITEMS // 256 // nb
    B = (cb if T == 1 else cf) + 77   # (T = 300: the forward alone is cut; its tensors take 80 GB)
    announce(f"recurrence B={B} T={T} D={D}")
    _room(100 << 30)
    x = torch.randn(B, T, D, device=DEV, dtype=torch.bfloat16)
    la = torch.rand(B, T, D, device=DEV).neg_()
    h0 = torch.randn(B, D, device=DEV)
    h, hT, ws = g2.gdr2_glr_fwd(x, la, h0)
    g = g2.gdr2_glr_bwd(x, la, x, ws, h0) if T == 1 else None
    for at in (0, cf - 50, B - 100):
        s = slice(at, at + 100)
        sx, sl, s0 = x[s].contiguous(), la[s].contiguous(), h0[s].contiguous()
        rh, rT, rws = g2.gdr2_glr_fwd(sx, sl, s0)
        assert torch.equal(h[s], rh) and torch.equal(hT[s], rT), at
        if g:
            r = g2.gdr2_glr_bwd(sx, sl, sx, rws, s0)
            for n in r:
                assert torch.equal(g[n][s], r[n]), (n, at)


def test_decode_sequences_beyond_a_launch():
    """One workgroup of 256 threads per sequence and key/value head."""
    N, d, W = MAX_ITEMS // 256 + 77, 64, 2
    announce(f"decode N={N}")
    _room(40 << 30)
    q, k, v = (torch.randn(N, 1, d, device=DEV, dtype=torch.bfloat16) for _ in range(3))
    kc = torch.randn(N, W, 1, d, device=DEV, dtype=torch.bfloat16)
    vc = torch.randn(N, W, 1, d, device=DEV, dtype=torch.bfloat16)
    pos = (torch.arange(N, device=DEV, dtype=torch.int32) % 5) - 1
    # 200 sequences around each place, before the call stores its tokens
    small = {at: [t[at:at + 200].clone() for t in (q, k, v, kc, vc, pos)] for at in (0, N - 200, MAX_ITEMS // 256 - 100)}
    o = g2.gdr2_swa_decode_step(q, k, v, kc, vc, pos)
    for at, s in small.items():
        want = g2.gdr2_swa_decode_step(*s)
        assert torch.equal(o[at:at + 200], want) and torch.equal(kc[at:at + 200], s[3]) and torch.equal(vc[at:at + 200], s[4]), at


def test_cache_fill_beyond_a_launch():
    """Caches of more than 64 GiB: one thread per 16 bytes.  Only the slots of 100 tokens per sequence are
    written, so the rest of the memory is never touched."""
    B, T, Hkv, d, W = 1100, 100, 8, 128, 32768
    assert B * W * Hkv * d * 2 // 16 > MAX_ITEMS
    announce(f"cache fill B={B} window={W}")
    _room(152 << 30)
    kc = torch.empty(B, W, Hkv, d, device=DEV, dtype=torch.bfloat16)
    vc = torch.empty_like(kc)
    k = torch.randn(B, T, Hkv, d, device=DEV, dtype=torch.bfloat16)
    v = torch.randn(B, T, Hkv, d, device=DEV, dtype=torch.bfloat16)
    kc[:, T] = 1.0
    vc[:, T] = 2.0
    lengths = torch.full((B,), T, device=DEV, dtype=torch.int32)
    lengths[-2], lengths[-1] = 0, T - 1
    kc[-2:, :T], vc[-2:, :T] = 3.0, 4.0
    g2.gdr2_swa_cache_fill(k, v, kc, vc, lengths=lengths)
    assert torch.equal(kc[:-2, :T], k[:-2]) and torch.equal(vc[:-2, :T], v[:-2])
    assert (kc[:, T] == 1.0).all() and (vc[:, T] == 2.0).all()
    assert (kc[-2, :T] == 3.0).all() and (vc[-2, :T] == 4.0).all()
    assert torch.equal(kc[-1, :T - 1], k[-1, :T - 1]) and (kc[-1, T - 1] == 3.0).all() and (vc[-1, T - 1] == 4.0).all()


def test_recurrence_rounds_once_per_group():
    """Nothing decays and every term is positive, so the relative error of a state is at most half a step
    (2^-24) per rounding on its way: 4 in a thread's run, 3 in the wave's scan, one per wave of the segment (8
    forward, 4 backward), 16 in a group's composition, one per group of 16 segments (of 256 / 128 tokens),
    and 8 where the state enters the segment, the wave and the run.  Rounding once per segment instead adds
    up to one per segment: 127 half steps were measured forward with these terms, above the 71 allowed."""
    T, D = 1 << 17, 64
    gen = torch.Generator().manual_seed(61)
    c, u = 1.0 + torch.rand(D, generator=gen), 1.0 + torch.rand(D, generator=gen)
    announce(f"recurrence of {T} equal terms")
    x, dh = (v.to(DEV).expand(1, T, D).contiguous() for v in (c, u))
    la = torch.zeros(1, T, D, device=DEV)
    h, hT, ws = g2.gdr2_glr_fwd(x, la)
    g = g2.gdr2_glr_bwd(x, la, dh, ws)
    t = torch.arange(1, T + 1, dtype=torch.float64, device=DEV)[:, None]
    c, u = c.double().to(DEV), u.double().to(DEV)
    nf, nb = (4 + 3 + w + 16 + T // (16 * s) + 8 for w, s in ((8, 256), (4, 128)))
    step = 2.0 ** -24 * 1.0001   # (terms of second order: 100 half steps of 2^-24)
    H, G = t * c, (T + 1 - t) * u
    assert ((h[0].double() - H).abs() <= nf * step * H).all()
    assert ((hT[0].double() - H[-1]).abs() <= nf * step * H[-1]).all()
    assert ((g["dx"][0].double() - G).abs() <= nb * step * G).all()
    assert ((g["dh0"][0].double() - G[0]).abs() <= nb * step * G[0]).all()
    # R_t h_{t-1}: the state rebuilt from the one that enters the segment of 128
    P = G * (H - c)
    assert ((g["dlog_a"][0].double() - P).abs() <= (nf + nb + 16) * step * P).all()


def test_statistics_at_four_byte_offsets():
    """mean, rstd and lse as slices of a larger buffer: an odd number of rows puts the second one off 16 bytes."""
    gen = torch.Generator().manual_seed(62)
    x, dy = (torch.randn(2, 13, 72, generator=gen).to(DEV) for _ in range(2))
    w = torch.randn(72, generator=gen).to(DEV)
    y, mean, rstd = g2.gdr2_layer_norm_fwd(x, w)
    q, k, v, dO = (torch.randn(1, 13, h, 64, generator=gen).to(DEV) for h in (3, 1, 1, 3))
    o, lse = g2.gdr2_swa_fwd(q, k, v, 5)
    buf = torch.zeros(26 + 26 + 39 + 1, device=DEV)
    m, r, s = buf[1:27].view(2, 13), buf[27:53].view(2, 13), buf[53:].view(1, 3, 13)
    for dst, src in ((m, mean), (r, rstd), (s, lse)):
        dst.copy_(src)
        assert dst.data_ptr() % 16
    a, b = g2.gdr2_layer_norm_bwd(x, w, m, r, dy), g2.gdr2_layer_norm_bwd(x, w, mean, rstd, dy)
    assert all(torch.equal(a[n], b[n]) for n in a)
    a, b = g2.gdr2_swa_bwd(q, k, v, o, s, dO, 5), g2.gdr2_swa_bwd(q, k, v, o, lse, dO, 5)
    assert all(torch.equal(a[n], b[n]) for n in a)
