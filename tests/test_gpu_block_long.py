"""Attention past 2^31 elements, every element of chosen heads against fp64 within the derived bounds: grouped
heads, sinks (their far queries, pieces and reduction), padded batches with an empty sequence, both types.
The fp64 form here works on the band of visible pairs, so that long sequences fit; it is itself compared
with the full one."""
import numpy as np
import pytest
import torch

import gated_delta_rule_gdr_amd as g2
from oracle import block
from tests._block import DT, swa_bounds, within
from tests._util import announce

DEV = "cuda:0"


def band(q, k, v, dO, window, sinks, scale, chunk=2048):
    """block.swa for one key/value head: q, dO [L, G, d], k, v [L, d] of one sequence (fp64, any device)."""
    L, G, d = q.shape
    r = {n: torch.zeros_like(q) for n in ("o", "o_abs", "dq", "dq_abs", "dq_delta")}
    r.update({n: torch.zeros_like(k) for n in ("dk", "dk_abs", "dk_delta", "dv", "dv_abs")})
    r["lse"] = torch.zeros(G, L, dtype=q.dtype, device=q.device)
    smax = 0.0
    for i0 in range(0, L, chunk):
        i = torch.arange(i0, min(i0 + chunk, L), device=q.device)[:, None]
        # the window's keys, then the sinks that lie before it
        j = torch.cat([i - torch.arange(window, device=q.device), torch.arange(sinks, device=q.device).expand(len(i), sinks)], 1)
        vis = j >= 0
        vis[:, window:] &= j[:, window:] <= i - window
        j = j.clamp(0, L - 1)   # (hidden pairs; a sequence may be shorter than its sinks)
        K, V, at = k[j], v[j], j[:, :window].reshape(-1)
        for h in range(G):
            Q, g = q[i[:, 0], h], dO[i[:, 0], h]
            S = (K * Q[:, None]).sum(-1) * scale
            smax = max(smax, float((K.abs() * Q.abs()[:, None]).sum(-1)[vis].max()) * scale)
            S = S.masked_fill(~vis, float("-inf"))
            m = S.amax(1, keepdim=True)
            P = torch.exp(S - m)
            z = P.sum(1, keepdim=True)
            P = P / z
            r["lse"][h, i[:, 0]] = (m + z.log())[:, 0]
            O, Oa = (P[..., None] * V).sum(1), (P[..., None] * V.abs()).sum(1)
            dS = P * ((V * g[:, None]).sum(-1) - (g * O).sum(1, keepdim=True))
            De = P * (g.abs() * (Oa + O.abs())).sum(1, keepdim=True)
            for n, val in (("o", O), ("o_abs", Oa), ("dq", scale * (dS[..., None] * K).sum(1)),
                           ("dq_abs", scale * (dS.abs()[..., None] * K.abs()).sum(1)),
                           ("dq_delta", scale * (De[..., None] * K.abs()).sum(1))):
                r[n][i[:, 0], h] = val
            for n, w, x in (("dk", scale * dS, Q), ("dk_abs", scale * dS.abs(), Q.abs()), ("dk_delta", scale * De, Q.abs()),
                            ("dv", P, g), ("dv_abs", P, g.abs())):
                val, s = w[..., None] * x[:, None], min(sinks, L)
                r[n].index_add_(0, at, val[:, :window].reshape(-1, d))
                r[n][:s] += val[:, window:window + s].sum(0)
    return dict({n: x.cpu().numpy() for n, x in r.items()}, smax=smax)


@pytest.mark.parametrize("L,window,sinks", [(1, 1, 0), (1, 64, 5), (4, 64, 5), (3, 1, 64), (200, 7, 3), (150, 64, 5), (90, 100, 64), (77, 30, 40)])
def test_band_is_the_definition(L, window, sinks):
    gen = torch.Generator().manual_seed(L)
    q, dO = (torch.randn(L, 2, 16, generator=gen, dtype=torch.float64) for _ in range(2))
    k, v = (torch.randn(L, 16, generator=gen, dtype=torch.float64) for _ in range(2))
    got = band(q, k, v, dO, window, sinks, 0.25, chunk=64)
    want = block.swa(*(t.numpy()[None] for t in (q, k[:, None], v[:, None])), window, sinks, 0.25, None, dO.numpy()[None])
    for n in got:
        w = want[n] if n == "smax" else want[n][0].reshape(got[n].shape)
        assert np.allclose(got[n], w, rtol=1e-11, atol=1e-12), n


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,H,Hkv,d,lengths", [("bf16", 128, 64, 128, [70001, 0, 131999]), ("f32", 256, 128, 64, [1, 131999])])
def test_attention_past_32_bit_offsets(dtype, H, Hkv, d, lengths):
    B, T, W, S = len(lengths), 132000, 64, 5
    announce(f"attention {dtype} B={B} T={T} H={H}/{Hkv} d={d} window={W} sinks={S} lengths={lengths}")
    torch.cuda.empty_cache()
    need = B * T * (5 * H + 4 * Hkv) * d * DT[dtype].itemsize + (8 << 30)
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip(f"needs {need >> 30} GiB of device memory")
    gen = torch.Generator(device=DEV).manual_seed(71)
    q, k, v, dO = (torch.empty(B, T, h, d, dtype=DT[dtype], device=DEV).normal_(generator=gen) for h in (H, Hkv, Hkv, H))
    # the last sequence starts past 2^31 elements of q, and its last keys lie there too
    assert (B - 1) * T * H * d > 1 << 31 and (B * T - 1000) * Hkv * d > 1 << 31
    for b, L in enumerate(lengths):
        for t in (q, k, v, dO):
            t[b, L:] = float("nan")
    ln = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    o, lse = g2.gdr2_swa_fwd(q, k, v, W, sinks=S, lengths=ln)
    g = g2.gdr2_swa_bwd(q, k, v, o, lse, dO, W, sinks=S, lengths=ln)
    torch.cuda.synchronize()
    G = H // Hkv
    for b, kvh in ((B - 1, Hkv - 1), (B - 1, 0), (0, Hkv - 1)):
        L, hs = lengths[b], slice(kvh * G, kvh * G + G)
        r = band(q[b, :L, hs].double(), k[b, :L, kvh].double(), v[b, :L, kvh].double(), dO[b, :L, hs].double(), W, S, d ** -0.5)
        bd = swa_bounds(r, dtype, d, W + S + L * G)
        # few terms meet in o and dq, and in all of dk and dv but the sinks'
        few = swa_bounds(r, dtype, d, W + S + (W + 128) * G)
        for n in ("o", "lse", "dq"):
            bd[n] = few[n]
        for n in ("dk", "dv"):
            bd[n][S:] = few[n][S:]
        name = f"[{b}, {kvh}]"
        announce(f"compared {name}")
        within("o" + name, o[b, :L, hs], r["o"], bd["o"])
        within("lse" + name, lse[b, hs, :L], r["lse"], bd["lse"])
        within("dq" + name, g["dq"][b, :L, hs], r["dq"], bd["dq"])
        within("dk" + name, g["dk"][b, :L, kvh], r["dk"], bd["dk"])
        within("dv" + name, g["dv"][b, :L, kvh], r["dv"], bd["dv"])
        for t in (o, g["dq"], g["dk"], g["dv"]):
            assert not t[b, L:].any()
        assert torch.isneginf(lse[b, :, L:]).all()
