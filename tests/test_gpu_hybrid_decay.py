"""The decay of linear attention's state where what was carried in outweighs what is added: keys and cotangents that are
zero but for a few tokens, entering states that are not.  Every element against the fp64 definitions of oracle/hybrid.py within
the bounds of tests/_hybrid.py, which are relative to the decayed state there."""
import numpy as np
import pytest
import torch

import gated_delta_rule_gdr_amd as g2
from oracle import hybrid
from tests._block import DT, f64, randn, within
from tests._hybrid import dla_bounds, dla_state_bounds
from tests._util import announce

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# e^(64 g) from 0.04 to 1e-14; on both sides of a half; and of segments of 128 to 512 tokens
FAST = [-0.05, -0.1, -0.15, -0.2, -0.25, -0.3, -0.4, -0.5]
HALF = [-1e-4, -0.005, -0.0107, -0.0109, -0.012, -0.02, 0.0, float("-inf")]
LONG = [-0.001, -0.002, -0.0027, -0.0054, -0.01, -0.02, -0.03, -0.06]


def _check(dtype, T, dk, dv, g, lengths, filled):
    """The forward and dq with keys that are zero behind the first `filled` tokens; dk, dv and dS0 with cotangents of o that are
    zero before the last `filled` of each sequence."""
    announce(f"dla carried state {dtype} T={T} dk={dk} dv={dv} lengths={lengths} filled={filled}")
    H, B = len(g), 1 if lengths is None else len(lengths)
    gen = torch.Generator().manual_seed(T + dk + filled)
    tok = lambda d: randn(gen, (B, T, H, d), dtype)  # noqa: E731
    x = dict(q=(dk ** -0.5 * tok(dk).float()).to(DT[dtype]), k=tok(dk), v=tok(dv), dO=tok(dv), S0=randn(gen, (B, H, dk, dv)),
             dS_T=randn(gen, (B, H, dk, dv)), g=torch.tensor(g))
    x["few_k"], x["few_dO"] = x["k"].clone(), x["dO"].clone()
    x["few_k"][:, filled:] = 0.0
    for b in range(B):
        x["few_dO"][b, :max(0, (T if lengths is None else lengths[b]) - filled)] = 0.0
    d = {n: t.to(DEV) for n, t in x.items()}
    f = {n: f64(t) for n, t in x.items()}
    for b, L in enumerate(lengths or ()):
        for n in ("q", "k", "v", "dO", "few_k", "few_dO"):
            f[n][b, L:] = 0.0
    Ld = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV)
    o, ST = g2.gdr2_dla_fwd(d["q"], d["few_k"], d["v"], d["g"], d["S0"], Ld)
    early = g2.gdr2_dla_bwd(d["q"], d["few_k"], d["v"], d["g"], d["dO"], d["S0"], d["dS_T"], Ld)
    late = g2.gdr2_dla_bwd(d["q"], d["k"], d["v"], d["g"], d["few_dO"], d["S0"], d["dS_T"], Ld)
    torch.cuda.synchronize()
    ro, rS = hybrid.dla_forward(f["q"], f["few_k"], f["v"], f["g"], f["S0"], lengths)
    rq = hybrid.dla_backward(f["q"], f["few_k"], f["v"], f["g"], f["dO"], f["S0"], f["dS_T"], lengths)
    rg = hybrid.dla_backward(f["q"], f["k"], f["v"], f["g"], f["few_dO"], f["S0"], f["dS_T"], lengths)
    flip = lambda t: np.swapaxes(t, -1, -2)  # noqa: E731
    for name, got, ref, (a, b, c), init, rev in (
            ("o", o, ro, ("q", "few_k", "v"), f["S0"], False), ("dq", early["dq"], rq["dq"], ("dO", "v", "few_k"), flip(f["S0"]), False),
            ("dk", late["dk"], rg["dk"], ("v", "few_dO", "q"), flip(f["dS_T"]), True),
            ("dv", late["dv"], rg["dv"], ("k", "q", "few_dO"), f["dS_T"], True)):
        r = hybrid.dla_sizes(f[a], f[b], f[c], f["g"], init, lengths, rev)
        within(name, got, ref, dla_bounds(r, ref, dtype, f[a].shape[-1], T))
        if name == "o":
            within("S_T", ST, rS, dla_state_bounds(r, dtype, dk, T))
        if name == "dv":
            r["state"] = r["state"] * np.exp(f["g"])[:, None, None]
            within("dS0", late["dS0"], rg["dS0"], dla_state_bounds(r, dtype, dk, T))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 128)])
@pytest.mark.parametrize("T,lengths", [(64, None), (65, [65, 62]), (200, [200, 129])])
@pytest.mark.parametrize("g", [FAST, HALF], ids=["fast", "half"])
def test_dla_carried_state(dtype, dk, dv, T, lengths, g):
    for filled in (0, 40):
        _check(dtype, T, dk, dv, g, lengths, filled)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128)])
@pytest.mark.parametrize("g", [LONG, FAST], ids=["long", "fast"])
def test_dla_carried_state_over_segments(dtype, dk, dv, g):
    assert g2.dla_fwd_workspace_bytes(1, 1024, 8, dk, dv, DT[dtype]) > 0 and g2.dla_bwd_workspace_bytes(1, 1024, 8, dk, dv, DT[dtype]) > 0
    _check(dtype, 1024, dk, dv, g, None, 0)
    _check(dtype, 1024, dk, dv, g, [1001], 40)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dla_many_steps_do_not_drift(dtype):
    """Slow decays over 10000 tokens, one by one, whose factors lie half a step of fp32 between two numbers: a rounded factor would be
    off by 2^-25 at every token, to one side, 2500 to 3000 u32 of the state in the end.  What remains are the two roundings that
    every step adds to the state, of either sign: sqrt(2 N / 3) u32 of a state that only grows; 4 sqrt(N) u32 leaves a
    factor of five (e^g - 1 itself, two u32 of it, adds 2 N |g| u32 < 2).  A prefill of the same tokens is as exact."""
    N, H, dk, dv = 10000, 4, 64, 64
    announce(f"dla {N} steps {dtype}")
    gen = torch.Generator().manual_seed(3)
    g = torch.tensor([-(j + 0.5) * 2.0 ** -24 for j in (1677, 500, 100, 16)])
    q = (dk ** -0.5 * randn(gen, (1, N, H, dk))).to(DT[dtype])
    k, v, S0 = (0.1 * randn(gen, (1, N, H, dk))).to(DT[dtype]), randn(gen, (1, N, H, dv), dtype), randn(gen, (1, H, dk, dv))
    qd, kd, vd, gd, S = (t.to(DEV) for t in (q, k, v, g, S0))
    _, ST = g2.gdr2_dla_fwd(qd, kd, vd, gd, S)
    S = S.clone()
    for t in range(N):
        g2.gdr2_dla_step(qd[:, t], kd[:, t], vd[:, t], gd, S)
    a, ref = torch.exp(g.double())[:, None, None], S0[0].double()
    for kt, vt in zip(k[0].double(), v[0].double()):
        ref = a * ref + kt[:, :, None] * vt[:, None, :]
    for name, got in (("steps", S), ("prefill", ST)):
        err = (got[0].cpu().double() - ref).flatten(1).norm(dim=1) / ref.flatten(1).norm(dim=1)
        assert (err <= 4 * N ** 0.5 * 2.0 ** -24).all(), f"{name}: {(err * 2 ** 24).tolist()} u32"
