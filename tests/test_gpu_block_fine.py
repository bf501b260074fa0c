"""bf16 gradients of the attention over short sequences: each rounded once from sums that are good to 16 bits."""
import numpy as np
import pytest
import torch

import gated_delta_rule_gdr_amd as g2
from oracle import block
from tests._block import U, U32, f64, randn, swa_bounds, within
from tests._util import announce

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,T,H,Hkv,window,sinks,lengths", [
    (1, 1, 2, 1, 5, 0, None), (1, 2, 2, 1, 145, 17, None), (4, 5, 2, 1, 2, 1, None), (1, 15, 12, 3, 2, 4, None), (3, 31, 6, 3, 9, 0, [31, 0, 20]),
    (2, 32, 3, 3, 64, 64, None), (1, 32, 1, 1, 20, 3, [30]), (2, 32, 4, 2, 64, 0, [32, 1]), (40, 32, 9, 9, 20, 2, None)])
def test_short_sequences_round_their_gradients_once(d, B, T, H, Hkv, window, sinks, lengths):
    """Probabilities and score gradients enter the products in two bf16 pieces: 2^-8 of 2^-8 is left of each, the sums
    are fp32, and delta is summed from the probabilities (fp32 terms, as the products').  So the bounds of
    tests/_block.py hold with 2^-16 in place of 2^-8 in the sums, and with no rounding of o in delta."""
    announce(f"swa fine B={B} T={T} H={H}/{Hkv} d={d} window={window} sinks={sinks} lengths={lengths}")
    gen = torch.Generator().manual_seed(T + window + sinks)
    q, k, v, dO = (randn(gen, (B, T, h, d), "bf16") for h in (H, Hkv, Hkv, H))
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV)
    dev = [t.to(DEV) for t in (q, k, v, dO)]
    o, lse = g2.gdr2_swa_fwd(*dev[:3], window, sinks=sinks, lengths=ln)
    g = g2.gdr2_swa_bwd(*dev[:3], o, lse, dev[3], window, sinks=sinks, lengths=ln)
    r = block.swa(f64(q), f64(k), f64(v), window, sinks, d ** -0.5, lengths, f64(dO))
    n = T * (H // Hkv) + T
    ep, up, uo = ((2 * d + 16) * r["smax"] + 128.0) * U32, 2.0 ** -16, U["bf16"]
    few = up + 4 * ep + (2 * n + 4 * d) * U32
    within("dv", g["dv"], r["dv"], few * r["dv_abs"] + uo * np.abs(r["dv"]) + 1e-30)
    for name in ("dq", "dk"):
        within(name, g[name], r[name], few * (r[name + "_abs"] + 4 * r[name + "_delta"]) + uo * np.abs(r[name]) + 1e-30)
    within("o", o, r["o"], swa_bounds(r, "bf16", d, n)["o"])
