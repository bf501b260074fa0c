"""Sequences of a padded batch of linear attention get the results of their own lengths, whatever the batch is padded to."""
import numpy as np
import pytest
import torch

import gated_delta_rule_gdr_amd as g2
from oracle import hybrid
from tests._block import DT, U, f64, randn, within
from tests._hybrid import dla_c32
from tests._util import announce

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64), (64, 128), (128, 128)])
@pytest.mark.parametrize("T", [129, 300, 1100])
def test_dla_short_sequences_of_a_longer_batch_round_once(T, dk, dv):
    """bf16: sequences of up to 128 tokens keep 16 bits of what their products take (2^-15 of the terms at most for each of three
    operands), and their bits are those of the sequence alone."""
    announce(f"dla short sequences padded to T={T} dk={dk} dv={dv}")
    lengths, H = [40, T, 128, 0, 129, 1], 3
    B = len(lengths)
    gen = torch.Generator().manual_seed(T + dk)
    x = dict(q=(dk ** -0.5 * randn(gen, (B, T, H, dk))).to(DT["bf16"]), k=randn(gen, (B, T, H, dk), "bf16"), v=randn(gen, (B, T, H, dv), "bf16"),
             dO=randn(gen, (B, T, H, dv), "bf16"), S0=randn(gen, (B, H, dk, dv)), dS_T=randn(gen, (B, H, dk, dv)))
    g = torch.tensor([-0.05, -0.3, -1e-3])
    d, gd = {n: t.to(DEV) for n, t in x.items()}, g.to(DEV)

    def run(L, rows, width):
        s = {n: (t[rows, :width] if n in ("q", "k", "v", "dO") else t[rows]).contiguous() for n, t in d.items()}
        L = None if L is None else torch.tensor(L, dtype=torch.int32, device=DEV)
        o, S = g2.gdr2_dla_fwd(s["q"], s["k"], s["v"], gd, s["S0"], L)
        return dict(g2.gdr2_dla_bwd(s["q"], s["k"], s["v"], gd, s["dO"], s["S0"], s["dS_T"], L), o=o, S_T=S)

    whole = run(lengths, list(range(B)), T)
    for b in (0, 2, 5):
        L = lengths[b]
        own = run(None, [b], L)
        for n, t in own.items():
            got = whole[n][b:b + 1, :L] if n in ("o", "dq", "dk", "dv") else whole[n][b:b + 1]
            assert torch.equal(got, t), (n, L)
        f = {n: f64(t[b:b + 1, :L] if n in ("q", "k", "v", "dO") else t[b:b + 1]) for n, t in x.items()}
        gn = f64(g)
        ro, _ = hybrid.dla_forward(f["q"], f["k"], f["v"], gn, f["S0"])
        rg = hybrid.dla_backward(f["q"], f["k"], f["v"], gn, f["dO"], f["S0"], f["dS_T"])
        flip = lambda t: np.swapaxes(t, -1, -2)  # noqa: E731
        for name, ref, (p, y, z), init, rev in (("o", ro, ("q", "k", "v"), f["S0"], False), ("dq", rg["dq"], ("dO", "v", "k"), flip(f["S0"]), False),
                                                ("dk", rg["dk"], ("v", "dO", "q"), flip(f["dS_T"]), True), ("dv", rg["dv"], ("k", "q", "dO"), f["dS_T"], True)):
            r = hybrid.dla_sizes(f[p], f[y], f[z], gn, init, None, rev)
            low = (3 * 2.0 ** -15 + dla_c32(f[p].shape[-1], L)) * r["all"]
            within(name, whole[name][b:b + 1, :L], ref, low + U["bf16"] * (1 + 2.0 ** -7) * np.abs(ref) + 1e-30)
    for n in ("o", "dq", "dk", "dv"):
        assert not whole[n][3].any() and not whole[n][0, 40:].any() and not whole[n][5, 1:].any()
