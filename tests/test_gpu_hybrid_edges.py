"""Paged decode at the ends of the scores' range."""
import pytest
import torch

import gated_delta_rule_gdr_amd as g2
from tests._util import announce

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("n", [1, 2, 300, 700])
def test_paged_decode_scores_near_the_largest_number(n, sign):
    """Every position's score, in powers of two, is the same: one key's product of 2.2e38 times log2 e is 3.2e38 of fp32's
    3.4e38.  Softmax weighs the positions alike, so whole-number values average exactly but for the sum's roundings and the
    division's (n + 2 half steps)."""
    announce(f"paged decode of {n} positions, scores {sign * 3.2e38}")
    H, Hkv, d, page = 4, 2, 64, 16
    pages = -(-n // page)
    gen = torch.Generator().manual_seed(n)
    kp = torch.zeros(pages, page, Hkv, d)
    kp[..., 0] = sign * 2.2e19
    vp = torch.randint(1, 9, (pages, page, Hkv, d), generator=gen).float()
    q, k = torch.zeros(1, H, d), torch.zeros(1, Hkv, d)
    q[..., 0], k[..., 0] = 1e19, sign * 2.2e19
    v = torch.randint(1, 9, (1, Hkv, d), generator=gen).float()
    table, pos = torch.arange(pages, dtype=torch.int32)[None], torch.tensor([n - 1], dtype=torch.int32)
    o = g2.gdr2_paged_decode_step(*(t.to(DEV) for t in (q, k, v, kp, vp, table, pos)), scale=1.0)
    rows = vp.view(-1, Hkv, d)[:n].double().clone()
    rows[n - 1] = v[0].double()
    ref = rows.mean(0).repeat_interleave(H // Hkv, dim=0)[None]
    assert ((o.cpu().double() - ref).abs() <= (n + 2) * 2.0 ** -24 * ref).all()
