"""Arguments of the operators around the mixer that are numbers: what does not fit the library's types is
refused by the binding instead of being cut to something else."""
import pytest
import torch

import gated_delta_rule_gdr_amd as g2

BF, I32 = torch.bfloat16, torch.int32


def _attention():
    q, k = torch.zeros(2, 5, 4, 64, dtype=BF), torch.zeros(2, 5, 2, 64, dtype=BF)
    return q, k, k.clone()


@pytest.mark.parametrize("name", ["window", "sinks"])
@pytest.mark.parametrize("bad,match", [((1 << 64) + 512, "64 bits"), (-(1 << 63) - 1, "64 bits"), (2.5, "whole number"),
                                       (float("nan"), "NaN")])
def test_window_and_sinks_are_not_cut(name, bad, match):
    q, k, v = _attention()
    lse, o, kc, pos = torch.zeros(2, 4, 5), q.clone(), torch.zeros(2, 9, 2, 64, dtype=BF), torch.zeros(2, dtype=I32)
    a = {"window": 3, "sinks": 1, name: bad}
    with pytest.raises(ValueError, match=match):
        g2.gdr2_swa_fwd(q, k, v, **a)
    with pytest.raises(ValueError, match=match):
        g2.gdr2_swa_bwd(q, k, v, o, lse, o.clone(), **a)
    with pytest.raises(ValueError, match=match):
        g2.swa_bwd_workspace_bytes(2, 5, 4, 2, 64, **a)
    with pytest.raises(ValueError, match=match):
        g2.swa_decode_workspace_bytes(2, 4, 2, 64, **a)
    if name == "sinks":
        with pytest.raises(ValueError, match=match):
            g2.gdr2_swa_cache_fill(k, v, kc, kc.clone(), sinks=bad)
        with pytest.raises(ValueError, match=match):
            g2.gdr2_swa_decode_step(*(t[:, 0].contiguous() for t in (q, k, v)), kc, kc.clone(), pos, sinks=bad)


def test_whole_numbers_of_other_types_stay_accepted():
    want = g2.swa_bwd_workspace_bytes(2, 300, 4, 2, 64, 100, 3)
    for w in (100.0, torch.tensor(100), True * 100):
        assert g2.swa_bwd_workspace_bytes(2, 300, 4, 2, 64, w, 3) == want
    assert g2.swa_bwd_workspace_bytes(2, 300, 4, 2, 64, (1 << 63) - 1, 3) > 0    # a window without an end
    q, k, v = _attention()
    with pytest.raises(ValueError, match="GPU tensors"):
        g2.gdr2_swa_fwd(q, k, v, 3.0, sinks=torch.tensor(1))


def test_empty_heads_have_a_scale():
    assert g2._swa_scale(None, 64) == 0.125 and g2._swa_scale(0.3, 0) == 0.3 and g2._swa_scale(None, 0) == 1.0
