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


def test_statistics_need_four_byte_alignment():
    """mean, rstd and lse are read and written as single numbers.  Refused calls only: a later check's status
    shows that the alignment passed."""
    lib = g2.load_library()
    at = lambda i: 0x100000 * (i + 1)  # noqa: E731
    E_ALIGN, E_ALIAS, E_WS = 5, 6, 7
    for off, alias, ws in ((4, E_ALIAS, E_WS), (2, E_ALIGN, E_ALIGN)):
        for m, r in ((at(3) + off, at(4)), (at(3), at(4) + off)):
            assert lib.gdr2_layer_norm_fwd(4, 64, 1, at(0), at(1), None, 1e-5, at(0), m, r, None) == alias
            assert lib.gdr2_layer_norm_bwd(4, 64, 1, at(0), at(1), m, r, at(5), at(6), at(7), None, at(8), 0, None) == ws
        q = (1, 8, 2, 1, 64, 1, 4, 0, 0.1, at(0), at(1), at(2), None)
        assert lib.gdr2_swa_fwd(*q, at(0), at(4) + off, None) == alias
        assert lib.gdr2_swa_bwd(*q, at(3), at(4) + off, at(5), at(6), at(7), at(8), at(9), 0, None) == ws
