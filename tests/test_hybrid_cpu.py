"""Refusals of the residual stream's norm, linear attention with a decay and the paged cache on a host without a
GPU: the C ABI rejects bad arguments before any launch, the binding wrong tensors before any library call."""
import ctypes

import pytest
import torch

import gated_delta_rule_gdr_amd as g2
from gated_delta_rule_gdr_amd import load_library

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
OK, E_NULL, E_SHAPE, E_DTYPE, E_UNSUP, E_ALIGN, E_ALIAS, E_WS, E_VALUE = 0, 1, 2, 3, 4, 5, 6, 7, 9


def at(i):
    """Distinct 16-byte aligned addresses that are never dereferenced."""
    return 0x10000000 * (i + 1)


# ------------------------------------------------------------------ C ABI
def test_rms_norm_abi():
    lib = load_library()

    def fwd(rows=4, D=64, dt=1, x=at(0), r=at(1), w=at(2), eps=1e-6, h=at(3), y=at(4), s=at(5)):
        return lib.gdr2_rms_norm_fwd(rows, D, dt, x, r, w, eps, h, y, s, None)

    def q8(rows=4, D=64, dt=1, group=32, x=at(0), r=at(1), w=at(2), eps=1e-6, h=at(3), y=at(4), s=at(5)):
        return lib.gdr2_rms_norm_q8_fwd(rows, D, dt, group, x, r, w, eps, h, y, s, None)
    for f in (fwd, q8):
        assert f(dt=2) == E_DTYPE and f(rows=-1) == f(rows=1 << 31) == E_SHAPE
        assert f(D=0) == f(D=60) == f(D=16392) == E_UNSUP
        assert f(eps=0.0) == f(eps=float("nan")) == f(eps=float("inf")) == E_VALUE
        assert f(r=None) == E_VALUE                                   # a stream to write, and nothing added
        assert f(x=None) == f(w=None) == f(y=None) == f(h=None) == E_NULL
        assert f(x=at(0) + 8) == f(r=at(1) + 8, h=at(3)) == f(s=at(5) + 2) == E_ALIGN
        assert f(y=at(0)) == f(h=at(0)) == f(h=at(1) + 16) == f(s=at(4)) == f(y=at(1), h=at(1)) == E_ALIAS
        assert f(rows=0, x=None) == OK
    assert q8(group=16) == q8(group=256) == q8(group=-32) == q8(group=1) == E_UNSUP and q8(s=None) == E_NULL
    need = lib.gdr2_rms_norm_bwd_workspace_bytes(4, 64)
    assert need > 0 and lib.gdr2_rms_norm_bwd_workspace_bytes(4, 63) == lib.gdr2_rms_norm_bwd_workspace_bytes(-4, 64) == 0

    def bwd(rows=4, D=64, dt=1, h=at(0), s=at(2), dy=at(3), dh=at(4), dx=at(5), dw=at(6), ws=at(7), n=need):
        return lib.gdr2_rms_norm_bwd(rows, D, dt, h, at(1), s, dy, dh, dx, dw, ws, n, None)
    assert bwd(dt=9) == E_DTYPE and bwd(D=12) == E_UNSUP and bwd(rows=-2) == E_SHAPE
    assert bwd(h=None) == bwd(s=None) == bwd(dy=None) == bwd(dx=None) == bwd(dw=None) == E_NULL
    assert bwd(ws=None) == bwd(n=need - 1) == E_WS
    assert bwd(dx=at(3)) == bwd(dx=at(4)) == bwd(dw=at(5)) == bwd(ws=at(0)) == E_ALIAS
    assert bwd(dx=at(5) + 4) == bwd(s=at(2) + 1) == E_ALIGN


def test_dla_abi():
    lib = load_library()
    need = lib.gdr2_dla_fwd_workspace_bytes(1, 4096, 1, 64, 128, 1)
    back = lib.gdr2_dla_bwd_workspace_bytes(1, 4096, 1, 64, 128, 1)
    assert need > 0 and back > 0                                      # few chains: the sequence is cut
    assert lib.gdr2_dla_fwd_workspace_bytes(64, 4096, 16, 128, 128, 1) == 0
    for bad in ((1, 1 << 31, 1, 64, 64, 1), (1 << 20, 64, 2, 64, 64, 1), (1 << 18, 1 << 20, 1, 64, 64, 1), (-1, 1, 1, 64, 64, 1),
                (1, 1, 1, 96, 64, 1), (1, 1, 1, 64, 256, 1), (1, 1, 1, 64, 64, 5)):
        assert lib.gdr2_dla_fwd_workspace_bytes(*bad) == lib.gdr2_dla_bwd_workspace_bytes(*bad) == 0

    def fwd(B=1, T=4096, H=1, dk=64, dv=128, dt=1, q=at(0), k=at(1), v=at(2), g=at(3), S0=None, L=None, o=at(4), ST=at(5), ws=at(6), n=need):
        return lib.gdr2_dla_fwd(B, T, H, dk, dv, dt, q, k, v, g, S0, L, o, ST, ws, n, None)
    assert fwd(dt=3) == E_DTYPE and fwd(dk=32) == fwd(dv=96) == E_UNSUP
    assert fwd(B=-1) == fwd(T=1 << 31) == fwd(B=1 << 21) == fwd(B=(1 << 19) + 1, T=64) == fwd(B=1 << 14, H=1 << 5) == fwd(B=1 << 40, H=1 << 40) == E_SHAPE
    assert fwd(q=None) == fwd(k=None) == fwd(v=None) == fwd(g=None) == fwd(o=None) == E_NULL
    assert fwd(ws=None) == fwd(n=need - 1) == E_WS
    assert fwd(o=at(0)) == fwd(ST=at(4)) == fwd(S0=at(5)) == fwd(ws=at(1)) == fwd(o=at(3)) == E_ALIAS
    assert fwd(q=at(0) + 8) == fwd(g=at(3) + 2) == fwd(L=at(7) + 1) == fwd(ST=at(5) + 4) == E_ALIGN
    assert fwd(B=0, q=None) == OK

    def bwd(T=4096, dt=1, q=at(0), g=at(3), S0=None, dO=at(4), dS=None, dq=at(5), dk=at(6), dv=at(7), dS0=None, ws=at(9), n=back):
        return lib.gdr2_dla_bwd(1, T, 1, 64, 128, dt, q, at(1), at(2), g, S0, None, dO, dS, dq, dk, dv, dS0, ws, n, None)
    assert bwd(dt=2) == E_DTYPE and bwd(T=-1) == E_SHAPE
    assert bwd(q=None) == bwd(g=None) == bwd(dO=None) == bwd(dq=None) == bwd(dk=None) == bwd(dv=None) == E_NULL
    assert bwd(ws=None) == bwd(n=back - 1) == E_WS
    assert bwd(dq=at(4)) == bwd(dk=at(5)) == bwd(S0=at(8), dS0=at(8)) == bwd(dS=at(8), dS0=at(8)) == bwd(ws=at(2)) == E_ALIAS
    assert bwd(dS=at(8) + 8) == E_ALIGN

    def step(N=2, H=2, dk=64, dv=64, dt=1, q=at(0), k=at(1), v=at(2), g=at(3), Si=at(4), So=at(4), o=at(5)):
        return lib.gdr2_dla_step(N, H, dk, dv, dt, q, k, v, g, Si, So, o, None)
    assert step(dt=4) == E_DTYPE and step(dk=80) == E_UNSUP and step(N=-1) == step(N=1 << 24, H=1) == step(N=1 << 40, H=1 << 40) == E_SHAPE
    assert step(q=None) == step(g=None) == step(So=None) == step(o=None) == E_NULL
    assert step(So=at(4) + 16) == step(o=at(4)) == step(o=at(0)) == E_ALIAS
    assert step(k=at(1) + 4) == step(g=at(3) + 1) == E_ALIGN
    assert step(N=0) == OK


def test_paged_abi():
    lib = load_library()

    def fill(B=2, T=8, Hkv=1, d=64, dt=1, page=16, pages=9, width=4, k=at(0), v=at(1), s=None, L=None, t=at(2), kp=at(3), vp=at(4)):
        return lib.gdr2_paged_cache_fill(B, T, Hkv, d, dt, page, pages, width, k, v, s, L, t, kp, vp, None)
    assert fill(dt=3) == E_DTYPE and fill(d=32) == E_UNSUP
    assert fill(page=0) == fill(page=24) == fill(page=-16) == E_VALUE
    assert fill(T=-1) == fill(B=-1) == fill(pages=-1) == fill(width=-1) == fill(pages=1 << 27) == fill(width=1 << 27) == E_SHAPE
    assert fill(B=1 << 20, T=1 << 20) == fill(B=1 << 31) == fill(Hkv=40000) == E_SHAPE
    assert fill(k=None) == fill(t=None) == fill(vp=None) == E_NULL
    assert fill(kp=at(0)) == fill(vp=at(3)) == fill(kp=at(2)) == fill(s=at(4)) == E_ALIAS
    assert fill(vp=at(4) + 8) == fill(s=at(5) + 2) == fill(L=at(5) + 1) == fill(t=at(2) + 3) == E_ALIGN
    assert fill(T=0, k=None) == fill(pages=0, kp=None, vp=None) == fill(width=0, t=None) == OK
    q = lib.gdr2_paged_decode_workspace_bytes
    need = q(1, 4, 1, 64, 16, 256)
    assert need > 0 and q(4096, 4, 1, 64, 16, 256) == 0
    assert q(1, 4, 3, 64, 16, 256) == q(1, 4, 1, 96, 16, 256) == q(1, 4, 1, 64, 15, 256) == q(-1, 4, 1, 64, 16, 256) == 0
    assert q(1 << 40, 4, 1, 64, 16, 256) == q(1, 4, 1, 64, 16, 1 << 27) == 0

    def dec(N=1, H=4, Hkv=1, d=64, dt=1, page=16, pages=300, width=256, sc=0.1, q=at(0), k=at(1), v=at(2), t=at(3), pos=at(4), kp=at(5),
            vp=at(6), o=at(7), ws=at(8), n=need):
        return lib.gdr2_paged_decode_step(N, H, Hkv, d, dt, page, pages, width, sc, q, k, v, t, pos, kp, vp, o, ws, n, None)
    assert dec(dt=2) == E_DTYPE and dec(d=256) == E_UNSUP and dec(H=3, Hkv=2) == dec(N=-1) == dec(N=1 << 40) == dec(H=0) == E_SHAPE
    assert dec(page=48) == dec(sc=0.0) == dec(sc=float("nan")) == dec(sc=float("inf")) == E_VALUE
    assert dec(q=None) == dec(k=None) == dec(t=None) == dec(pos=None) == dec(kp=None) == dec(o=None) == E_NULL
    assert dec(ws=None) == dec(n=need - 1) == E_WS
    assert dec(vp=at(5)) == dec(o=at(0)) == dec(k=at(5)) == dec(ws=at(7)) == dec(t=at(6)) == E_ALIAS
    assert dec(pos=at(4) + 1) == dec(t=at(3) + 2) == dec(o=at(7) + 8) == E_ALIGN
    assert dec(N=0, q=None) == OK


# ------------------------------------------------------------------ binding
def test_rms_norm_binding():
    x, w = torch.zeros(3, 4, 64, dtype=BF), torch.ones(64)
    for f in (g2.gdr2_rms_norm_fwd, g2.gdr2_rms_norm_q8_fwd):
        with pytest.raises(TypeError, match="weight has dtype"):
            f(x, w.to(BF))
        with pytest.raises(TypeError, match="unsupported dtype"):
            f(x.half(), w)
        with pytest.raises(ValueError, match="x must be contiguous"):
            f(x.transpose(0, 1), w)
        with pytest.raises(ValueError, match="residual has shape"):
            f(x, w, x[:2])
        with pytest.raises(TypeError, match="residual has dtype"):
            f(x, w, x.float())
        with pytest.raises(ValueError, match="h_out needs a residual"):
            f(x, w, h_out=x.clone())
        with pytest.raises(ValueError, match="GPU tensors"):
            f(x, w, x.clone())
    for bad, match in ((2.5, "whole number"), (1 << 64, "64 bits")):
        with pytest.raises(ValueError, match=match):
            g2.gdr2_rms_norm_q8_fwd(x, w, group=bad)
    st = torch.zeros(3, 4)
    with pytest.raises(ValueError, match="rstd has shape"):
        g2.gdr2_rms_norm_bwd(x, w, torch.zeros(3), x.clone())
    with pytest.raises(TypeError, match="dh has dtype"):
        g2.gdr2_rms_norm_bwd(x, w, st, x.clone(), x.float())
    with pytest.raises(TypeError, match="workspace must be a 1-D uint8"):
        g2.gdr2_rms_norm_bwd(x, w, st, x.clone(), workspace=st)


def test_dla_binding():
    q, v, g = torch.zeros(2, 5, 3, 64, dtype=BF), torch.zeros(2, 5, 3, 128, dtype=BF), torch.zeros(3)
    S = torch.zeros(2, 3, 64, 128)
    with pytest.raises(ValueError, match="log_decay has shape"):
        g2.gdr2_dla_fwd(q, q, v, torch.zeros(2, 5, 3))
    with pytest.raises(TypeError, match="log_decay has dtype"):
        g2.gdr2_dla_fwd(q, q, v, g.double())
    with pytest.raises(ValueError, match="k has shape"):
        g2.gdr2_dla_fwd(q, v, v, g)
    with pytest.raises(ValueError, match="v has shape"):
        g2.gdr2_dla_fwd(q, q, v[:, :4].contiguous(), g)
    with pytest.raises(ValueError, match="S0 has shape"):
        g2.gdr2_dla_fwd(q, q, v, g, S0=S.transpose(2, 3).contiguous())
    with pytest.raises(TypeError, match="S0 has dtype"):
        g2.gdr2_dla_fwd(q, q, v, g, S0=S.to(BF))
    with pytest.raises(TypeError, match="lengths has dtype"):
        g2.gdr2_dla_fwd(q, q, v, g, lengths=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="GPU tensors"):
        g2.gdr2_dla_fwd(q, q, v, g, S0=S)
    with pytest.raises(ValueError, match="dO has shape"):
        g2.gdr2_dla_bwd(q, q, v, g, q)
    with pytest.raises(ValueError, match="dS_T has shape"):
        g2.gdr2_dla_bwd(q, q, v, g, v.clone(), dS_T=S[:1])
    with pytest.raises(TypeError, match="unsupported dtype"):
        g2.dla_fwd_workspace_bytes(1, 1, 1, 64, 64, torch.float16)
    with pytest.raises(ValueError, match="3-D"):
        g2.gdr2_dla_step(q, q, v, g)
    t = lambda x: x[:, 0].contiguous()  # noqa: E731
    with pytest.raises(ValueError, match="S_out has shape"):
        g2.gdr2_dla_step(t(q), t(q), t(v), g, S, S[:1])


def test_paged_binding():
    k, q = torch.zeros(2, 5, 2, 64, dtype=BF), torch.zeros(2, 4, 64, dtype=BF)
    kp, t = torch.zeros(7, 16, 2, 64, dtype=BF), torch.zeros(2, 3, dtype=I32)
    one, pos = k[:, 0].contiguous(), torch.zeros(2, dtype=I32)
    for call in (lambda **a: g2.gdr2_paged_cache_fill(*[{**dict(k=k, v=k.clone(), kp=kp, vp=kp.clone(), t=t), **a}[n] for n in ("k", "v", "kp", "vp", "t")]),
                 lambda **a: g2.gdr2_paged_decode_step(*[{**dict(q=q, k=one, v=one.clone(), kp=kp, vp=kp.clone(), t=t, pos=pos), **a}[n]
                                                         for n in ("q", "k", "v", "kp", "vp", "t", "pos")])):
        with pytest.raises(ValueError, match="v_pages has shape"):
            call(vp=kp[:6])
        with pytest.raises(ValueError, match="k_pages has shape"):
            call(kp=torch.zeros(7, 16, 1, 64, dtype=BF))
        with pytest.raises(TypeError, match="k_pages has dtype"):
            call(kp=kp.float())
        with pytest.raises(TypeError, match="page_table has dtype"):
            call(t=t.long())
        with pytest.raises(ValueError, match="page_table has shape"):
            call(t=t[:1])
        with pytest.raises(ValueError, match="page_table must be contiguous"):
            call(t=torch.zeros(3, 2, dtype=I32).t())
        with pytest.raises(ValueError, match="GPU tensors"):
            call()
    with pytest.raises(ValueError, match="start has shape"):
        g2.gdr2_paged_cache_fill(k, k.clone(), kp, kp.clone(), t, start=torch.zeros(3, dtype=I32))
    with pytest.raises(TypeError, match="pos has dtype"):
        g2.gdr2_paged_decode_step(q, one, one.clone(), kp, kp.clone(), t, pos.float())


def test_every_new_entry_point_is_bound():
    lib = load_library()
    for n in ("gdr2_rms_norm_fwd", "gdr2_rms_norm_q8_fwd", "gdr2_rms_norm_bwd", "gdr2_dla_fwd", "gdr2_dla_bwd", "gdr2_dla_step",
              "gdr2_paged_cache_fill", "gdr2_paged_decode_step"):
        assert n in g2.__all__ and getattr(lib, n).argtypes and getattr(lib, n).restype is ctypes.c_int
