"""Refusals of the operators around the mixer on a host without a GPU: the C ABI rejects bad arguments
before any launch, the binding rejects wrong tensors before any library call."""
import ctypes

import pytest
import torch

import gated_delta_rule_gdr_amd as g2
from gated_delta_rule_gdr_amd import load_library

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
OK, E_NULL, E_SHAPE, E_DTYPE, E_UNSUP, E_ALIGN, E_ALIAS, E_WS, E_VALUE = 0, 1, 2, 3, 4, 5, 6, 7, 9


def at(i):
    """Distinct 16-byte aligned addresses that are never dereferenced."""
    return 0x100000 * (i + 1)


# ------------------------------------------------------------------ C ABI
def test_layer_norm_abi():
    lib = load_library()

    def fwd(rows=4, D=64, dt=1, x=at(0), w=at(1), b=None, eps=1e-5, y=at(2), m=at(3), r=at(4)):
        return lib.gdr2_layer_norm_fwd(rows, D, dt, x, w, b, eps, y, m, r, None)
    assert fwd(dt=2) == E_DTYPE
    assert fwd(rows=-1) == fwd(rows=1 << 40) == E_SHAPE
    assert fwd(D=0) == fwd(D=60) == fwd(D=16392) == E_UNSUP
    assert fwd(eps=0.0) == fwd(eps=float("nan")) == fwd(eps=float("inf")) == E_VALUE
    assert fwd(x=None) == fwd(w=None) == fwd(y=None) == E_NULL
    assert fwd(x=at(0) + 8) == fwd(b=at(5) + 4) == E_ALIGN
    assert fwd(y=at(0)) == fwd(m=at(1)) == fwd(r=at(3)) == E_ALIAS
    assert fwd(rows=0, x=None) == OK
    need = lib.gdr2_layer_norm_bwd_workspace_bytes(4, 64)
    assert need > 0 and lib.gdr2_layer_norm_bwd_workspace_bytes(4, 63) == 0

    def bwd(rows=4, D=64, dt=1, dy=at(4), dx=at(5), dw=at(6), db=None, ws=at(8), n=need):
        return lib.gdr2_layer_norm_bwd(rows, D, dt, at(0), at(1), at(2), at(3), dy, dx, dw, db, ws, n, None)
    assert bwd(dt=9) == E_DTYPE and bwd(D=12) == E_UNSUP and bwd(rows=-2) == E_SHAPE
    assert bwd(dw=None) == bwd(dy=None) == bwd(dx=None) == E_NULL
    assert bwd(ws=None) == bwd(n=need - 1) == E_WS
    assert bwd(dx=at(4)) == bwd(db=at(6)) == bwd(ws=at(0)) == E_ALIAS
    assert bwd(dx=at(5) + 2) == E_ALIGN


def test_glr_abi():
    lib = load_library()
    fn, bn = lib.gdr2_glr_fwd_workspace_bytes(1, 300, 64), lib.gdr2_glr_bwd_workspace_bytes(1, 300, 64)
    assert fn > bn > 0 and lib.gdr2_glr_bwd_workspace_bytes(1, 100, 64) == 0
    for bad in ((1, 1 << 40, 64), (1 << 31, 1, 64), (1, 1 << 37, 1 << 20), (-1, 1, 64), (1, 1, 60)):
        assert lib.gdr2_glr_fwd_workspace_bytes(*bad) == lib.gdr2_glr_bwd_workspace_bytes(*bad) == 0

    def fwd(B=1, T=300, D=64, dt=1, x=at(0), la=at(1), h0=None, h=at(3), hT=None, ws=at(5), n=fn):
        return lib.gdr2_glr_fwd(B, T, D, dt, x, la, h0, h, hT, ws, n, None)
    assert fwd(dt=5) == E_DTYPE and fwd(D=36) == E_UNSUP and fwd(T=-1) == fwd(T=1 << 50) == E_SHAPE
    assert fwd(x=None) == fwd(la=None) == fwd(h=None) == E_NULL
    assert fwd(ws=None) == fwd(n=fn - 1) == E_WS
    assert fwd(h=at(0)) == fwd(h0=at(2), hT=at(2)) == fwd(ws=at(1)) == E_ALIAS
    assert fwd(h0=at(2) + 4) == E_ALIGN
    assert fwd(B=0, x=None) == OK

    def bwd(T=300, x=at(0), fws=at(2), f=fn, dh=at(3), dx=at(4), dla=at(5), dh0=None, ws=at(6), n=bn):
        return lib.gdr2_glr_bwd(1, T, 64, 1, x, at(1), fws, f, dh, None, dx, dla, dh0, ws, n, None)
    assert bwd(x=None) == bwd(dh=None) == bwd(dx=None) == bwd(dla=None) == E_NULL
    assert bwd(fws=None) == bwd(f=fn - 1) == bwd(ws=None) == bwd(n=bn - 1) == E_WS
    assert bwd(dx=at(3)) == bwd(dla=at(2)) == bwd(dh0=at(4)) == E_ALIAS
    assert bwd(dla=at(5) + 8) == E_ALIGN

    def step(N=2, D=64, dt=1, x=at(0), la=at(1), hi=at(2), ho=at(2), h=at(4)):
        return lib.gdr2_glr_step(N, D, dt, x, la, hi, ho, h, None)
    assert step(dt=4) == E_DTYPE and step(N=-1) == step(N=1 << 40) == E_SHAPE and step(D=4) == E_UNSUP
    assert step(ho=None) == step(h=None) == E_NULL
    assert step(ho=at(2) + 16) == step(h=at(2)) == step(h=at(0)) == E_ALIAS
    assert step(N=0) == OK


def test_swa_abi():
    lib = load_library()

    def fwd(B=1, T=8, H=2, Hkv=1, d=64, dt=1, w=4, s=0, sc=0.1, q=at(0), k=at(1), v=at(2), L=None, o=at(4), lse=at(5)):
        return lib.gdr2_swa_fwd(B, T, H, Hkv, d, dt, w, s, sc, q, k, v, L, o, lse, None)
    assert fwd(dt=2) == E_DTYPE and fwd(d=96) == E_UNSUP
    assert fwd(B=-1) == fwd(T=1 << 31) == fwd(H=3, Hkv=2) == fwd(Hkv=0) == fwd(H=1 << 16) == E_SHAPE
    assert fwd(B=1 << 30, T=1 << 20) == E_SHAPE
    assert fwd(w=0) == fwd(s=-1) == fwd(s=65) == fwd(sc=0.0) == fwd(sc=float("nan")) == fwd(sc=float("inf")) == E_VALUE
    assert fwd(q=None) == fwd(k=None) == fwd(o=None) == fwd(lse=None) == E_NULL
    assert fwd(o=at(0)) == fwd(lse=at(2)) == fwd(lse=at(4)) == E_ALIAS
    assert fwd(v=at(2) + 8) == fwd(L=at(6) + 2) == E_ALIGN
    assert fwd(T=0, q=None) == OK
    need = lib.gdr2_swa_bwd_workspace_bytes(1, 8, 2, 1, 64, 4, 0)
    assert need > 0 and lib.gdr2_swa_bwd_workspace_bytes(1, 8, 2, 1, 64, 0, 0) == 0
    # pieces for the sinks' gradients once queries lie behind the window
    assert lib.gdr2_swa_bwd_workspace_bytes(8, 8192, 16, 16, 64, 512, 4) > lib.gdr2_swa_bwd_workspace_bytes(8, 8192, 16, 16, 64, 512, 0)

    def bwd(H=2, w=4, s=0, sc=0.1, o=at(3), lse=at(4), dO=at(5), dq=at(6), dk=at(7), dv=at(8), ws=at(9), n=need):
        return lib.gdr2_swa_bwd(1, 8, H, 1, 64, 1, w, s, sc, at(0), at(1), at(2), None, o, lse, dO, dq, dk, dv, ws, n, None)
    assert bwd(w=0) == bwd(s=65) == bwd(sc=-1.0) == E_VALUE
    assert bwd(o=None) == bwd(lse=None) == bwd(dO=None) == bwd(dq=None) == bwd(dk=None) == bwd(dv=None) == E_NULL
    assert bwd(ws=None) == bwd(n=need - 1) == E_WS
    assert bwd(dq=at(5)) == bwd(dk=at(7), dv=at(7)) == bwd(ws=at(4)) == E_ALIAS
    assert bwd(dq=at(6) + 4) == E_ALIGN


def test_swa_cache_abi():
    lib = load_library()

    def fill(B=1, T=8, Hkv=1, d=64, dt=1, w=4, s=0, k=at(0), v=at(1), L=None, kc=at(2), vc=at(3)):
        return lib.gdr2_swa_cache_fill(B, T, Hkv, d, dt, w, s, k, v, L, kc, vc, None)
    assert fill(dt=3) == E_DTYPE and fill(d=32) == E_UNSUP and fill(T=-1) == fill(w=1 << 33) == E_SHAPE
    assert fill(w=0) == fill(s=65) == E_VALUE
    assert fill(k=None) == fill(vc=None) == E_NULL
    assert fill(kc=at(0)) == fill(kc=at(2), vc=at(2)) == E_ALIAS and fill(vc=at(3) + 8) == E_ALIGN
    assert fill(T=0) == OK
    need = lib.gdr2_swa_decode_workspace_bytes(1, 4, 1, 64, 4096, 4)
    assert need > 0                                             # few jobs: the slots are cut into parts
    assert lib.gdr2_swa_decode_workspace_bytes(512, 4, 1, 64, 4096, 4) == 0

    def dec(N=1, H=4, Hkv=1, d=64, dt=1, w=4096, s=4, sc=0.1, q=at(0), k=at(1), v=at(2), kc=at(3), vc=at(10), pos=at(20),
            o=at(21), ws=at(22), n=need):
        return lib.gdr2_swa_decode_step(N, H, Hkv, d, dt, w, s, sc, q, k, v, kc, vc, pos, o, ws, n, None)
    assert dec(dt=2) == E_DTYPE and dec(d=256) == E_UNSUP and dec(N=-1) == dec(H=3, Hkv=2) == dec(N=1 << 40) == E_SHAPE
    assert dec(w=0) == dec(s=99) == dec(sc=0.0) == E_VALUE
    assert dec(q=None) == dec(kc=None) == dec(pos=None) == dec(o=None) == E_NULL
    assert dec(ws=None) == dec(n=need - 1) == E_WS
    assert dec(vc=at(3)) == dec(o=at(0)) == dec(k=at(3)) == dec(ws=at(21)) == E_ALIAS
    assert dec(pos=at(20) + 1) == dec(o=at(21) + 8) == E_ALIGN
    assert dec(N=0) == OK


# ------------------------------------------------------------------ binding
def test_layer_norm_binding():
    x, w = torch.zeros(3, 4, 64, dtype=BF), torch.ones(64)
    with pytest.raises(TypeError, match="weight has dtype"):
        g2.gdr2_layer_norm_fwd(x, w.to(BF))
    with pytest.raises(ValueError, match="weight has shape"):
        g2.gdr2_layer_norm_fwd(x, torch.ones(32))
    with pytest.raises(ValueError, match="bias has shape"):
        g2.gdr2_layer_norm_fwd(x, w, torch.ones(1))
    with pytest.raises(TypeError, match="unsupported dtype"):
        g2.gdr2_layer_norm_fwd(x.half(), w)
    with pytest.raises(ValueError, match="x must be contiguous"):
        g2.gdr2_layer_norm_fwd(x.transpose(0, 1), w)
    with pytest.raises(TypeError, match="x must be a tensor"):
        g2.gdr2_layer_norm_fwd(None, w)
    with pytest.raises(ValueError, match="GPU tensors"):
        g2.gdr2_layer_norm_fwd(x, w)
    st = torch.zeros(3, 4)
    with pytest.raises(ValueError, match="rstd has shape"):
        g2.gdr2_layer_norm_bwd(x, w, st, torch.zeros(3), x.clone())
    with pytest.raises(TypeError, match="dy has dtype"):
        g2.gdr2_layer_norm_bwd(x, w, st, st.clone(), x.float())
    with pytest.raises(TypeError, match="workspace must be a 1-D uint8"):
        g2.gdr2_layer_norm_bwd(x, w, st, st.clone(), x.clone(), workspace=st)


def test_glr_binding():
    x, la, st = torch.zeros(2, 5, 64, dtype=BF), torch.zeros(2, 5, 64), torch.zeros(2, 64)
    ws = torch.zeros(16, dtype=torch.uint8)
    with pytest.raises(TypeError, match="log_a has dtype"):
        g2.gdr2_glr_fwd(x, la.to(BF))
    with pytest.raises(ValueError, match="3-D"):
        g2.gdr2_glr_fwd(x[0], la[0])
    with pytest.raises(ValueError, match="h0 has shape"):
        g2.gdr2_glr_fwd(x, la, h0=st[:, :32].contiguous())
    with pytest.raises(ValueError, match="GPU tensors"):
        g2.gdr2_glr_fwd(x, la, h0=st)
    with pytest.raises(TypeError, match="dh has dtype"):
        g2.gdr2_glr_bwd(x, la, la, ws)
    with pytest.raises(TypeError, match="fwd_ws must be a 1-D uint8"):
        g2.gdr2_glr_bwd(x, la, x.clone(), None)
    with pytest.raises(ValueError, match="dh_T has shape"):
        g2.gdr2_glr_bwd(x, la, x.clone(), ws, dh_T=torch.zeros(2))
    with pytest.raises(TypeError, match="h_in has dtype"):
        g2.gdr2_glr_step(x[:, 0].contiguous(), la[:, 0].contiguous(), st.to(BF))
    with pytest.raises(ValueError, match="2-D"):
        g2.gdr2_glr_step(x, la)


def test_swa_binding():
    q, k = torch.zeros(2, 5, 4, 64, dtype=BF), torch.zeros(2, 5, 2, 64, dtype=BF)
    v, lse = k.clone(), torch.zeros(2, 4, 5)
    with pytest.raises(ValueError, match="v has shape"):
        g2.gdr2_swa_fwd(q, k, v[:, :, :1].contiguous(), 3)
    with pytest.raises(ValueError, match="k has shape"):
        g2.gdr2_swa_fwd(q, k[:, :4].contiguous(), v, 3)
    with pytest.raises(TypeError, match="k has dtype"):
        g2.gdr2_swa_fwd(q, k.float(), v, 3)
    with pytest.raises(TypeError, match="lengths has dtype"):
        g2.gdr2_swa_fwd(q, k, v, 3, lengths=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="lengths has shape"):
        g2.gdr2_swa_fwd(q, k, v, 3, lengths=torch.zeros(5, dtype=I32))
    with pytest.raises(ValueError, match="GPU tensors"):
        g2.gdr2_swa_fwd(q, k, v, 3)
    with pytest.raises(ValueError, match="lse has shape"):
        g2.gdr2_swa_bwd(q, k, v, q.clone(), lse.transpose(1, 2).contiguous(), q.clone(), 3)
    with pytest.raises(ValueError, match="dO has shape"):
        g2.gdr2_swa_bwd(q, k, v, q.clone(), lse, k.clone(), 3)
    kc = torch.zeros(2, 9, 2, 64, dtype=BF)
    with pytest.raises(ValueError, match="v_cache has shape"):
        g2.gdr2_swa_cache_fill(k, v, kc, kc[:, :8].contiguous())
    with pytest.raises(TypeError, match="k_cache has dtype"):
        g2.gdr2_swa_cache_fill(k, v, kc.float(), kc.clone())
    t = lambda x: x[:, 0].contiguous()  # noqa: E731
    pos = torch.zeros(2, dtype=I32)
    with pytest.raises(TypeError, match="pos has dtype"):
        g2.gdr2_swa_decode_step(t(q), t(k), t(v), kc, kc.clone(), pos.long())
    with pytest.raises(ValueError, match="k_cache has shape"):
        g2.gdr2_swa_decode_step(t(q), t(k), t(v), kc[:1].contiguous(), kc.clone(), pos)
    with pytest.raises(ValueError, match="GPU tensors"):
        g2.gdr2_swa_decode_step(t(q), t(k), t(v), kc, kc.clone(), pos, sinks=2)


def test_every_new_entry_point_is_bound():
    lib = load_library()
    for n in ("gdr2_layer_norm_fwd", "gdr2_layer_norm_bwd", "gdr2_glr_fwd", "gdr2_glr_bwd", "gdr2_glr_step", "gdr2_swa_fwd",
              "gdr2_swa_bwd", "gdr2_swa_cache_fill", "gdr2_swa_decode_step"):
        assert n in g2.__all__ and getattr(lib, n).argtypes and getattr(lib, n).restype is ctypes.c_int
