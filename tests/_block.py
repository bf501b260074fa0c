"""Inputs, bounds and checks shared by the tests of the operators around the mixer.

Bounds are derived, per element, from the sums of the terms' absolute values that oracle/block.py
returns.  u16 is half a step of bf16 relative to the value (2^-8), u32 that of fp32 (2^-24).

Attention.  A score is an fp32 sum of d products and one scaling: its error is at most (d + 4) u32
smax (smax: the largest sum of |q_c k_c| times the scale), the exponent's argument s - m (at most
2 smax + 16 in magnitude, in units of log 2) and the exponential itself (1 ulp) add (4 smax + 32) u32,
the reference of a lane or lse the same once more; so a probability is off by at most a relative
e_p = (2 d + 16) smax u32 + 128 u32, twice that with its denominator (n terms: n u32).
With bf16 products every probability and every ds is rounded once to bf16 (u16), and every output
once (u16):
    o   : (u_p + 2 e_p + 2 n u32) o_abs + u_out |o|
    dv  : (u_p + 2 e_p + 2 n u32) dv_abs + u_out |dv|
    dq  : (u_p + 4 e_p + (2 n + 4 d) u32) (dq_abs + dq_delta) + (u_p + u_out) dq_delta + u_out |dq|
where the term in dq_delta is the rounding of o, which delta is formed from, and u_p = u_out = u16 for
bf16, 0 and u32 for fp32 (dp - delta cancels: its terms' error is bounded through dq_delta, whose
weights |dO| (o_abs + |o|) bound |dp| on average; a factor 4 covers single terms).  dk as dq.
"""
import numpy as np
import torch

U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
U32 = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def randn(gen, shape, dtype="f32"):
    return torch.randn(shape, generator=gen).to(DT[dtype])


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def within(name, got, ref, bound):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, f"{name}: shape {got.shape}, expected {ref.shape}"
    if not got.size:
        return
    same = (got == ref)  # infinities included
    with np.errstate(invalid="ignore"):
        over = np.where(same, 0.0, np.abs(got - ref) - bound)
    over = np.where(np.isnan(over), np.inf, over)
    at = np.unravel_index(int(over.argmax()), over.shape)
    assert over[at] <= 0.0, (f"{name}: at {tuple(int(x) for x in at)} got {got[at]:.9g}, expected {ref[at]:.9g}, bound "
                             f"{np.broadcast_to(bound, ref.shape)[at]:.3g}; {int((over > 0).sum())} elements over")


def swa_bounds(r, dtype, d, n):
    up = U[dtype] if dtype == "bf16" else 0.0
    uo = U[dtype]
    ep = ((2 * d + 16) * r["smax"] + 128.0) * U32
    tiny = 1e-30
    b = {"o": (up + 2 * ep + 2 * n * U32) * r["o_abs"] + uo * np.abs(r["o"]) + tiny,
         "lse": ep + 4 * U32 * np.abs(np.where(np.isinf(r["lse"]), 0.0, r["lse"])) + n * U32}
    if "dq" in r:
        b["dv"] = (up + 2 * ep + 2 * n * U32) * r["dv_abs"] + uo * np.abs(r["dv"]) + tiny
        for g in ("dq", "dk"):
            b[g] = ((up + 4 * ep + (2 * n + 4 * d) * U32) * (r[g + "_abs"] + 4 * (0.0 if up else 1.0) * r[g + "_delta"])
                    + (up + (4 * ep + (2 * n + 4 * d) * U32) + uo) * r[g + "_delta"] + uo * np.abs(r[g]) + tiny)
    return b
