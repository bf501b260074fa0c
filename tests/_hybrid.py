"""Bounds shared by the tests of the RMS norm, linear attention with a decay and the paged cache, derived from
the sums of absolute values that oracle/hybrid.py returns (u16 = 2^-8, u32 = 2^-24: half a step).

Linear attention.  A term a^(t - s) (x . y) z of an output passes, in fp32, a dot product of K terms (K + 4
roundings, of |x| . |y|), its weight (a hardware exponential: 4 roundings, and the rounding of its argument
n g, at most |n g| <= 64 |g| inside a chunk; weights that small are bounded by n|g| e^(-n|g|) <= 1, and by 32 where a
state's power is formed from one argument), a sum over 64 tokens, and one rounding of the state per later
chunk (at most ceil(T / 64), and as many for segments): c32 = (2 K + 128 + 4 ceil(T / 64) + 64) u32, times `all`.
With bf16 the scores of a chunk and the state as it is read are each rounded once (u16: `score`, `read`), the
state's decayed operand keeps 16 bits, cut (2^-15, times `all`; 24 bits, 2^-23 times `state`, for a final state),
and outputs are rounded once.

Normwise: roundings of a half step are at most u / sqrt(3) of the value in the mean square for each of three
roundings whose errors add in squares where terms have either sign: below u16 = sqrt(3) u16 / sqrt(3); 2 u16 leaves room for
few terms.  fp32: c32's roundings add likewise, sqrt(2 K + 192 + 4 ceil(T / 64)) u32 and twice that at most.
"""
import numpy as np

from tests._block import U, U32, f64

U16 = 2.0 ** -8


def dla_c32(K, T):
    return (2 * K + 128 + 4 * -(-T // 64) + 64) * U32


def dla_bounds(r, ref, dtype, K, T):
    c = dla_c32(K, T) + (2.0 ** -15 if dtype == "bf16" else 0.0)
    low = U16 * (1 + 2.0 ** -7) * (r["score"] + r["read"]) if dtype == "bf16" else 0.0
    return low + c * r["all"] + U[dtype] * np.abs(ref) * (1 + 2.0 ** -7) + 1e-30


def dla_state_bounds(r, dtype, K, T):
    return (dla_c32(K, T) + (2.0 ** -23 if dtype == "bf16" else 0.0)) * r["state"] + 1e-30


def norm_close(name, got, ref, dtype, K, T):
    got = f64(got)
    lim = 2 * U16 if dtype == "bf16" else 2 * np.sqrt(2 * K + 192 + 4 * -(-T // 64)) * U32
    n = np.linalg.norm(ref)
    assert np.linalg.norm(got - ref) <= lim * n + 1e-30, f"{name}: normwise {np.linalg.norm(got - ref) / n:.3g} over {lim:.3g}"
