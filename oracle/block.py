"""fp64 definitions of the operators around the mixer (layer norm, gated linear recurrence,
sliding-window attention and its bounded cache), in numpy.  Test infrastructure only.

Beside each result stands the sum of the absolute values of its terms, from which the tests derive
how far a correctly rounding kernel can be off.
"""
import numpy as np


# ------------------------------------------------------------------ layer norm
def layer_norm_forward(x, w, b, eps):
    mu = x.mean(-1, keepdims=True)
    rstd = 1.0 / np.sqrt(((x - mu) ** 2).mean(-1, keepdims=True) + eps)
    return (x - mu) * rstd * w + (0.0 if b is None else b), mu[..., 0], rstd[..., 0]


def layer_norm_backward(x, w, eps, dy):
    _, mu, rstd = layer_norm_forward(x, w, None, eps)
    n, a = (x - mu[..., None]) * rstd[..., None], dy * w
    dx = rstd[..., None] * (a - a.mean(-1, keepdims=True) - n * (a * n).mean(-1, keepdims=True))
    D = x.shape[-1]
    return dict(dx=dx, dweight=(dy * n).reshape(-1, D).sum(0), dbias=dy.reshape(-1, D).sum(0))


# ------------------------------------------------------------------ gated linear recurrence
def glr_forward(x, la, h0):
    """h [B, T, D] and, per element, err: the sum over the terms of h_t of |term| (64 + sum of
    (1 + |log a|) over the decays it went through): 2^-23 err bounds the rounding of an fp32 scan
    whose every term passes at most 64 further roundings of half a step or better."""
    B, T, D = x.shape
    h = np.zeros((B, D)) if h0 is None else h0.copy()
    habs, cnt = np.abs(h), np.zeros((B, D))
    out, err = np.empty_like(x), np.empty_like(x)
    for t in range(T):
        a = np.exp(la[:, t])
        cnt = a * (cnt + (1.0 + np.where(np.isinf(la[:, t]), 0.0, np.abs(la[:, t]))) * habs)
        habs = a * habs + np.abs(x[:, t])
        h = a * h + x[:, t]
        out[:, t], err[:, t] = h, cnt + 64.0 * habs
    return out, h, err


def glr_backward(x, la, h0, dh, dhT):
    B, T, D = x.shape
    h, _, herr = glr_forward(x, la, h0)
    zero = np.zeros((B, 1, D))
    prev = np.concatenate([zero if h0 is None else h0[:, None], h[:, :-1]], 1)
    perr = np.concatenate([64.0 * np.abs(prev[:, :1]), herr[:, :-1]], 1)
    R = np.zeros((B, D)) if dhT is None else dhT.copy()
    rabs, cnt = np.abs(R), np.zeros((B, D))
    g = {n: np.empty_like(x) for n in ("dx", "dx_err", "dlog_a", "dlog_a_err")}
    for t in range(T - 1, -1, -1):
        a, la_t = np.exp(la[:, t]), np.where(np.isinf(la[:, t]), 0.0, np.abs(la[:, t]))
        G, gabs = dh[:, t] + R, np.abs(dh[:, t]) + rabs
        g["dx"][:, t], g["dx_err"][:, t] = G, cnt + 64.0 * gabs
        R, rabs, cnt = a * G, a * gabs, a * (cnt + (1.0 + la_t) * gabs)
        g["dlog_a"][:, t] = R * prev[:, t]
        rerr = cnt + 64.0 * rabs
        g["dlog_a_err"][:, t] = rerr * np.abs(prev[:, t]) + np.abs(R) * perr[:, t]
    return dict(g, dh0=R, dh0_err=cnt + 64.0 * rabs)


# ------------------------------------------------------------------ sliding-window attention
def swa_visible(T, L, window, sinks):
    i, j = np.arange(T)[:, None], np.arange(T)[None, :]
    return (j <= i) & (i < L) & ((i - j < window) | (j < sinks))


def swa(q, k, v, window, sinks, scale, lengths=None, dO=None):
    """o, lse and (with dO) dq, dk, dv of [B, T, H, d] inputs, rows at and behind a length ignored.
    *_abs: sums of the terms' absolute values: o_abs = sum_j p |v|; with D_i = sum_c |dO| (o_abs +
    |o|): dq_abs = scale sum_j |ds| |k|, dq_delta = scale sum_j p D_i |k|, dk likewise over the
    queries with |q|, dv_abs = sum_i p |dO|; smax: the largest sum_c |q_c k_c| scale."""
    B, T, H, d = q.shape
    Hkv = k.shape[2]
    r = {n: np.zeros_like(q) for n in ("o", "o_abs")}
    r["lse"] = np.full((B, H, T), -np.inf)
    r["smax"] = 0.0
    if dO is not None:
        for n in ("dq", "dq_abs", "dq_delta"):
            r[n] = np.zeros_like(q)
        for n in ("dk", "dk_abs", "dk_delta", "dv", "dv_abs"):
            r[n] = np.zeros_like(k)
    for b in range(B):
        L = T if lengths is None else min(max(int(lengths[b]), 0), T)
        if L == 0:
            continue
        vis = swa_visible(L, L, window, sinks)
        for h in range(H):
            g = h // (H // Hkv)
            Q, K, V = q[b, :L, h], k[b, :L, g], v[b, :L, g]
            S = np.where(vis, Q @ K.T * scale, -np.inf)
            r["smax"] = max(r["smax"], float((np.where(vis, np.abs(Q) @ np.abs(K).T, 0.0)).max()) * scale)
            m = S.max(1, keepdims=True)
            P = np.exp(S - m)
            z = P.sum(1, keepdims=True)
            P /= z
            r["lse"][b, h, :L] = (m + np.log(z))[:, 0]
            O, Oa = P @ V, P @ np.abs(V)
            r["o"][b, :L, h], r["o_abs"][b, :L, h] = O, Oa
            if dO is None:
                continue
            G = dO[b, :L, h]
            dS = P * (G @ V.T - (G * O).sum(1, keepdims=True))
            De = (np.abs(G) * (Oa + np.abs(O))).sum(1, keepdims=True)
            r["dq"][b, :L, h] = scale * dS @ K
            r["dq_abs"][b, :L, h] = scale * np.abs(dS) @ np.abs(K)
            r["dq_delta"][b, :L, h] = scale * (P * De) @ np.abs(K)
            r["dk"][b, :L, g] += scale * dS.T @ Q
            r["dk_abs"][b, :L, g] += scale * np.abs(dS).T @ np.abs(Q)
            r["dk_delta"][b, :L, g] += scale * (P * De).T @ np.abs(Q)
            r["dv"][b, :L, g] += P.T @ G
            r["dv_abs"][b, :L, g] += P.T @ np.abs(G)
    return r


def swa_cache(k, v, kc, vc, window, sinks, lengths=None):
    """The caches after a prefill of k, v: the last position of every slot."""
    kc, vc = kc.copy(), vc.copy()
    for b in range(k.shape[0]):
        L = k.shape[1] if lengths is None else min(max(int(lengths[b]), 0), k.shape[1])
        for p in range(L):
            slot = p if p < sinks else sinks + (p - sinks) % window
            kc[b, slot], vc[b, slot] = k[b, p], v[b, p]
    return kc, vc
