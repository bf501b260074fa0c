"""fp64 definitions of the residual stream's RMS norm, linear attention with a decay per head, and attention of
one token over a paged cache, in numpy.  Test infrastructure only.

Beside results stand the sums of the absolute values that the tests derive bounds from.
"""
import numpy as np

CHUNK = 64


# ------------------------------------------------------------------ RMS norm of a stream h
def rms_forward(h, w, eps):
    rstd = 1.0 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    return h * rstd * w, rstd[..., 0]


def rms_backward(h, w, eps, dy, dh):
    rstd = rms_forward(h, w, eps)[1][..., None]
    n, a = h * rstd, dy * w
    dx = rstd * (a - n * (a * n).mean(-1, keepdims=True)) + (0.0 if dh is None else dh)
    return dict(dx=dx, dweight=(dy * n).reshape(-1, h.shape[-1]).sum(0))


# ------------------------------------------------------------------ linear attention with a decay per head
def dla_forward(q, k, v, g, S0=None, lengths=None):
    """Token by token: o [B, T, H, dv] and the state at each sequence's length."""
    B, T, H, dk = q.shape
    a = np.exp(g)[:, None, None]
    o = np.zeros(v.shape)
    S = np.zeros((B, H, dk, v.shape[-1])) if S0 is None else S0.copy()
    for b in range(B):
        for t in range(_length(lengths, b, T)):
            S[b] = a * S[b] + k[b, t][:, :, None] * v[b, t][:, None, :]
            o[b, t] = np.einsum("hkv,hk->hv", S[b], q[b, t])
    return o, S


def dla_backward(q, k, v, g, dO, S0=None, dS_T=None, lengths=None):
    """Reverse mode of dla_forward, token by token."""
    B, T, H, dk = q.shape
    a = np.exp(g)[:, None, None]
    r = dict(dq=np.zeros(q.shape), dk=np.zeros(q.shape), dv=np.zeros(v.shape))
    R = np.zeros((B, H, dk, v.shape[-1])) if dS_T is None else dS_T.copy()
    for b in range(B):
        L = _length(lengths, b, T)
        S = np.zeros(R[b].shape) if S0 is None else S0[b].copy()
        for t in range(L):
            S = a * S + k[b, t][:, :, None] * v[b, t][:, None, :]
            r["dq"][b, t] = np.einsum("hkv,hv->hk", S, dO[b, t])
        for t in range(L - 1, -1, -1):
            R[b] += q[b, t][:, :, None] * dO[b, t][:, None, :]
            r["dk"][b, t] = np.einsum("hkv,hv->hk", R[b], v[b, t])
            r["dv"][b, t] = np.einsum("hkv,hk->hv", R[b], k[b, t])
            R[b] = a * R[b]
    return dict(r, dS0=R)


def _length(lengths, b, T):
    return T if lengths is None else min(max(int(lengths[b]), 0), T)


def _powers(g, n):
    """exp(n g) with a^0 = 1 for g = -inf too."""
    with np.errstate(invalid="ignore"):
        return np.where(n == 0, 1.0, np.exp(n * g))


def dla_sizes(x, y, z, g, init=None, lengths=None, reverse=False):
    """What bounds the error of out_t = sum over s <= t of a^(t - s) (x_t . y_s) z_s + init's part (time turned round
    with `reverse`, init then undecayed at the first token), per element of out:
      score  sum of a^(t - s) |x_t . y_s| |z_s| over the tokens of t's chunk of 64
      read   sum_k |x_k| |S_k| of the state S entering the chunk, decayed to t
      all    the same double sum with |x| . |y|, and |x| |init|
    and per element of the final state: state = sum of a^(L - 1 - s) |y| |z| and a^L |init|.  [B, T, H, .] and [B, H, ., .]."""
    B, T, H, K = x.shape
    V = z.shape[-1]
    r = {n: np.zeros((B, T, H, V)) for n in ("score", "read", "all")}
    r["state"] = np.zeros((B, H, K, V))
    for b in range(B):
        L = _length(lengths, b, T)
        order = np.arange(L)[::-1] if reverse else np.arange(L)
        early = 1 if reverse else 0
        for h in range(H):
            X, Y, Z = x[b, order, h], y[b, order, h], z[b, order, h]
            I = np.zeros((K, V)) if init is None else init[b, h]
            lag = np.arange(L)[:, None] - np.arange(L)[None, :]
            with np.errstate(over="ignore"):
                W = np.where(lag >= 0, _powers(g[h], np.maximum(lag, 0)), 0.0)
            same = np.arange(L)[:, None] // CHUNK == np.arange(L)[None, :] // CHUNK
            score = (np.abs(X @ Y.T) * W * same) @ np.abs(Z)
            full = (np.abs(X) @ np.abs(Y).T * W) @ np.abs(Z)
            full += _powers(g[h], np.arange(L) + 1 - early)[:, None] * (np.abs(X) @ np.abs(I))
            read = np.zeros((L, V))
            for t0 in range(0, L, CHUNK):
                t = np.arange(t0, min(L, t0 + CHUNK))
                s = np.arange(t0)
                # the state before token t0, decayed to it
                S = (Y[s] * _powers(g[h], t0 - s)[:, None]).T @ Z[s] + _powers(g[h], np.array(t0 + 1 - early)) * I
                read[t] = _powers(g[h], t - t0)[:, None] * (np.abs(X[t]) @ np.abs(S))
            for n, val in (("score", score), ("read", read), ("all", full)):
                r[n][b, order, h] = val
            left = _powers(g[h], L - 1 - np.arange(L)) if L else np.zeros(0)
            r["state"][b, h] = (np.abs(Y) * left[:, None]).T @ np.abs(Z) + _powers(g[h], np.array(max(L - early, 0))) * np.abs(I)
    return r


# ------------------------------------------------------------------ paged cache
def paged_rows(table, page, pages, positions):
    """The row (page * size + offset) of each position, -1 where the table names none."""
    out = []
    for p in positions:
        e = int(table[p // page]) if 0 <= p and p // page < len(table) else -1
        out.append(e * page + p % page if 0 <= e < pages else -1)
    return np.array(out, dtype=np.int64)


def paged_fill(k, v, kp, vp, table, start=None, lengths=None):
    """The pages [pages, page, Hkv, d] after the fill."""
    pages, page = kp.shape[:2]
    kf, vf = kp.reshape(-1, *kp.shape[2:]).copy(), vp.reshape(-1, *vp.shape[2:]).copy()
    for b in range(k.shape[0]):
        L = _length(lengths, b, k.shape[1])
        rows = paged_rows(table[b], page, pages, [(0 if start is None else int(start[b])) + t for t in range(L)])
        for t, r in enumerate(rows):
            if r >= 0:
                kf[r], vf[r] = k[b, t], v[b, t]
    return kf.reshape(kp.shape), vf.reshape(vp.shape)


def paged_decode(q, k, v, kp, vp, table, pos, scale):
    """o, o_abs (sum of p |v|), smax (the largest sum of |q_c k_c| scale) and the pages afterwards."""
    N, H, d = q.shape
    Hkv = k.shape[1]
    pages, page = kp.shape[:2]
    kf, vf = kp.reshape(-1, Hkv, d).copy(), vp.reshape(-1, Hkv, d).copy()
    r = dict(o=np.zeros(q.shape), o_abs=np.zeros(q.shape), smax=0.0)
    for n in range(N):
        p = int(pos[n])
        if p < 0:
            continue
        last = min(p, len(table[n]) * page)
        rows = paged_rows(table[n], page, pages, range(last))
        rows = rows[rows >= 0]
        K, V = np.concatenate([kf[rows], k[n:n + 1]]), np.concatenate([vf[rows], v[n:n + 1]])
        for h in range(H):
            Kh, Vh = K[:, h // (H // Hkv)], V[:, h // (H // Hkv)]
            s = Kh @ q[n, h] * scale
            r["smax"] = max(r["smax"], float((np.abs(Kh) @ np.abs(q[n, h])).max()) * scale)
            w = np.exp(s - s.max())
            w /= w.sum()
            r["o"][n, h], r["o_abs"][n, h] = w @ Vh, w @ np.abs(Vh)
    for n in range(N):
        row = paged_rows(table[n], page, pages, [int(pos[n])])[0] if pos[n] >= 0 else -1
        if row >= 0:
            kf[row], vf[row] = k[n], v[n]
    return dict(r, k_pages=kf.reshape(kp.shape), v_pages=vf.reshape(vp.shape))
