"""The operators around the Gated Delta Rule-2 mixer, as cases to measure.

A hybrid stack alternates the recurrent mixer with sliding-window attention, normalises the input
of every mixer, and may use an elementwise gated recurrence in the recurrent mixer's place.  Each
case is one of:

  swa_train    sliding-window attention with always-visible first tokens (sinks): forward and
               gradients of q, k, v
  swa_prefill  the forward alone, and the bounded cache that decoding continues from
  swa_decode   one token per sequence against the bounded cache (a ring of `window` rows behind
               `sinks` fixed rows), which receives the token's key and value
  glr_train    gated linear recurrence h_t = exp(log_a_t) h_{t-1} + x_t: forward and gradients
  glr_step     one token of it per sequence
  ln_train     layer normalisation over the last axis: forward and gradients
  ln_fwd       its forward alone

Token tensors are [B, T, heads, d] (attention) or [B, T, D]; lengths are int32, one per sequence,
and rows at and behind a sequence's length are padding.
"""
import math

import torch

own = False

DEV = "cuda"
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the attention layer of the hybrid at the 1.3B layer's shape (4 x 4096 tokens, 16 heads
        # of 128, the 2K window), training
        dict(name="swa_train_layer", op="swa_train", B=4, T=4096, H=16, Hkv=16, d=128, window=2048,
             sinks=4, ragged=False, dtype="bf16"),
        # grouped key/value heads of 64, a padded batch of odd lengths, a short window, training
        dict(name="swa_train_gqa_ragged", op="swa_train", B=3, T=1537, H=12, Hkv=3, d=64, window=500,
             sinks=1, ragged=True, dtype="bf16"),
        # the same in fp32 at the size of a numerics test
        dict(name="swa_train_f32", op="swa_train", B=2, T=777, H=6, Hkv=2, d=64, window=256, sinks=8,
             ragged=True, dtype="f32"),
        # prefill of the long-context workload (32K tokens), four heads to a key/value head
        dict(name="swa_prefill_long", op="swa_prefill", B=1, T=32768, H=16, Hkv=4, d=128, window=2048,
             sinks=4, ragged=False, dtype="bf16"),
        # one user's token: latency
        dict(name="swa_decode_single", op="swa_decode", N=1, H=16, Hkv=4, d=128, window=2048, sinks=4,
             ragged=False, dtype="bf16"),
        # the decode workload's 256 sequences of 16 heads, all positions different
        dict(name="swa_decode_batch", op="swa_decode", N=256, H=16, Hkv=4, d=128, window=2048, sinks=4,
             ragged=True, dtype="bf16"),
        # the recurrence over the 1.3B layer's tokens and its 16 x 128 channels, training
        dict(name="glr_train_layer", op="glr_train", B=4, T=4096, D=2048, dtype="bf16"),
        # one long sequence of odd length in fp32: few channels, a long scan
        dict(name="glr_train_long_f32", op="glr_train", B=1, T=32749, D=1024, dtype="f32"),
        # the recurrence's token of the decode workload
        dict(name="glr_step_batch", op="glr_step", N=256, D=2048, dtype="bf16"),
        # the norm before the 1.3B layer's mixer, training
        dict(name="ln_train_layer", op="ln_train", rows=16384, D=2048, bias=True, dtype="bf16"),
        # a row width that is no power of two, an odd number of rows, no bias, fp32
        dict(name="ln_train_odd_f32", op="ln_train", rows=4099, D=1000, bias=False, dtype="f32"),
        # the norm of one decode step: latency
        dict(name="ln_decode", op="ln_fwd", rows=256, D=2048, bias=True, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["swa_train", "swa_train", "swa_prefill", "swa_decode", "swa_decode", "glr_train",
                     "glr_train", "glr_step", "ln_train", "ln_train", "ln_fwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("swa_train", "swa_prefill"):
        Hkv = rng.randint(1, 4)
        c = dict(op=op, B=rng.randint(1, 4), T=_log(rng, 1, 4096), H=Hkv * rng.randint(1, 4), Hkv=Hkv,
                 d=rng.choice([64, 128]), window=_log(rng, 1, 2048), sinks=rng.choice([0, 1, 4, 17, 64]),
                 ragged=rng.random() < 0.5, dtype=dtype)
        if dtype == "f32":
            c["T"] = min(c["T"], 1500)
        return c
    if op == "swa_decode":
        Hkv = rng.randint(1, 8)
        return dict(op=op, N=_log(rng, 1, 128), H=Hkv * rng.choice([1, 2, 3, 4, 8]), Hkv=Hkv,
                    d=rng.choice([64, 128]), window=_log(rng, 1, 2048),
                    sinks=rng.choice([0, 1, 4, 17, 64]), ragged=rng.random() < 0.7, dtype=dtype)
    if op == "glr_train":
        B, D = rng.randint(1, 4), 8 * _log(rng, 1, 256)
        return dict(op=op, B=B, T=_log(rng, 1, min(32768, 33554432 // (B * D))), D=D, dtype=dtype)
    if op == "glr_step":
        return dict(op=op, N=_log(rng, 1, 1024), D=8 * _log(rng, 1, 512), dtype=dtype)
    D = 8 * _log(rng, 1, 1024)
    return dict(op=op, rows=_log(rng, 1, min(65536, 33554432 // D)), D=D, bias=rng.random() < 0.5,
                dtype=dtype)


def _lengths(case):
    """Sequence lengths: the whole T, or (ragged) falling from T to about a third of it."""
    B, T = case["B"], case["T"]
    if not case["ragged"]:
        return [T] * B
    return [T - (2 * T * b) // (3 * B) for b in range(B)]


def _positions(case):
    """Tokens already cached: a full window, or (ragged) anything from none to several windows."""
    N, cap = case["N"], case["window"] + case["sinks"]
    if not case["ragged"]:
        return [2 * cap + 1] * N
    return [(n * 7919 + 13) % (3 * cap) if n else 3 * cap for n in range(N)]


# ---------------------------------------------------------------------------------------- inputs
def _randn(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _log_decay(gen, shape):
    """Log decays -0.1 softplus(N(0, 1)); an eighth of the channels never decays, an eighth forgets
    within a token."""
    la = -0.1 * torch.nn.functional.softplus(_randn(gen, shape, torch.float32))
    D = shape[-1]
    la[..., : D // 8] = 0.0
    la[..., D // 8: D // 4] *= 200.0
    return la


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt = _DT[case["dtype"]]
    op = case["op"]
    st = dict(case=case)
    if op in ("swa_train", "swa_prefill"):
        B, T, H, Hkv, d = (case[n] for n in ("B", "T", "H", "Hkv", "d"))
        st["q"] = _randn(gen, (B, T, H, d), dt)
        st["k"] = _randn(gen, (B, T, Hkv, d), dt)
        st["v"] = _randn(gen, (B, T, Hkv, d), dt)
        if op == "swa_train":
            st["dO"] = _randn(gen, (B, T, H, d), dt)
        else:
            cap = case["window"] + case["sinks"]
            st["k_cache"] = torch.zeros((B, cap, Hkv, d), dtype=dt, device=DEV)
            st["v_cache"] = torch.zeros((B, cap, Hkv, d), dtype=dt, device=DEV)
        st["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device=DEV) if case["ragged"] else None
    elif op == "swa_decode":
        N, H, Hkv, d = (case[n] for n in ("N", "H", "Hkv", "d"))
        cap = case["window"] + case["sinks"]
        st["q"] = _randn(gen, (N, H, d), dt)
        st["k"] = _randn(gen, (N, Hkv, d), dt)
        st["v"] = _randn(gen, (N, Hkv, d), dt)
        st["k_cache"] = _randn(gen, (N, cap, Hkv, d), dt)
        st["v_cache"] = _randn(gen, (N, cap, Hkv, d), dt)
        st["pos"] = torch.tensor(_positions(case), dtype=torch.int32, device=DEV)
    elif op == "glr_train":
        shape = (case["B"], case["T"], case["D"])
        st["x"] = _randn(gen, shape, dt)
        st["log_a"] = _log_decay(gen, shape)
        st["h0"] = _randn(gen, (shape[0], shape[2]), torch.float32)
        st["dh"] = _randn(gen, shape, dt)
        st["dh_T"] = _randn(gen, (shape[0], shape[2]), torch.float32)
    elif op == "glr_step":
        shape = (case["N"], case["D"])
        st["x"] = _randn(gen, shape, dt)
        st["log_a"] = _log_decay(gen, shape)
        st["h_in"] = _randn(gen, shape, torch.float32)
        st["h_out"] = torch.empty(shape, dtype=torch.float32, device=DEV)
    else:
        shape = (case["rows"], case["D"])
        # rows of different scale and mean, as a residual stream has
        mu = _randn(gen, (shape[0], 1), torch.float32)
        sd = torch.exp(_randn(gen, (shape[0], 1), torch.float32))
        st["x"] = (mu + sd * _randn(gen, shape, torch.float32)).to(dt)
        st["weight"] = 1.0 + 0.1 * _randn(gen, (shape[1],), torch.float32)
        st["bias"] = 0.1 * _randn(gen, (shape[1],), torch.float32) if case["bias"] else None
        if op == "ln_train":
            st["dy"] = _randn(gen, shape, dt)
    return st


# ---------------------------------------------------------------------------------------- one pass
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(st):
    import gated_delta_rule_gdr_amd as g2
    c = st["case"]
    op = c["op"]
    if op == "swa_train":
        o, lse = g2.gdr2_swa_fwd(st["q"], st["k"], st["v"], c["window"], sinks=c["sinks"], lengths=st["lengths"])
        g = g2.gdr2_swa_bwd(st["q"], st["k"], st["v"], o, lse, st["dO"], c["window"], sinks=c["sinks"],
                            lengths=st["lengths"])
        return dict(o=o, dq=g["dq"], dk=g["dk"], dv=g["dv"])
    if op == "swa_prefill":
        o, _ = g2.gdr2_swa_fwd(st["q"], st["k"], st["v"], c["window"], sinks=c["sinks"], lengths=st["lengths"])
        g2.gdr2_swa_cache_fill(st["k"], st["v"], st["k_cache"], st["v_cache"], sinks=c["sinks"],
                               lengths=st["lengths"])
        return dict(o=o, k_cache=st["k_cache"], v_cache=st["v_cache"])
    if op == "swa_decode":
        o = g2.gdr2_swa_decode_step(st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"], st["pos"],
                                    sinks=c["sinks"])
        return dict(o=o, k_cache=st["k_cache"], v_cache=st["v_cache"])
    if op == "glr_train":
        h, h_T, ws = g2.gdr2_glr_fwd(st["x"], st["log_a"], h0=st["h0"])
        g = g2.gdr2_glr_bwd(st["x"], st["log_a"], st["dh"], ws, dh_T=st["dh_T"])
        return dict(h=h, h_T=h_T, dx=g["dx"], dlog_a=g["dlog_a"], dh0=g["dh0"])
    if op == "glr_step":
        h, h_out = g2.gdr2_glr_step(st["x"], st["log_a"], h_in=st["h_in"], h_out=st["h_out"])
        return dict(h=h, h_out=h_out)
    y, mean, rstd = g2.gdr2_layer_norm_fwd(st["x"], st["weight"], st["bias"])
    if op == "ln_fwd":
        return dict(y=y)
    g = g2.gdr2_layer_norm_bwd(st["x"], st["weight"], mean, rstd, st["dy"], want_dbias=c["bias"])
    out = dict(y=y, dx=g["dx"], dweight=g["dweight"])
    if c["bias"]:
        out["dbias"] = g["dbias"]
    return out


# The plain forms: fp32 throughout, rounded once at the end.

def _plain_swa_blocks(T, window, sinks, step=1024):
    """Blocks of queries with the key rows any of them may see: the sinks, then a run."""
    for i0 in range(0, T, step):
        i1 = min(T, i0 + step)
        lo = max(0, i0 - window + 1)
        yield i0, i1, torch.cat([torch.arange(0, min(sinks, lo), device=DEV), torch.arange(lo, i1, device=DEV)])


def _plain_swa(st, train):
    c = st["case"]
    B, T, H, Hkv, d = (c[n] for n in ("B", "T", "H", "Hkv", "d"))
    W, sinks, G, scale = c["window"], c["sinks"], H // Hkv, d ** -0.5
    dt = st["q"].dtype
    heads = lambda t: t.float().transpose(1, 2).contiguous()  # noqa: E731   [B, heads, T, d]
    q, k, v = heads(st["q"]), heads(st["k"]), heads(st["v"])
    k = k.repeat_interleave(G, dim=1)
    v = v.repeat_interleave(G, dim=1)
    L = st["lengths"].long() if st["lengths"] is not None else torch.full((B,), T, device=q.device)
    o = torch.zeros_like(q)
    if train:
        dO = heads(st["dO"])
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q)
    for i0, i1, j in _plain_swa_blocks(T, W, sinks):
        i = torch.arange(i0, i1, device=q.device)
        near = (j[None, :] <= i[:, None]) & ((i[:, None] - j[None, :] < W) | (j[None, :] < sinks))
        vis = near[None] & (i[None, :, None] < L[:, None, None])          # [B, queries, keys]
        vis = vis[:, None]
        kb, vb, qb = k[:, :, j], v[:, :, j], q[:, :, i0:i1]
        s = torch.matmul(qb, kb.transpose(-1, -2).contiguous()) * scale
        s = s.masked_fill(~vis, float("-inf"))
        m = s.amax(-1, keepdim=True)
        m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
        p = torch.exp(s - m)
        z = p.sum(-1, keepdim=True)
        p = p / torch.where(z > 0, z, torch.ones_like(z))
        ob = torch.matmul(p, vb)
        o[:, :, i0:i1] = ob
        if train:
            dOb = dO[:, :, i0:i1]
            dp = torch.matmul(dOb, vb.transpose(-1, -2).contiguous())
            ds = p * (dp - (dOb * ob).sum(-1, keepdim=True)) * scale
            dq[:, :, i0:i1] = torch.matmul(ds, kb)
            dk[:, :, j] += torch.matmul(ds.transpose(-1, -2).contiguous(), qb)
            dv[:, :, j] += torch.matmul(p.transpose(-1, -2).contiguous(), dOb)
    back = lambda t: t.transpose(1, 2).to(dt).contiguous()  # noqa: E731
    if not train:
        return back(o)
    group = lambda t: t.view(B, Hkv, G, T, d).sum(2)  # noqa: E731
    return dict(o=back(o), dq=back(dq), dk=back(group(dk)), dv=back(group(dv)))


def _plain_fill(st):
    c = st["case"]
    T, W, sinks = c["T"], c["window"], c["sinks"]
    for b, L in enumerate(_lengths(c)):
        p = torch.cat([torch.arange(0, min(sinks, L), device=DEV),
                       torch.arange(min(max(sinks, L - W), L), L, device=DEV)])
        slot = torch.where(p < sinks, p, sinks + (p - sinks) % W)
        st["k_cache"][b, slot] = st["k"][b, p]
        st["v_cache"][b, slot] = st["v"][b, p]


def _plain_decode(st):
    c = st["case"]
    N, H, Hkv, d, W, sinks = (c[n] for n in ("N", "H", "Hkv", "d", "window", "sinks"))
    cap = W + sinks
    pos = st["pos"].long()
    slot = torch.where(pos < sinks, pos, sinks + (pos - sinks) % W)
    n = torch.arange(N, device=pos.device)
    st["k_cache"][n, slot] = st["k"]
    st["v_cache"][n, slot] = st["v"]
    held = torch.arange(cap, device=pos.device)[None] < (pos + 1).clamp(max=cap)[:, None]  # [N, cap]
    k = st["k_cache"].float().transpose(1, 2).contiguous()     # [N, Hkv, cap, d]
    v = st["v_cache"].float().transpose(1, 2).contiguous()
    q = st["q"].float().view(N, Hkv, H // Hkv, d)
    s = torch.matmul(q, k.transpose(-1, -2).contiguous()) * d ** -0.5
    s = s.masked_fill(~held[:, None, None], float("-inf"))
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    o = torch.matmul(p, v).view(N, H, d)
    return dict(o=o.to(st["q"].dtype), k_cache=st["k_cache"], v_cache=st["v_cache"])


def _plain_scan(a, x):
    """h_t = a_t h_{t-1} + x_t along axis 1 by doubling (h_{-1} = 0)."""
    T, n = x.shape[1], 1
    while n < T:
        x = torch.cat([x[:, :n], x[:, n:] + a[:, n:] * x[:, :-n]], 1)
        a = torch.cat([a[:, :n], a[:, n:] * a[:, :-n]], 1)
        n *= 2
    return x


def _plain_glr(st):
    dt = st["x"].dtype
    a, x, h0 = torch.exp(st["log_a"]), st["x"].float(), st["h0"]
    first = x[:, :1] + a[:, :1] * h0[:, None]
    h = _plain_scan(a, torch.cat([first, x[:, 1:]], 1))
    dh = st["dh"].float()
    dh = torch.cat([dh[:, :-1], dh[:, -1:] + st["dh_T"][:, None]], 1)
    # g_t = dh_t + a_{t+1} g_{t+1}: the same scan with time reversed
    nxt = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    g = _plain_scan(nxt.flip(1), dh.flip(1)).flip(1)
    prev = torch.cat([h0[:, None], h[:, :-1]], 1)
    return dict(h=h.to(dt), h_T=h[:, -1].contiguous(), dx=g.to(dt), dlog_a=g * a * prev,
                dh0=(a[:, 0] * g[:, 0]).contiguous())


def _plain_ln(st, train):
    dt, x, w, eps = st["x"].dtype, st["x"].float(), st["weight"], 1e-5
    xc = x - x.mean(-1, keepdim=True)
    rstd = 1.0 / torch.sqrt((xc * xc).mean(-1, keepdim=True) + eps)
    n = xc * rstd
    y = n * w
    if st["bias"] is not None:
        y = y + st["bias"]
    out = dict(y=y.to(dt))
    if train:
        dy = st["dy"].float()
        a = dy * w
        dx = rstd * (a - a.mean(-1, keepdim=True) - n * (a * n).mean(-1, keepdim=True))
        out["dx"] = dx.to(dt)
        out["dweight"] = (dy * n).sum(0)
        if st["bias"] is not None:
            out["dbias"] = dy.sum(0)
    return out


def _run_plain(st):
    op = st["case"]["op"]
    if op == "swa_train":
        return _plain_swa(st, True)
    if op == "swa_prefill":
        o = _plain_swa(st, False)
        _plain_fill(st)
        return dict(o=o, k_cache=st["k_cache"], v_cache=st["v_cache"])
    if op == "swa_decode":
        return _plain_decode(st)
    if op == "glr_train":
        return _plain_glr(st)
    if op == "glr_step":
        h = torch.exp(st["log_a"]) * st["h_in"] + st["x"].float()
        st["h_out"].copy_(h)
        return dict(h=h.to(st["x"].dtype), h_out=st["h_out"])
    return _plain_ln(st, op == "ln_train")


# ---------------------------------------------------------------------------------------- work
def _pairs(L, window, sinks):
    """Visible (query, key) pairs of one sequence of L tokens."""
    inside = min(L, window)
    n = inside * (inside + 1) // 2 + (L - inside) * window
    # sinks outside the window: query i sees min(sinks, i - window + 1) more of them
    out = max(0, L - window)
    ramp = min(out, sinks)
    return n + ramp * (ramp + 1) // 2 + (out - ramp) * sinks


def work(case):
    op, es = case["op"], 4 if case["dtype"] == "f32" else 2
    if op in ("swa_train", "swa_prefill"):
        H, Hkv, d, W, sinks = (case[n] for n in ("H", "Hkv", "d", "window", "sinks"))
        Ls = _lengths(case)
        tok, whole = sum(Ls), case["B"] * case["T"]
        pairs = H * sum(_pairs(L, W, sinks) for L in Ls)
        if op == "swa_train":   # q, k, v, dO read; o, dq, dk, dv written (padding rows too)
            return dict(bytes=es * d * (tok * (2 * H + 2 * Hkv) + whole * (2 * H + 2 * Hkv)), flops=14 * d * pairs)
        kept = sum(min(L, W + sinks) for L in Ls)
        return dict(bytes=es * d * (tok * (H + 2 * Hkv) + whole * H + 2 * kept * Hkv), flops=4 * d * pairs)
    if op == "swa_decode":
        N, H, Hkv, d = (case[n] for n in ("N", "H", "Hkv", "d"))
        cap = case["window"] + case["sinks"]
        rows = sum(min(p + 1, cap) for p in _positions(case))
        return dict(bytes=es * d * (2 * Hkv * rows + 2 * Hkv * N + 2 * N * H), flops=4 * d * rows * H)
    if op == "glr_train":
        n, s = case["B"] * case["T"] * case["D"], case["B"] * case["D"]
        return dict(bytes=n * (4 * es + 8) + 16 * s, flops=9 * n)
    if op == "glr_step":
        return dict(bytes=case["N"] * case["D"] * (2 * es + 12), flops=3 * case["N"] * case["D"])
    rows, D = case["rows"], case["D"]
    if op == "ln_fwd":
        return dict(bytes=2 * rows * D * es + 8 * D, flops=8 * rows * D)
    return dict(bytes=4 * rows * D * es + 16 * D, flops=20 * rows * D)


# ---------------------------------------------------------------------------------------- exact
# From the definitions, in fp64 on inputs widened once.

def _exact_swa(st, train):
    """Softmax over the visible keys of every query, one sequence and one key/value head at a time,
    in blocks of queries against every key up to the block's end."""
    c = st["case"]
    B, T, H, Hkv, d = (c[n] for n in ("B", "T", "H", "Hkv", "d"))
    W, sinks, G = c["window"], c["sinks"], H // Hkv
    f = {n: st[n].double() for n in ("q", "k", "v")}
    out = dict(o=torch.zeros_like(f["q"]))
    if train:
        f["dO"] = st["dO"].double()
        out.update(dq=torch.zeros_like(f["q"]), dk=torch.zeros_like(f["k"]), dv=torch.zeros_like(f["v"]))
    sc = 1.0 / math.sqrt(d)
    for b, L in enumerate(_lengths(c)):
        for kv in range(Hkv):
            hs = slice(kv * G, (kv + 1) * G)
            for i0 in range(0, L, 2048):
                i1 = min(L, i0 + 2048)
                base = 0 if sinks > 0 and i0 < 2 * W + 2048 else max(0, i0 - W + 1)
                far = torch.arange(0, min(sinks, base), device=DEV)
                j = torch.cat([far, torch.arange(base, i1, device=DEV)])
                i = torch.arange(i0, i1, device=DEV)[:, None]
                hidden = (j > i) | ((i - j >= W) & (j >= sinks))
                K, V = f["k"][b, j, kv], f["v"][b, j, kv]
                for h in range(hs.start, hs.stop):
                    Q = f["q"][b, i0:i1, h]
                    S = (Q @ K.t()) * sc
                    S[hidden] = float("-inf")
                    P = torch.softmax(S, dim=1)
                    O = P @ V
                    out["o"][b, i0:i1, h] = O
                    if train:
                        dO = f["dO"][b, i0:i1, h]
                        dS = P * (dO @ V.t() - (dO * O).sum(1, keepdim=True))
                        out["dq"][b, i0:i1, h] = dS @ K * sc
                        out["dk"][b, :, kv].index_add_(0, j, dS.t() @ Q * sc)
                        out["dv"][b, :, kv].index_add_(0, j, P.t() @ dO)
    return out


def _exact_cache(case, k, v, kc, vc):
    """The cache that holds, in their slots, the last `window` positions behind the sinks."""
    W, sinks = case["window"], case["sinks"]
    for b, L in enumerate(_lengths(case)):
        for p in list(range(0, min(L, sinks))) + list(range(max(sinks, L - W), L)):
            slot = p if p < sinks else sinks + (p - sinks) % W
            kc[b, slot], vc[b, slot] = k[b, p], v[b, p]
    return kc, vc


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "swa_train":
        return _exact_swa(st, True)
    if op == "swa_prefill":
        kc, vc = (st[n].double().cpu() for n in ("k_cache", "v_cache"))
        kc, vc = _exact_cache(case, st["k"].double().cpu(), st["v"].double().cpu(), kc, vc)
        return dict(o=_exact_swa(st, False)["o"], k_cache=kc.to(DEV), v_cache=vc.to(DEV))
    if op == "swa_decode":
        N, H, Hkv, d, W, sinks = (case[n] for n in ("N", "H", "Hkv", "d", "window", "sinks"))
        kc, vc = st["k_cache"].double(), st["v_cache"].double()
        o = torch.zeros((N, H, d), dtype=torch.float64, device=DEV)
        q = st["q"].double()
        for n, p in enumerate(_positions(case)):
            slot = p if p < sinks else sinks + (p - sinks) % W
            kc[n, slot], vc[n, slot] = st["k"][n].double(), st["v"][n].double()
            rows = min(p + 1, W + sinks)
            for kv in range(Hkv):
                hs = slice(kv * (H // Hkv), (kv + 1) * (H // Hkv))
                P = torch.softmax(q[n, hs] @ kc[n, :rows, kv].t() / math.sqrt(d), dim=1)
                o[n, hs] = P @ vc[n, :rows, kv]
        return dict(o=o, k_cache=kc, v_cache=vc)
    if op == "glr_train":
        a, x, dh = st["log_a"].double().exp(), st["x"].double(), st["dh"].double()
        h = st["h0"].double()
        hs, prev = torch.empty_like(x), torch.empty_like(x)
        for t in range(case["T"]):
            prev[:, t] = h
            h = a[:, t] * h + x[:, t]
            hs[:, t] = h
        g, dx = st["dh_T"].double(), torch.empty_like(x)
        for t in range(case["T"] - 1, -1, -1):
            g = g + dh[:, t]
            dx[:, t] = g
            g = a[:, t] * g
        return dict(h=hs, h_T=h, dx=dx, dlog_a=dx * a * prev, dh0=g)
    if op == "glr_step":
        h = st["log_a"].double().exp() * st["h_in"].double() + st["x"].double()
        return dict(h=h, h_out=h)
    x, w = st["x"].double(), st["weight"].double()
    var, mu = torch.var_mean(x, dim=1, unbiased=False, keepdim=True)
    sd = torch.sqrt(var + 1e-5)
    y = (x - mu) / sd * w + (0.0 if st["bias"] is None else st["bias"].double())
    if op == "ln_fwd":
        return dict(y=y)
    dy = st["dy"].double()
    n, u = (x - mu) / sd, dy * w
    out = dict(y=y, dx=(u - u.mean(1, keepdim=True) - n * (u * n).mean(1, keepdim=True)) / sd,
               dweight=(dy * n).sum(0))
    if st["bias"] is not None:
        out["dbias"] = dy.sum(0)
    return out
