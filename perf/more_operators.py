"""More operators of a hybrid stack around the Gated Delta Rule-2 mixer, as cases to measure.

A pre-norm block adds the previous layer's output to the residual stream and normalises the sum, in
serving with an 8-bit result for the products behind it; a linear-attention layer with one fixed decay
per head stands where the recurrent mixer does; full-attention layers decode against a cache of pages.
Each case is one of:

  rms_train     h = x + residual in the stream's type, y = h / sqrt(mean h^2 + eps) weight: forward, and
                gradients from the cotangents of y and of the stream h
  rms_q8        the forward alone, y as e4m3 values with one fp32 scale per row or per group of channels
  dla_train     linear attention with a decay per head, S_t = a S_{t-1} + k_t v_t^T, o_t = S_t^T q_t:
                forward and gradients
  dla_prefill   the forward alone, with the state that decoding continues from
  dla_step      one token per sequence
  paged_fill    a prefill's (or one of its pieces') keys and values into the cache's pages
  paged_decode  one token per sequence over everything its pages hold, the token's own key and value
                stored first

Token tensors are [B, T, heads, d] or [rows, D]; lengths, starts, positions and page tables are int32.
"""
import math

import torch

own = False

DEV = "cuda"
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-6
_E4M3_MAX = 448.0


# ---------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the norm before the 1.3B layer's mixer with the residual stream, training
        dict(name="rms_train_layer", op="rms_train", rows=16384, D=2048, residual=True, dtype="bf16"),
        # a row width that is no power of two, an odd number of rows, no residual, fp32
        dict(name="rms_train_odd_f32", op="rms_train", rows=4099, D=1000, residual=False, dtype="f32"),
        # the same norm in a prefill of 16K tokens, 8-bit output with a scale per 128 channels
        dict(name="rms_q8_prefill", op="rms_q8", rows=16384, D=2048, residual=True, group=128, dtype="bf16"),
        # and of one decode step, a scale per token: latency
        dict(name="rms_q8_decode", op="rms_q8", rows=256, D=2048, residual=True, group=0, dtype="bf16"),
        # linear attention in the mixer's place at the 1.3B layer's shape, training
        dict(name="dla_train_layer", op="dla_train", B=4, T=4096, H=16, dk=128, dv=128, ragged=False, dtype="bf16"),
        # a padded batch of odd lengths, keys narrower than values, fp32
        dict(name="dla_train_ragged_f32", op="dla_train", B=3, T=777, H=6, dk=64, dv=128, ragged=True, dtype="f32"),
        # prefill of the long-context workload: few chains, 32K tokens each
        dict(name="dla_prefill_long", op="dla_prefill", B=1, T=32768, H=16, dk=128, dv=128, ragged=False, dtype="bf16"),
        # the decode workload's token: 256 sequences of 16 heads
        dict(name="dla_step_batch", op="dla_step", N=256, H=16, dk=128, dv=128, dtype="bf16"),
        # a padded prefill batch stored in pages of 16, two sequences continuing earlier pieces
        dict(name="paged_fill_ragged", op="paged_fill", B=4, T=4096, Hkv=4, d=128, page=16, ragged=True, dtype="bf16"),
        # one user's token over a 32K-token context: latency, the length split
        dict(name="paged_decode_single", op="paged_decode", N=1, H=16, Hkv=4, d=128, page=64, longest=32768, mixed=False,
             dtype="bf16"),
        # a serving batch: 256 sequences of lengths from one token to 4K, pages of 16
        dict(name="paged_decode_batch", op="paged_decode", N=256, H=16, Hkv=4, d=128, page=16, longest=4096, mixed=True,
             dtype="bf16"),
        # a small batch in fp32 with odd lengths, three heads of 64 to a key/value head, one slot idle
        dict(name="paged_decode_f32", op="paged_decode", N=13, H=12, Hkv=4, d=64, page=32, longest=2777, mixed=True,
             dtype="f32"),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rms_train", "rms_train", "rms_q8", "rms_q8", "dla_train", "dla_train", "dla_prefill", "dla_prefill",
                     "dla_step", "paged_fill", "paged_decode", "paged_decode", "paged_decode"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("rms_train", "rms_q8"):
        D = 8 * _log(rng, 1, 1024)
        c = dict(op=op, rows=_log(rng, 1, min(65536, 33554432 // D)), D=D, residual=rng.random() < 0.7, dtype=dtype)
        if op == "rms_q8":
            c["group"] = rng.choice([0, 32, 64, 128])
        return c
    if op in ("dla_train", "dla_prefill"):
        B, H = rng.randint(1, 4), rng.randint(1, 16)
        most = 262144 // (B * H) if dtype == "bf16" else 16384 // (B * H)
        return dict(op=op, B=B, T=_log(rng, 1, min(32768, most)), H=H, dk=rng.choice([64, 128]), dv=rng.choice([64, 128]),
                    ragged=rng.random() < 0.5, dtype=dtype)
    if op == "dla_step":
        H = rng.randint(1, 16)
        return dict(op=op, N=_log(rng, 1, 4096 // H), H=H, dk=rng.choice([64, 128]), dv=rng.choice([64, 128]), dtype=dtype)
    Hkv, d, page = rng.randint(1, 8), rng.choice([64, 128]), rng.choice([1, 8, 16, 32, 64, 128, 256])
    if op == "paged_fill":
        B = rng.randint(1, 8)
        return dict(op=op, B=B, T=_log(rng, 1, 16384 // B), Hkv=Hkv, d=d, page=page, ragged=rng.random() < 0.7, dtype=dtype)
    N = _log(rng, 1, 256)
    most = min(32768, 2097152 // (N * Hkv * (2 if dtype == "f32" else 1)))
    return dict(op=op, N=N, H=Hkv * rng.choice([1, 2, 3, 4, 8]), Hkv=Hkv, d=d, page=page, longest=_log(rng, 1, most),
                mixed=rng.random() < 0.7, dtype=dtype)


def _lengths(case):
    """Sequence lengths: the whole T, or (ragged) falling from T to about a third of it."""
    B, T = case["B"], case["T"]
    return [T - (2 * T * b) // (3 * B) if case["ragged"] else T for b in range(B)]


def _starts(case):
    """Positions a piece starts at: zero, or (ragged) for every other sequence some odd position."""
    return [(b * 777 + 5) % 1500 if case["ragged"] and b % 2 else 0 for b in range(case["B"])]


def _positions(case):
    """The new token's position: the last of `longest`, or (mixed) anything below it, every thirteenth
    slot of the batch without a token."""
    N, L = case["N"], case["longest"]
    if not case["mixed"]:
        return [L - 1] * N
    return [-1 if n % 13 == 12 else (n * 7919 + 13) % L if n else L - 1 for n in range(N)]


# ---------------------------------------------------------------------------------------- inputs
def _randn(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _pages(gen, case, held):
    """A cache whose pages hold `held` rows per sequence, in any order, and its table; entries behind a
    sequence's last page name none."""
    page, shape = case["page"], (case["page"], case["Hkv"], case["d"])
    need = [(n + page - 1) // page for n in held]
    width = max(1, max(need))
    used = torch.arange(width, device=DEV)[None] < torch.tensor(need, device=DEV)[:, None]
    table = torch.full((len(held), width), -1, dtype=torch.int32, device=DEV)
    total = sum(need) + 3
    table[used] = torch.randperm(total, generator=gen, device=DEV)[: sum(need)].int()
    dt = _DT[case["dtype"]]
    return dict(table=table, k_pages=_randn(gen, (total,) + shape, dt), v_pages=_randn(gen, (total,) + shape, dt))


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt = _DT[case["dtype"]]
    op = case["op"]
    st = dict(case=case)
    if op in ("rms_train", "rms_q8"):
        shape = (case["rows"], case["D"])
        # rows of different scale, a stream that is larger than what a layer adds, outlying channels
        sd = torch.exp(_randn(gen, (shape[0], 1), torch.float32))
        out = 1.0 + 10.0 * (torch.rand((1, shape[1]), generator=gen, device=DEV) < 0.01).float()
        st["x"] = (sd * out * _randn(gen, shape, torch.float32)).to(dt)
        st["residual"] = (2.0 * sd * out * _randn(gen, shape, torch.float32)).to(dt) if case["residual"] else None
        st["weight"] = 1.0 + 0.1 * _randn(gen, (shape[1],), torch.float32)
        if op == "rms_train":
            st["dy"] = _randn(gen, shape, dt)
            st["dh"] = _randn(gen, shape, dt) if case["residual"] else None
    elif op in ("dla_train", "dla_prefill", "dla_step"):
        H, dk, dv = case["H"], case["dk"], case["dv"]
        tok = (case["N"], H) if op == "dla_step" else (case["B"], case["T"], H)
        st["q"] = (dk ** -0.5 * _randn(gen, tok + (dk,), torch.float32)).to(dt)
        st["k"] = _randn(gen, tok + (dk,), dt)
        st["v"] = _randn(gen, tok + (dv,), dt)
        # a memory of two tokens for the first head to a few hundred for the last, jittered
        slope = 2.0 ** (-8.0 * torch.arange(1, H + 1, device=DEV, dtype=torch.float32) / H)
        st["log_decay"] = -slope * (0.5 + torch.rand((H,), generator=gen, device=DEV))
        st["S0"] = _randn(gen, (tok[0], H, dk, dv), torch.float32)
        if op == "dla_step":
            st["S_out"] = torch.empty_like(st["S0"])
        else:
            st["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device=DEV) if case["ragged"] else None
        if op == "dla_train":
            st["dO"] = _randn(gen, tok + (dv,), dt)
            st["dS_T"] = _randn(gen, (tok[0], H, dk, dv), torch.float32)
    elif op == "paged_fill":
        shape = (case["B"], case["T"], case["Hkv"], case["d"])
        st["k"] = _randn(gen, shape, dt)
        st["v"] = _randn(gen, shape, dt)
        st.update(_pages(gen, case, [s + n for s, n in zip(_starts(case), _lengths(case))]))
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV) if case["ragged"] else None  # noqa: E731
        st["start"], st["lengths"] = ints(_starts(case)), ints(_lengths(case))
    else:
        N, H, Hkv, d = (case[n] for n in ("N", "H", "Hkv", "d"))
        st["q"] = _randn(gen, (N, H, d), dt)
        st["k"] = _randn(gen, (N, Hkv, d), dt)
        st["v"] = _randn(gen, (N, Hkv, d), dt)
        st["pos"] = torch.tensor(_positions(case), dtype=torch.int32, device=DEV)
        st.update(_pages(gen, case, [p + 1 for p in _positions(case)]))
    return st


# ---------------------------------------------------------------------------------------- one pass
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(st):
    import gated_delta_rule_gdr_amd as g2
    c = st["case"]
    op = c["op"]
    if op == "rms_train":
        y, h, rstd = g2.gdr2_rms_norm_fwd(st["x"], st["weight"], residual=st["residual"], eps=_EPS)
        g = g2.gdr2_rms_norm_bwd(h, st["weight"], rstd, st["dy"], dh=st["dh"])
        return dict(y=y, h=h, dx=g["dx"], dweight=g["dweight"])
    if op == "rms_q8":
        y8, scale, h = g2.gdr2_rms_norm_q8_fwd(st["x"], st["weight"], residual=st["residual"], eps=_EPS, group=c["group"])
        return dict(y8=y8, scale=scale, h=h)
    if op == "dla_train":
        o, S_T = g2.gdr2_dla_fwd(st["q"], st["k"], st["v"], st["log_decay"], S0=st["S0"], lengths=st["lengths"])
        g = g2.gdr2_dla_bwd(st["q"], st["k"], st["v"], st["log_decay"], st["dO"], S0=st["S0"], dS_T=st["dS_T"],
                            lengths=st["lengths"])
        return dict(o=o, S_T=S_T, dq=g["dq"], dk=g["dk"], dv=g["dv"], dS0=g["dS0"])
    if op == "dla_prefill":
        o, S_T = g2.gdr2_dla_fwd(st["q"], st["k"], st["v"], st["log_decay"], S0=st["S0"], lengths=st["lengths"])
        return dict(o=o, S_T=S_T)
    if op == "dla_step":
        o, S_out = g2.gdr2_dla_step(st["q"], st["k"], st["v"], st["log_decay"], S_in=st["S0"], S_out=st["S_out"])
        return dict(o=o, S_out=S_out)
    if op == "paged_fill":
        g2.gdr2_paged_cache_fill(st["k"], st["v"], st["k_pages"], st["v_pages"], st["table"], start=st["start"],
                                 lengths=st["lengths"])
        return dict(k_pages=st["k_pages"], v_pages=st["v_pages"])
    o = g2.gdr2_paged_decode_step(st["q"], st["k"], st["v"], st["k_pages"], st["v_pages"], st["table"], st["pos"])
    return dict(o=o, k_pages=st["k_pages"], v_pages=st["v_pages"])


# The plain forms: fp32 throughout, rounded once at the end (powers of a decay in fp64, since their
# exponents reach the length of the sequence).

def _plain_rms(st, train):
    dt, w = st["x"].dtype, st["weight"]
    h = st["x"].float()
    if st["residual"] is not None:
        # the stream is kept in its type, and what is kept is what is normalised
        h = h + st["residual"].float()
    h = h.to(dt)
    x = h.float()
    rstd = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + _EPS)
    n = x * rstd
    y = n * w
    if train:
        dy = st["dy"].float()
        a = dy * w
        dx = rstd * (a - n * (a * n).mean(-1, keepdim=True))
        if st["dh"] is not None:
            dx = dx + st["dh"].float()
        return dict(y=y.to(dt), h=h, dx=dx.to(dt), dweight=(dy * n).sum(0))
    rows, D = x.shape
    group = st["case"]["group"] or D
    pad = torch.zeros((rows, -D % group), device=y.device)
    yg = torch.cat([y, pad], 1).view(rows, -1, group)
    scale = yg.abs().amax(-1) / _E4M3_MAX
    y8 = (yg / scale.clamp(min=1e-37)[..., None]).view(rows, -1)[:, :D].to(torch.float8_e4m3fn)
    return dict(y8=y8, scale=scale if st["case"]["group"] else scale[:, 0].contiguous(), h=h)


def _powers(g, n):
    """exp(n g) for decays g [H] and whole numbers n >= 0 of any shape: [H, *n.shape], fp32."""
    return torch.exp(g.double().view(-1, *([1] * n.dim())) * n.double()).float()


def _plain_la(x, y, z, g, C=256):
    """sum over s <= t of a^(t - s) (x_t . y_s) z_s for [B, H, T, .] fp32: within chunks of C tokens by their
    scores, before them by the chunks' states, whose carry is a product with the powers of a^C."""
    B, H, T = x.shape[:3]
    n = (T + C - 1) // C
    cut = lambda t: torch.nn.functional.pad(t, (0, 0, 0, n * C - T)).view(B, H, n, C, t.shape[-1])  # noqa: E731
    x, y, z = cut(x), cut(y), cut(z)
    i = torch.arange(C, device=x.device)
    lag = i[:, None] - i[None, :]
    near = torch.where(lag >= 0, _powers(g, lag.clamp(min=0)), torch.zeros((), device=x.device))      # [H, C, C]
    out = torch.matmul(torch.matmul(x, y.transpose(-1, -2).contiguous()) * near[None, :, None], z)
    late = (y * _powers(g, C - 1 - i)[None, :, None, :, None]).transpose(-1, -2).contiguous()
    local = torch.matmul(late, z)                                                                     # [B, H, n, K, V]
    c = torch.arange(n, device=x.device)
    far = c[:, None] - 1 - c[None, :]
    carry = torch.where(far >= 0, _powers(g, C * far.clamp(min=0)), torch.zeros((), device=x.device))  # [H, n, n]
    state = torch.matmul(carry[None], local.flatten(-2)).view_as(local)                # the state behind chunk c - 1
    out = out + torch.matmul(x * _powers(g, i + 1)[None, :, None, :, None], state)
    return out.view(B, H, n * C, -1)[:, :, :T]


def _plain_dla(st, train):
    c = st["case"]
    B, T, g, dt = c["B"], c["T"], st["log_decay"], st["q"].dtype
    L = st["lengths"] if st["lengths"] is not None else torch.full((B,), T, device=DEV, dtype=torch.int32)
    t = torch.arange(T, device=DEV)
    live = (t[None] < L[:, None])[:, None, :, None]                                                    # [B, 1, T, 1]
    heads = lambda u: torch.where(live, u.float().transpose(1, 2), 0.0).contiguous()                   # noqa: E731
    back = lambda u: torch.where(live, u, 0.0).transpose(1, 2).to(dt).contiguous()                     # noqa: E731
    q, k, v, S0 = heads(st["q"]), heads(st["k"]), heads(st["v"]), st["S0"]
    left = (L[:, None] - 1 - t[None]).clamp(min=0)                                                     # [B, T]
    to_end = _powers(g, left).transpose(0, 1)[..., None]                                               # [B, H, T, 1]
    from_start = _powers(g, t + 1)[None, ..., None]                                                    # [1, H, T, 1]
    whole = _powers(g, L).transpose(0, 1)[..., None, None]                                             # [B, H, 1, 1]
    o = _plain_la(q, k, v, g) + from_start * torch.matmul(q, S0)
    S_T = torch.matmul((k * to_end).transpose(-1, -2).contiguous(), v) + whole * S0
    out = dict(o=back(o), S_T=S_T)
    if not train:
        return out
    dO, dS = heads(st["dO"]), st["dS_T"]
    turn = lambda u: u.flip(2)  # noqa: E731
    S0t, dSt = S0.transpose(-1, -2).contiguous(), dS.transpose(-1, -2).contiguous()
    dq = _plain_la(dO, v, k, g) + from_start * torch.matmul(dO, S0t)
    dk = turn(_plain_la(turn(v), turn(dO), turn(q), g)) + to_end * torch.matmul(v, dSt)
    dv = turn(_plain_la(turn(k), turn(q), turn(dO), g)) + to_end * torch.matmul(k, dS)
    dS0 = torch.matmul((q * from_start).transpose(-1, -2).contiguous(), dO) + whole * dS
    return dict(out, dq=back(dq), dk=back(dk), dv=back(dv), dS0=dS0)


def _plain_fill(st):
    c = st["case"]
    B, T, page = c["B"], c["T"], c["page"]
    t = torch.arange(T, device=DEV)
    L = st["lengths"] if st["lengths"] is not None else torch.full((B,), T, device=DEV, dtype=torch.int32)
    start = st["start"] if st["start"] is not None else torch.zeros_like(L)
    b, i = (t[None] < L[:, None]).nonzero(as_tuple=True)
    p = (start.long()[b] + i)
    at = st["table"].long()[b, p // page], p % page
    st["k_pages"][at] = st["k"][b, i]
    st["v_pages"][at] = st["v"][b, i]
    return dict(k_pages=st["k_pages"], v_pages=st["v_pages"])


def _plain_decode(st):
    c = st["case"]
    N, H, Hkv, d, page = (c[n] for n in ("N", "H", "Hkv", "d", "page"))
    pos, table = st["pos"].long(), st["table"].long()
    n = (pos >= 0).nonzero()[:, 0]
    at = table[n, pos[n] // page], pos[n] % page
    st["k_pages"][at] = st["k"][n]
    st["v_pages"][at] = st["v"][n]
    rows = lambda t: t[table.clamp(min=0)].view(N, -1, Hkv, d).float().transpose(1, 2).contiguous()  # noqa: E731
    k, v = rows(st["k_pages"]), rows(st["v_pages"])
    held = torch.arange(k.shape[2], device=DEV)[None] <= pos[:, None]
    s = torch.matmul(st["q"].float().view(N, Hkv, H // Hkv, d), k.transpose(-1, -2).contiguous()) * d ** -0.5
    s = s.masked_fill(~held[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p / torch.where(z > 0, z, torch.ones_like(z)), v).view(N, H, d)
    return dict(o=o.to(st["q"].dtype), k_pages=st["k_pages"], v_pages=st["v_pages"])


def _run_plain(st):
    op = st["case"]["op"]
    if op in ("rms_train", "rms_q8"):
        return _plain_rms(st, op == "rms_train")
    if op in ("dla_train", "dla_prefill"):
        return _plain_dla(st, op == "dla_train")
    if op == "dla_step":
        S = torch.exp(st["log_decay"])[None, :, None, None] * st["S0"]
        S = S + st["k"].float()[..., None] * st["v"].float()[..., None, :]
        st["S_out"].copy_(S)
        o = (S * st["q"].float()[..., None]).sum(-2)
        return dict(o=o.to(st["q"].dtype), S_out=st["S_out"])
    if op == "paged_fill":
        return _plain_fill(st)
    return _plain_decode(st)


# ---------------------------------------------------------------------------------------- work
def work(case):
    op, es = case["op"], 4 if case["dtype"] == "f32" else 2
    if op in ("rms_train", "rms_q8"):
        rows, D = case["rows"], case["D"]
        n, res = rows * D * es, 1 if case["residual"] else 0
        if op == "rms_train":   # x, residual, dy, dh read; y, h, dx written (without a residual h is x)
            return dict(bytes=n * (4 + 3 * res) + 8 * D, flops=(12 + 2 * res) * rows * D)
        scales = rows * (-(-D // case["group"]) if case["group"] else 1)
        return dict(bytes=n * (1 + 2 * res) + rows * D + 4 * scales + 4 * D, flops=(7 + res) * rows * D)
    if op == "dla_step":
        n, dk, dv = case["N"] * case["H"], case["dk"], case["dv"]
        return dict(bytes=n * (8 * dk * dv + es * (2 * dk + 2 * dv)), flops=5 * n * dk * dv)
    if op in ("dla_train", "dla_prefill"):
        H, dk, dv = case["H"], case["dk"], case["dv"]
        tok, whole, state = sum(_lengths(case)) * H, case["B"] * case["T"] * H, case["B"] * H * dk * dv * 4
        if op == "dla_train":   # q, k, v, dO read; o, dq, dk, dv written (padding rows too); four states
            return dict(bytes=es * (tok + whole) * (2 * dk + 2 * dv) + 4 * state, flops=12 * tok * dk * dv)
        return dict(bytes=es * (tok * (2 * dk + dv) + whole * dv) + 2 * state, flops=4 * tok * dk * dv)
    if op == "paged_fill":
        return dict(bytes=4 * sum(_lengths(case)) * case["Hkv"] * case["d"] * es, flops=0)
    N, H, Hkv, d = (case[n] for n in ("N", "H", "Hkv", "d"))
    held = sum(p + 1 for p in _positions(case))
    # the pages' rows read, the new rows read and written, queries and outputs
    return dict(bytes=es * d * (2 * Hkv * held + 2 * Hkv * N + 2 * N * H), flops=4 * d * held * H)


# ---------------------------------------------------------------------------------------- exact
# From the definitions, in fp64 on inputs widened once.

def _exact_rms(st, train):
    x, w = st["x"].double(), st["weight"].double()
    s = x if st["residual"] is None else x + st["residual"].double()
    h = s.to(st["x"].dtype).double()                 # the stream as it is kept
    ms = torch.einsum("rd,rd->r", h, h)[:, None] / h.shape[1] + _EPS
    y = h * w / ms.sqrt()
    if train:
        dy = st["dy"].double()
        # d/dh_j of sum_i dy_i w_i h_i ms^(-1/2)
        u = dy * w
        dx = u / ms.sqrt() - h * (u * h).sum(1, keepdim=True) / (h.shape[1] * ms ** 1.5)
        if st["dh"] is not None:
            dx = dx + st["dh"].double()
        return dict(y=y, h=s, dx=dx, dweight=(dy * h / ms.sqrt()).sum(0))
    group = st["case"]["group"] or h.shape[1]
    cols = [y[:, c: c + group] for c in range(0, h.shape[1], group)]
    scale = torch.stack([c.abs().max(1).values / _E4M3_MAX for c in cols], 1)
    y8 = torch.cat([torch.where(scale[:, i: i + 1] > 0, c / scale[:, i: i + 1], 0.0) for i, c in enumerate(cols)], 1)
    return dict(y8=y8, scale=scale if st["case"]["group"] else scale[:, 0], h=s)


def _exact_dla(st, train):
    """Token by token: S_t, and backwards R_t = dL/dS_t."""
    c = st["case"]
    B, T, H, dk, dv = (c[n] for n in ("B", "T", "H", "dk", "dv"))
    L = torch.tensor(_lengths(c), device=DEV)
    a = st["log_decay"].double().exp()[None, :, None, None]
    q, k, v = (st[n].double() for n in ("q", "k", "v"))
    S = st["S0"].double()
    out = dict(o=torch.zeros((B, T, H, dv), dtype=torch.float64, device=DEV))
    if train:
        dO = st["dO"].double()
        out.update(dq=torch.zeros_like(q))
    for t in range(T):
        on = (t < L)[:, None, None, None]
        new = a * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        S = torch.where(on, new, S)
        out["o"][:, t] = torch.where(on[..., 0], (S * q[:, t, :, :, None]).sum(2), 0.0)
        if train:
            out["dq"][:, t] = torch.where(on[..., 0], (S * dO[:, t, :, None, :]).sum(3), 0.0)
    out["S_T"] = S
    if not train:
        return out
    R = st["dS_T"].double()
    out.update(dk=torch.zeros_like(k), dv=torch.zeros_like(v))
    for t in range(T - 1, -1, -1):
        on = (t < L)[:, None, None, None]
        G = R + q[:, t, :, :, None] * dO[:, t, :, None, :]
        out["dk"][:, t] = torch.where(on[..., 0], (G * v[:, t, :, None, :]).sum(3), 0.0)
        out["dv"][:, t] = torch.where(on[..., 0], (G * k[:, t, :, :, None]).sum(2), 0.0)
        R = torch.where(on, a * G, R)
    return dict(out, dS0=R)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("rms_train", "rms_q8"):
        return _exact_rms(st, op == "rms_train")
    if op in ("dla_train", "dla_prefill"):
        out = _exact_dla(st, op == "dla_train")
        return {n: out[n] for n in (("o", "S_T", "dq", "dk", "dv", "dS0") if op == "dla_train" else ("o", "S_T"))}
    if op == "dla_step":
        S = st["log_decay"].double().exp()[None, :, None, None] * st["S0"].double()
        S = S + st["k"].double()[..., None] * st["v"].double()[..., None, :]
        return dict(o=torch.einsum("nhkv,nhk->nhv", S, st["q"].double()), S_out=S)
    kp, vp, table, page = st["k_pages"].double(), st["v_pages"].double(), st["table"].long().tolist(), case["page"]
    if op == "paged_fill":
        kf, vf = kp.view(-1, case["Hkv"], case["d"]), vp.view(-1, case["Hkv"], case["d"])
        for b, (s, n) in enumerate(zip(_starts(case), _lengths(case))):
            slot = torch.tensor([table[b][p // page] * page + p % page for p in range(s, s + n)], device=DEV)
            kf[slot], vf[slot] = st["k"][b, :n].double(), st["v"][b, :n].double()
        return dict(k_pages=kp, v_pages=vp)
    N, H, Hkv, d = (case[n] for n in ("N", "H", "Hkv", "d"))
    o = torch.zeros((N, H, d), dtype=torch.float64, device=DEV)
    q = st["q"].double()
    for n, p in enumerate(_positions(case)):
        if p < 0:
            continue
        pages = torch.tensor(table[n][: p // page + 1], device=DEV)
        kp[pages[-1], p % page], vp[pages[-1], p % page] = st["k"][n].double(), st["v"][n].double()
        K, V = kp[pages].reshape(-1, Hkv, d)[: p + 1], vp[pages].reshape(-1, Hkv, d)[: p + 1]
        for g in range(Hkv):
            hs = slice(g * (H // Hkv), (g + 1) * (H // Hkv))
            P = torch.softmax(q[n, hs] @ K[:, g].t() / math.sqrt(d), dim=1)
            o[n, hs] = P @ V[:, g]
    return dict(o=o, k_pages=kp, v_pages=vp)
