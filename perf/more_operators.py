"""The gated delta rule (prompts, backward, single tokens), the norms around a block with its
gate and residual scale (forward, backward) and rotary positions, as they are measured.

Where `own` is false, run() computes them in elementary torch operations in float32 (sums of
log decays, their differences and angles in float64); where it is true it calls the
framework.  exact() is the definition itself in float64: the recurrences token by token, the
norms differentiated, the rotation as a complex product.
"""
import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
CHUNK = 64  # tokens per chunk of the plain chunked form


def _act(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


# ----------------------------------------------------------------------------- cases


def listed():
    return [
        # forward of a mixer shard's tokens: 2 rows of 8192, 32 heads, 128 key and 64
        # value channels (the SSD shard's state size)
        _gd("gd_fwd_shard", batch=2, tokens=8192, heads=32, kheads=32, dk=128, dv=64),
        # packed prompts of 512 to 8192 tokens, four value heads to a key head, q, k and v as
        # views of one projection; every prompt continues from a state and leaves one
        _gd("gd_fwd_packed", tokens=32768, lo=512, hi=8192, heads=32, kheads=8, dk=128, dv=128,
            fused=True, init=True),
        # a handful of short float32 prompts of odd lengths: latency
        _gd("gd_fwd_ragged_f32", tokens=256, lo=1, hi=97, heads=4, kheads=4, dk=64, dv=64,
            act="f32", init=True),
        # training step of the shard, two value heads to a key head
        _gd("gd_bwd_shard", kind="gd_bwd", batch=2, tokens=8192, heads=32, kheads=16, dk=128, dv=128),
        # training step of a small packed batch of odd lengths with state gradients
        _gd("gd_bwd_ragged", kind="gd_bwd", tokens=1000, lo=1, hi=301, heads=8, kheads=2, dk=64,
            dv=64, init=True),
        # one user's next token
        _step("gd_step_one", rows=1, slots=1, heads=32, kheads=32, dk=128, dv=128),
        # a full serving batch with a pool of states, a few rows of padding
        _step("gd_step_batch", rows=256, slots=300, heads=32, kheads=8, dk=128, dv=128),
        # around the shard's mixer: its output normalised, gated and scaled into a float32
        # residual stream, whose norm is the next block's input
        _bn("bn_fwd_shard", "bn_fwd", rows=16384, channels=2048, gate="silu", res="f32"),
        # its backward in training
        _bn("bn_bwd_shard", "bn_bwd", rows=16384, channels=2048, gate="silu", res="f32"),
        # a decode batch of a model in float32, centred norms, odd sizes: latency
        _bn("bn_fwd_decode_f32", "bn_fwd", rows=33, channels=1120, gate="none", res="f32", center=True,
            act="f32"),
        # queries and keys of the shard's linear attention
        _rope("rope_fwd_shard", "rope_fwd", batch=2, tokens=8192, heads=32, kheads=8, dim=128, rot=128,
              style="half"),
        # gradients of a packed batch far into long contexts, half of each head rotated
        _rope("rope_bwd_packed", "rope_bwd", batch=1, tokens=5003, heads=8, kheads=2, dim=128, rot=64,
              style="interleaved", places="far", scaling="yarn"),
    ]


def _named(name, c):
    return dict(c, name=name) if name else c


def _gd(name=None, kind="gd_fwd", batch=1, tokens=0, lo=0, hi=0, heads=1, kheads=1, dk=64, dv=64,
        act="bf16", fused=False, init=False):
    return _named(name, dict(kind=kind, batch=batch, tokens=tokens, lo=lo, hi=hi, heads=heads,
                             kheads=kheads, dk=dk, dv=dv, act=act, fused=fused, init=init))


def _step(name, rows, slots, heads, kheads, dk, dv, act="bf16"):
    return _named(name, dict(kind="gd_step", rows=rows, slots=slots, heads=heads, kheads=kheads,
                             dk=dk, dv=dv, act=act))


def _bn(name, kind, rows, channels, gate, res, center=False, act="bf16", post=True, pre=True):
    return _named(name, dict(kind=kind, rows=rows, channels=channels, gate=gate, res=res,
                             center=center, act=act, post=post, pre=pre))


def _rope(name, kind, batch, tokens, heads, kheads, dim, rot, style, places="rows", scaling="none",
          act="bf16"):
    return _named(name, dict(kind=kind, batch=batch, tokens=tokens, heads=heads, kheads=kheads,
                             dim=dim, rot=rot, style=style, places=places, scaling=scaling, act=act))


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    kind = rng.choice(["gd_fwd", "gd_fwd", "gd_bwd", "gd_step", "bn_fwd", "bn_bwd", "rope_fwd",
                       "rope_bwd"])
    act = rng.choice(["bf16", "bf16", "f32"])
    if kind in ("gd_fwd", "gd_bwd"):
        kheads = rng.choice([1, 2, 4, 8])
        heads = kheads * rng.choice([1, 2, 4])
        dk, dv = rng.choice([64, 128]), rng.choice([64, 128])
        tokens = _log_int(rng, 16, (32768 if kind == "gd_fwd" else 12288) // (2 if act == "f32" else 1))
        fused, init = rng.random() < 0.5, rng.random() < 0.5
        if rng.random() < 0.4:
            batch = rng.choice([1, 2, 3])
            return _gd(None, kind, batch, max(1, tokens // batch), 0, 0, heads, kheads, dk, dv, act,
                       fused, init)
        hi = _log_int(rng, max(8, tokens // 64), 8192)
        return _gd(None, kind, 1, tokens, max(1, hi // 16), hi, heads, kheads, dk, dv, act, fused, init)
    if kind == "gd_step":
        rows, kheads = _log_int(rng, 1, 256), rng.choice([1, 2, 4, 8])
        return _step(None, rows, rows + rng.randrange(0, 45), kheads * rng.choice([1, 2, 4]), kheads,
                     rng.choice([64, 128]), rng.choice([64, 128]), act)
    if kind in ("bn_fwd", "bn_bwd"):
        post = rng.random() < 0.6
        return _bn(None, kind, _log_int(rng, 1, 8192), _log_int(rng, 96, 4096),
                   rng.choice(["none", "linear", "sigmoid", "silu"]), rng.choice(["act", "f32"]),
                   rng.random() < 0.5, act, post, not post or rng.random() < 0.8)
    kheads, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 80, 96, 128])
    return _rope(None, kind, rng.choice([1, 2, 3]), _log_int(rng, 1, 5000), kheads * rng.choice([1, 2, 4]),
                 kheads, dim, 2 * rng.randrange(8, dim // 2 + 1), rng.choice(["half", "interleaved"]),
                 rng.choice(["rows", "far"]), rng.choice(["none", "linear", "ntk", "yarn"]), act)


# ---------------------------------------------------------------------------- inputs


class _Gen:
    """Seeded draws on the device."""

    def __init__(self, seed):
        self.g = torch.Generator(device=DEV)
        self.g.manual_seed(int(seed))

    def normal(self, *shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=self.g, device=DEV) * scale).to(dtype)

    def uniform(self, lo, hi, *shape):
        return torch.rand(*shape, generator=self.g, device=DEV) * (hi - lo) + lo

    def unit(self, *shape, dtype):
        """Rows of length one, as a model's norm of its queries and keys leaves them."""
        x = self.normal(*shape)
        return (x / x.norm(dim=-1, keepdim=True)).to(dtype)

    def gates(self, *shape):
        """(log decays, betas) of the last dimension's heads: -A softplus(a + dt0) with A in
        (0, 16) and time steps from 1e-3 to 1e-1, and a sigmoid."""
        H = shape[-1]
        dt0 = torch.exp(self.uniform(math.log(1e-3), math.log(0.1), H))
        step = torch.log1p(torch.exp(self.normal(*shape) + torch.log(torch.expm1(dt0))))
        return -self.uniform(0.0, 16.0, H) * step, torch.sigmoid(self.normal(*shape))


def _sequences(case):
    """How many sequences a case has: as many of the middle length as its tokens hold."""
    if not case["hi"]:
        return case["batch"]
    return max(1, min(case["tokens"], round(2 * case["tokens"] / (case["lo"] + case["hi"]))))


def _lengths(case, seed):
    """Sequence lengths of a packed case: uniform draws from [lo, hi], scaled to the tokens."""
    g = torch.Generator()
    g.manual_seed(int(seed) * 7 + 3)
    n, total = _sequences(case), case["tokens"]
    w = torch.randint(case["lo"], case["hi"] + 1, (n,), generator=g).double()
    ends = torch.cumsum(w, 0) / w.sum() * (total - n)
    ends = [0] + [int(e) for e in ends[:-1]] + [total - n]
    return [b - a + 1 for a, b in zip(ends, ends[1:])]


def _prepare_gd(case, seed):
    g = _Gen(seed)
    act = _act(case["act"])
    b, L, H, Hk, Dk, Dv = (case[k] for k in ("batch", "tokens", "heads", "kheads", "dk", "dv"))
    q, k, v = g.unit(b, L, Hk, Dk, dtype=act), g.unit(b, L, Hk, Dk, dtype=act), g.normal(b, L, H, Dv, dtype=act)
    if case["fused"]:  # views of one projection's output rows
        w = [Hk * Dk, Hk * Dk, H * Dv]
        qkv = torch.cat([x.flatten(2) for x in (q, k, v)], dim=-1)
        q, k, v = (x.unflatten(-1, s) for x, s in zip(qkv.split(w, dim=-1),
                                                      ((Hk, Dk), (Hk, Dk), (H, Dv))))
    log_decay, beta = g.gates(b, L, H)
    s = dict(kind=case["kind"], q=q, k=k, v=v, g=log_decay, beta=beta, scale=Dk ** -0.5,
             act=case["act"], cu=None, init=None)
    if case["hi"]:
        lens = _lengths(case, seed)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
    else:
        lens = [L] * b
    S = len(lens)
    # the plain form's plan: every sequence at the start of a row of whole chunks
    n = torch.tensor(lens, device=DEV)
    wide = -(-max(lens) // CHUNK) * CHUNK
    first = torch.cumsum(n, 0) - n
    at = torch.arange(wide, device=DEV)[None, :]
    s["lens"], s["first"], s["longest"] = n, first, max(lens)
    s["live"] = at < n[:, None]
    s["rows"] = torch.where(s["live"], first[:, None] + at, 0)
    if case["init"]:
        s["init"] = g.normal(S, H, Dv, Dk, scale=Dk ** -0.5)
    if case["kind"] == "gd_bwd":
        s["do"] = g.normal(b, L, H, Dv, dtype=act)
        if case["init"]:
            s["dfinal"] = g.normal(S, H, Dv, Dk, scale=Dk ** -0.5)
    return s


def _prepare_step(case, seed):
    g = _Gen(seed)
    act = _act(case["act"])
    n, H, Hk, Dk, Dv = (case[k] for k in ("rows", "heads", "kheads", "dk", "dv"))
    gc = torch.Generator()
    gc.manual_seed(int(seed) * 11 + 5)
    ids = torch.randperm(case["slots"], generator=gc)[:n]
    live = n - 3 if n >= 16 else n  # of 16 rows or more, the last three are padding
    ids[live:] = -1
    log_decay, beta = g.gates(n, 1, H)
    return dict(kind="gd_step", q=g.unit(n, 1, Hk, Dk, dtype=act), k=g.unit(n, 1, Hk, Dk, dtype=act),
                v=g.normal(n, 1, H, Dv, dtype=act), g=log_decay, beta=beta, scale=Dk ** -0.5,
                state=g.normal(case["slots"], H, Dv, Dk, scale=Dk ** -0.5),
                slots=ids.to(torch.int32).to(DEV), live=live, act=case["act"],
                o=torch.zeros(n, 1, H, Dv, dtype=act, device=DEV))


def _prepare_bn(case, seed):
    g = _Gen(seed)
    act = _act(case["act"])
    res = act if case["res"] == "act" else torch.float32
    n, C = case["rows"], case["channels"]
    s = dict(kind=case["kind"], act=case["act"], res=case["res"], gate=case["gate"], eps=1e-5,
             center=case["center"], alpha=1.0, x=g.normal(n, C, scale=2.0, dtype=res),
             y=g.normal(n, C, dtype=act), z=None, scale=0.5 + g.normal(C, scale=0.2),
             post=None, pre=None)
    if case["gate"] != "none":
        # z is the first part of the input projection's rows, [z | xBC]
        s["z"] = g.normal(n, 2 * C, dtype=act)[:, :C]
    for name in ("post", "pre"):
        if case[name]:
            s[name] = (1.0 + g.normal(C, scale=0.2), g.normal(C, scale=0.2))
    if case["kind"] == "bn_bwd":
        s["dr"] = g.normal(n, C, dtype=res)
        s["dh"] = g.normal(n, C, dtype=act) if case["pre"] else None
    return s


BASE, TRAINED, FACTOR = 10000.0, 4096, 16.0


def _frequencies(rot, scaling):
    """(radians per position of every pair in float64, factor of the rotated channels), with
    contexts of TRAINED positions stretched by FACTOR."""
    f = BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if scaling == "linear":
        return f / FACTOR, 1.0
    if scaling == "ntk":
        wide = BASE * FACTOR ** (rot / (rot - 2))
        return wide ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot), 1.0
    if scaling == "yarn":  # pairs of 32 turns or more keep theirs, of one turn or less are stretched
        place = lambda turns: rot * math.log(TRAINED / (2 * math.pi * turns)) / (2 * math.log(BASE))  # noqa: E731
        lo, hi = max(0, math.floor(place(32.0))), min(rot - 1, math.ceil(place(1.0)))
        ramp = ((torch.arange(rot // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return f * (1 - ramp) + f / FACTOR * ramp, 0.1 * math.log(FACTOR) + 1.0
    return f, 1.0


def _prepare_rope(case, seed):
    g = _Gen(seed)
    act = _act(case["act"])
    b, L, H, Hk, D = (case[k] for k in ("batch", "tokens", "heads", "kheads", "dim"))
    qkv = g.normal(b, L, (H + 2 * Hk) * D, dtype=act)  # one projection's output rows
    q, k, _ = qkv.split([H * D, Hk * D, Hk * D], dim=-1)
    f, m = _frequencies(case["rot"], case["scaling"])
    pos = None
    if case["places"] == "far":
        gc = torch.Generator()
        gc.manual_seed(int(seed) * 13 + 1)
        pos = (torch.randint(0, 1 << 20, (b, 1), generator=gc) + torch.arange(L)[None]).to(torch.int32).to(DEV)
    return dict(kind=case["kind"], act=case["act"], q=q.unflatten(-1, (H, D)), k=k.unflatten(-1, (Hk, D)),
                frequencies=f.to(DEV), factor=m, rot=case["rot"], style=case["style"], positions=pos)


def prepare(case, seed):
    kind = case["kind"]
    if kind in ("gd_fwd", "gd_bwd"):
        return _prepare_gd(case, seed)
    if kind == "gd_step":
        return _prepare_step(case, seed)
    if kind in ("bn_fwd", "bn_bwd"):
        return _prepare_bn(case, seed)
    return _prepare_rope(case, seed)


# ---------------------------------------------------------------------- plain forms


def _chunks(x, s, repeat=1):
    """Token rows [b, L, h, ...] as float32 [S, h * repeat, chunks, CHUNK, ...], zero where a
    sequence has no token."""
    x = x.flatten(0, 1).float()[s["rows"]]
    x = x * s["live"].reshape(*s["live"].shape, *([1] * (x.dim() - 2)))
    if repeat > 1:
        x = x.repeat_interleave(repeat, dim=2)
    return x.transpose(1, 2).unflatten(2, (-1, CHUNK)).contiguous()


def _tokens(x, s, shape, dtype):
    """The chunks' values back at their tokens."""
    out = torch.zeros(shape[0] * shape[1], *shape[2:], device=x.device)
    out[s["rows"][s["live"]]] = x.flatten(2, 3).transpose(1, 2)[s["live"]]
    return out.reshape(shape).to(dtype)


def _t(x):
    return x.transpose(-1, -2).contiguous()


def _unit_lower_inverse(A):
    """(I + A)^-1 of strictly lower triangular A: blocks of 1, 2, 4, .. are joined."""
    n = A.shape[-1]
    T = torch.eye(n, device=A.device).expand_as(A).clone()
    m = 1
    while m < n:
        for i in range(0, n, 2 * m):
            a, b = slice(i, i + m), slice(i + m, i + 2 * m)
            T[..., b, a] = -torch.matmul(T[..., b, b], torch.matmul(A[..., b, a], T[..., a, a]))
        m *= 2
    return T


def _gd_parts(s):
    """What the chunks' products are made of."""
    r = s["v"].shape[2] // s["k"].shape[2]
    p = dict(q=_chunks(s["q"], s, r), k=_chunks(s["k"], s, r), v=_chunks(s["v"], s))
    beta = _chunks(s["beta"], s)
    cum = torch.cumsum(_chunks(s["g"], s).double(), -1)
    i = torch.arange(CHUNK, device=cum.device)
    low = i[:, None] >= i[None, :]
    p["M"] = torch.exp((cum[..., :, None] - cum[..., None, :]).float().masked_fill(~low, -math.inf))
    p["before"] = i[:, None] > i[None, :]
    p["kk"] = torch.matmul(p["k"], _t(p["k"])) * p["M"] * p["before"]
    p["P"] = torch.matmul(p["q"], _t(p["k"])) * p["M"] * s["scale"]
    p["T"] = _unit_lower_inverse(beta[..., None] * p["kk"])
    p["b"] = beta[..., None]
    p["in"] = torch.exp(cum.float())[..., None]
    p["out"] = torch.exp((cum[..., -1:] - cum).float())[..., None]
    p["all"] = torch.exp(cum[..., -1].float())[..., None, None]
    return p


def _gd_walk(s, p, want_o):
    """(outputs, entering states, u of the chunks, last state [S, H, Dk, Dv])."""
    S, H, n, _, Dk = p["k"].shape
    M = _t(s["init"]) if s["init"] is not None else torch.zeros(S, H, Dk, p["v"].shape[-1], device=DEV)
    q_in, k_in, k_out = p["q"] * p["in"] * s["scale"], p["k"] * p["in"], _t(p["k"] * p["out"])
    o, states, us = [], [], []
    for c in range(n):
        u = torch.matmul(p["T"][:, :, c], p["b"][:, :, c] * (p["v"][:, :, c] - torch.matmul(k_in[:, :, c], M)))
        if want_o:
            o.append(torch.matmul(q_in[:, :, c], M) + torch.matmul(p["P"][:, :, c], u))
        else:
            states.append(M)
            us.append(u)
        M = p["all"][:, :, c] * M + torch.matmul(k_out[:, :, c], u)
    return o, states, us, M


def _plain_gd(s):
    act, (b, L, H, Dv) = _act(s["act"]), s["v"].shape
    Hk, Dk = s["k"].shape[2:]
    r = H // Hk
    p = _gd_parts(s)
    o, states, us, M = _gd_walk(s, p, s["kind"] == "gd_fwd")
    if s["kind"] == "gd_fwd":
        return {"o": _tokens(torch.stack(o, 2), s, (b, L, H, Dv), act), "final_state": _t(M)}
    do = _chunks(s["do"], s)
    n, scale = len(states), s["scale"]
    G = _t(s["dfinal"]) if s.get("dfinal") is not None else torch.zeros_like(M)
    du_o, Tt = torch.matmul(_t(p["P"]), do), _t(p["T"])
    qdo = torch.matmul(_t(p["q"] * p["in"] * scale), do)
    k_out, k_in = p["k"] * p["out"], _t(p["k"] * p["in"])
    zs, behind = [None] * n, [None] * n
    for c in range(n - 1, -1, -1):
        behind[c] = G
        zs[c] = torch.matmul(Tt[:, :, c], du_o[:, :, c] + torch.matmul(k_out[:, :, c], G))
        G = p["all"][:, :, c] * G + qdo[:, :, c] - torch.matmul(k_in[:, :, c], p["b"][:, :, c] * zs[c])
    M0, G1, u, z = (torch.stack(x, 2) for x in (states, behind, us, zs))
    dv = p["b"] * z
    E = torch.matmul(do, _t(u)) * p["M"] * scale
    F = torch.matmul(z, _t(u))
    N = p["b"] * F * p["M"] * p["before"]
    dq = torch.matmul(do * p["in"] * scale, _t(M0)) + torch.matmul(E, p["k"])
    dk = (torch.matmul(_t(E), p["q"]) + torch.matmul(u * p["out"], _t(G1))
          - torch.matmul(dv * p["in"], _t(M0)) - torch.matmul(N, p["k"]) - torch.matmul(_t(N), p["k"]))
    x = p["v"] - torch.matmul(p["k"] * p["in"], M0)
    dbeta = (z * x).sum(-1) - (F * p["kk"]).sum(-1)
    # a decay of token t scales the queries from t on and the state behind the chunk, and
    # unscales the values from t on
    last = (p["all"] * M0 + torch.matmul(_t(k_out), u)) * G1
    own_g = (p["q"] * dq).sum(-1) - (p["v"] * dv).sum(-1)
    dg = own_g.flip(-1).cumsum(-1).flip(-1) + last.sum((-1, -2))[..., None]
    group = lambda t: t.unflatten(1, (Hk, r)).sum(2)  # noqa: E731
    return {"dq": _tokens(group(dq), s, (b, L, Hk, Dk), act), "dk": _tokens(group(dk), s, (b, L, Hk, Dk), act),
            "dv": _tokens(dv, s, (b, L, H, Dv), act), "dg": _tokens(dg, s, (b, L, H), torch.float32),
            "dbeta": _tokens(dbeta, s, (b, L, H), torch.float32), "dinit": _t(G)}


def _plain_step(s):
    live, H = s["live"], s["v"].shape[2]
    r = H // s["k"].shape[2]
    at = s["slots"][:live].long()
    q = s["q"][:live, 0].float().repeat_interleave(r, dim=1)
    k = s["k"][:live, 0].float().repeat_interleave(r, dim=1)
    v = s["v"][:live, 0].float()
    old = s["state"][at] * torch.exp(s["g"][:live, 0])[..., None, None]
    u = s["beta"][:live, 0][..., None] * (v - (old * k[..., None, :]).sum(-1))
    new = old + u[..., :, None] * k[..., None, :]
    s["state"][at] = new
    s["o"][:live, 0] = ((new * q[..., None, :]).sum(-1) * s["scale"]).to(s["o"].dtype)
    return {"o": s["o"], "state": s["state"]}


def _norm(u, center, eps):
    """(normalised rows, 1 / their deviation)"""
    if center:
        u = u - u.mean(-1, keepdim=True)
    rstd = torch.rsqrt(u.square().mean(-1, keepdim=True) + eps)
    return u * rstd, rstd


def _norm_back(g, xh, rstd, center):
    d = g - xh * (g * xh).mean(-1, keepdim=True)
    if center:
        d = d - g.mean(-1, keepdim=True)
    return d * rstd


def _gate(z, kind):
    """(factor, its derivative)"""
    if kind == "linear":
        return z, torch.ones_like(z)
    sig = torch.sigmoid(z)
    if kind == "sigmoid":
        return sig, sig * (1 - sig)
    return z * sig, sig * (1 + z * (1 - sig))


def _plain_bn(s):
    act = _act(s["act"])
    x, y = s["x"].float(), s["y"].float()
    if s["post"]:
        yh, y_rstd = _norm(y, s["center"], s["eps"])
        u = yh * s["post"][0] + s["post"][1]
    else:
        u = y
    m = u
    if s["z"] is not None:
        f, df = _gate(s["z"].float(), s["gate"])
        m = u * f
    r = s["alpha"] * x + s["scale"] * m
    if s["pre"]:
        rh, r_rstd = _norm(r, s["center"], s["eps"])
    if s["kind"] == "bn_fwd":
        out = {"r": r.to(s["x"].dtype)}
        return dict(out, h=(rh * s["pre"][0] + s["pre"][1]).to(act)) if s["pre"] else out
    G, out = s["dr"].float(), {}
    if s["pre"]:
        dh = s["dh"].float()
        G = G + _norm_back(dh * s["pre"][0], rh, r_rstd, s["center"])
        out.update(dpre_weight=(dh * rh).sum(0), dpre_bias=dh.sum(0))
    out.update(dx=(s["alpha"] * G).to(s["x"].dtype), dscale=(G * m).sum(0))
    du = s["scale"] * G
    if s["z"] is not None:
        out["dz"] = (du * u * df).to(act)
        du = du * f
    if s["post"]:
        out.update(dpost_weight=(du * yh).sum(0), dpost_bias=du.sum(0))
        du = _norm_back(du * s["post"][0], yh, y_rstd, s["center"])
    return dict(out, dy=du.to(act))


def _plain_rope(s):
    b, L = s["q"].shape[:2]
    pos = torch.arange(L, device=DEV)[None].expand(b, L) if s["positions"] is None else s["positions"]
    angle = pos.double()[..., None] * s["frequencies"]
    turn = -1.0 if s["kind"] == "rope_bwd" else 1.0
    cos = (torch.cos(angle) * s["factor"]).float()[:, :, None, :]
    sin = (torch.sin(angle) * s["factor"] * turn).float()[:, :, None, :]
    out = {}
    for name in ("q", "k"):
        x = s[name].float()
        rot, rest = x[..., :s["rot"]], x[..., s["rot"]:]
        if s["style"] == "half":
            a, c = rot.chunk(2, dim=-1)
            new = torch.cat([a * cos - c * sin, c * cos + a * sin], dim=-1)
        else:
            a, c = rot[..., 0::2], rot[..., 1::2]
            new = torch.stack([a * cos - c * sin, c * cos + a * sin], dim=-1).flatten(-2)
        out[name] = torch.cat([new, rest], dim=-1).to(s[name].dtype)
    return out


# ------------------------------------------------------------------ the framework's


def _own_gd(s):
    import mamba2_ssd_chunked_amd as ssd
    (b, L, H, Dv), (Hk, Dk) = s["v"].shape, s["k"].shape[2:]
    p = ssd.make_gdelta(batch=b, seqlen=L, nheads=H, nkheads=Hk, keydim=Dk, valdim=Dv, act=s["act"],
                        scale=s["scale"])
    if s["kind"] == "gd_fwd":
        f = ssd.gdelta_forward(p, s["q"], s["k"], s["v"], s["g"], s["beta"], cu_seqlens=s["cu"],
                               init=s["init"], want_final=True)
        return {"o": f.o, "final_state": f.final_state}
    g = ssd.gdelta_backward(p, s["q"], s["k"], s["v"], s["g"], s["beta"], s["do"], cu_seqlens=s["cu"],
                            init=s["init"], dfinal=s.get("dfinal"), want_dinit=True)
    return {"dq": g.dq, "dk": g.dk, "dv": g.dv, "dg": g.dg, "dbeta": g.dbeta, "dinit": g.dinit}


def _own_step(s):
    import mamba2_ssd_chunked_amd as ssd
    (n, _, H, Dv), (Hk, Dk) = s["v"].shape, s["k"].shape[2:]
    p = ssd.make_gdelta(batch=n, seqlen=1, nheads=H, nkheads=Hk, keydim=Dk, valdim=Dv, act=s["act"],
                        scale=s["scale"])
    ssd.ssd_gdelta_step(p, s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], s["o"],
                        slots=s["slots"])
    return {"o": s["o"], "state": s["state"]}


def _own_bn(s):
    import mamba2_ssd_chunked_amd as ssd
    n, C = s["y"].shape
    p = ssd.make_block_norm(rows=n, channels=C, act=s["act"], res=s["act"] if s["res"] == "act" else "f32",
                            post=s["post"] is not None, pre=s["pre"] is not None, gate=s["gate"],
                            center=s["center"], alpha=s["alpha"], eps=s["eps"])
    w = dict(z=s["z"], scale=s["scale"])
    for name in ("post", "pre"):
        if s[name]:
            w[name + "_weight"], w[name + "_bias"] = s[name]
    if s["kind"] == "bn_fwd":
        r, h = ssd.block_norm_forward(p, s["x"], s["y"], **w)
        return {"r": r, "h": h} if s["pre"] else {"r": r}
    g = ssd.block_norm_backward(p, s["x"], s["y"], s["dr"], dh=s["dh"], **w)
    out = {"dx": g.dx, "dscale": g.dscale, "dy": g.dy}
    if s["pre"]:
        out.update(dpre_weight=g.dpre_weight, dpre_bias=g.dpre_bias)
    if s["z"] is not None:
        out["dz"] = g.dz
    if s["post"]:
        out.update(dpost_weight=g.dpost_weight, dpost_bias=g.dpost_bias)
    return out


def _own_rope(s):
    import mamba2_ssd_chunked_amd as ssd
    b, L, H, D = s["q"].shape
    p = ssd.make_rope(batch=b, seqlen=L, nheads=H, nkheads=s["k"].shape[2], headdim=D, rotdim=s["rot"],
                      act=s["act"], style=s["style"], factor=s["factor"])
    call = ssd.rope_forward if s["kind"] == "rope_fwd" else ssd.rope_backward
    q, k = call(p, s["q"], s["k"], s["frequencies"], positions=s["positions"])
    return {"q": q, "k": k}


def run(state):
    kind = state["kind"]
    if own:
        if kind in ("gd_fwd", "gd_bwd"):
            return _own_gd(state)
        if kind == "gd_step":
            return _own_step(state)
        if kind in ("bn_fwd", "bn_bwd"):
            return _own_bn(state)
        return _own_rope(state)
    if kind in ("gd_fwd", "gd_bwd"):
        return _plain_gd(state)
    if kind == "gd_step":
        return _plain_step(state)
    if kind in ("bn_fwd", "bn_bwd"):
        return _plain_bn(state)
    return _plain_rope(state)


# ------------------------------------------------------------------------------ work


def work(case):
    kind = case["kind"]
    e = 2 if case["act"] == "bf16" else 4
    if kind in ("gd_fwd", "gd_bwd"):
        b, L, H, Hk, Dk, Dv = (case[k] for k in ("batch", "tokens", "heads", "kheads", "dk", "dv"))
        T = b * L
        states, gates = _sequences(case) * H * Dk * Dv * 4, T * H * 8
        qk, vo = 2 * T * Hk * Dk * e, 2 * T * H * Dv * e
        if kind == "gd_fwd":  # read q, k, v, the gates (and init), write o and the final state
            return {"bytes": qk + vo + gates + states * (2 if case["init"] else 1),
                    "flops": 6.0 * T * H * Dk * Dv}
        # read q, k, v, do, the gates (and the states), write their gradients
        return {"bytes": 2 * qk + vo * 3 // 2 + 2 * gates + states * (3 if case["init"] else 1),
                "flops": 16.0 * T * H * Dk * Dv}
    if kind == "gd_step":
        n, H, Hk, Dk, Dv = (case[k] for k in ("rows", "heads", "kheads", "dk", "dv"))
        n = n - 3 if n >= 16 else n
        state = n * H * Dk * Dv
        return {"bytes": 8 * state + n * (2 * Hk * Dk + 2 * H * Dv) * e + n * H * 8, "flops": 7.0 * state}
    if kind in ("bn_fwd", "bn_bwd"):
        n = case["rows"] * case["channels"]
        res = e if case["res"] == "act" else 4
        z, pre = case["gate"] != "none", case["pre"]
        if kind == "bn_fwd":  # read x, y, z, write r, h
            return {"bytes": n * (2 * res + e * (1 + z + pre)), "flops": 16.0 * n}
        # read x, y, z, dr, dh, write dx, dy, dz
        return {"bytes": n * (3 * res + e * (2 + 2 * z + pre)), "flops": 40.0 * n}
    n = case["batch"] * case["tokens"] * (case["heads"] + case["kheads"]) * case["dim"]
    return {"bytes": 2 * n * e, "flops": 3.0 * n}


# ----------------------------------------------------------------------------- exact


def _token_rows(s, t):
    """(rows of the sequences' token t, which of them have one)"""
    alive = t < s["lens"]
    return torch.where(alive, s["first"] + t, s["first"]), alive


def _exact_gd(case, s):
    (b, L, H, Dv), (Hk, Dk) = s["v"].shape, s["k"].shape[2:]
    r, scale = H // Hk, s["scale"]
    flat = lambda x: x.flatten(0, 1).double()  # noqa: E731
    q, k = flat(s["q"]).repeat_interleave(r, 1), flat(s["k"]).repeat_interleave(r, 1)
    v, a, beta = flat(s["v"]), torch.exp(flat(s["g"])), flat(s["beta"])
    M = torch.zeros(len(s["lens"]), H, Dv, Dk, dtype=torch.float64, device=q.device)
    if s["init"] is not None:
        M = s["init"].double()

    def step(M, t):
        row, alive = _token_rows(s, t)
        kept = a[row][..., None, None] * M
        miss = v[row] - (kept * k[row][..., None, :]).sum(-1)
        new = kept + (beta[row][..., None] * miss)[..., :, None] * k[row][..., None, :]
        return row, alive, kept, miss, torch.where(alive[:, None, None, None], new, M)

    if case["kind"] == "gd_fwd":
        o = torch.zeros(b * L, H, Dv, dtype=torch.float64, device=q.device)
        for t in range(s["longest"]):
            row, alive, _, _, M = step(M, t)
            o[row[alive]] = scale * (M * q[row][..., None, :]).sum(-1)[alive]
        return {"o": o.reshape(b, L, H, Dv), "final_state": M}
    do = flat(s["do"])
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(v)
    dg, dbeta = torch.zeros_like(a), torch.zeros_like(a)
    G = torch.zeros_like(M) if s.get("dfinal") is None else s["dfinal"].double()
    marks, every = [], 64
    for t in range(s["longest"]):
        if t % every == 0:
            marks.append(M)
        M = step(M, t)[-1]
    for c in range(len(marks) - 1, -1, -1):
        tokens, M = [], marks[c]
        for t in range(c * every, min((c + 1) * every, s["longest"])):
            tokens.append(step(M, t))
            M = tokens[-1][-1]
        for row, alive, kept, miss, M in reversed(tokens):
            D = G + scale * do[row][..., :, None] * q[row][..., None, :]
            du = (D * k[row][..., None, :]).sum(-1)
            w = -beta[row][..., None] * du
            B = D + w[..., :, None] * k[row][..., None, :]  # of the decayed state
            at = row[alive]
            dq[at] = scale * (M * do[row][..., :, None]).sum(-2)[alive]
            dk[at] = ((D * (beta[row][..., None] * miss)[..., :, None]).sum(-2)
                      + (kept * w[..., :, None]).sum(-2))[alive]
            dv[at] = -w[alive]
            dbeta[at] = (du * miss).sum(-1)[alive]
            dg[at] = (B * kept).sum((-1, -2))[alive]
            G = torch.where(alive[:, None, None, None], a[row][..., None, None] * B, G)
    group = lambda x: x.reshape(b, L, Hk, r, Dk).sum(3)  # noqa: E731
    return {"dq": group(dq), "dk": group(dk), "dv": dv.reshape(b, L, H, Dv), "dg": dg.reshape(b, L, H),
            "dbeta": dbeta.reshape(b, L, H), "dinit": G}


def _exact_step(s):
    o, state = s["o"].double(), s["state"].double()
    r = s["v"].shape[2] // s["k"].shape[2]
    for i, slot in enumerate(s["slots"].tolist()):
        if slot < 0:
            continue
        q, k = (s[n][i, 0].double().repeat_interleave(r, 0) for n in ("q", "k"))
        kept = torch.exp(s["g"][i, 0].double())[:, None, None] * state[slot]
        u = s["beta"][i, 0].double()[:, None] * (s["v"][i, 0].double() - (kept * k[:, None, :]).sum(-1))
        state[slot] = kept + u[:, :, None] * k[:, None, :]
        o[i, 0] = s["scale"] * (state[slot] * q[:, None, :]).sum(-1)
    return {"o": o, "state": state}


def _exact_bn(s):
    """The gradients come from differentiating the definition in float64."""
    leaf = lambda t: None if t is None else t.double().requires_grad_(True)  # noqa: E731
    x, y, z, scale = leaf(s["x"]), leaf(s["y"]), leaf(s["z"]), leaf(s["scale"])
    post, pre = ([leaf(t) for t in s[n] or ()] for n in ("post", "pre"))

    def norm(u, w, b):
        mean = u.mean(-1, keepdim=True) if s["center"] else 0.0
        return (u - mean) / torch.sqrt(((u - mean) ** 2).mean(-1, keepdim=True) + s["eps"]) * w + b

    m = norm(y, *post) if post else y
    if z is not None:
        m = m * {"linear": z, "sigmoid": 1 / (1 + torch.exp(-z)), "silu": z / (1 + torch.exp(-z))}[s["gate"]]
    r = s["alpha"] * x + scale * m
    h = norm(r, *pre) if pre else None
    if s["kind"] == "bn_fwd":
        return {"r": r.detach()} if h is None else {"r": r.detach(), "h": h.detach()}
    names = dict(dx=x, dscale=scale, dy=y)
    if pre:
        names.update(dpre_weight=pre[0], dpre_bias=pre[1])
    if z is not None:
        names["dz"] = z
    if post:
        names.update(dpost_weight=post[0], dpost_bias=post[1])
    of, by = ([r], [s["dr"].double()]) if h is None else ([r, h], [s["dr"].double(), s["dh"].double()])
    return dict(zip(names, torch.autograd.grad(of, list(names.values()), by)))


def _exact_rope(s):
    b, L = s["q"].shape[:2]
    pos = torch.arange(L, device=DEV).expand(b, L) if s["positions"] is None else s["positions"]
    angle = pos.double()[..., None, None] * s["frequencies"]
    turn = torch.polar(torch.full_like(angle, s["factor"]), angle if s["kind"] == "rope_fwd" else -angle)
    out = {}
    for name in ("q", "k"):
        x = s[name].double().clone()
        R = s["rot"]
        first, second = ((slice(0, R // 2), slice(R // 2, R)) if s["style"] == "half"
                         else (slice(0, R, 2), slice(1, R, 2)))
        c = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
        x[..., first], x[..., second] = c.real, c.imag
        out[name] = x
    return out


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind in ("gd_fwd", "gd_bwd"):
        return _exact_gd(case, s)
    if kind == "gd_step":
        return _exact_step(s)
    if kind in ("bn_fwd", "bn_bwd"):
        return _exact_bn(s)
    return _exact_rope(s)
