"""The operators beside the SSD scan, as they are measured: linear attention with a
decay per head (prompts, backward, single tokens), the gated group norm of a mixer's
output (forward, backward) and the SSD scan's single-token step.

Where `own` is false, run() computes them in elementary torch operations in float32
(decay powers in float64, rounded once); where it is true it calls the framework.
exact() is the definition itself, token by token in float64.
"""
import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
CHUNK = 64  # tokens per chunk of the plain chunked form
DT_MIN, DT_MAX = 1e-3, 0.1


def _act(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


# ----------------------------------------------------------------------------- cases


def listed():
    return [
        # forward of a mixer shard's tokens: 2 rows of 8192, 32 heads, 128 key and 64
        # value channels (the SSD shard's state size)
        _la("la_fwd_shard", batch=2, tokens=8192, lo=0, hi=0, heads=32, kv=32, dk=128, dv=64),
        # packed prompts of 512 to 8192 tokens, four heads to a key/value head, q, k and v
        # as views of one projection; every prompt continues from a state
        _la("la_fwd_packed", tokens=32768, lo=512, hi=8192, heads=32, kv=8, dk=128, dv=128,
            fused=True, init=True),
        # a handful of short float32 prompts of odd lengths: latency
        _la("la_fwd_ragged_f32", tokens=256, lo=1, hi=97, heads=4, kv=4, dk=64, dv=64, act="f32",
            init=True),
        # training step of the shard, shared keys and values
        _la("la_bwd_shard", kind="la_bwd", batch=2, tokens=8192, lo=0, hi=0, heads=32, kv=32,
            dk=128, dv=64),
        # training step of a small packed batch of odd lengths with state gradients
        _la("la_bwd_ragged", kind="la_bwd", tokens=1000, lo=1, hi=301, heads=8, kv=2, dk=64, dv=64,
            init=True),
        # one user's next token
        _step("la_step_one", "la_step", rows=1, slots=1, heads=32, kv=32, dk=128, dv=128),
        # a full serving batch with a pool of states, a few rows of padding
        _step("la_step_batch", "la_step", rows=256, slots=300, heads=32, kv=8, dk=128, dv=128),
        # the shard's output norm: y gated by a slice of the input projection, one group
        _norm("norm_fwd_shard", "norm_fwd", rows=16384, channels=2048, groups=1, mode="before"),
        # its backward in training
        _norm("norm_bwd_shard", "norm_bwd", rows=16384, channels=2048, groups=1, mode="before"),
        # a decode batch's per-head norm in float32, centred, odd sizes: latency
        _norm("norm_fwd_heads_f32", "norm_fwd", rows=33, channels=1120, groups=7, mode="after",
              center=True, act="f32"),
        # one user's next token through the SSD mixer core
        _step("ssd_step_one", "ssd_step", rows=1, slots=1, heads=32, kv=1, dk=128, dv=64),
        # a full serving batch, 64 heads in 8 groups
        _step("ssd_step_batch", "ssd_step", rows=256, slots=300, heads=64, kv=8, dk=128, dv=64),
    ]


def _la(name=None, kind="la_fwd", batch=1, tokens=0, lo=0, hi=0, heads=1, kv=1, dk=64, dv=64,
        act="bf16", fused=False, init=False):
    c = dict(kind=kind, batch=batch, tokens=tokens, lo=lo, hi=hi, heads=heads, kv=kv, dk=dk, dv=dv,
             act=act, fused=fused, init=init)
    return dict(c, name=name) if name else c


def _step(name, kind, rows, slots, heads, kv, dk, dv, act="bf16"):
    c = dict(kind=kind, rows=rows, slots=slots, heads=heads, kv=kv, dk=dk, dv=dv, act=act)
    return dict(c, name=name) if name else c


def _norm(name, kind, rows, channels, groups, mode, center=False, act="bf16"):
    c = dict(kind=kind, rows=rows, channels=channels, groups=groups, mode=mode, center=center,
             act=act)
    return dict(c, name=name) if name else c


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    kind = rng.choice(["la_fwd", "la_fwd", "la_bwd", "la_step", "norm_fwd", "norm_bwd", "ssd_step"])
    act = rng.choice(["bf16", "bf16", "f32"])
    if kind in ("la_fwd", "la_bwd"):
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 4])
        dk, dv = rng.choice([64, 128]), rng.choice([64, 128])
        tokens = _log_int(rng, 16, (32768 if kind == "la_fwd" else 12288) // (2 if act == "f32" else 1))
        if rng.random() < 0.4:
            batch = rng.choice([1, 2, 3])
            return _la(None, kind, batch, max(1, tokens // batch), 0, 0, heads, kv, dk, dv, act,
                       rng.random() < 0.5, rng.random() < 0.5)
        hi = _log_int(rng, max(8, tokens // 64), 8192)
        return _la(None, kind, 1, tokens, max(1, hi // 16), hi, heads, kv, dk, dv, act,
                   rng.random() < 0.5, rng.random() < 0.5)
    if kind == "la_step":
        rows = _log_int(rng, 1, 256)
        kv = rng.choice([1, 2, 4, 8])
        return _step(None, kind, rows, rows + rng.randrange(0, 45), kv * rng.choice([1, 2, 4]), kv,
                     rng.choice([64, 128]), rng.choice([64, 128]), act)
    if kind == "ssd_step":
        rows = _log_int(rng, 1, 256)
        kv = rng.choice([1, 2, 4, 8])
        return _step(None, kind, rows, rows + rng.randrange(0, 45), kv * rng.choice([1, 2, 4, 8]),
                     kv, rng.choice([64, 128]), 64, act)
    groups = rng.choice([1, 2, 4, 8, 16, 32])
    width = _log_int(rng, 24, 2048 // groups * 2 if groups > 1 else 2048)
    return _norm(None, kind, _log_int(rng, 1, 8192), groups * width, groups,
                 rng.choice(["before", "after", "silu", "none"]), rng.random() < 0.5, act)


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


def _decays(g, heads):
    """log decays -2^(-8 (h + 1) / H), with some jitter: from half-lives of one token to
    a few hundred."""
    h = torch.arange(1, heads + 1, device=DEV, dtype=torch.float32)
    return -torch.exp2(-8.0 * h / heads) * g.uniform(0.7, 1.3, heads)


def _prepare_la(case, seed):
    g = _Gen(seed)
    act = _act(case["act"])
    b, L, H, Hk, Dk, Dv = (case[k] for k in ("batch", "tokens", "heads", "kv", "dk", "dv"))
    if case["fused"]:  # views of one projection's output rows
        w = [H * Dk, Hk * Dk, Hk * Dv]
        qkv = g.normal(b, L, sum(w), dtype=act)
        q, k, v = (x.unflatten(-1, s) for x, s in zip(qkv.split(w, dim=-1),
                                                      ((H, Dk), (Hk, Dk), (Hk, Dv))))
    else:
        q, k, v = (g.normal(b, L, h, n, dtype=act) for h, n in ((H, Dk), (Hk, Dk), (Hk, Dv)))
    s = dict(kind=case["kind"], q=q, k=k, v=v, log_decay=_decays(g, H), scale=Dk ** -0.5,
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
    # the plain form's plan: every sequence right-aligned in a row of whole chunks
    n = torch.tensor(lens, device=DEV)
    wide = -(-max(lens) // CHUNK) * CHUNK
    first = torch.cumsum(n, 0) - n
    at = torch.arange(wide, device=DEV)[None, :] - (wide - n)[:, None]  # place in the sequence
    s["lens"], s["first"], s["longest"] = n, first, max(lens)
    s["place"] = at
    s["rows"] = torch.where(at >= 0, first[:, None] + at, 0)
    s["rows_rev"] = torch.where(at >= 0, first[:, None] + (n[:, None] - 1 - at), 0)
    if case["init"]:
        s["init"] = g.normal(S, H, Dv, Dk)
    if case["kind"] == "la_bwd":
        s["do"] = g.normal(b, L, H, Dv, dtype=act)
        if case["init"]:
            s["dfinal"] = g.normal(S, H, Dv, Dk)
    return s


def _slots(rows, slots, seed):
    """A slot of the pool for every row; of 16 rows or more, the last three are padding."""
    g = torch.Generator()
    g.manual_seed(int(seed) * 11 + 5)
    ids = torch.randperm(slots, generator=g)[:rows]
    live = rows - 3 if rows >= 16 else rows
    ids[live:] = -1
    return ids.to(torch.int32).to(DEV), live


def _prepare_la_step(case, seed):
    g = _Gen(seed)
    act = _act(case["act"])
    n, H, Hk, Dk, Dv = (case[k] for k in ("rows", "heads", "kv", "dk", "dv"))
    ids, live = _slots(n, case["slots"], seed)
    return dict(kind="la_step", q=g.normal(n, 1, H, Dk, dtype=act), k=g.normal(n, 1, Hk, Dk, dtype=act),
                v=g.normal(n, 1, Hk, Dv, dtype=act), log_decay=_decays(g, H), scale=Dk ** -0.5,
                state=g.normal(case["slots"], H, Dv, Dk), slots=ids, live=live, act=case["act"],
                o=torch.zeros(n, 1, H, Dv, dtype=act, device=DEV))


def _prepare_ssd_step(case, seed):
    g = _Gen(seed)
    act = _act(case["act"])
    n, H, G, N, P = (case[k] for k in ("rows", "heads", "kv", "dk", "dv"))
    C, W = H * P + 2 * G * N, 4
    ids, live = _slots(n, case["slots"], seed)
    gc = torch.Generator()
    gc.manual_seed(int(seed) * 13 + 1)
    pos = torch.randint(1, 100000, (n,), generator=gc)
    pos[::7] = torch.arange(len(pos[::7])) % 3  # some sequences have only begun
    dt0 = torch.exp(g.uniform(math.log(1e-3), math.log(0.1), H))
    return dict(kind="ssd_step", act=case["act"], xBC=g.normal(n, 1, C, dtype=act),
                conv_w=g.normal(C, W, scale=0.5), dt_raw=g.normal(n, 1, H, dtype=act),
                dt_bias=dt0 + torch.log(-torch.expm1(-dt0)), A_log=g.uniform(0.0, math.log(16.0), H),
                D=g.normal(H), conv_ring=g.normal(case["slots"], W, C, dtype=act),
                state=g.normal(case["slots"], H, P, N), slots=ids, live=live,
                positions=pos.to(torch.int32).to(DEV),
                y=torch.zeros(n, 1, H, P, dtype=act, device=DEV), groups=G)


def _prepare_norm(case, seed):
    g = _Gen(seed)
    act = _act(case["act"])
    n, C, mode = case["rows"], case["channels"], case["mode"]
    s = dict(kind=case["kind"], mode=mode, center=case["center"], groups=case["groups"], eps=1e-5,
             act=case["act"], x=g.normal(n, C, dtype=act), z=None,
             weight=1.0 + g.normal(C, scale=0.2), bias=g.normal(C, scale=0.2))
    if mode in ("before", "after"):
        # z is the first part of the input projection's rows, [z | xBC]
        s["z"] = g.normal(n, 2 * C, dtype=act)[:, :C]
    if case["kind"] == "norm_bwd":
        s["dy"] = g.normal(n, C, dtype=act)
    return s


def prepare(case, seed):
    kind = case["kind"]
    if kind in ("la_fwd", "la_bwd"):
        return _prepare_la(case, seed)
    if kind == "la_step":
        return _prepare_la_step(case, seed)
    if kind == "ssd_step":
        return _prepare_ssd_step(case, seed)
    return _prepare_norm(case, seed)


# ---------------------------------------------------------------------- plain forms


def _powers(log_decay, e):
    """exp(log_decay[h])^e[...] for e >= 0, [H, ...] float32 (computed in float64)."""
    ld = log_decay.double().reshape(-1, *([1] * e.dim()))
    return torch.exp(ld * e.double()).float()


def _scan_chunks(q, k, v, s0, log_decay, place, lens, e0):
    """(scan of q, k, v, state after the last token) for padded rows [S, H, wide, D]:
    o_t = S_t q_t with the given first state decayed t + e0 times, S_t = l S_(t-1) +
    v_t k_t^T.  Padding comes first and holds zeros."""
    S, H, wide, Dk = q.shape
    Dv = v.shape[-1]
    n = wide // CHUNK
    q, k, v = (x.reshape(S, H, n, CHUNK, -1) for x in (q, k, v))
    i = torch.arange(CHUNK, device=q.device)
    d = i[:, None] - i[None, :]
    mask = _powers(log_decay, d.clamp(min=0)) * (d >= 0)
    intra = torch.matmul(torch.matmul(q, k.transpose(-1, -2).contiguous()) * mask[None, :, None], v)
    kw = (k * _powers(log_decay, CHUNK - 1 - i)[None, :, None, :, None]).transpose(-1, -2).contiguous()
    own_states = torch.matmul(kw, v).reshape(S, H, n, Dk * Dv)
    c = torch.arange(n, device=q.device)
    gap = c[:, None] - 1 - c[None, :]
    mix = _powers(log_decay, CHUNK * gap.clamp(min=0)) * (gap >= 0)
    entering = torch.matmul(mix[None], own_states).reshape(S, H, n, Dk, Dv)
    inter = torch.matmul(q * _powers(log_decay, i + 1)[None, :, None, :, None], entering)
    o = (intra + inter).reshape(S, H, wide, Dv)
    last = (own_states * _powers(log_decay, CHUNK * (n - 1 - c))[None, :, :, None]).sum(2)
    last = last.reshape(S, H, Dk, Dv)
    if s0 is not None:
        w = _powers(log_decay, place.clamp(min=0) + e0).permute(1, 0, 2)[..., None]
        o = o + torch.matmul(q.reshape(S, H, wide, Dk) * w, s0)
        last = last + s0 * _powers(log_decay, lens - 1 + e0).permute(1, 0)[:, :, None, None]
    return o, last


def _padded(x, rows, place, repeat=1):
    """Token rows [b, L, h, D] as float32 [S, h * repeat, wide, D], zero before the start."""
    x = x.flatten(0, 1).float()[rows] * (place >= 0)[..., None, None]
    x = x.permute(0, 2, 1, 3)
    return x.repeat_interleave(repeat, dim=1) if repeat > 1 else x


def _back(o, s, rows, like):
    """The padded rows' values back at their tokens."""
    out = torch.zeros(like[0] * like[1], *like[2:], device=o.device)
    keep = s["place"] >= 0
    out[rows[keep]] = o.permute(0, 2, 1, 3)[keep]
    return out.reshape(like)


def _t(x):
    return None if x is None else x.transpose(-1, -2).contiguous()


def _plain_la(s):
    act, ld, scale = _act(s["act"]), s["log_decay"], s["scale"]
    (b, L, H, Dk), Hk, Dv = s["q"].shape, s["k"].shape[2], s["v"].shape[3]
    r, plan = H // Hk, (s["place"], s["lens"])
    rows, place = s["rows"], s["place"]
    if s["kind"] == "la_fwd":
        q, k, v = _padded(s["q"], rows, place), _padded(s["k"], rows, place, r), _padded(s["v"], rows, place, r)
        o, last = _scan_chunks(q, k, v, _t(s["init"]), ld, *plan, 1)
        return {"o": _back(o * scale, s, rows, (b, L, H, Dv)).to(act), "final_state": _t(last)}
    # dq: the forward scan of (do, v, k) and the transposed state
    k, v, do = (_padded(s["k"], rows, place, r), _padded(s["v"], rows, place, r),
                _padded(s["do"], rows, place))
    dq, _ = _scan_chunks(do, v, k, s["init"], ld, *plan, 1)
    dq = _back(dq * scale, s, rows, (b, L, H, Dk)).to(act)
    # dv, dk: the scans of (k, q, do) and (v, do, q) from the last token back
    rows = s["rows_rev"]
    q, k, v, do = (_padded(s["q"], rows, place) * scale, _padded(s["k"], rows, place, r),
                   _padded(s["v"], rows, place, r), _padded(s["do"], rows, place))
    dfinal = s.get("dfinal")
    dv, first = _scan_chunks(k, q, do, _t(dfinal), ld, *plan, 0)
    dk, _ = _scan_chunks(v, do, q, dfinal, ld, *plan, 0)
    dv = _back(dv, s, rows, (b, L, H, Dv)).reshape(b, L, Hk, r, Dv).sum(3).to(act)
    dk = _back(dk, s, rows, (b, L, H, Dk)).reshape(b, L, Hk, r, Dk).sum(3).to(act)
    dinit = _t(first) * torch.exp(ld.double()).float()[None, :, None, None]
    return {"dq": dq, "dk": dk, "dv": dv, "dinit": dinit}


def _plain_la_step(s):
    live, H = s["live"], s["q"].shape[2]
    r = H // s["k"].shape[2]
    at = s["slots"][:live].long()
    q = s["q"][:live, 0].float()
    k = s["k"][:live, 0].float().repeat_interleave(r, dim=1)
    v = s["v"][:live, 0].float().repeat_interleave(r, dim=1)
    new = (s["state"][at] * torch.exp(s["log_decay"])[None, :, None, None]
           + v[..., :, None] * k[..., None, :])
    s["state"][at] = new
    s["o"][:live, 0] = ((new * q[..., None, :]).sum(-1) * s["scale"]).to(s["o"].dtype)
    return {"o": s["o"], "state": s["state"]}


def _plain_ssd_step(s):
    live, G, W = s["live"], s["groups"], s["conv_w"].shape[1]
    H, P, N = s["state"].shape[1:]
    R, C = s["conv_ring"].shape[1:]
    at, pos = s["slots"][:live].long(), s["positions"][:live].long()
    x = s["xBC"][:live, 0]
    s["conv_ring"][at, pos % R] = x
    back = torch.arange(W - 1, -1, -1, device=x.device)  # tap kk reads the token W - 1 - kk back
    src = pos[:, None] - back[None, :]
    taps = s["conv_ring"][at[:, None], src % R].float() * (src >= 0)[..., None]  # [n, W, C]
    u = (taps * s["conv_w"].t()[None]).sum(1)
    u = u * torch.sigmoid(u)
    xs = u[:, :H * P].reshape(live, H, P)
    B = u[:, H * P:H * P + G * N].reshape(live, G, N).repeat_interleave(H // G, dim=1)
    Cc = u[:, H * P + G * N:].reshape(live, G, N).repeat_interleave(H // G, dim=1)
    zz = s["dt_raw"][:live, 0].float() + s["dt_bias"]
    dt = (zz.clamp(min=0) + torch.log1p(torch.exp(-zz.abs()))).clamp(DT_MIN, DT_MAX)
    a = torch.exp(-dt * torch.exp(s["A_log"])) * (pos > 0)[:, None]
    new = s["state"][at] * a[..., None, None] + (dt[..., None] * xs)[..., None] * B[:, :, None, :]
    s["state"][at] = new
    y = (new * Cc[:, :, None, :]).sum(-1) + s["D"][None, :, None] * xs
    s["y"][:live, 0] = y.to(s["y"].dtype)
    return {"y": s["y"], "state": s["state"], "conv_ring": s["conv_ring"]}


def _norm_parts(s, dtype):
    n, C = s["x"].shape
    G = s["groups"]
    x = s["x"].to(dtype)
    sig = act = None
    if s["z"] is not None:
        z = s["z"].to(dtype)
        sig = torch.sigmoid(z)
        act = z * sig
    u = x * act if s["mode"] == "before" else x
    ug = u.reshape(n, G, C // G)
    if s["center"]:
        ug = ug - ug.mean(-1, keepdim=True)
    rstd = torch.rsqrt(ug.square().mean(-1, keepdim=True) + s["eps"])
    xh = (ug * rstd).reshape(n, C)
    return x, sig, act, xh, rstd, xh * s["weight"].to(dtype) + s["bias"].to(dtype)


def _norm_fwd(s, dtype):
    _, _, act, _, _, lin = _norm_parts(s, dtype)
    if s["mode"] == "after":
        return lin * act
    return lin * torch.sigmoid(lin) if s["mode"] == "silu" else lin


def _norm_bwd(s, dtype):
    x, sig, act, xh, rstd, lin = _norm_parts(s, dtype)
    n, C = x.shape
    G, mode = s["groups"], s["mode"]
    dy = s["dy"].to(dtype)
    dz = None
    if sig is not None:
        dsilu = sig * (1 + s["z"].to(dtype) * (1 - sig))
    if mode == "after":
        dz = dy * lin * dsilu
        dy = dy * act
    elif mode == "silu":
        g = torch.sigmoid(lin)
        dy = dy * g * (1 + lin * (1 - g))
    dw, db = (dy * xh).sum(0), dy.sum(0)
    gh = (dy * s["weight"].to(dtype)).reshape(n, G, C // G)
    xg = xh.reshape(n, G, C // G)
    du = gh - xg * (gh * xg).mean(-1, keepdim=True)
    if s["center"]:
        du = du - gh.mean(-1, keepdim=True)
    du = (du * rstd).reshape(n, C)
    dx = du
    if mode == "before":
        dx, dz = du * act, du * x * dsilu
    return dx, dz, dw, db


def _plain_norm(s):
    act = _act(s["act"])
    if s["kind"] == "norm_fwd":
        return {"y": _norm_fwd(s, torch.float32).to(act)}
    dx, dz, dw, db = _norm_bwd(s, torch.float32)
    out = {"dx": dx.to(act), "dweight": dw, "dbias": db}
    return out if dz is None else dict(out, dz=dz.to(act))


# ------------------------------------------------------------------ the framework's


def _own_la(s):
    import mamba2_ssd_chunked_amd as ssd
    (b, L, H, Dk), Hk, Dv = s["q"].shape, s["k"].shape[2], s["v"].shape[3]
    p = ssd.make_linattn(batch=b, seqlen=L, nheads=H, nkvheads=Hk, keydim=Dk, valdim=Dv,
                         act=s["act"], scale=s["scale"])
    if s["kind"] == "la_fwd":
        f = ssd.linattn_forward(p, s["q"], s["k"], s["v"], s["log_decay"], cu_seqlens=s["cu"],
                                init=s["init"], want_final=True)
        return {"o": f.o, "final_state": f.final_state}
    g = ssd.linattn_backward(p, s["q"], s["k"], s["v"], s["log_decay"], s["do"],
                             cu_seqlens=s["cu"], init=s["init"], dfinal=s.get("dfinal"),
                             want_dinit=True)
    return {"dq": g.dq, "dk": g.dk, "dv": g.dv, "dinit": g.dinit}


def _own_la_step(s):
    import mamba2_ssd_chunked_amd as ssd
    n, H, Dk = s["q"].shape[0], s["q"].shape[2], s["q"].shape[3]
    p = ssd.make_linattn(batch=n, seqlen=1, nheads=H, nkvheads=s["k"].shape[2], keydim=Dk,
                         valdim=s["v"].shape[3], act=s["act"], scale=s["scale"])
    ssd.ssd_linattn_step(p, s["q"], s["k"], s["v"], s["log_decay"], s["state"], s["o"],
                         slots=s["slots"])
    return {"o": s["o"], "state": s["state"]}


def _own_ssd_step(s):
    import mamba2_ssd_chunked_amd as ssd
    H, P, N = s["state"].shape[1:]
    p = ssd.make_problem(batch=s["xBC"].shape[0], seqlen=1, nheads=H, headdim=P, dstate=N,
                         ngroups=s["groups"], chunk=64, conv_width=s["conv_w"].shape[1],
                         act=s["act"], dt_min=DT_MIN, dt_max=DT_MAX)
    ssd.ssd_token_step(p, s["xBC"], s["conv_w"], s["dt_raw"], s["dt_bias"], s["A_log"], s["D"],
                       s["conv_ring"], s["state"], s["positions"], s["y"], slots=s["slots"])
    return {"y": s["y"], "state": s["state"], "conv_ring": s["conv_ring"]}


def _own_norm(s):
    import mamba2_ssd_chunked_amd as ssd
    n, C = s["x"].shape
    p = ssd.make_norm(rows=n, channels=C, ngroups=s["groups"], act=s["act"], mode=s["mode"],
                      center=s["center"], eps=s["eps"])
    if s["kind"] == "norm_fwd":
        return {"y": ssd.norm_forward(p, s["x"], s["weight"], bias=s["bias"], z=s["z"])}
    g = ssd.norm_backward(p, s["x"], s["weight"], s["dy"], bias=s["bias"], z=s["z"])
    out = {"dx": g.dx, "dweight": g.dweight, "dbias": g.dbias}
    return out if g.dz is None else dict(out, dz=g.dz)


def run(state):
    kind = state["kind"]
    if own:
        if kind in ("la_fwd", "la_bwd"):
            return _own_la(state)
        if kind == "la_step":
            return _own_la_step(state)
        if kind == "ssd_step":
            return _own_ssd_step(state)
        return _own_norm(state)
    if kind in ("la_fwd", "la_bwd"):
        return _plain_la(state)
    if kind == "la_step":
        return _plain_la_step(state)
    if kind == "ssd_step":
        return _plain_ssd_step(state)
    return _plain_norm(state)


# ------------------------------------------------------------------------------ work


def work(case):
    kind = case["kind"]
    e = 2 if case["act"] == "bf16" else 4
    if kind in ("la_fwd", "la_bwd"):
        b, L, H, Hk, Dk, Dv = (case[k] for k in ("batch", "tokens", "heads", "kv", "dk", "dv"))
        T = b * L
        states = _sequences(case) * H * Dk * Dv * 4
        qo, kv = T * H * (Dk + Dv) * e, T * Hk * (Dk + Dv) * e
        if kind == "la_fwd":  # read q, k, v (and init), write o and the final state
            return {"bytes": qo + kv + states * (2 if case["init"] else 1),
                    "flops": 4.0 * T * H * Dk * Dv}
        # read q, do, k, v (and the states), write dq, dk, dv and dinit
        return {"bytes": qo + T * H * Dk * e + 2 * kv + states * (3 if case["init"] else 1),
                "flops": 10.0 * T * H * Dk * Dv}
    if kind in ("la_step", "ssd_step"):
        n, H, G, Dk, Dv = (case[k] for k in ("rows", "heads", "kv", "dk", "dv"))
        n = n - 3 if n >= 16 else n
        state = n * H * Dk * Dv
        if kind == "la_step":
            return {"bytes": 8 * state + n * (H + G) * (Dk + Dv) * e, "flops": 5.0 * state}
        C = H * Dv + 2 * G * Dk
        return {"bytes": 8 * state + n * (C * 5 + H + H * Dv) * e, "flops": 5.0 * state}
    n = case["rows"] * case["channels"]
    gated = case["mode"] in ("before", "after")
    if kind == "norm_fwd":
        return {"bytes": n * e * (3 if gated else 2), "flops": 8.0 * n}
    return {"bytes": n * e * (5 if gated else 3), "flops": 20.0 * n}


# ----------------------------------------------------------------------------- exact


def _walk_tokens(a, b, c, state, decay, first, lens, longest, back, late):
    """Token by token in float64, all sequences at once: M <- decay M + c_t b_t^T, out_t =
    M a_t, from the last token where `back`; with `late` the given state is not decayed
    before its first use."""
    T, H, Da = a.shape
    out = torch.zeros(T, H, c.shape[-1], dtype=torch.float64, device=a.device)
    M = state
    for t in range(longest):
        alive = t < lens
        row = first + (lens - 1 - t if back else t)
        row = torch.where(alive, row, first)
        keep = 1.0 if late and t == 0 else decay[None, :, None, None]
        new = M * keep + c[row][..., :, None] * b[row][..., None, :]
        M = torch.where(alive[:, None, None, None], new, M)
        o = (M * a[row][..., None, :]).sum(-1)
        out[row[alive]] = o[alive]
    return out, M


def _exact_la(case, s):
    (b, L, H, Dk), Hk, Dv = s["q"].shape, s["k"].shape[2], s["v"].shape[3]
    r, S = H // Hk, len(s["lens"])
    flat = lambda x: x.flatten(0, 1).double()  # noqa: E731
    q, k, v = flat(s["q"]), flat(s["k"]).repeat_interleave(r, 1), flat(s["v"]).repeat_interleave(r, 1)
    decay = torch.exp(s["log_decay"].double())
    zero = torch.zeros(S, H, Dv, Dk, dtype=torch.float64, device=q.device)
    S0 = zero if s["init"] is None else s["init"].double()
    seqs = (s["first"], s["lens"], s["longest"])
    if case["kind"] == "la_fwd":
        o, last = _walk_tokens(q, k, v, S0, decay, *seqs, False, False)
        return {"o": (o * s["scale"]).reshape(b, L, H, Dv), "final_state": last}
    do = flat(s["do"])
    qs = q * s["scale"]
    G0 = zero if s.get("dfinal") is None else s["dfinal"].double()
    St = S0.transpose(-1, -2).contiguous()
    dq, _ = _walk_tokens(do * s["scale"], v, k, St, decay, *seqs, False, False)
    dv, G = _walk_tokens(k, qs, do, G0, decay, *seqs, True, True)
    dk, _ = _walk_tokens(v, do, qs, G0.transpose(-1, -2).contiguous(), decay, *seqs, True, True)
    return {"dq": dq.reshape(b, L, H, Dk), "dk": dk.reshape(b, L, Hk, r, Dk).sum(3),
            "dv": dv.reshape(b, L, Hk, r, Dv).sum(3), "dinit": G * decay[None, :, None, None]}


def _exact_la_step(s):
    o, state = s["o"].double(), s["state"].double()
    r = s["q"].shape[2] // s["k"].shape[2]
    decay = torch.exp(s["log_decay"].double())
    for i, slot in enumerate(s["slots"].tolist()):
        if slot < 0:
            continue
        k, v = (s[n][i, 0].double().repeat_interleave(r, 0) for n in ("k", "v"))
        state[slot] = state[slot] * decay[:, None, None] + v[:, :, None] * k[:, None, :]
        o[i, 0] = s["scale"] * (state[slot] * s["q"][i, 0].double()[:, None, :]).sum(-1)
    return {"o": o, "state": state}


def _exact_ssd_step(s):
    y, state, ring = s["y"].double(), s["state"].double(), s["conv_ring"].double()
    H, P, N = state.shape[1:]
    G, W, R = s["groups"], s["conv_w"].shape[1], ring.shape[1]
    w, A = s["conv_w"].double(), -torch.exp(s["A_log"].double())
    where = zip(s["slots"].tolist(), s["positions"].tolist())
    for i, (slot, pos) in enumerate(where):
        if slot < 0:
            continue
        x = s["xBC"][i, 0].double()
        u = w[:, W - 1] * x
        for back in range(1, min(W, pos + 1)):
            u = u + w[:, W - 1 - back] * ring[slot, (pos - back) % R]
        ring[slot, pos % R] = x
        u = u / (1 + torch.exp(-u))
        xs = u[:H * P].reshape(H, P)
        B, C = (u[H * P + o * G * N:H * P + (o + 1) * G * N].reshape(G, N).repeat_interleave(H // G, 0)
                for o in (0, 1))
        dt = torch.nn.functional.softplus(s["dt_raw"][i, 0].double() + s["dt_bias"].double())
        dt = dt.clamp(DT_MIN, DT_MAX)
        old = state[slot] * torch.exp(dt * A)[:, None, None] if pos > 0 else 0.0
        state[slot] = old + (dt[:, None] * xs)[:, :, None] * B[:, None, :]
        y[i, 0] = (state[slot] * C[:, None, :]).sum(-1) + s["D"].double()[:, None] * xs
    return {"y": y, "state": state, "conv_ring": ring}


def _exact_norm(s):
    """The gradients come from differentiating the definition in float64."""
    leaf = lambda t: None if t is None else t.double().requires_grad_(True)  # noqa: E731
    x, z, w, b = leaf(s["x"]), leaf(s["z"]), leaf(s["weight"]), leaf(s["bias"])
    n, C = x.shape
    gate = None if z is None else z / (1 + torch.exp(-z))
    u = (x * gate if s["mode"] == "before" else x).reshape(n, s["groups"], -1)
    mean = u.mean(-1, keepdim=True) if s["center"] else 0.0
    second = ((u - mean) ** 2).mean(-1, keepdim=True)
    lin = ((u - mean) / torch.sqrt(second + s["eps"])).reshape(n, C) * w + b
    y = lin
    if s["mode"] == "after":
        y = lin * gate
    elif s["mode"] == "silu":
        y = lin / (1 + torch.exp(-lin))
    if s["kind"] == "norm_fwd":
        return {"y": y.detach()}
    leaves = [t for t in (x, w, b, z) if t is not None]
    got = torch.autograd.grad(y, leaves, s["dy"].double())
    out = {"dx": got[0], "dweight": got[1], "dbias": got[2]}
    return out if z is None else dict(out, dz=got[3])


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind in ("la_fwd", "la_bwd"):
        return _exact_la(case, s)
    if kind == "la_step":
        return _exact_la_step(s)
    if kind == "ssd_step":
        return _exact_ssd_step(s)
    return _exact_norm(s)
