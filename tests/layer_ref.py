"""The operators of include/ssd_layer.h from their definitions, in float64 on the CPU.

Written from the header's formulas; nothing here comes from the library.  `sequences` is a list of
(first token, length).
"""
from __future__ import annotations

import torch


def f64(t):
    return None if t is None else t.detach().to("cpu", torch.float64)


def gdelta_fwd(q, k, v, g, beta, scale, sequences, init=None):
    """(o, final states, largest |u|, largest state norm) for q, k [T, Hk, Dk], v [T, H, Dv], g and
    beta [T, H]; rows outside every sequence are 0."""
    q, k, v, g, beta, init = (f64(x) for x in (q, k, v, g, beta, init))
    T, H, Dv = v.shape
    r, Dk = H // k.shape[1], k.shape[2]
    q, k = q.repeat_interleave(r, 1), k.repeat_interleave(r, 1)
    o = torch.zeros(T, H, Dv, dtype=torch.float64)
    fin = torch.zeros(len(sequences), H, Dv, Dk, dtype=torch.float64)
    umax = smax = 0.0
    for s, (at, n) in enumerate(sequences):
        S = fin[s] if init is None else init[s].clone()
        smax = max(smax, float(S.flatten(1).norm(dim=1).max()))
        for t in range(at, at + n):
            kept = torch.exp(g[t])[:, None, None] * S
            u = beta[t][:, None] * (v[t] - (kept * k[t][:, None, :]).sum(-1))
            S = kept + u[:, :, None] * k[t][:, None, :]
            o[t] = scale * (S * q[t][:, None, :]).sum(-1)
            umax = max(umax, float(u.abs().max()))
            smax = max(smax, float(S.flatten(1).norm(dim=1).max()))
        fin[s] = S
    return o, fin, umax, smax


def gdelta_bwd(q, k, v, g, beta, scale, sequences, do, init=None, dfinal=None):
    """dict of dq, dk, dv, dg, dbeta, dinit: the adjoint of every token's step."""
    q, k, v, g, beta, do, init, dfinal = (f64(x) for x in (q, k, v, g, beta, do, init, dfinal))
    T, H, Dv = v.shape
    Hk, Dk = k.shape[1:]
    r = H // Hk
    q, k = q.repeat_interleave(r, 1), k.repeat_interleave(r, 1)
    out = dict(dq=torch.zeros_like(q), dk=torch.zeros_like(k), dv=torch.zeros_like(v),
               dg=torch.zeros_like(g), dbeta=torch.zeros_like(g),
               dinit=torch.zeros(len(sequences), H, Dv, Dk, dtype=torch.float64))
    for s, (at, n) in enumerate(sequences):
        S = torch.zeros(H, Dv, Dk, dtype=torch.float64) if init is None else init[s]
        G = torch.zeros_like(S) if dfinal is None else dfinal[s]
        before = []
        for t in range(at, at + n):
            before.append(S)
            kept = torch.exp(g[t])[:, None, None] * S
            u = beta[t][:, None] * (v[t] - (kept * k[t][:, None, :]).sum(-1))
            S = kept + u[:, :, None] * k[t][:, None, :]
        for t in range(at + n - 1, at - 1, -1):
            a = torch.exp(g[t])[:, None, None]
            kept = a * before[t - at]
            miss = v[t] - (kept * k[t][:, None, :]).sum(-1)
            u = beta[t][:, None] * miss
            S = kept + u[:, :, None] * k[t][:, None, :]
            D = G + scale * do[t][:, :, None] * q[t][:, None, :]
            du = (D * k[t][:, None, :]).sum(-1)
            w = beta[t][:, None] * du
            B = D - w[:, :, None] * k[t][:, None, :]
            out["dq"][t] = scale * (S * do[t][:, :, None]).sum(1)
            out["dk"][t] = (D * u[:, :, None]).sum(1) - (kept * w[:, :, None]).sum(1)
            out["dv"][t] = w
            out["dbeta"][t] = (du * miss).sum(-1)
            out["dg"][t] = (B * kept).sum((1, 2))
            G = a * B
        out["dinit"][s] = G
    for name in ("dq", "dk"):
        out[name] = out[name].reshape(T, Hk, r, Dk).sum(2)
    return out


def _norm(u, w, b, center, eps):
    m = u.mean(-1, keepdim=True) if center else 0.0
    n = (u - m) / torch.sqrt(((u - m) ** 2).mean(-1, keepdim=True) + eps)
    return n * w + (0.0 if b is None else b)


def act(kind, z):
    return {"linear": z, "sigmoid": 1 / (1 + torch.exp(-z)), "silu": z / (1 + torch.exp(-z))}[kind]


def block_norm(t, *, gate, center, alpha, eps):
    """(r, h) of float64 tensors t: x, y and what there is of z, scale, post_weight, post_bias,
    pre_weight, pre_bias."""
    u = t["y"]
    if t.get("post_weight") is not None:
        u = _norm(u, t["post_weight"], t.get("post_bias"), center, eps)
    if gate != "none":
        u = u * act(gate, t["z"])
    r = alpha * t["x"] + (1.0 if t.get("scale") is None else t["scale"]) * u
    if t.get("pre_weight") is None:
        return r, None
    return r, _norm(r, t["pre_weight"], t.get("pre_bias"), center, eps)


def rope(x, angles, factor, rotdim, style, inverse):
    """x [..., heads, dim] float64 turned by angles [..., rotdim / 2]."""
    y = x.clone()
    a, b = ((slice(0, rotdim // 2), slice(rotdim // 2, rotdim)) if style == "half"
            else (slice(0, rotdim, 2), slice(1, rotdim, 2)))
    c, s = torch.cos(angles)[..., None, :] * factor, torch.sin(angles)[..., None, :] * factor
    if inverse:
        s = -s
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y
