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
