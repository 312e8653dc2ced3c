"""The operators around the scan from their definitions, in float64 on the CPU.

Token by token, head by head, written from the formulas of include/ssd_mixer.h; nothing
here comes from the library.  `sequences` is a list of (first token, length).
"""
from __future__ import annotations

import torch


def f64(t):
    return None if t is None else t.detach().to("cpu", torch.float64)


def linattn_fwd(q, k, v, log_decay, scale, sequences, init=None):
    """(o, final states) for q [T, H, Dk], k, v [T, Hk, .]; rows outside every sequence are 0."""
    q, k, v, init = f64(q), f64(k), f64(v), f64(init)
    T, H, Dk = q.shape
    r, Dv = H // k.shape[1], v.shape[2]
    k, v = k.repeat_interleave(r, 1), v.repeat_interleave(r, 1)
    lam = torch.exp(f64(log_decay))
    o = torch.zeros(T, H, Dv, dtype=torch.float64)
    fin = torch.zeros(len(sequences), H, Dv, Dk, dtype=torch.float64)
    for s, (at, n) in enumerate(sequences):
        S = fin[s] if init is None else init[s].clone()
        for t in range(at, at + n):
            S = lam[:, None, None] * S + v[t][:, :, None] * k[t][:, None, :]
            o[t] = scale * (S * q[t][:, None, :]).sum(-1)
        fin[s] = S
    return o, fin


def linattn_bwd(q, k, v, log_decay, scale, sequences, do, init=None, dfinal=None):
    """(dq, dk, dv, dinit)."""
    q, k, v, do, init, dfinal = (f64(x) for x in (q, k, v, do, init, dfinal))
    T, H, Dk = q.shape
    Hk, Dv = k.shape[1], v.shape[2]
    r = H // Hk
    kr, vr = k.repeat_interleave(r, 1), v.repeat_interleave(r, 1)
    lam = torch.exp(f64(log_decay))[:, None, None]
    dq = torch.zeros(T, H, Dk, dtype=torch.float64)
    dk, dv = torch.zeros_like(dq), torch.zeros(T, H, Dv, dtype=torch.float64)
    dinit = torch.zeros(len(sequences), H, Dv, Dk, dtype=torch.float64)
    for s, (at, n) in enumerate(sequences):
        S = torch.zeros(H, Dv, Dk, dtype=torch.float64) if init is None else init[s].clone()
        for t in range(at, at + n):
            S = lam * S + vr[t][:, :, None] * kr[t][:, None, :]
            dq[t] = scale * (S * do[t][:, :, None]).sum(1)
        G = torch.zeros(H, Dv, Dk, dtype=torch.float64) if dfinal is None else dfinal[s].clone()
        for i, t in enumerate(range(at + n - 1, at - 1, -1)):
            G = (G if i == 0 else lam * G) + scale * do[t][:, :, None] * q[t][:, None, :]
            dv[t] = (G * kr[t][:, None, :]).sum(-1)
            dk[t] = (G * vr[t][:, :, None]).sum(1)
        dinit[s] = lam * G if n else G
    return (dq, dk.reshape(T, Hk, r, Dk).sum(2), dv.reshape(T, Hk, r, Dv).sum(2), dinit)


def token_step(xBC, conv_w, dt_raw, dt_bias, A_log, D, history, state, pos, groups, dt_min,
               dt_max):
    """One sequence's new tokens xBC [n, C] at places pos ..: (y [n, H, P], state).
    `history` [pos, C]: every earlier input, the last W - 1 of which are read."""
    xBC, conv_w, dt_raw, dt_bias, A_log, D = (f64(x) for x in (xBC, conv_w, dt_raw, dt_bias,
                                                               A_log, D))
    S = f64(state).clone()
    H, P, N = S.shape
    W = conv_w.shape[1]
    rows = torch.cat([f64(history), xBC])
    if pos == 0:
        S.zero_()
    y = torch.zeros(len(xBC), H, P, dtype=torch.float64)
    for i in range(len(xBC)):
        u = torch.zeros(xBC.shape[1], dtype=torch.float64)
        for back in range(W):
            if len(rows) - len(xBC) + i - back >= 0 and pos + i - back >= 0:
                u += conv_w[:, W - 1 - back] * rows[len(rows) - len(xBC) + i - back]
        u = u / (1 + torch.exp(-u))
        x = u[:H * P].reshape(H, P)
        B = u[H * P:H * P + groups * N].reshape(groups, N).repeat_interleave(H // groups, 0)
        C = u[H * P + groups * N:].reshape(groups, N).repeat_interleave(H // groups, 0)
        dt = torch.log1p(torch.exp(dt_raw[i] + dt_bias)).clamp(dt_min, dt_max)
        S = torch.exp(-dt * torch.exp(A_log))[:, None, None] * S + (
            dt[:, None, None] * x[:, :, None] * B[:, None, :])
        y[i] = (S * C[:, None, :]).sum(-1) + D[:, None] * x
    return y, S


def norm(x, weight, bias, z, groups, mode, center, eps):
    """The norm of [rows, C] float64 leaves (differentiable)."""
    n, C = x.shape
    gate = None if z is None else z / (1 + torch.exp(-z))
    u = (x * gate if mode == "before" else x).reshape(n, groups, C // groups)
    m = u.mean(-1, keepdim=True) if center else 0.0
    r = 1 / torch.sqrt(((u - m) ** 2).mean(-1, keepdim=True) + eps)
    lin = ((u - m) * r).reshape(n, C) * weight
    if bias is not None:
        lin = lin + bias
    if mode == "after":
        return lin * gate
    return lin / (1 + torch.exp(-lin)) if mode == "silu" else lin
