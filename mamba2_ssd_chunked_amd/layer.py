"""Python binding of include/ssd_layer.h: more operators of a layer around a recurrent mixer.

  gdelta_forward / gdelta_backward / ssd_gdelta_step   the gated delta rule: a state with a
      decay and an update rate per token and head; prompts, their gradients, single tokens
  block_norm_forward / block_norm_backward             the norms before and after a block with
      its gate and residual scale
  rope_forward / rope_backward / rope_frequencies      rotary positions of queries and keys

Checks, streams and buffers are those of mixer.py.
"""
from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass
from typing import Optional, Tuple

import torch

from ._lib import (SSD_GATE_LINEAR, SSD_GATE_NONE, SSD_GATE_SIGMOID, SSD_GATE_SILU, SSD_ROPE_HALF,
                   SSD_ROPE_INTERLEAVED, SSD_WS_BACKWARD, SSD_WS_FORWARD, BlockNorm, GatedDelta, Rope,
                   SSDError)
from .mixer import _TORCH_ACT, _act_code, _Args, _entry, _made_for, _new_states, _nseq, _state_shape

_GATE = {"none": SSD_GATE_NONE, "linear": SSD_GATE_LINEAR, "sigmoid": SSD_GATE_SIGMOID,
         "silu": SSD_GATE_SILU}
_STYLE = {"half": SSD_ROPE_HALF, "interleaved": SSD_ROPE_INTERLEAVED}

# --------------------------------------------------------------------- gated delta rule


def make_gdelta(*, batch: int, seqlen: int, nheads: int, keydim: int, valdim: int, act: str | int,
                nkheads: Optional[int] = None, scale: Optional[float] = None) -> GatedDelta:
    """Sizes of a gated delta rule: `nheads` heads of values, gates and states over `nkheads`
    (default: as many) heads of queries and keys; scale defaults to keydim ** -0.5."""
    return GatedDelta(batch, seqlen, nheads, nheads if nkheads is None else nkheads, keydim, valdim,
                      _act_code(act), keydim ** -0.5 if scale is None else scale)


def _gate_rows(a: _Args, t, name, p: GatedDelta):
    """(pointer, elements between tokens; 0 packed) of float32 rows [batch, tokens, nheads]."""
    act, a.act = a.act, torch.float32
    try:
        return a.tokens(t, name, (p.batch, p.seqlen, p.nheads))
    finally:
        a.act = act


def _gd_inputs(a: _Args, p: GatedDelta, c: GatedDelta, q, k, v, g, beta):
    """Pointers of the tokens' inputs; their strides go into `c`."""
    b, L, H, K, Dk, Dv = p.batch, p.seqlen, p.nheads, p.nkheads, p.keydim, p.valdim
    qp, c.q_stride = a.tokens(q, "q", (b, L, K, Dk))
    kp, c.k_stride = a.tokens(k, "k", (b, L, K, Dk))
    vp, c.v_stride = a.tokens(v, "v", (b, L, H, Dv))
    gp, c.g_stride = _gate_rows(a, g, "g", p)
    bp, c.beta_stride = _gate_rows(a, beta, "beta", p)
    return qp, kp, vp, gp, bp


def ssd_gdelta_workspace_bytes(problem: GatedDelta, nseq: int, kind: int = SSD_WS_FORWARD) -> int:
    return int(_entry("ssd_gdelta_workspace_bytes")(ctypes.byref(problem), nseq, kind))


def ssd_gdelta_fwd(problem: GatedDelta, q, k, v, g, beta, cu_seqlens, init, o, final_state, ws,
                   stream=None):
    p, n = problem, _nseq(problem, cu_seqlens)
    a, c = _Args(p.act_dtype), GatedDelta.from_buffer_copy(p)  # the caller's stays as it is
    ins = _gd_inputs(a, p, c, q, k, v, g, beta)
    op, c.o_stride = a.tokens(o, "o", (p.batch, p.seqlen, p.nheads, p.valdim))
    cu = a.flat(cu_seqlens, "cu_seqlens", (n + 1,), torch.int32, optional=True)
    ini = a.flat(init, "init", _state_shape(p, n), optional=True)
    fin = a.flat(final_state, "final_state", _state_shape(p, n), optional=True)
    wp, wn = a.scratch(ws, "ws")
    a.call("ssd_gdelta_fwd", stream, ctypes.byref(c), n, *ins, cu, ini, op, fin, wp, wn)


def ssd_gdelta_bwd(problem: GatedDelta, q, k, v, g, beta, cu_seqlens, do, init, dfinal, dq, dk, dv,
                   dg, dbeta, dinit, ws, stream=None):
    p, n = problem, _nseq(problem, cu_seqlens)
    a, c = _Args(p.act_dtype), GatedDelta.from_buffer_copy(p)
    b, L, H, K, Dk, Dv = p.batch, p.seqlen, p.nheads, p.nkheads, p.keydim, p.valdim
    ins = _gd_inputs(a, p, c, q, k, v, g, beta)
    dop, c.o_stride = a.tokens(do, "do", (b, L, H, Dv))
    dqp, c.dq_stride = a.tokens(dq, "dq", (b, L, K, Dk))
    dkp, c.dk_stride = a.tokens(dk, "dk", (b, L, K, Dk))
    dvp, c.dv_stride = a.tokens(dv, "dv", (b, L, H, Dv))
    dgp, dbp = a.flat(dg, "dg", (b, L, H)), a.flat(dbeta, "dbeta", (b, L, H))
    cu = a.flat(cu_seqlens, "cu_seqlens", (n + 1,), torch.int32, optional=True)
    st = _state_shape(p, n)
    ini, dfin = a.flat(init, "init", st, optional=True), a.flat(dfinal, "dfinal", st, optional=True)
    dini = a.flat(dinit, "dinit", st, optional=True)
    wp, wn = a.scratch(ws, "ws")
    a.call("ssd_gdelta_bwd", stream, ctypes.byref(c), n, *ins, cu, dop, ini, dfin, dqp, dkp, dvp,
           dgp, dbp, dini, wp, wn)


def ssd_gdelta_step(problem: GatedDelta, q, k, v, g, beta, state, o, slots=None, positions=None,
                    stream=None):
    """The next `seqlen` tokens (1, or a few) of `batch` rows; `state` [slots, H, valdim,
    keydim] float32 is updated in place, `slots` [batch] int32 says where each row's is, and a
    row at position 0 (`positions` [batch] int32) starts from zero."""
    p = problem
    a, c = _Args(p.act_dtype), GatedDelta.from_buffer_copy(p)
    ins = _gd_inputs(a, p, c, q, k, v, g, beta)
    op, c.o_stride = a.tokens(o, "o", (p.batch, p.seqlen, p.nheads, p.valdim))
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state must have shape (slots, nheads, valdim, keydim)")
    sp = a.flat(state, "state", _state_shape(p, state.shape[0]))
    sl = a.flat(slots, "slots", (p.batch,), torch.int32, optional=True)
    po = a.flat(positions, "positions", (p.batch,), torch.int32, optional=True)
    a.call("ssd_gdelta_step", stream, ctypes.byref(c), *ins, sl, state.shape[0], po, sp, op)


def _gd_workspace(p: GatedDelta, nseq: int, kind: int, device):
    n = ssd_gdelta_workspace_bytes(p, nseq, kind)
    if n == 0:
        raise SSDError("ssd_gdelta_workspace_bytes", -2)
    return torch.empty(n, dtype=torch.uint8, device=device)


@dataclass
class GatedDeltaForwardBuffers:
    o: torch.Tensor
    final_state: Optional[torch.Tensor]  # [nseq][H][valdim][keydim] float32
    ws: torch.Tensor

    @staticmethod
    def allocate(problem: GatedDelta, nseq: int, device, final: bool = True) -> "GatedDeltaForwardBuffers":
        """Buffers of gdelta_forward; without `final` they have no final_state."""
        p = problem
        ws = _gd_workspace(p, nseq, SSD_WS_FORWARD, device)
        return GatedDeltaForwardBuffers(
            o=torch.empty((p.batch, p.seqlen, p.nheads, p.valdim), dtype=_TORCH_ACT[p.act_dtype],
                          device=device),
            final_state=_new_states(p, nseq, device) if final else None, ws=ws)


def gdelta_forward(problem: GatedDelta, q, k, v, g, beta, cu_seqlens=None, init=None,
                   bufs: Optional[GatedDeltaForwardBuffers] = None, stream=None,
                   want_final: bool = False) -> GatedDeltaForwardBuffers:
    """o = scale S_t q_t with S_t = a_t S_(t-1) + u_t k_t^T, u_t = beta_t (v_t - a_t S_(t-1) k_t)
    and a_t = exp(g_t); returns the buffers.

    q, k [b, L, nkheads, keydim], v [b, L, H, valdim], g and beta [b, L, H] float32; every row
    is a sequence, or with cu_seqlens (int32 [nseq + 1], b = 1) the packed sequences are.
    init       : optional [nseq, H, valdim, keydim] float32 states before the sequences.
    want_final : also write bufs.final_state (None in buffers made here without it).
    Rows of bufs.o outside every sequence are left as they were.
    """
    if bufs is None:
        bufs = GatedDeltaForwardBuffers.allocate(problem, _nseq(problem, cu_seqlens), q.device,
                                                 final=want_final)
        _made_for(stream, q.device, bufs.o, bufs.final_state, bufs.ws)
    elif want_final and bufs.final_state is None:
        raise ValueError("the buffers have no final_state")
    ssd_gdelta_fwd(problem, q, k, v, g, beta, cu_seqlens, init, bufs.o,
                   bufs.final_state if want_final else None, bufs.ws, stream)
    return bufs


@dataclass
class GatedDeltaBackwardBuffers:
    dq: torch.Tensor
    dk: torch.Tensor
    dv: torch.Tensor
    dg: torch.Tensor     # [b][L][H] float32
    dbeta: torch.Tensor  # [b][L][H] float32
    dinit: Optional[torch.Tensor]  # [nseq][H][valdim][keydim] float32
    ws: torch.Tensor

    @staticmethod
    def allocate(problem: GatedDelta, nseq: int, device, dinit: bool = True) -> "GatedDeltaBackwardBuffers":
        """Buffers of gdelta_backward; without `dinit` they have none."""
        p = problem
        ws = _gd_workspace(p, nseq, SSD_WS_BACKWARD, device)
        new = lambda *s, dtype=_TORCH_ACT[p.act_dtype]: torch.empty((p.batch, p.seqlen, *s), dtype=dtype,  # noqa: E731
                                                                    device=device)
        return GatedDeltaBackwardBuffers(
            dq=new(p.nkheads, p.keydim), dk=new(p.nkheads, p.keydim), dv=new(p.nheads, p.valdim),
            dg=new(p.nheads, dtype=torch.float32), dbeta=new(p.nheads, dtype=torch.float32),
            dinit=_new_states(p, nseq, device) if dinit else None, ws=ws)


def gdelta_backward(problem: GatedDelta, q, k, v, g, beta, do, cu_seqlens=None, init=None,
                    dfinal=None, bufs: Optional[GatedDeltaBackwardBuffers] = None, stream=None,
                    want_dinit: bool = False) -> GatedDeltaBackwardBuffers:
    """Gradients of gdelta_forward (its inputs, `init` included, given again); returns the
    buffers.

    dfinal     : optional gradient of the final states.
    want_dinit : also write bufs.dinit, the gradient of `init` (None in buffers made here
                 without it).
    """
    if bufs is None:
        bufs = GatedDeltaBackwardBuffers.allocate(problem, _nseq(problem, cu_seqlens), q.device,
                                                  dinit=want_dinit)
        _made_for(stream, q.device, bufs.dq, bufs.dk, bufs.dv, bufs.dg, bufs.dbeta, bufs.dinit, bufs.ws)
    elif want_dinit and bufs.dinit is None:
        raise ValueError("the buffers have no dinit")
    ssd_gdelta_bwd(problem, q, k, v, g, beta, cu_seqlens, do, init, dfinal, bufs.dq, bufs.dk, bufs.dv,
                   bufs.dg, bufs.dbeta, bufs.dinit if want_dinit else None, bufs.ws, stream)
    return bufs


# ------------------------------------------------------------------ norms around a block


def make_block_norm(*, rows: int, channels: int, act: str | int, res: str | int | None = None,
                    post: bool = True, pre: bool = True, gate: str | int = "none",
                    center: bool = False, alpha: float = 1.0, eps: float = 1e-5) -> BlockNorm:
    """The norms around a block: `post` of what the block gives, `pre` of the residual stream before
    the next block; gate: "none", "linear", "sigmoid" or "silu" of z; alpha: factor of the residual
    stream x, whose type is `res` (default: act)."""
    act = _act_code(act)
    return BlockNorm(rows, channels, act, act if res is None else _act_code(res), int(bool(post)),
                     int(bool(pre)), _GATE[gate] if isinstance(gate, str) else gate,
                     int(bool(center)), alpha, eps)


def _block_rows(a: _Args, t, name, rows: int, channels: int, dtype):
    """(pointer, elements between rows; 0 packed) of [rows, channels] with contiguous channels."""
    a._base(t, name, dtype, (rows, channels))
    if t.is_contiguous():
        return t.data_ptr(), 0
    if channels > 1 and t.stride(1) != 1:
        raise ValueError(f"the channels of a row of {name} must be contiguous")
    step = t.stride(0) if rows > 1 else channels
    if step < channels:
        raise ValueError(f"the rows of {name} overlap")
    return t.data_ptr(), step


def _block_vectors(a: _Args, p: BlockNorm, z, scale, post_weight, post_bias, pre_weight, pre_bias):
    """Pointers of the channels' vectors; what the problem has no use for is refused."""
    if not p.post and (post_weight is not None or post_bias is not None):
        raise ValueError("the problem has no use for post_weight and post_bias")
    if not p.pre and (pre_weight is not None or pre_bias is not None):
        raise ValueError("the problem has no use for pre_weight and pre_bias")
    if not p.gate and z is not None:
        raise ValueError("the problem has no use for z")
    C, f = (p.channels,), a.flat
    return (None if scale is None else f(scale, "scale", C),
            f(post_weight, "post_weight", C) if p.post else None,
            None if post_bias is None else f(post_bias, "post_bias", C),
            f(pre_weight, "pre_weight", C) if p.pre else None,
            None if pre_bias is None else f(pre_bias, "pre_bias", C))


def ssd_block_norm_fwd(problem: BlockNorm, x, y, z, scale, post_weight, post_bias, pre_weight, pre_bias,
                       r, h, stream=None):
    p, n, C = problem, problem.rows, problem.channels
    a, c, res = _Args(p.act_dtype), BlockNorm.from_buffer_copy(p), _TORCH_ACT[p.res_dtype]
    xp, c.x_stride = _block_rows(a, x, "x", n, C, res)
    yp, c.y_stride = _block_rows(a, y, "y", n, C, a.act)
    vectors = _block_vectors(a, p, z, scale, post_weight, post_bias, pre_weight, pre_bias)
    zp, c.z_stride = _block_rows(a, z, "z", n, C, a.act) if p.gate else (None, 0)
    rp, c.r_stride = _block_rows(a, r, "r", n, C, res)
    if not p.pre and h is not None:
        raise ValueError("the problem has no use for h")
    hp, c.h_stride = _block_rows(a, h, "h", n, C, a.act) if p.pre else (None, 0)
    a.call("ssd_block_norm_fwd", stream, ctypes.byref(c), xp, yp, zp, *vectors, rp, hp)


def ssd_block_norm_workspace_bytes(problem: BlockNorm) -> int:
    return int(_entry("ssd_block_norm_workspace_bytes")(ctypes.byref(problem)))


def ssd_block_norm_bwd(problem: BlockNorm, x, y, z, scale, post_weight, post_bias, pre_weight, dr, dh,
                       dx, dy, dz, dscale, dpost_weight, dpost_bias, dpre_weight, dpre_bias, ws,
                       stream=None):
    p, n, C = problem, problem.rows, problem.channels
    a, c, res = _Args(p.act_dtype), BlockNorm.from_buffer_copy(p), _TORCH_ACT[p.res_dtype]
    xp, c.x_stride = _block_rows(a, x, "x", n, C, res)
    yp, c.y_stride = _block_rows(a, y, "y", n, C, a.act)
    vectors = _block_vectors(a, p, z, scale, post_weight, post_bias, pre_weight, None)[:-1]
    zp, c.z_stride = _block_rows(a, z, "z", n, C, a.act) if p.gate else (None, 0)
    if dr is None and not p.pre:
        raise ValueError("dr is required")
    drp, c.r_stride = (None, 0) if dr is None else _block_rows(a, dr, "dr", n, C, res)
    if not p.pre and dh is not None:
        raise ValueError("the problem has no use for dh")
    dhp, c.h_stride = _block_rows(a, dh, "dh", n, C, a.act) if p.pre else (None, 0)
    dxp, c.dx_stride = _block_rows(a, dx, "dx", n, C, res)
    dyp, c.dy_stride = _block_rows(a, dy, "dy", n, C, a.act)
    dzp, c.dz_stride = _block_rows(a, dz, "dz", n, C, a.act) if p.gate else (None, 0)
    sums = [a.flat(t, n, (p.channels,), optional=True)
            for n, t in (("dscale", dscale), ("dpost_weight", dpost_weight), ("dpost_bias", dpost_bias),
                         ("dpre_weight", dpre_weight), ("dpre_bias", dpre_bias))]
    wp, wn = a.scratch(ws, "ws")
    a.call("ssd_block_norm_bwd", stream, ctypes.byref(c), xp, yp, zp, *vectors, drp, dhp, dxp, dyp, dzp,
           *sums, wp, wn)


def block_norm_forward(problem: BlockNorm, x, y, z=None, scale=None, post_weight=None, post_bias=None,
                       pre_weight=None, pre_bias=None, r=None, h=None, stream=None):
    """(r, h): r = alpha x + scale act(z) norm(y), h = norm(r) (None without `pre`).

    x, r [rows, channels] of the residual's type, y, z and h of the activations'; scale, weights
    and biases [channels] float32, biases and scale optional.  `r` and `h`: tensors to write
    to (r may be x, h may be y or z).
    """
    p, made_r, made_h = problem, None, None
    if r is None:
        r = made_r = torch.empty((p.rows, p.channels), dtype=_TORCH_ACT[p.res_dtype], device=x.device)
    if h is None and p.pre:
        h = made_h = torch.empty((p.rows, p.channels), dtype=_TORCH_ACT[p.act_dtype], device=x.device)
    _made_for(stream, x.device, made_r, made_h)
    ssd_block_norm_fwd(p, x, y, z, scale, post_weight, post_bias, pre_weight, pre_bias, r, h, stream)
    return r, h


@dataclass
class BlockNormBackwardBuffers:
    dx: torch.Tensor
    dy: torch.Tensor
    dz: Optional[torch.Tensor]            # None without a gate
    dscale: torch.Tensor
    dpost_weight: Optional[torch.Tensor]  # None without `post`
    dpost_bias: Optional[torch.Tensor]
    dpre_weight: Optional[torch.Tensor]   # None without `pre`
    dpre_bias: Optional[torch.Tensor]
    ws: torch.Tensor

    @staticmethod
    def allocate(problem: BlockNorm, device) -> "BlockNormBackwardBuffers":
        p = problem
        n = ssd_block_norm_workspace_bytes(p)
        if n == 0:
            raise SSDError("ssd_block_norm_workspace_bytes", -2)
        new = lambda t: torch.empty((p.rows, p.channels), dtype=_TORCH_ACT[t], device=device)  # noqa: E731
        vec = lambda want: torch.empty(p.channels, dtype=torch.float32, device=device) if want else None  # noqa: E731
        return BlockNormBackwardBuffers(
            dx=new(p.res_dtype), dy=new(p.act_dtype), dz=new(p.act_dtype) if p.gate else None,
            dscale=vec(True), dpost_weight=vec(p.post), dpost_bias=vec(p.post), dpre_weight=vec(p.pre),
            dpre_bias=vec(p.pre), ws=torch.empty(n, dtype=torch.uint8, device=device))


def block_norm_backward(problem: BlockNorm, x, y, dr, dh=None, z=None, scale=None, post_weight=None,
                        post_bias=None, pre_weight=None, pre_bias=None,
                        bufs: Optional[BlockNormBackwardBuffers] = None, stream=None) -> BlockNormBackwardBuffers:
    """Gradients of block_norm_forward (its inputs given again); returns the buffers.  dr: gradient
    of r, or None (zero) where there is dh; dh: gradient of h, with `pre`.  pre_bias is not read."""
    if bufs is None:
        bufs = BlockNormBackwardBuffers.allocate(problem, x.device)
        _made_for(stream, x.device, bufs.dx, bufs.dy, bufs.dz, bufs.dscale, bufs.dpost_weight, bufs.dpost_bias,
                  bufs.dpre_weight, bufs.dpre_bias, bufs.ws)
    ssd_block_norm_bwd(problem, x, y, z, scale, post_weight, post_bias, pre_weight, dr, dh, bufs.dx, bufs.dy,
                       bufs.dz, bufs.dscale, bufs.dpost_weight, bufs.dpost_bias, bufs.dpre_weight,
                       bufs.dpre_bias, bufs.ws, stream)
    return bufs


# ------------------------------------------------------------------------ rotary positions


def make_rope(*, batch: int, seqlen: int, nheads: int, headdim: int, act: str | int, nkheads: int = 0,
              rotdim: Optional[int] = None, style: str | int = "half", factor: float = 1.0) -> Rope:
    """Rotary positions of `nheads` heads of queries and `nkheads` of keys: the first `rotdim`
    (default: all) channels of a head are turned in pairs (i, i + rotdim / 2) ("half") or (2 i, 2 i
    + 1) ("interleaved") and multiplied by `factor`."""
    return Rope(batch, seqlen, nheads, nkheads, headdim, headdim if rotdim is None else rotdim,
                _act_code(act), _STYLE[style] if isinstance(style, str) else style, factor)


def rope_frequencies(rotdim: int, base: float = 10000.0, scaling: str = "none", stretch: float = 1.0,
                     trained: int = 4096, fast: float = 32.0, slow: float = 1.0,
                     device=None) -> Tuple[torch.Tensor, float]:
    """(radians per position of the pairs [rotdim / 2] float64, factor for make_rope): base^(-2 i /
    rotdim), for contexts `stretch` times as long as the `trained` positions changed by

      "linear"  positions divided by `stretch`
      "ntk"     a wider base, so that the slowest pair is stretched and the fastest keeps its own
      "yarn"    pairs that turn `fast` times or more within `trained` positions keep their own, those
                that turn `slow` times or less are stretched, in between by a ramp; the factor is
                0.1 ln(stretch) + 1
    """
    if rotdim < 2 or rotdim % 2:
        raise ValueError("rotdim must be even")
    if not stretch >= 1.0 or not base > 1.0:
        raise ValueError("stretch must be 1 or more and base above 1")
    i = torch.arange(0, rotdim, 2, dtype=torch.float64)
    f, factor = base ** (-i / rotdim), 1.0
    if scaling == "linear":
        f = f / stretch
    elif scaling == "ntk":
        if rotdim < 4:
            raise ValueError("ntk needs two pairs or more")
        f = (base * stretch ** (rotdim / (rotdim - 2))) ** (-i / rotdim)
    elif scaling == "yarn":
        place = lambda turns: rotdim * math.log(trained / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(0, math.floor(place(fast))), min(rotdim - 1, math.ceil(place(slow)))
        ramp = ((i / 2 - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = f * (1 - ramp) + f / stretch * ramp
        factor = 0.1 * math.log(stretch) + 1.0
    elif scaling != "none":
        raise ValueError(f"unknown scaling {scaling!r}")
    return f.to(device), factor


def ssd_rope(problem: Rope, q, k, frequencies, positions, cu_seqlens, inverse, q_out, k_out, stream=None):
    p = problem
    a, c = _Args(p.act_dtype), Rope.from_buffer_copy(p)
    b, L, D = p.batch, p.seqlen, p.headdim
    if not p.nkheads and (k is not None or k_out is not None):
        raise ValueError("the problem has no keys")
    qp, c.q_stride = a.tokens(q, "q", (b, L, p.nheads, D))
    qo, c.qo_stride = a.tokens(q_out, "q_out", (b, L, p.nheads, D))
    kp, c.k_stride = a.tokens(k, "k", (b, L, p.nkheads, D)) if p.nkheads else (None, 0)
    ko, c.ko_stride = a.tokens(k_out, "k_out", (b, L, p.nkheads, D)) if p.nkheads else (None, 0)
    fp = a.flat(frequencies, "frequencies", (p.rotdim // 2,), torch.float64)
    pos = a.flat(positions, "positions", (b, L), torch.int32, optional=True)
    n = _nseq(p, cu_seqlens)
    cu = a.flat(cu_seqlens, "cu_seqlens", (n + 1,), torch.int32, optional=True)
    a.call("ssd_rope", stream, ctypes.byref(c), qp, kp, fp, pos, cu, n, int(bool(inverse)), qo, ko)


def _rope(problem, q, k, frequencies, positions, cu_seqlens, inverse, out, stream):
    p = problem
    if out is None:
        new = lambda h: torch.empty((p.batch, p.seqlen, h, p.headdim), dtype=_TORCH_ACT[p.act_dtype],  # noqa: E731
                                    device=q.device)
        out = new(p.nheads), new(p.nkheads) if p.nkheads else None
        _made_for(stream, q.device, *out)
    ssd_rope(p, q, k, frequencies, positions, cu_seqlens, inverse, out[0], out[1], stream)
    return out


def rope_forward(problem: Rope, q, k, frequencies, positions=None, cu_seqlens=None, out=None, stream=None):
    """(q, k) with rotary positions, new or in `out` (which may be (q, k)); k is None where the
    problem has no keys.

    q [b, L, nheads, headdim], k [b, L, nkheads, headdim], frequencies [rotdim / 2] float64;
    positions [b, L] int32, or None: a token's place in its row, or in its sequence of
    cu_seqlens (int32 [nseq + 1], b = 1).  Tokens outside every sequence are left as they were.
    """
    return _rope(problem, q, k, frequencies, positions, cu_seqlens, False, out, stream)


def rope_backward(problem: Rope, dq, dk, frequencies, positions=None, cu_seqlens=None, out=None,
                  stream=None):
    """Gradients of rope_forward's q and k from those of its outputs, new or in `out`."""
    return _rope(problem, dq, dk, frequencies, positions, cu_seqlens, True, out, stream)
