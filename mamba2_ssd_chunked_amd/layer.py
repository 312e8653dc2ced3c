"""Python binding of include/ssd_layer.h: more operators of a layer around a recurrent mixer.

  gdelta_forward / gdelta_backward / ssd_gdelta_step   the gated delta rule: a state with a
      decay and an update rate per token and head; prompts, their gradients, single tokens

Checks, streams and buffers are those of mixer.py.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional

import torch

from ._lib import SSD_WS_BACKWARD, SSD_WS_FORWARD, GatedDelta, SSDError
from .mixer import _TORCH_ACT, _act_code, _Args, _entry, _made_for, _new_states, _nseq, _state_shape

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
