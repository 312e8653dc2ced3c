"""Python binding of include/ssd_mixer.h: the operators that stand around the SSD scan.

  linattn_forward / linattn_backward / ssd_linattn_step   linear attention with a fixed
      decay per head: prompts of any length, their gradients, single tokens
  ssd_token_step                                          the conv1d + SSD path token by
      token, continuing from forward()'s final state (StepState holds what it carries)
  norm_forward / norm_backward                            the group norm with an activation
      over a mixer's output, channels last

As in ops.py, one function per entry point with the same name checks every tensor's
size, dtype, device and layout and passes pointers; the functions without the prefix
also make the buffers.  Token arrays may be views of wider rows (a slice of a
projection): their channels have to be contiguous.  Work goes to the current stream of
the tensors' device, or to `stream` (of that device).
"""
from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass
from typing import Optional, Tuple

import torch

from . import _lib
from ._lib import (SSD_BF16, SSD_F32, SSD_NORM_AFTER, SSD_NORM_BEFORE, SSD_NORM_NONE,
                   SSD_NORM_SILU, SSD_WS_BACKWARD, SSD_WS_FORWARD, LinAttn, Norm, Problem,
                   SSDError)

_TORCH_ACT = {SSD_F32: torch.float32, SSD_BF16: torch.bfloat16}
_ACT = {"f32": SSD_F32, "float32": SSD_F32, "bf16": SSD_BF16, "bfloat16": SSD_BF16}
_MODE = {"none": SSD_NORM_NONE, "silu": SSD_NORM_SILU, "before": SSD_NORM_BEFORE,
         "after": SSD_NORM_AFTER}


# ------------------------------------------------------------------ argument checks


_calls = {}  # entry points by name, once the library is loaded


def _entry(fn):
    f = _calls.get(fn)
    if f is None:
        f = _calls[fn] = getattr(_lib.load(), fn)
    return f


class _Args:
    """The checked tensors of one call: all of them on one device."""

    __slots__ = ("act", "device", "index")

    def __init__(self, act):
        self.act = _TORCH_ACT[act]
        self.device = self.index = None

    def _base(self, t, name, dtype, shape):
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name} is required")
        if t.get_device() != self.index:  # -1 where there is no device
            if not t.is_cuda:
                raise ValueError(f"{name} must be a device tensor")
            if self.device is not None:
                raise ValueError(f"{name} is on {t.device}, other tensors on {self.device}")
            self.device, self.index = t.device, t.get_device()
        if t.dtype is not dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")

    def flat(self, t, name, shape, dtype=torch.float32, optional=False):
        """A contiguous tensor of the given shape."""
        if t is None and optional:
            return None
        self._base(t, name, dtype, shape)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t.data_ptr()

    def tokens(self, t, name, shape) -> Tuple[int, int]:
        """(pointer, elements between tokens; 0 packed) of an activation tensor [batch, tokens,
        *channels] whose channels are contiguous and whose rows follow each other."""
        self._base(t, name, self.act, shape)
        if t.is_contiguous():
            return t.data_ptr(), 0
        st, want = t.stride(), 1
        for n, s in zip(reversed(shape[2:]), reversed(st[2:])):
            if n > 1 and s != want:
                raise ValueError(f"the channels of a token of {name} must be contiguous")
            want *= n
        step = st[1] if shape[1] > 1 else (st[0] if shape[0] > 1 else want)
        if step < want:
            raise ValueError(f"the tokens of {name} overlap")
        if shape[0] > 1 and st[0] != shape[1] * step:
            raise ValueError(f"the rows of {name} must follow each other at its token stride")
        return t.data_ptr(), step

    def scratch(self, t, name):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous device tensor")
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, other tensors on {self.device}")
        return t.data_ptr(), t.numel() * t.element_size()

    def call(self, fn, stream, *args):
        """The library call on the tensors' device; the stream comes last."""
        if stream is None:
            handle = torch._C._cuda_getCurrentRawStream(self.index)
        else:
            handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        if self.index == torch._C._cuda_getDevice():
            rc = _entry(fn)(*args, handle)
        else:
            with torch.cuda.device(self.device):
                rc = _entry(fn)(*args, handle)
        if rc != 0:
            raise SSDError(fn, rc)


def _made_for(stream, device, *tensors):
    """Tensors made here (on the current stream) and used on `stream`: the allocator must
    not hand their memory out again before that stream is done with it."""
    if stream is None:
        return
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    if stream.cuda_stream != torch.cuda.current_stream(device).cuda_stream:
        stream.wait_stream(torch.cuda.current_stream(device))
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _act_code(act) -> int:
    return _ACT[act] if isinstance(act, str) else act


# ------------------------------------------------------- linear attention with decay


def make_linattn(*, batch: int, seqlen: int, nheads: int, keydim: int, valdim: int,
                 act: str | int, nkvheads: Optional[int] = None,
                 scale: Optional[float] = None) -> LinAttn:
    """Sizes of a linear attention: `nheads` query heads over `nkvheads` (default: as many)
    key/value heads; scale defaults to keydim ** -0.5."""
    return LinAttn(batch, seqlen, nheads, nheads if nkvheads is None else nkvheads, keydim, valdim,
                   _act_code(act), keydim ** -0.5 if scale is None else scale)


def _strided(p: LinAttn, q, k, v, o, dq=0, dk=0, dv=0) -> LinAttn:
    """The problem with the tensors' strides (a copy: the caller's stays as it is)."""
    c = LinAttn.from_buffer_copy(p)
    c.q_stride, c.k_stride, c.v_stride, c.o_stride = q, k, v, o
    c.dq_stride, c.dk_stride, c.dv_stride = dq, dk, dv
    return c


def _nseq(p: LinAttn, cu_seqlens) -> int:
    return p.batch if cu_seqlens is None else max(0, cu_seqlens.numel() - 1)


def _state_shape(p: LinAttn, n: int):
    return (n, p.nheads, p.valdim, p.keydim)


def _new_states(p: LinAttn, n: int, device):
    return torch.empty(_state_shape(p, n), dtype=torch.float32, device=device)


def ssd_linattn_workspace_bytes(problem: LinAttn, nseq: int, kind: int = SSD_WS_FORWARD) -> int:
    return int(_entry("ssd_linattn_workspace_bytes")(ctypes.byref(problem), nseq, kind))


def ssd_linattn_fwd(problem: LinAttn, q, k, v, log_decay, cu_seqlens, init, o, final_state, ws,
                    stream=None):
    p, n = problem, _nseq(problem, cu_seqlens)
    a = _Args(p.act_dtype)
    b, L, H, K, Dk, Dv = p.batch, p.seqlen, p.nheads, p.nkvheads, p.keydim, p.valdim
    qp, qs = a.tokens(q, "q", (b, L, H, Dk))
    kp, ks = a.tokens(k, "k", (b, L, K, Dk))
    vp, vs = a.tokens(v, "v", (b, L, K, Dv))
    op, os_ = a.tokens(o, "o", (b, L, H, Dv))
    ld = a.flat(log_decay, "log_decay", (H,))
    cu = a.flat(cu_seqlens, "cu_seqlens", (n + 1,), torch.int32, optional=True)
    ini = a.flat(init, "init", _state_shape(p, n), optional=True)
    fin = a.flat(final_state, "final_state", _state_shape(p, n), optional=True)
    wp, wn = a.scratch(ws, "ws")
    p = _strided(p, qs, ks, vs, os_)
    a.call("ssd_linattn_fwd", stream, ctypes.byref(p), n, qp, kp, vp, ld, cu, ini, op, fin, wp, wn)


def ssd_linattn_bwd(problem: LinAttn, q, k, v, log_decay, cu_seqlens, do, init, dfinal, dq, dk, dv,
                    dinit, ws, stream=None):
    p, n = problem, _nseq(problem, cu_seqlens)
    a = _Args(p.act_dtype)
    b, L, H, K, Dk, Dv = p.batch, p.seqlen, p.nheads, p.nkvheads, p.keydim, p.valdim
    shapes = dict(q=(q, (b, L, H, Dk)), k=(k, (b, L, K, Dk)), v=(v, (b, L, K, Dv)),
                  do=(do, (b, L, H, Dv)), dq=(dq, (b, L, H, Dk)), dk=(dk, (b, L, K, Dk)),
                  dv=(dv, (b, L, K, Dv)))
    t = {name: a.tokens(x, name, s) for name, (x, s) in shapes.items()}
    ld = a.flat(log_decay, "log_decay", (H,))
    cu = a.flat(cu_seqlens, "cu_seqlens", (n + 1,), torch.int32, optional=True)
    st = _state_shape(p, n)
    ini, dfin = a.flat(init, "init", st, optional=True), a.flat(dfinal, "dfinal", st, optional=True)
    dini = a.flat(dinit, "dinit", st, optional=True)
    wp, wn = a.scratch(ws, "ws")
    p = _strided(p, *(t[name][1] for name in ("q", "k", "v", "do", "dq", "dk", "dv")))
    a.call("ssd_linattn_bwd", stream, ctypes.byref(p), n, t["q"][0], t["k"][0], t["v"][0], ld, cu,
           t["do"][0], ini, dfin, t["dq"][0], t["dk"][0], t["dv"][0], dini, wp, wn)


def ssd_linattn_step(problem: LinAttn, q, k, v, log_decay, state, o, slots=None, positions=None,
                     stream=None):
    """The next `seqlen` tokens (1, or a few) of `batch` rows; `state` [slots, H, valdim,
    keydim] float32 is updated in place, `slots` [batch] int32 says where each row's is."""
    p = problem
    a = _Args(p.act_dtype)
    b, L, H, K, Dk, Dv = p.batch, p.seqlen, p.nheads, p.nkvheads, p.keydim, p.valdim
    qp, qs = a.tokens(q, "q", (b, L, H, Dk))
    kp, ks = a.tokens(k, "k", (b, L, K, Dk))
    vp, vs = a.tokens(v, "v", (b, L, K, Dv))
    op, os_ = a.tokens(o, "o", (b, L, H, Dv))
    ld = a.flat(log_decay, "log_decay", (H,))
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state must have shape (slots, nheads, valdim, keydim)")
    sp = a.flat(state, "state", _state_shape(p, state.shape[0]))
    sl = a.flat(slots, "slots", (b,), torch.int32, optional=True)
    po = a.flat(positions, "positions", (b,), torch.int32, optional=True)
    p = _strided(p, qs, ks, vs, os_)
    a.call("ssd_linattn_step", stream, ctypes.byref(p), qp, kp, vp, ld, sl, state.shape[0], po, sp,
           op)


@dataclass
class LinAttnForwardBuffers:
    o: torch.Tensor
    final_state: Optional[torch.Tensor]  # [nseq][H][valdim][keydim] float32
    ws: torch.Tensor

    @staticmethod
    def allocate(problem: LinAttn, nseq: int, device, final: bool = True) -> "LinAttnForwardBuffers":
        """Buffers of linattn_forward; without `final` they have no final_state."""
        p = problem
        n = ssd_linattn_workspace_bytes(p, nseq, SSD_WS_FORWARD)
        if n == 0:
            raise SSDError("ssd_linattn_workspace_bytes", -2)
        return LinAttnForwardBuffers(
            o=torch.empty((p.batch, p.seqlen, p.nheads, p.valdim), dtype=_TORCH_ACT[p.act_dtype],
                          device=device),
            final_state=_new_states(p, nseq, device) if final else None,
            ws=torch.empty(n, dtype=torch.uint8, device=device))


def linattn_forward(problem: LinAttn, q, k, v, log_decay, cu_seqlens=None, init=None,
                    bufs: Optional[LinAttnForwardBuffers] = None, stream=None,
                    want_final: bool = False) -> LinAttnForwardBuffers:
    """o = scale S_t q_t with S_t = exp(log_decay) S_(t-1) + v_t k_t^T; returns the buffers.

    q [b, L, H, keydim], k and v [b, L, nkvheads, keydim or valdim]; every row is a
    sequence, or with cu_seqlens (int32 [nseq + 1], b = 1) the packed sequences are.
    init       : optional [nseq, H, valdim, keydim] float32 states before the sequences.
    want_final : also write bufs.final_state (None in buffers made here without it).
    Rows of bufs.o outside every sequence are left as they were.
    """
    if bufs is None:
        bufs = LinAttnForwardBuffers.allocate(problem, _nseq(problem, cu_seqlens), q.device,
                                              final=want_final)
        _made_for(stream, q.device, bufs.o, bufs.final_state, bufs.ws)
    elif want_final and bufs.final_state is None:
        raise ValueError("the buffers have no final_state")
    ssd_linattn_fwd(problem, q, k, v, log_decay, cu_seqlens, init, bufs.o,
                    bufs.final_state if want_final else None, bufs.ws, stream)
    return bufs


@dataclass
class LinAttnBackwardBuffers:
    dq: torch.Tensor
    dk: torch.Tensor
    dv: torch.Tensor
    dinit: Optional[torch.Tensor]  # [nseq][H][valdim][keydim] float32
    ws: torch.Tensor

    @staticmethod
    def allocate(problem: LinAttn, nseq: int, device, dinit: bool = True) -> "LinAttnBackwardBuffers":
        """Buffers of linattn_backward; without `dinit` they have none."""
        p = problem
        n = ssd_linattn_workspace_bytes(p, nseq, SSD_WS_BACKWARD)
        if n == 0:
            raise SSDError("ssd_linattn_workspace_bytes", -2)
        new = lambda h, d: torch.empty((p.batch, p.seqlen, h, d), dtype=_TORCH_ACT[p.act_dtype],  # noqa: E731
                                       device=device)
        return LinAttnBackwardBuffers(
            dq=new(p.nheads, p.keydim), dk=new(p.nkvheads, p.keydim), dv=new(p.nkvheads, p.valdim),
            dinit=_new_states(p, nseq, device) if dinit else None,
            ws=torch.empty(n, dtype=torch.uint8, device=device))


def linattn_backward(problem: LinAttn, q, k, v, log_decay, do, cu_seqlens=None, init=None,
                     dfinal=None, bufs: Optional[LinAttnBackwardBuffers] = None, stream=None,
                     want_dinit: bool = False) -> LinAttnBackwardBuffers:
    """Gradients of linattn_forward (its inputs, `init` included, given again); returns the
    buffers.  The decays are constants and get none.

    dfinal     : optional gradient of the final states.
    want_dinit : also write bufs.dinit, the gradient of `init` (None in buffers made here
                 without it).
    """
    if bufs is None:
        bufs = LinAttnBackwardBuffers.allocate(problem, _nseq(problem, cu_seqlens), q.device,
                                               dinit=want_dinit)
        _made_for(stream, q.device, bufs.dq, bufs.dk, bufs.dv, bufs.dinit, bufs.ws)
    elif want_dinit and bufs.dinit is None:
        raise ValueError("the buffers have no dinit")
    ssd_linattn_bwd(problem, q, k, v, log_decay, cu_seqlens, do, init, dfinal, bufs.dq, bufs.dk,
                    bufs.dv, bufs.dinit if want_dinit else None, bufs.ws, stream)
    return bufs


# ------------------------------------------------- the conv1d + SSD path token by token


def ssd_token_step(problem: Problem, xBC, conv_w, dt_raw, dt_bias, A_log, D, conv_ring, state,
                   positions, y, slots=None, stream=None):
    """The next `problem.seqlen` tokens (1, or a few) of `problem.batch` rows through conv1d,
    dt, the scan and D x; conv_ring [slots, ring, C] and state [slots, H, P, N] are updated
    in place (StepState).  positions [batch] int32: the place of each row's first new token
    in its sequence; slots [batch] int32: where each row's state is (row r's in slot r if
    None)."""
    p = problem
    a = _Args(p.act_dtype)
    b, L, H, P, N = p.batch, p.seqlen, p.nheads, p.headdim, p.dstate
    C = H * P + 2 * p.ngroups * N
    if not isinstance(conv_ring, torch.Tensor) or conv_ring.dim() != 3:
        raise ValueError("conv_ring must have shape (slots, ring, channels)")
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state must have shape (slots, nheads, headdim, dstate)")
    n, ring = state.shape[0], conv_ring.shape[1]
    ins = (a.flat(xBC, "xBC", (b, L, C), a.act), a.flat(conv_w, "conv_w", (C, p.conv_width)),
           a.flat(dt_raw, "dt_raw", (b, L, H), a.act), a.flat(dt_bias, "dt_bias", (H,)),
           a.flat(A_log, "A_log", (H,)), a.flat(D, "D", (H,)),
           a.flat(slots, "slots", (b,), torch.int32, optional=True))
    pos = a.flat(positions, "positions", (b,), torch.int32)
    rp = a.flat(conv_ring, "conv_ring", (n, ring, C), a.act)
    sp = a.flat(state, "state", (n, H, P, N))
    yp = a.flat(y, "y", (b, L, H, P), a.act)
    a.call("ssd_token_step", stream, ctypes.byref(p), *ins, n, pos, rp, ring, sp, yp)


@dataclass
class StepState:
    """What ssd_token_step carries from token to token, for a pool of sequences."""
    conv_ring: torch.Tensor  # [slots][ring][C], the input of token t at entry t % ring
    state: torch.Tensor      # [slots][H][P][N] float32

    @staticmethod
    def allocate(problem: Problem, nslots: int, device, tokens: int = 1) -> "StepState":
        """Room for `nslots` sequences and steps of up to `tokens` tokens.  Nothing has to be
        cleared: a sequence that starts at position 0 reads nothing from its slot."""
        p = problem
        C = p.nheads * p.headdim + 2 * p.ngroups * p.dstate
        return StepState(
            conv_ring=torch.empty((nslots, p.conv_width - 1 + tokens, C),
                                  dtype=_TORCH_ACT[p.act_dtype], device=device),
            state=torch.empty((nslots, p.nheads, p.headdim, p.dstate), dtype=torch.float32,
                              device=device))

    def load(self, problem: Problem, xBC, final_state, slots=None, stream=None) -> torch.Tensor:
        """Takes over rows that forward(..., want_final=True) has run, in the order of their
        tokens: the last inputs of xBC [batch, seqlen, C] and final_state [batch, H, P, N] go to
        `slots` (rows r to slot r if None).  Returns the rows' positions.

        As in the steps that follow, a row whose slot is outside the pool is padding and of
        several rows with one slot only the first counts: the others go nowhere, and their
        position is -1, so that the steps skip them too.  Work goes to the current stream, or to
        `stream` (which waits for the current one first); give a step the same one."""
        b, L = problem.batch, problem.seqlen
        n, ring, C = self.conv_ring.shape
        if xBC.shape != (b, L, C) or xBC.dtype is not self.conv_ring.dtype:
            raise ValueError(f"xBC must be {self.conv_ring.dtype} of shape {(b, L, C)}, got "
                             f"{xBC.dtype} of {tuple(xBC.shape)}")
        if final_state.shape != (b, *self.state.shape[1:]) or final_state.dtype is not torch.float32:
            raise ValueError("final_state must be torch.float32 of shape "
                             f"{(b, *self.state.shape[1:])}")
        if slots is None:
            if b > n:
                raise ValueError(f"{b} rows need slots: the pool has {n}")
        elif slots.shape != (b,) or slots.dtype not in (torch.int32, torch.int64):
            raise ValueError(f"slots must be int32 or int64 of shape {(b,)}")
        dev = self.state.device
        positions = torch.empty((b,), dtype=torch.int32, device=dev)
        if stream is None:
            self._load(problem, xBC, final_state, slots, positions)
            return positions
        _made_for(stream, dev, positions)
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=dev)
        with torch.cuda.stream(stream):
            self._load(problem, xBC, final_state, slots, positions)
        return positions

    def _load(self, problem, xBC, final_state, slots, positions):
        b, L = problem.batch, problem.seqlen
        n, ring, _ = self.conv_ring.shape
        rows = torch.arange(b, device=positions.device)
        last = torch.arange(max(0, L - (problem.conv_width - 1)), L, device=positions.device)
        entry = (last % ring)[None, :]
        if slots is None:
            self.conv_ring[rows[:, None], entry] = xBC[:, last]
            self.state[rows] = final_state
            positions.fill_(L)
            return
        slots = slots.to(positions.device, torch.int64)
        live = (slots >= 0) & (slots < n)
        spot = torch.where(live, slots, n)
        owner = torch.full((n + 1,), b, dtype=torch.int64, device=positions.device)
        owner.scatter_reduce_(0, spot, rows, "amin")
        live &= owner[spot] == rows
        # Rows that go nowhere write the first live row's values a second time, or, if there is
        # none, a slot's own: nothing has to come back to the host to leave them out.  (`first`
        # of one element, since an index without dimensions is read by the host.)
        first = live.to(torch.int32).argmax(0, keepdim=True)
        src = torch.where(live, rows, first)
        at = torch.where(live, slots, slots[first]).clamp(0, n - 1)
        some = live.any()
        ring_at = (at[:, None], entry)
        self.conv_ring[ring_at] = torch.where(some, xBC[src[:, None], last[None, :]],
                                              self.conv_ring[ring_at])
        self.state[at] = torch.where(some, final_state[src], self.state[at])
        positions.copy_(torch.where(live, L, -1))


# ------------------------------------------- group norm with an activation, channels last


def make_norm(*, rows: int, channels: int, act: str | int, ngroups: int = 1,
              mode: str | int = "before", center: bool = False, eps: float = 1e-5) -> Norm:
    """A group norm over the channels of every row: RMS, or centred (`center`).
    mode: "none", "silu" (of the result), "before" (x silu(z) is normalised) or "after" (the
    result is multiplied by silu(z))."""
    return Norm(rows, channels, ngroups, _act_code(act), _MODE[mode] if isinstance(mode, str) else mode,
                int(bool(center)), eps)


def _norm_rows(a: _Args, t, name, p: Norm):
    a._base(t, name, a.act, (p.rows, p.channels))
    if p.channels > 1 and t.stride(1) != 1:
        raise ValueError(f"the channels of a row of {name} must be contiguous")
    step = t.stride(0) if p.rows > 1 else p.channels
    if step < p.channels:
        raise ValueError(f"the rows of {name} overlap")
    return t.data_ptr(), step


def _gated(p: Norm) -> bool:
    return p.mode in (SSD_NORM_BEFORE, SSD_NORM_AFTER)


def _norm_z(a, p, t, name):
    if _gated(p):
        return _norm_rows(a, t, name, p)
    if t is not None:
        raise ValueError(f"{name} is only for the gated modes")
    return None, 0


def ssd_norm_fwd(problem: Norm, x, z, weight, bias, y, stream=None):
    p = problem
    a = _Args(p.act_dtype)
    xp, xs = _norm_rows(a, x, "x", p)
    zp, zs = _norm_z(a, p, z, "z")
    yp, ys = _norm_rows(a, y, "y", p)
    w = a.flat(weight, "weight", (p.channels,))
    b = a.flat(bias, "bias", (p.channels,), optional=True)
    p = Norm.from_buffer_copy(p)
    p.x_stride, p.z_stride, p.y_stride = xs, zs, ys
    a.call("ssd_norm_fwd", stream, ctypes.byref(p), xp, zp, w, b, yp)


def ssd_norm_workspace_bytes(problem: Norm) -> int:
    return int(_entry("ssd_norm_workspace_bytes")(ctypes.byref(problem)))


def ssd_norm_bwd(problem: Norm, x, z, weight, bias, dy, dx, dz, dweight, dbias, ws, stream=None):
    p = problem
    a = _Args(p.act_dtype)
    xp, xs = _norm_rows(a, x, "x", p)
    zp, zs = _norm_z(a, p, z, "z")
    dyp, ys = _norm_rows(a, dy, "dy", p)
    dxp, dxs = _norm_rows(a, dx, "dx", p)
    dzp, dzs = _norm_z(a, p, dz, "dz")
    w = a.flat(weight, "weight", (p.channels,))
    b = a.flat(bias, "bias", (p.channels,), optional=True)
    dw = a.flat(dweight, "dweight", (p.channels,))
    db = a.flat(dbias, "dbias", (p.channels,), optional=True)
    wp, wn = a.scratch(ws, "ws")
    p = Norm.from_buffer_copy(p)
    p.x_stride, p.z_stride, p.y_stride, p.dx_stride, p.dz_stride = xs, zs, ys, dxs, dzs
    a.call("ssd_norm_bwd", stream, ctypes.byref(p), xp, zp, w, b, dyp, dxp, dzp, dw, db, wp, wn)


def norm_forward(problem: Norm, x, weight, bias=None, z=None, out=None, stream=None):
    """The normalised rows [rows, channels] (`out`, or a new tensor)."""
    if out is None:
        out = torch.empty((problem.rows, problem.channels), dtype=_TORCH_ACT[problem.act_dtype],
                          device=x.device)
        _made_for(stream, x.device, out)
    ssd_norm_fwd(problem, x, z, weight, bias, out, stream)
    return out


@dataclass
class NormBackwardBuffers:
    dx: torch.Tensor
    dz: Optional[torch.Tensor]  # None where the mode has no gate
    dweight: torch.Tensor
    dbias: torch.Tensor
    ws: torch.Tensor

    @staticmethod
    def allocate(problem: Norm, device) -> "NormBackwardBuffers":
        p = problem
        n = ssd_norm_workspace_bytes(p)
        if n == 0:
            raise SSDError("ssd_norm_workspace_bytes", -2)
        new = lambda: torch.empty((p.rows, p.channels), dtype=_TORCH_ACT[p.act_dtype], device=device)  # noqa: E731
        return NormBackwardBuffers(
            dx=new(), dz=new() if _gated(p) else None,
            dweight=torch.empty(p.channels, dtype=torch.float32, device=device),
            dbias=torch.empty(p.channels, dtype=torch.float32, device=device),
            ws=torch.empty(n, dtype=torch.uint8, device=device))


def norm_backward(problem: Norm, x, weight, dy, bias=None, z=None,
                  bufs: Optional[NormBackwardBuffers] = None, stream=None) -> NormBackwardBuffers:
    """Gradients of norm_forward; returns the buffers (dweight and dbias summed over rows)."""
    if bufs is None:
        bufs = NormBackwardBuffers.allocate(problem, x.device)
        _made_for(stream, x.device, bufs.dx, bufs.dz, bufs.dweight, bufs.dbias, bufs.ws)
    ssd_norm_bwd(problem, x, z, weight, bias, dy, bufs.dx, bufs.dz, bufs.dweight, bufs.dbias,
                 bufs.ws, stream)
    return bufs
