"""Refusals of the operators around the scan: host-side validation, no GPU.

Every call is made with arguments that fail a check, so nothing is launched (a launch
would return SSD_ERR_HIP here).
"""
import ctypes

import pytest
import torch

import mamba2_ssd_chunked_amd as ssd
from mamba2_ssd_chunked_amd import _lib

FAKE = 0x100000        # never dereferenced
MISALIGNED = 0x100004
BIG = 1 << 45


def la(**kw):
    base = dict(batch=1, seqlen=1000, nheads=8, nkvheads=2, keydim=128, valdim=64, act="bf16")
    strides = {k: kw.pop(k) for k in list(kw) if k.endswith("_stride")}
    p = ssd.make_linattn(**dict(base, **kw))
    for k, v in strides.items():
        setattr(p, k, v)
    return p


def fwd(p, nseq=3, q=FAKE, k=FAKE, v=FAKE, ld=FAKE, cu=FAKE, init=None, o=FAKE, fin=None, ws=FAKE,
        n=BIG):
    return _lib.load().ssd_linattn_fwd(None if p is None else ctypes.byref(p), nseq, q, k, v, ld, cu,
                                       init, o, fin, ws, n, None)


def bwd(p, nseq=3, cu=FAKE, ws=FAKE, n=BIG, **kw):
    t = dict(q=FAKE, k=FAKE, v=FAKE, ld=FAKE, do=FAKE, init=None, dfinal=None, dq=FAKE, dk=FAKE,
             dv=FAKE, dinit=None)
    t.update(kw)
    return _lib.load().ssd_linattn_bwd(None if p is None else ctypes.byref(p), nseq, t["q"], t["k"],
                                       t["v"], t["ld"], cu, t["do"], t["init"], t["dfinal"],
                                       t["dq"], t["dk"], t["dv"], t["dinit"], ws, n, None)


def step(p, slots=FAKE, nslots=4, pos=None, **kw):
    t = dict(q=FAKE, k=FAKE, v=FAKE, ld=FAKE, state=FAKE, o=FAKE)
    t.update(kw)
    return _lib.load().ssd_linattn_step(None if p is None else ctypes.byref(p), t["q"], t["k"],
                                        t["v"], t["ld"], slots, nslots, pos, t["state"], t["o"], None)


def test_struct_layouts():
    assert ctypes.sizeof(_lib.LinAttn) == 96
    assert ctypes.sizeof(_lib.Norm) == 72


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), -2), (dict(seqlen=0), -2), (dict(nheads=7), -2), (dict(nheads=65536), -2),
    (dict(nkvheads=0), -2), (dict(keydim=96), -3), (dict(valdim=48), -3), (dict(act=2), -3),
    (dict(seqlen=1 << 31), -2), (dict(batch=1 << 20, seqlen=1 << 20), -2),
    (dict(q_stride=1000), -2), (dict(k_stride=260), -4), (dict(v_stride=1 << 23), -2),
    (dict(o_stride=-512), -2), (dict(dq_stride=1028), -4),
])
def test_linattn_problem(kw, code):
    p = la(**kw)
    assert fwd(p) == code and bwd(p) == code and step(p) == code
    assert ssd.ssd_linattn_workspace_bytes(p, 3) == 0


def test_linattn_sequences_and_pointers():
    p = la()
    assert fwd(None) == -1 and bwd(None) == -1 and step(None) == -1
    assert fwd(p, nseq=0) == -7 and fwd(p, nseq=(1 << 24) + 1) == -7
    assert fwd(p, nseq=3, cu=None) == -7            # rows are sequences: nseq is the batch
    assert fwd(la(batch=3), nseq=3, cu=FAKE) == -7  # packed sequences: one row
    assert fwd(la(nheads=65535, nkvheads=1), nseq=1 << 20) == -2  # more workgroups than a grid holds
    for name in ("q", "k", "v", "ld", "o"):
        assert fwd(p, **{name: None}) == -1
    for name in ("q", "k", "v", "ld", "do", "dq", "dk", "dv"):
        assert bwd(p, **{name: None}) == -1
    for name in ("q", "k", "v", "init", "o", "fin", "ws"):
        assert fwd(p, **{name: MISALIGNED}) == -4
    for name in ("q", "do", "init", "dfinal", "dq", "dk", "dv", "dinit", "ws"):
        assert bwd(p, **{name: MISALIGNED}) == -4
    assert fwd(p, cu=FAKE + 2) == -4 and fwd(p, ld=FAKE + 1) == -4
    for kind, call in ((ssd.SSD_WS_FORWARD, fwd), (ssd.SSD_WS_BACKWARD, bwd)):
        need = ssd.ssd_linattn_workspace_bytes(p, 3, kind)
        assert need > 0
        assert call(p, ws=None) == -5
        if need > 256:
            assert call(p, n=need - 1) == -5
    assert ssd.ssd_linattn_workspace_bytes(p, 3, 2) == 0
    assert ssd.ssd_linattn_workspace_bytes(p, 0) == 0


def test_linattn_step_refusals():
    p = la(batch=4, seqlen=1)
    for name in ("q", "k", "v", "ld", "state", "o"):
        assert step(p, **{name: None}) == -1
    assert step(p, nslots=0) == -2 and step(p, slots=None, nslots=3) == -2
    assert step(p, state=MISALIGNED) == -4 and step(p, slots=FAKE + 2) == -4
    assert step(p, pos=FAKE + 1) == -4
    assert step(la(batch=1 << 20, seqlen=1, nheads=64), nslots=1 << 20) == -2


def token(p, slots=FAKE, nslots=4, pos=FAKE, ring=FAKE, R=4, **kw):
    t = dict(x=FAKE, w=FAKE, dt=FAKE, db=FAKE, A=FAKE, D=FAKE, state=FAKE, y=FAKE)
    t.update(kw)
    return _lib.load().ssd_token_step(None if p is None else ctypes.byref(p), t["x"], t["w"],
                                      t["dt"], t["db"], t["A"], t["D"], slots, nslots, pos, ring, R,
                                      t["state"], t["y"], None)


def test_token_step_refusals():
    def prob(**kw):
        base = dict(batch=4, seqlen=1, nheads=8, headdim=64, dstate=128, ngroups=2, chunk=64,
                    conv_width=4, act="bf16")
        return ssd.make_problem(**dict(base, **kw))
    assert token(None) == -1
    for kw, code in [(dict(batch=0), -2), (dict(ngroups=3), -2), (dict(nheads=65536), -2),
                     (dict(act=2), -3), (dict(headdim=48), -3), (dict(dstate=16), -3),
                     (dict(conv_width=9), -3), (dict(conv_width=0), -2), (dict(dt_min=-1.0), -2),
                     (dict(seqlen=2), -2), (dict(seqlen=1 << 32), -2), (dict(batch=1 << 32), -2),
                     (dict(batch=1 << 22), -2)]:
        assert token(prob(**kw), nslots=1 << 33) == code, kw
    p = prob()
    for name in ("x", "w", "dt", "db", "A", "D", "state", "y"):
        assert token(p, **{name: None}) == -1
    assert token(p, pos=None) == -1 and token(p, ring=None) == -1
    assert token(p, R=3) == -2 and token(p, nslots=0) == -2
    assert token(p, slots=None, nslots=3) == -2
    assert token(p, state=MISALIGNED) == -4 and token(p, pos=FAKE + 2) == -4


def norm(rows=8, channels=512, ngroups=4, act="bf16", mode="before", center=False, eps=1e-5, **st):
    p = ssd.make_norm(rows=rows, channels=channels, ngroups=ngroups, act=act, mode=mode,
                      center=center, eps=eps)
    for k, v in st.items():
        setattr(p, k, v)
    return p


def nfwd(p, x=FAKE, z=FAKE, w=FAKE, b=FAKE, y=FAKE):
    return _lib.load().ssd_norm_fwd(None if p is None else ctypes.byref(p), x, z, w, b, y, None)


def nbwd(p, ws=FAKE, n=BIG, **kw):
    t = dict(x=FAKE, z=FAKE, w=FAKE, b=FAKE, dy=FAKE, dx=FAKE, dz=FAKE, dw=FAKE, db=FAKE)
    t.update(kw)
    return _lib.load().ssd_norm_bwd(None if p is None else ctypes.byref(p), t["x"], t["z"], t["w"],
                                    t["b"], t["dy"], t["dx"], t["dz"], t["dw"], t["db"], ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), -2), (dict(channels=0), -2), (dict(ngroups=3), -2), (dict(ngroups=0), -2),
    (dict(channels=1 << 21, ngroups=1), -2), (dict(rows=1 << 31), -2), (dict(rows=1 << 30), -2),
    (dict(channels=65536, ngroups=65536), -2), (dict(act=2), -3), (dict(mode=4), -3),
    (dict(mode=-1), -3), (dict(eps=0.0), -2), (dict(eps=float("nan")), -2),
    (dict(eps=float("inf")), -2), (dict(x_stride=511), -2), (dict(dz_stride=1 << 28), -2),
])
def test_norm_problem(kw, code):
    p = norm(**kw)
    assert nfwd(p) == code and nbwd(p) == code
    assert ssd.ssd_norm_workspace_bytes(p) == 0


def test_norm_pointers():
    p = norm()
    p2 = norm()
    p2.center = 2
    assert nfwd(p2) == -2 and nfwd(None) == -1 and nbwd(None) == -1
    for name in ("x", "z", "w", "y"):
        assert nfwd(p, **{name: None}) == -1
    for name in ("x", "z", "w", "dy", "dx", "dz", "dw"):
        assert nbwd(p, **{name: None}) == -1
    assert nfwd(p, x=FAKE + 1) == -4 and nfwd(p, w=FAKE + 2) == -4
    assert nbwd(p, dx=FAKE + 1) == -4 and nbwd(p, ws=FAKE + 2) == -4
    need = ssd.ssd_norm_workspace_bytes(p)
    assert nbwd(p, ws=None) == -5 and nbwd(p, n=need - 1) == -5


def test_binding_refuses_before_the_library():
    """Host tensors, and missing ones, are refused in Python."""
    x = torch.zeros(2, 8, 4, 64)
    ld = torch.zeros(4)
    p = ssd.make_linattn(batch=2, seqlen=8, nheads=4, keydim=64, valdim=64, act="f32")
    assert p.nkvheads == 4 and p.scale == 0.125
    with pytest.raises(ValueError, match="q must be a device tensor"):
        ssd.ssd_linattn_fwd(p, x, x, x, ld, None, None, x, None, x)
    with pytest.raises(ValueError, match="state must have shape"):
        ssd.ssd_token_step(ssd.make_problem(batch=1, seqlen=1, nheads=1, headdim=16, dstate=16,
                                            ngroups=1, chunk=64, conv_width=4, act="f32"),
                           x, x, x, x, x, x, x[0], None, x, x)
    pn = ssd.make_norm(rows=2, channels=8, act="f32", mode="none")
    with pytest.raises(ValueError, match="x must be a device tensor"):
        ssd.ssd_norm_fwd(pn, torch.zeros(2, 8), None, torch.zeros(8), None, torch.zeros(2, 8))
    with pytest.raises(KeyError):
        ssd.make_norm(rows=1, channels=8, act="f32", mode="gelu")


def _meta(shape, stride=None):
    """A stand-in with a layout, to see what the layout checks say without a GPU."""
    t = torch.empty(shape) if stride is None else torch.empty_strided(shape, stride)

    class OnDevice:
        is_cuda, device, dtype = True, "cuda:0", torch.float32
        shape = t.shape
        stride = staticmethod(t.stride)
        is_contiguous = staticmethod(t.is_contiguous)
        data_ptr = staticmethod(lambda: 4096)
    return OnDevice()


@pytest.mark.parametrize("shape,stride,want", [
    ((2, 8, 4, 16), None, 0),                   # packed
    ((2, 8, 4, 16), (800, 100, 16, 1), 100),
    ((1, 8, 4, 16), (1, 100, 16, 1), 100),      # one row: its stride says nothing
    ((2, 1, 4, 16), (96, 1, 16, 1), 96),        # one token: the next row is the next token
    ((2, 8, 4, 16), (900, 100, 16, 1), None),   # rows further apart than their tokens
    ((2, 8, 4, 16), (800, 100, 20, 1), None),   # heads apart
    ((2, 8, 4, 16), (64, 128, 16, 1), None),    # token-major batch
    ((2, 8, 4, 16), (512, 0, 16, 1), None),     # a broadcast token
])
def test_token_layouts(shape, stride, want, monkeypatch):
    from mamba2_ssd_chunked_amd import mixer
    monkeypatch.setattr(mixer._Args, "_base", lambda self, t, name, dtype, shape: None)
    a = mixer._Args(ssd.SSD_F32)
    t = _meta(shape, stride)
    if want is None:
        with pytest.raises(ValueError):
            a.tokens(t, "q", shape)
    else:
        assert a.tokens(t, "q", shape) == (4096, want)
