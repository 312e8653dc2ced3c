"""Refusals of the operators of include/ssd_layer.h: host-side validation, no GPU.

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


def gd(**kw):
    base = dict(batch=1, seqlen=1000, nheads=8, nkheads=2, keydim=128, valdim=64, act="bf16")
    strides = {k: kw.pop(k) for k in list(kw) if k.endswith("_stride")}
    p = ssd.make_gdelta(**dict(base, **kw))
    for k, v in strides.items():
        setattr(p, k, v)
    return p


def ref(p):
    return None if p is None else ctypes.byref(p)


def gd_fwd(p, nseq=3, cu=FAKE, ws=FAKE, n=BIG, **kw):
    t = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, beta=FAKE, init=None, o=FAKE, fin=None)
    t.update(kw)
    return _lib.load().ssd_gdelta_fwd(ref(p), nseq, t["q"], t["k"], t["v"], t["g"], t["beta"], cu,
                                      t["init"], t["o"], t["fin"], ws, n, None)


def gd_bwd(p, nseq=3, cu=FAKE, ws=FAKE, n=BIG, **kw):
    t = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, beta=FAKE, do=FAKE, init=None, dfinal=None, dq=FAKE, dk=FAKE,
             dv=FAKE, dg=FAKE, dbeta=FAKE, dinit=None)
    t.update(kw)
    return _lib.load().ssd_gdelta_bwd(ref(p), nseq, t["q"], t["k"], t["v"], t["g"], t["beta"], cu, t["do"],
                                      t["init"], t["dfinal"], t["dq"], t["dk"], t["dv"], t["dg"],
                                      t["dbeta"], t["dinit"], ws, n, None)


def gd_step(p, slots=FAKE, nslots=4, pos=None, **kw):
    t = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, beta=FAKE, state=FAKE, o=FAKE)
    t.update(kw)
    return _lib.load().ssd_gdelta_step(ref(p), t["q"], t["k"], t["v"], t["g"], t["beta"], slots, nslots,
                                       pos, t["state"], t["o"], None)


def test_gdelta_struct_layout():
    assert ctypes.sizeof(_lib.GatedDelta) == 112


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), -2), (dict(seqlen=0), -2), (dict(nheads=7), -2), (dict(nheads=65536), -2),
    (dict(nkheads=0), -2), (dict(keydim=96), -3), (dict(valdim=48), -3), (dict(act=2), -3),
    (dict(seqlen=1 << 31), -2), (dict(batch=1 << 20, seqlen=1 << 20), -2),
    (dict(q_stride=250), -2), (dict(k_stride=260), -4), (dict(v_stride=1 << 22), -2),
    (dict(o_stride=-512), -2), (dict(dq_stride=300), -4), (dict(g_stride=7), -2),
    (dict(beta_stride=1 << 22), -2),
])
def test_gdelta_problem(kw, code):
    p = gd(**kw)
    assert gd_fwd(p) == code and gd_bwd(p) == code and gd_step(p) == code
    assert ssd.ssd_gdelta_workspace_bytes(p, 3) == 0


def test_gdelta_sequences_and_pointers():
    p = gd()
    assert gd_fwd(None) == -1 and gd_bwd(None) == -1 and gd_step(None) == -1
    assert gd_fwd(p, nseq=0) == -7 and gd_fwd(p, nseq=(1 << 24) + 1) == -7
    assert gd_fwd(p, nseq=3, cu=None) == -7               # rows are sequences: nseq is the batch
    assert gd_fwd(gd(batch=3), nseq=3, cu=FAKE) == -7     # packed sequences: one row
    assert gd_fwd(gd(nheads=65535, nkheads=1), nseq=1 << 20) == -2  # more workgroups than a grid holds
    for name in ("q", "k", "v", "g", "beta", "o"):
        assert gd_fwd(p, **{name: None}) == -1
    for name in ("q", "k", "v", "g", "beta", "do", "dq", "dk", "dv", "dg", "dbeta"):
        assert gd_bwd(p, **{name: None}) == -1
    for name in ("q", "k", "v", "init", "o", "fin", "ws"):
        assert gd_fwd(p, **{name: MISALIGNED}) == -4
    for name in ("q", "do", "init", "dfinal", "dq", "dk", "dv", "dinit", "ws"):
        assert gd_bwd(p, **{name: MISALIGNED}) == -4
    assert gd_fwd(p, cu=FAKE + 2) == -4 and gd_fwd(p, g=FAKE + 1) == -4 and gd_bwd(p, dbeta=FAKE + 2) == -4
    for kind, call in ((ssd.SSD_WS_FORWARD, gd_fwd), (ssd.SSD_WS_BACKWARD, gd_bwd)):
        need = ssd.ssd_gdelta_workspace_bytes(p, 3, kind)
        assert need > 0 and call(p, ws=None) == -5 and call(p, n=need - 1) == -5
    assert ssd.ssd_gdelta_workspace_bytes(p, 3, 2) == 0
    assert ssd.ssd_gdelta_workspace_bytes(p, 0) == 0


def test_gdelta_workspace_does_not_grow_with_the_sequences():
    p = gd(seqlen=32768)
    for kind in (ssd.SSD_WS_FORWARD, ssd.SSD_WS_BACKWARD):
        assert ssd.ssd_gdelta_workspace_bytes(p, 4096, kind) <= ssd.ssd_gdelta_workspace_bytes(p, 1, kind)


def test_gdelta_step_refusals():
    p = gd(batch=4, seqlen=1)
    for name in ("q", "k", "v", "g", "beta", "state", "o"):
        assert gd_step(p, **{name: None}) == -1
    assert gd_step(p, nslots=0) == -2 and gd_step(p, slots=None, nslots=3) == -2
    assert gd_step(p, state=MISALIGNED) == -4 and gd_step(p, slots=FAKE + 2) == -4
    assert gd_step(p, pos=FAKE + 1) == -4
    assert gd_step(gd(batch=1 << 20, seqlen=1, nheads=64), nslots=1 << 20) == -2


def test_tensors_on_the_host_are_refused():
    p = gd(seqlen=3)
    q, v, g = torch.zeros(1, 3, 2, 128, dtype=torch.bfloat16), torch.zeros(1, 3, 8, 64, dtype=torch.bfloat16), torch.zeros(1, 3, 8)
    with pytest.raises(ValueError, match="device tensor"):
        ssd.gdelta_forward(p, q, q, v, g, g)


def block(rows=8, channels=512, act="bf16", res="f32", gate="silu", **kw):
    strides = {k: kw.pop(k) for k in list(kw) if k.endswith("_stride")}
    fields = {k: kw.pop(k) for k in list(kw) if k in ("post_", "center_")}
    p = ssd.make_block_norm(rows=rows, channels=channels, act=act, res=res, gate=gate, **kw)
    for k, v in strides.items():
        setattr(p, k, v)
    for k, v in fields.items():
        setattr(p, k[:-1], v)
    return p


def block_fwd(p, **kw):
    t = dict(x=FAKE, y=FAKE, z=FAKE, scale=FAKE, pw=FAKE, pb=FAKE, w=FAKE, b=FAKE, r=FAKE, h=FAKE)
    t.update(kw)
    return _lib.load().ssd_block_norm_fwd(ref(p), *[t[n] for n in ("x", "y", "z", "scale", "pw", "pb", "w", "b", "r", "h")],
                                          None)


def block_bwd(p, ws=FAKE, n=BIG, **kw):
    names = ("x", "y", "z", "scale", "pw", "pb", "w", "dr", "dh", "dx", "dy", "dz", "ds", "dpw", "dpb", "dw", "db")
    t = dict.fromkeys(names, FAKE)
    t.update(kw)
    return _lib.load().ssd_block_norm_bwd(ref(p), *[t[n_] for n_ in names], ws, n, None)


def test_other_struct_layouts():
    assert ctypes.sizeof(_lib.BlockNorm) == 112 and ctypes.sizeof(_lib.Rope) == 80


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), -2), (dict(rows=1 << 31), -2), (dict(channels=0), -2), (dict(channels=16385), -3),
    (dict(act=2), -3), (dict(act="f32", res="bf16"), -3), (dict(gate=4), -3), (dict(post_=2), -2),
    (dict(center_=-1), -2), (dict(eps=0.0), -2), (dict(eps=float("nan")), -2), (dict(x_stride=511), -2),
    (dict(dz_stride=1 << 28), -2),
])
def test_block_norm_problem(kw, code):
    p = block(**kw)
    assert block_fwd(p) == code and block_bwd(p) == code
    assert ssd.ssd_block_norm_workspace_bytes(p) == 0


def test_block_norm_pointers():
    p = block()
    assert block_fwd(None) == -1 and block_bwd(None) == -1
    for name in ("x", "y", "z", "pw", "w", "r", "h"):
        assert block_fwd(p, **{name: None}) == -1
    for name in ("x", "y", "z", "pw", "w", "dh", "dx", "dy", "dz"):
        assert block_bwd(p, **{name: None}) == -1
    assert block_bwd(block(pre=False), dr=None) == -1
    for name in ("x", "r", "scale", "b"):
        assert block_fwd(p, **{name: FAKE + 2}) == -4
    for name in ("y", "z", "h"):
        assert block_fwd(p, **{name: FAKE + 1}) == -4
    assert block_bwd(p, dr=FAKE + 2) == -4 and block_bwd(p, dpw=FAKE + 1) == -4
    need = ssd.ssd_block_norm_workspace_bytes(p)
    assert need > 0 and block_bwd(p, n=need - 1) == -5 and block_bwd(p, ws=None) == -5


def rope(**kw):
    base = dict(batch=2, seqlen=9, nheads=4, nkheads=2, headdim=64, rotdim=32, act="bf16")
    strides = {k: kw.pop(k) for k in list(kw) if k.endswith("_stride")}
    p = ssd.make_rope(**dict(base, **kw))
    for k, v in strides.items():
        setattr(p, k, v)
    return p


def rope_call(p, nseq=0, inverse=0, **kw):
    t = dict(q=FAKE, k=FAKE, f=FAKE, pos=None, cu=None, qo=FAKE, ko=FAKE)
    t.update(kw)
    return _lib.load().ssd_rope(ref(p), t["q"], t["k"], t["f"], t["pos"], t["cu"], nseq, inverse, t["qo"], t["ko"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), -2), (dict(seqlen=0), -2), (dict(nheads=0), -2), (dict(nkheads=-1), -2),
    (dict(nheads=65536), -2), (dict(headdim=1025), -3), (dict(rotdim=31), -2), (dict(rotdim=66), -2),
    (dict(rotdim=0), -2), (dict(act=2), -3), (dict(style=2), -3), (dict(seqlen=1 << 31), -2),
    (dict(q_stride=255), -2), (dict(ko_stride=1 << 28), -2),
])
def test_rope_problem(kw, code):
    assert rope_call(rope(**kw)) == code


def test_rope_pointers():
    p = rope()
    assert rope_call(None) == -1
    for name in ("q", "k", "f", "qo", "ko"):
        assert rope_call(p, **{name: None}) == -1
    assert rope_call(p, inverse=2) == -2
    assert rope_call(p, cu=FAKE, nseq=2) == -7 and rope_call(rope(batch=1), cu=FAKE, nseq=0) == -7
    assert rope_call(p, q=FAKE + 1) == -4 and rope_call(p, f=FAKE + 4) == -4 and rope_call(p, pos=FAKE + 2) == -4


def test_frequencies():
    f, m = ssd.rope_frequencies(8, base=16.0)
    assert torch.allclose(f, torch.tensor([1.0, 0.5, 0.25, 0.125]).double()) and m == 1.0
    assert torch.allclose(ssd.rope_frequencies(8, scaling="linear", stretch=4.0)[0] * 4, ssd.rope_frequencies(8)[0])
    plain, ntk = ssd.rope_frequencies(64)[0], ssd.rope_frequencies(64, scaling="ntk", stretch=8.0)[0]
    assert ntk[0] == plain[0] and abs(float(ntk[-1] * 8 / plain[-1]) - 1) < 1e-12
    f, m = ssd.rope_frequencies(128, scaling="yarn", stretch=16.0)
    plain = ssd.rope_frequencies(128)[0]
    assert torch.equal(f[:20], plain[:20]) and torch.allclose(f[50:] * 16, plain[50:]) and 1.27 < m < 1.28
    for bad in (dict(rotdim=7), dict(rotdim=8, scaling="other"), dict(rotdim=8, stretch=0.5)):
        with pytest.raises(ValueError):
            ssd.rope_frequencies(**bad)
