"""Group norms that no team of lanes holds: groups wider than 16384 channels, and odd numbers of
more than 512 groups.  They read a group again for every sweep.  Also the gradient of a bias that
is not there.

Tolerances: those of test_gpu_norm, with one magnitude larger.  A centred value is u - m with m =
sum(u) / gs, and float32 leaves the sum off by up to gs 2^-24 of sum |u|, not of |sum u|: of a
group (-1.43, 0.0004, 1.43) the mean of 0.0002 is off by 2^-24 of 0.95, 1e-7 of its middle value's
distance to it.  So the magnitude that goes into u - m is |u| + mean |u|, not |u| + |m|.
"""
import pytest
import torch

import mixer_ref as R
import test_gpu_norm as TN

pytestmark = pytest.mark.gpu


def magnitudes(x, G, mode, center, eps):
    """Magnitudes of y, dx, dz, dweight and dbias (see above and test_gpu_norm)."""
    X, z, w, b = R.f64(x["x"]), R.f64(x["z"]), R.f64(x["w"]).abs(), R.f64(x["b"]).abs()
    n, C = X.shape
    gate = torch.ones_like(X) if z is None else z / (1 + torch.exp(-z))
    u = (X * gate if mode == "before" else X).reshape(n, G, C // G)
    m = u.mean(-1, keepdim=True) * center
    r = 1 / torch.sqrt(((u - m) ** 2).mean(-1, keepdim=True) + eps)
    nn = (u.abs() + u.abs().mean(-1, keepdim=True) * center) * r
    lin = nn.reshape(n, C) * w + b
    dy = R.f64(x["dy"]).abs()
    e = dy * (gate.abs() if mode == "after" else (1.1 + lin if mode == "silu" else 1))
    gw = (e * w).reshape(n, G, C // G)
    du = r * (gw + gw.mean(-1, keepdim=True) + nn * (gw * nn).mean(-1, keepdim=True))
    du = du.reshape(n, C)
    out = dict(y=lin * gate.abs() if mode == "after" else lin,
               dx=du * (gate.abs() if mode == "before" else 1),
               dweight=(e * nn.reshape(n, C)).sum(0), dbias=e.sum(0))
    if z is not None:
        out["dz"] = 1.1 * (du * X.abs() if mode == "before" else dy * lin)
    return out


def assert_norm(x, G, mode, center, act):
    """As in test_gpu_norm, with dbias compared without a bias too (the bias is then zero)."""
    import mamba2_ssd_chunked_amd as ssd
    rows, C = x["x"].shape
    p = ssd.make_norm(rows=rows, channels=C, ngroups=G, act=act, mode=mode, center=center)
    y = ssd.norm_forward(p, x["x"], x["w"], bias=x["b"], z=x["z"])
    g = ssd.norm_backward(p, x["x"], x["w"], x["dy"], bias=x["b"], z=x["z"])
    torch.cuda.synchronize()
    ref = x if x["b"] is not None else dict(x, b=torch.zeros_like(x["w"]))
    want, mag = TN.reference(ref, G, mode, center), magnitudes(ref, G, mode, center, 1e-5)
    got = dict(y=y, dx=g.dx, dz=g.dz, dweight=g.dweight, dbias=g.dbias)
    assert set(want) == {n for n, t in got.items() if t is not None}
    for n in want:
        TN.check(n, got[n], want[n], mag[n], act, C // G, rows if n in ("dweight", "dbias") else 0)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("mode", TN.MODES)
@pytest.mark.parametrize("C,G", [(16385, 1), (40000, 2), (2050, 1025)])
def test_swept_groups(C, G, mode, center, act):
    assert_norm(TN.make(3, C, mode, act), G, mode, center, act)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("C,G,rows", [(16385, 1, 1), (16390, 1, 700), (1539, 513, 2500)])
def test_swept_rows(C, G, rows, act):
    """Fewer and more rows than workgroups that share them; strided and without a bias."""
    assert_norm(TN.make(rows, C, "after", act, bias=False, strided=6), G, "after", True, act)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("mode", TN.MODES)
@pytest.mark.parametrize("C,G", [(512, 4), (333, 3), (5120, 1), (9000, 1), (16384, 1), (16380, 2), (3577, 7)])
def test_without_a_bias(C, G, mode, act):
    assert_norm(TN.make(21, C, mode, act, bias=False), G, mode, mode != "none", act)


def test_swept_groups_in_place():
    """y written over x, gradients crosswise over their inputs."""
    import mamba2_ssd_chunked_amd as ssd
    for mode in ("before", "after"):
        x = TN.make(4, 20000, mode, "bf16")
        p = ssd.make_norm(rows=4, channels=20000, act="bf16", mode=mode, center=True)
        y = ssd.norm_forward(p, x["x"], x["w"], bias=x["b"], z=x["z"])
        g = ssd.norm_backward(p, x["x"], x["w"], x["dy"], bias=x["b"], z=x["z"])
        b = ssd.NormBackwardBuffers.allocate(p, "cuda")
        b.dz, b.dx = x["x"].clone(), x["z"].clone()
        ssd.norm_backward(p, b.dz, x["w"], x["dy"], bias=x["b"], z=b.dx, bufs=b)
        ssd.norm_forward(p, x["x"], x["w"], bias=x["b"], z=x["z"], out=x["x"])
        torch.cuda.synchronize()
        assert torch.equal(x["x"], y) and torch.equal(b.dx, g.dx) and torch.equal(b.dz, g.dz)
        assert torch.equal(b.dweight, g.dweight) and torch.equal(b.dbias, g.dbias)
