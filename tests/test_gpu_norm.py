"""Group norm with an activation on the GPU against the float64 definition and its
differentiation.

Tolerances.  With u half a step of the activation type (2^-8 bf16, 2^-24 float32), exp and
reciprocals good to 2^-21 (SiLU's exp has an argument of up to about 6, off by 2^-24 of it),
and gs channels to a sum: outputs are off by u of their value once, plus e = (gs + 64) 2^-23
of the magnitudes that went into them (fixed-order partial sums: far below gs steps).  The
magnitudes: |n| |w| + |b| for y, |r| (|g| + mean |g| + |n| mean |g n|) for dx; with
centring n itself is a difference, so |u| + |m| over the deviation takes the place of |n|.
"""
import pytest
import torch

import mixer_ref as R
from ssd_testlib import log

pytestmark = pytest.mark.gpu
ACT = {"bf16": torch.bfloat16, "f32": torch.float32}
MODES = ["none", "silu", "before", "after"]


def make(rows, C, mode, act, bias=True, strided=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(900 + seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    dt = ACT[act]
    wide = lambda: rnd(rows, C + strided).to(dt)[:, strided // 2:strided // 2 + C]  # noqa: E731
    return dict(x=wide(), z=wide() if mode in ("before", "after") else None, w=1 + 0.3 * rnd(C),
                b=0.3 * rnd(C) if bias else None, dy=wide())


def magnitudes(x, G, mode, center, eps):
    """(n, |n| with what cancels in it, r, e-gradient magnitudes) in float64."""
    X, z, w, b = R.f64(x["x"]), R.f64(x["z"]), R.f64(x["w"]).abs(), R.f64(x["b"])
    n, C = X.shape
    gate = torch.ones_like(X) if z is None else z / (1 + torch.exp(-z))
    u = (X * gate if mode == "before" else X).reshape(n, G, C // G)
    m = u.mean(-1, keepdim=True) if center else torch.zeros_like(u[..., :1])
    r = 1 / torch.sqrt(((u - m) ** 2).mean(-1, keepdim=True) + eps)
    nn = (u.abs() + m.abs()) * r
    lin = nn.reshape(n, C) * w + (0 if b is None else b.abs())
    y = lin * gate.abs() if mode == "after" else lin
    e = R.f64(x["dy"]).abs() * (gate.abs() if mode == "after" else (1.1 + lin if mode == "silu" else 1))
    gw = (e * w).reshape(n, G, C // G)
    du = r * (gw + gw.mean(-1, keepdim=True) + nn * (gw * nn).mean(-1, keepdim=True))
    du = du.reshape(n, C)
    out = dict(y=y, dx=du * (gate.abs() if mode == "before" else 1),
               dweight=(e * nn.reshape(n, C)).sum(0), dbias=e.sum(0))
    if z is not None:
        out["dz"] = 1.1 * (du * X.abs() if mode == "before" else R.f64(x["dy"]).abs() * lin)
    return out


def check(what, got, want, mag, act, gs, rows=0):
    got = got.detach().double().cpu()
    e = (gs + rows + 64) * 2.0 ** -23
    u = 2.0 ** -8 if act == "bf16" and what in ("y", "dx", "dz") else 2.0 ** -24
    bad = ((got - want).abs() - u * want.abs()) / (mag + 1e-30)
    log(f"  {what}: worst (|error| - half a step) / magnitudes {float(bad.max()):.2e} "
        f"(tolerance {e:.2e})")
    assert torch.isfinite(got).all(), what
    assert float(bad.max()) <= e, (what, float(bad.max()), e)


def reference(x, G, mode, center, eps=1e-5):
    leaf = lambda t: None if t is None else R.f64(t).requires_grad_(True)  # noqa: E731
    X, z, w, b = leaf(x["x"]), leaf(x["z"]), leaf(x["w"]), leaf(x["b"])
    y = R.norm(X, w, b, z, G, mode, center, eps)
    names = [n for n, t in zip(("dx", "dz", "dweight", "dbias"), (X, z, w, b)) if t is not None]
    grads = torch.autograd.grad(y, [t for t in (X, z, w, b) if t is not None], R.f64(x["dy"]))
    return dict(zip(names, grads), y=y.detach())


def assert_norm(x, G, mode, center, act):
    import mamba2_ssd_chunked_amd as ssd
    rows, C = x["x"].shape
    p = ssd.make_norm(rows=rows, channels=C, ngroups=G, act=act, mode=mode, center=center)
    y = ssd.norm_forward(p, x["x"], x["w"], bias=x["b"], z=x["z"])
    g = ssd.norm_backward(p, x["x"], x["w"], x["dy"], bias=x["b"], z=x["z"])
    torch.cuda.synchronize()
    want = reference(x, G, mode, center)
    mag = magnitudes(x, G, mode, center, 1e-5)
    got = dict(y=y, dx=g.dx, dz=g.dz, dweight=g.dweight, dbias=g.dbias)
    if x["b"] is None:
        want["dbias"] = mag["dbias"] * 0 + R.f64(g.dbias)
    for n in want:
        check(n, got[n], want[n], mag[n], act, C // G, rows if n in ("dweight", "dbias") else 0)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("mode", MODES)
def test_modes(mode, center, act):
    assert_norm(make(37, 512, mode, act), 4, mode, center, act)


# channels per group around every lane and vector border, odd ones among them
@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("C,G", [(1, 1), (2, 2), (7, 1), (24, 3), (40, 5), (64, 1), (96, 2),
                                 (160, 1), (333, 3), (504, 1), (512, 8), (1000, 1), (1032, 1),
                                 (2048, 1), (2056, 1), (4096, 2), (4104, 1), (8192, 1), (10000, 1), (84, 2),
                                 (2004, 1), (8190, 1)])
def test_widths(C, G, act):
    if C // G < 2:
        # a centred group of one channel has no spread: its norm is 0 and not differentiated
        assert_norm(make(5, C, "before", act), G, "before", False, act)
        return
    assert_norm(make(5, C, "before", act), G, "before", True, act)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 2, 63, 257, 2500])
def test_rows(rows, act):
    assert_norm(make(rows, 256, "after", act), 2, "after", True, act)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("strided", [16, 6, 1])
@pytest.mark.parametrize("C,G", [(256, 2), (2048, 1)])
def test_strided_rows(C, G, strided, act):
    """Slices of wider rows, aligned to 16 bytes or to their elements only, without a bias."""
    assert_norm(make(9, C, "before", act, bias=False, strided=strided), G, "before", False, act)


def test_in_place_and_zero_rows():
    """y written over x, gradients over their inputs; a row of zeros gives b and finite grads."""
    import mamba2_ssd_chunked_amd as ssd
    for C, G in ((512, 4), (333, 3)):
        x = make(20, C, "before", "bf16")
        x["x"][3] = 0
        p = ssd.make_norm(rows=20, channels=C, ngroups=G, act="bf16", mode="before")
        y = ssd.norm_forward(p, x["x"], x["w"], bias=x["b"], z=x["z"])
        g = ssd.norm_backward(p, x["x"], x["w"], x["dy"], bias=x["b"], z=x["z"])
        xi, zi = x["x"].clone(), x["z"].clone()
        b = ssd.NormBackwardBuffers.allocate(p, "cuda")
        b.dx, b.dz = zi, xi
        ssd.norm_backward(p, xi, x["w"], x["dy"], bias=x["b"], z=zi, bufs=b)
        ssd.norm_forward(p, x["x"], x["w"], bias=x["b"], z=x["z"], out=x["x"])
        torch.cuda.synchronize()
        assert torch.equal(x["x"], y) and torch.equal(b.dx, g.dx) and torch.equal(b.dz, g.dz)
        assert torch.equal(b.dweight, g.dweight)
        assert torch.equal(y[3], x["b"].to(torch.bfloat16))
        assert torch.isfinite(g.dx).all() and torch.isfinite(g.dz).all()


def test_large_values_and_non_finite_rows():
    """Values far from the others (gates of +-80, x of 1e4) and a row that holds NaN or infinity:
    the other rows are as without it."""
    import mamba2_ssd_chunked_amd as ssd
    x = make(12, 512, "before", "f32")
    x["z"][0, ::2], x["z"][0, 1::2] = 80.0, -80.0
    x["x"][1] *= 1e4
    assert_norm(x, 4, "before", False, "f32")
    p = ssd.make_norm(rows=12, channels=512, ngroups=4, act="f32", mode="before")
    a = ssd.norm_forward(p, x["x"], x["w"], bias=x["b"], z=x["z"])
    x["x"][5, 7], x["x"][8, 300] = float("nan"), float("inf")
    b = ssd.norm_forward(p, x["x"], x["w"], bias=x["b"], z=x["z"])
    torch.cuda.synchronize()
    keep = [i for i in range(12) if i not in (5, 8)]
    assert torch.equal(a[keep], b[keep])
    assert torch.equal(a[5, 128:], b[5, 128:]) and not torch.isfinite(b[5, :128]).any()


def test_repeated_and_replayed_runs_are_bitwise_equal():
    import mamba2_ssd_chunked_amd as ssd
    x = make(3000, 384, "after", "bf16")
    p = ssd.make_norm(rows=3000, channels=384, ngroups=3, act="bf16", mode="after")
    out = torch.empty(3000, 384, dtype=torch.bfloat16, device="cuda")
    b = ssd.NormBackwardBuffers.allocate(p, "cuda")

    def run(out=None, bufs=None):
        y = ssd.norm_forward(p, x["x"], x["w"], bias=x["b"], z=x["z"], out=out)
        return y, ssd.norm_backward(p, x["x"], x["w"], x["dy"], bias=x["b"], z=x["z"], bufs=bufs)

    y, g = run()
    run(out, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(out, b)
    for _ in range(3):
        for t in (out, b.dx, b.dz, b.dweight, b.dbias):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, y)
        for n in ("dx", "dz", "dweight", "dbias"):
            assert torch.equal(getattr(b, n), getattr(g, n)), n
        run()
        torch.cuda.synchronize()


@pytest.mark.parametrize("C,G", [(192, 3), (21, 1), (40000, 1)])
def test_rows_far_apart(C, G):
    """Rows that reach beyond 2^31 elements give what packed ones give."""
    import mamba2_ssd_chunked_amd as ssd
    rows, step = 9, (1 << 28) - 8
    x = make(rows, C, "before", "bf16")
    p = ssd.make_norm(rows=rows, channels=C, ngroups=G, act="bf16", mode="before")
    want = ssd.norm_forward(p, x["x"], x["w"], x["b"], x["z"])
    wg = ssd.norm_backward(p, x["x"], x["w"], x["dy"], x["b"], x["z"])
    far = lambda t: torch.empty(rows * step, dtype=t.dtype, device="cuda").as_strided(  # noqa: E731
        t.shape, (step, 1)).copy_(t)
    out, xx = far(torch.zeros_like(want)), far(x["x"])
    ssd.norm_forward(p, xx, x["w"], x["b"], x["z"], out=out)
    bufs = ssd.NormBackwardBuffers.allocate(p, "cuda")
    bufs.dx = far(bufs.dx)
    got = out.clone()
    ssd.norm_backward(p, xx, x["w"], out.copy_(x["dy"]), x["b"], x["z"], bufs=bufs)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    for n in ("dx", "dz", "dweight", "dbias"):
        assert torch.equal(getattr(bufs, n), getattr(wg, n)), n
