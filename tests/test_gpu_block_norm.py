"""The norms around a block on the GPU against the definition, differentiated, in float64.

Tolerances.  A row's statistics are sums of up to 16384 float32 terms, 32 to a thread and then in pairs:
at most 46 steps of 2^-24 on positive terms, so factors of a row are good to 2^-18; exp and 1 / x add
2^-22.  Outputs are compared element by element with 2^-18 of the terms that they are made of (for the
norms' inputs: the gradient before them, its row's mean size and its projection on the row) and, in
bf16, half a step (2^-8) of their value.  Sums over rows, of n terms in some order: n 2^-24 of
the terms' sizes on top of the terms' own 2^-18.
"""
import pytest
import torch

import layer_ref as R

pytestmark = pytest.mark.gpu

ACT = {"bf16": torch.bfloat16, "f32": torch.float32}
CASES = [
    dict(rows=1, C=8, act="f32", res="f32", gate="none"),
    dict(rows=5, C=2048, act="bf16", res="f32", gate="silu"),
    dict(rows=33, C=1120, act="f32", res="f32", gate="none", center=True),
    dict(rows=17, C=291, act="bf16", res="bf16", gate="sigmoid", center=True),
    dict(rows=9, C=1641, act="f32", res="f32", gate="linear", alpha=0.5),
    dict(rows=3, C=4104, act="bf16", res="bf16", gate="silu", alpha=2.0),
    dict(rows=2, C=8200, act="bf16", res="f32", gate="linear"),
    dict(rows=2, C=16384, act="f32", res="f32", gate="silu", center=True),
    dict(rows=2, C=16383, act="bf16", res="f32", gate="none"),
    dict(rows=2100, C=96, act="bf16", res="f32", gate="silu"),
    dict(rows=1100, C=65, act="f32", res="f32", gate="sigmoid"),
    dict(rows=6, C=512, act="bf16", res="bf16", gate="silu", post=False),
    dict(rows=6, C=512, act="bf16", res="f32", gate="none", pre=False),
    dict(rows=6, C=520, act="f32", res="f32", gate="none", post=False, pre=False),
    dict(rows=7, C=640, act="bf16", res="f32", gate="silu", bare=True),
]


def make(rows, C, act, res, gate, center=False, alpha=1.0, post=True, pre=True, bare=False, eps=1e-5, seed=0):
    g = torch.Generator(device="cuda").manual_seed(900 + seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    wide = rnd(rows, 2 * C + 8).to(ACT[act])
    x = dict(x=2 * rnd(rows, C).to(ACT[res]), y=wide[:, :C])
    if gate != "none":
        x["z"] = wide[:, C + 8:] if C % 8 == 0 else wide[:, C + 3:2 * C + 3]
    if not bare:
        x["scale"] = 0.5 + 0.2 * rnd(C)
    for name, want in (("post", post), ("pre", pre)):
        if want:
            x[name + "_weight"] = 1.0 + 0.2 * rnd(C)
            if not bare:
                x[name + "_bias"] = 0.2 * rnd(C)
    return x, dict(gate=gate, center=center, alpha=alpha, eps=eps), dict(
        rows=rows, channels=C, act=act, res=res, post=post, pre=pre, gate=gate, center=center, alpha=alpha, eps=eps)


def grads(x, how, dr, dh):
    """({name: gradient}, {name: size of the terms it is made of}) in float64."""
    t = {n: R.f64(v).requires_grad_(True) for n, v in x.items()}
    r, h = R.block_norm(t, **how)
    outs = [(r, dr)] + ([(h, dh)] if h is not None else [])
    outs = [(o, R.f64(d)) for o, d in outs if d is not None]
    got = torch.autograd.grad([o for o, _ in outs], list(t.values()), [d for _, d in outs])
    return dict(zip(t, got))


def close(name, got, want, terms, extra=0.0, n=0):
    u = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -23
    err = (got.cpu().double() - want).abs()
    bound = u * want.abs() + (2.0 ** -18 + n * 2.0 ** -24) * terms + extra
    assert torch.isfinite(got).all() and (err <= bound).all(), (name, float((err / bound).max()))


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c['act']}-{c['rows']}x{c['C']}-{c['gate']}")
def test_forward(case):
    import mamba2_ssd_chunked_amd as ssd
    x, how, sizes = make(**case)
    r, h = ssd.block_norm_forward(ssd.make_block_norm(**sizes), **x)
    t = {n: R.f64(v) for n, v in x.items()}
    want_r, want_h = R.block_norm(t, **how)
    size = want_r.abs() + 4 * (t["x"].abs() + want_r.abs())
    close("r", r, want_r, size)
    assert (h is None) == (want_h is None)
    if h is not None:
        rms = want_r.square().mean(-1, keepdim=True).sqrt()
        close("h", h, want_h, want_h.abs() + 4 * (1 + size / rms) * (t["pre_weight"].abs() + 1))


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c['act']}-{c['rows']}x{c['C']}-{c['gate']}")
def test_backward(case):
    import mamba2_ssd_chunked_amd as ssd
    x, how, sizes = make(**case)
    rows, C = case["rows"], case["C"]
    g = torch.Generator(device="cuda").manual_seed(77)
    dr = torch.randn(rows, C, generator=g, device="cuda").to(ACT[case["res"]])
    dh = torch.randn(rows, C, generator=g, device="cuda").to(ACT[case["act"]]) if case.get("pre", True) else None
    got = ssd.block_norm_backward(ssd.make_block_norm(**sizes), x["x"], x["y"], dr, dh=dh,
                                  **{n: v for n, v in x.items() if n not in ("x", "y")})
    want = grads(x, how, dr, dh)
    # sizes of terms: G of the residual; du of the block's output; both with their rows' means
    t = {n: R.f64(v) for n, v in x.items()}
    row = lambda v: v.abs() + v.abs().mean(-1, keepdim=True)  # noqa: E731
    r, _ = R.block_norm(t, **how)
    hat = lambda v: 1 + v.abs() / v.square().mean(-1, keepdim=True).sqrt().clamp(min=1e-3)  # noqa: E731
    G = R.f64(dr).abs()
    if dh is not None:
        e = R.f64(dh) * t["pre_weight"]
        rstd = 1 / (r.var(-1, keepdim=True, unbiased=False) if case.get("center") else r.square().mean(-1, keepdim=True)).clamp(min=1e-5).sqrt()
        G = G + 4 * rstd * (row(e) + hat(r) * (e.abs() * hat(r)).mean(-1, keepdim=True))
    close("dx", got.dx, want["x"], 4 * how["alpha"] * G)
    scale = t.get("scale", torch.ones(C, dtype=torch.float64)).abs()
    z = t.get("z")
    f = R.act(how["gate"], z).abs() if z is not None else torch.ones_like(G)
    u = t["y"].abs()
    if case.get("post", True):  # norm(y) w + b may cancel: the sizes of both count
        u = R._norm(t["y"], t["post_weight"], None, how["center"], how["eps"]).abs()
        u = u + t.get("post_bias", torch.zeros(C, dtype=torch.float64)).abs()
    du = scale * G * f
    if z is not None:
        close("dz", got.dz, want["z"], 8 * scale * G * u * (1 + z.abs()))
    dy = du
    if case.get("post", True):
        y = t["y"]
        d = du * t["post_weight"].abs()
        std = (y.var(-1, keepdim=True, unbiased=False) if case.get("center") else y.square().mean(-1, keepdim=True)).clamp(min=1e-5).sqrt()
        dy = 4 * (row(d) + hat(y) * (d * hat(y)).mean(-1, keepdim=True)) / std
    close("dy", got.dy, want["y"], 4 * dy)
    if "scale" in x:
        close("dscale", got.dscale, want["scale"], (4 * G * u * f).sum(0), n=rows)
    for name in ("post", "pre"):
        if name + "_weight" not in x:
            assert getattr(got, f"d{name}_weight") is None
            continue
        base, n_hat = (du, hat(t["y"])) if name == "post" else (R.f64(dh).abs(), hat(r))
        close(name + "_weight", getattr(got, f"d{name}_weight"), want[name + "_weight"], (8 * base * n_hat).sum(0), n=rows)
        if name + "_bias" in x:
            close(name + "_bias", getattr(got, f"d{name}_bias"), want[name + "_bias"], (8 * base).sum(0), n=rows)


def test_in_place_without_dr_streams_and_graphs():
    import mamba2_ssd_chunked_amd as ssd
    x, how, sizes = make(300, 1024, "bf16", "bf16", "silu")
    p = ssd.make_block_norm(**sizes)
    r, h = ssd.block_norm_forward(p, **x)
    y = dict(x, x=x["x"].clone(), y=x["y"].contiguous().clone())
    r2, h2 = ssd.block_norm_forward(p, **y, r=y["x"], h=y["y"])
    assert r2 is y["x"] and torch.equal(r, r2) and torch.equal(h, h2)
    dh = torch.randn_like(h)
    rest = {n: v for n, v in x.items() if n not in ("x", "y")}
    a = ssd.block_norm_backward(p, x["x"], x["y"], None, dh=dh, **rest)
    b = ssd.block_norm_backward(p, x["x"], x["y"], torch.zeros_like(r), dh=dh, **rest, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    names = ("dx", "dy", "dz", "dscale", "dpost_weight", "dpost_bias", "dpre_weight", "dpre_bias")
    for n in names:
        assert torch.equal(getattr(a, n), getattr(b, n)), n
    want = [getattr(a, n).clone() for n in names]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ssd.block_norm_backward(p, x["x"], x["y"], None, dh=dh, **rest, bufs=a)
    for _ in range(3):
        for n in names:
            getattr(a, n).zero_()
        a.ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(getattr(a, n), w) for n, w in zip(names, want))


def test_rows_that_are_not_finite_stay_their_own():
    import mamba2_ssd_chunked_amd as ssd
    x, how, sizes = make(6, 264, "bf16", "f32", "silu")
    p = ssd.make_block_norm(**sizes)
    r, h = ssd.block_norm_forward(p, **x)
    x["y"][2, 3] = float("inf")
    x["x"][4, 7] = float("nan")
    r2, h2 = ssd.block_norm_forward(p, **x)
    ok = [0, 1, 3, 5]
    assert torch.equal(r[ok], r2[ok]) and torch.equal(h[ok], h2[ok])
    assert torch.isnan(h2[2]).any() and torch.isnan(h2[4]).all()


def test_more_rows_than_a_grid_holds_workgroups():
    """2^22 + 5 rows of workgroups of 1024 threads are more threads than a launch may have; in place.  Every y is
    one, so that its norm is 1 / sqrt(1 + eps), one in bf16."""
    import mamba2_ssd_chunked_amd as ssd
    rows, C = (1 << 22) + 5, 3842
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB of free device memory")
    x = torch.zeros(rows, C, dtype=torch.bfloat16, device="cuda")
    y = torch.ones_like(x)
    p = ssd.make_block_norm(rows=rows, channels=C, act="bf16", pre=False, post=True, gate="none", eps=1e-6)
    ssd.block_norm_forward(p, x, y, post_weight=torch.ones(C, device="cuda"), r=x)
    good = all(bool((part == 1).all()) for part in x.split(1 << 18))
    del x, y
    torch.cuda.empty_cache()
    assert good
