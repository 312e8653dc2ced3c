"""Rotary positions on the GPU against the definition in float64.

Tolerances.  An angle is formed in float64 and loses 2^-53 of its turns (positions up to 2^31, 2^29
turns: 2^-24 of a turn, 2^-21 of the angle's sine); its sine and cosine, the factor, two products and a
sum are seven float32 steps: 2^-21 of the pair's size for positions below 2^20, 2^-19 for all.  bf16
outputs are rounded once, 2^-8 of their value.
"""
import pytest
import torch

import layer_ref as R

pytestmark = pytest.mark.gpu

ACT = {"bf16": torch.bfloat16, "f32": torch.float32}
CASES = [
    dict(b=2, L=33, H=4, K=2, D=128, rot=128, style="half", act="bf16"),
    dict(b=1, L=1, H=1, K=0, D=64, rot=64, style="interleaved", act="f32"),
    dict(b=3, L=7, H=3, K=1, D=80, rot=76, style="interleaved", act="bf16"),
    dict(b=1, L=50, H=2, K=2, D=97, rot=34, style="half", act="f32"),
    dict(b=2, L=5, H=2, K=1, D=96, rot=32, style="half", act="bf16", far=True, factor=1.28),
    dict(b=2, L=9, H=16, K=4, D=128, rot=64, style="interleaved", act="f32", far=True, factor=1.28),
    dict(b=1, L=3, H=1, K=1, D=1024, rot=1024, style="half", act="bf16"),
    dict(b=1, L=4, H=1, K=1, D=2, rot=2, style="half", act="f32", far=True),
    dict(b=4, L=1, H=8, K=2, D=64, rot=64, style="half", act="bf16", far=True),
]


def make(b, L, H, K, D, rot, style, act, far=False, factor=1.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(40 + seed)
    qkv = torch.randn(b, L, (H + 2 * K) * D + 1, generator=g, device="cuda").to(ACT[act])
    q, k = qkv[..., :H * D].unflatten(-1, (H, D)), qkv[..., H * D:(H + K) * D].unflatten(-1, (K, D))
    pos = None
    if far:
        pos = torch.randint(-(1 << 20), 1 << 20, (b, L), generator=g, device="cuda", dtype=torch.int32)
        pos[0, 0] = (1 << 31) - 1
    return q, k if K else None, pos, dict(batch=b, seqlen=L, nheads=H, nkheads=K, headdim=D, rotdim=rot, act=act,
                                          style=style, factor=factor)


def check(got, x, angles, sizes, inverse=False, rows=None):
    want = R.rope(R.f64(x), angles, sizes["factor"], sizes["rotdim"], sizes["style"], inverse)
    rot = sizes["rotdim"]
    a, b = ((slice(0, rot // 2), slice(rot // 2, rot)) if sizes["style"] == "half" else (slice(0, rot, 2), slice(1, rot, 2)))
    pair = torch.zeros_like(want)
    pair[..., a] = pair[..., b] = sizes["factor"] * (R.f64(x)[..., a].abs() + R.f64(x)[..., b].abs())
    u = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
    far = float(angles.abs().max()) > 2.0 ** 21
    err = (got.cpu().double() - want).abs()
    bound = u * want.abs() + 2.0 ** (-19 if far else -21) * pair
    if rows is not None:
        err, bound = err[rows], bound[rows]
    assert (err <= bound).all(), float((err / bound.clamp(min=1e-300)).max())
    assert torch.equal(got[..., rot:], x[..., rot:]) or rows is not None


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c['act']}-{c['D']}-{c['rot']}-{c['style']}")
def test_rope(case, inverse):
    import mamba2_ssd_chunked_amd as ssd
    q, k, pos, sizes = make(**case)
    p = ssd.make_rope(**sizes)
    f, _ = ssd.rope_frequencies(case["rot"], device="cuda")
    call = ssd.rope_backward if inverse else ssd.rope_forward
    gq, gk = call(p, q, k, f, positions=pos)
    b, L = case["b"], case["L"]
    place = torch.arange(L).expand(b, L) if pos is None else pos.cpu()
    angles = place.double()[..., None] * f.cpu()
    check(gq, q, angles, sizes, inverse)
    if k is None:
        assert gk is None
        return
    check(gk, k, angles, sizes, inverse)
    q2, k2 = q.clone(), k.clone()  # in place
    assert call(p, q2, k2, f, positions=pos, out=(q2, k2))[0] is q2
    assert torch.equal(q2, gq) and torch.equal(k2, gk)


def test_packed_sequences():
    import mamba2_ssd_chunked_amd as ssd
    q, k, _, sizes = make(1, 60, 2, 1, 64, 48, "half", "f32")
    p = ssd.make_rope(**sizes)
    f, _ = ssd.rope_frequencies(48, device="cuda")
    cu = torch.tensor([3, 3, 20, 20, 21, 50], dtype=torch.int32, device="cuda")
    out = torch.full_like(q.contiguous(), 7.0), torch.full_like(k.contiguous(), 7.0)
    ssd.rope_forward(p, q, k, f, cu_seqlens=cu, out=out)
    place = torch.cat([torch.zeros(3), torch.arange(17), torch.arange(1), torch.arange(29), torch.zeros(10)])
    rows = torch.zeros(1, 60, dtype=torch.bool)
    rows[:, 3:50] = True
    for got, x in zip(out, (q, k)):
        check(got, x, (place.double()[:, None] * f.cpu())[None], sizes, rows=rows)
        assert (got.cpu()[~rows] == 7.0).all()


def test_gradient_is_the_transposed_turn_and_streams_and_graphs():
    import mamba2_ssd_chunked_amd as ssd
    q, k, pos, sizes = make(2, 30, 4, 2, 128, 96, "interleaved", "f32", far=True, factor=1.3)
    p = ssd.make_rope(**sizes)
    f, _ = ssd.rope_frequencies(96, scaling="yarn", stretch=8.0, device="cuda")
    out = ssd.rope_forward(p, q, k, f, positions=pos)
    d = [torch.randn_like(t) for t in out]
    back = ssd.rope_backward(p, *d, f, positions=pos)
    for x, o, g, b in zip((q, k), out, d, back):  # <out, d> = <x, back>
        lhs, rhs = (o.double() * g.double()).sum(), (x.double() * b.double()).sum()
        assert abs(lhs - rhs) <= 2.0 ** -20 * (o.double().norm() * g.double().norm())
    side = torch.cuda.Stream()
    again = ssd.rope_forward(p, q, k, f, positions=pos, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, again))
    want = [t.clone() for t in out]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ssd.rope_forward(p, q, k, f, positions=pos, out=out)
    for _ in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
