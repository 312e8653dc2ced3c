"""Calls of the layer's operators on two streams at once, and captured ones that share no workspace, give the
bits that they give one after the other."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def calls(seed, L=600, H=8, Hk=2, D=64):
    """A function of a stream that runs every operator on its own inputs and returns its outputs."""
    import mamba2_ssd_chunked_amd as ssd
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).bfloat16()  # noqa: E731
    q, k, v, do = unit(rnd(2, L, Hk, D)), unit(rnd(2, L, Hk, D)), rnd(2, L, H, D).bfloat16(), rnd(2, L, H, D).bfloat16()
    gates, beta = -torch.rand(2, L, H, generator=g, device="cuda"), torch.rand(2, L, H, generator=g, device="cuda")
    x, y, z = rnd(2 * L, H * D), rnd(2 * L, H * D).bfloat16(), rnd(2 * L, H * D).bfloat16()
    w1, w2 = rnd(H * D), rnd(H * D)
    freq, _ = ssd.rope_frequencies(D, device="cuda")
    rule = ssd.make_gdelta(batch=2, seqlen=L, nheads=H, nkheads=Hk, keydim=D, valdim=D, act="bf16")
    rope = ssd.make_rope(batch=2, seqlen=L, nheads=Hk, nkheads=Hk, headdim=D, act="bf16")
    norm = ssd.make_block_norm(rows=2 * L, channels=H * D, act="bf16", res="f32", gate="silu")
    torch.cuda.synchronize()

    def run(stream=None):
        a, b = ssd.rope_forward(rope, q, k, freq, stream=stream)
        f = ssd.gdelta_forward(rule, a, b, v, gates, beta, want_final=True, stream=stream)
        d = ssd.gdelta_backward(rule, a, b, v, gates, beta, do, stream=stream)
        r, h = ssd.block_norm_forward(norm, x, y, z=z, post_weight=w1, pre_weight=w2, stream=stream)
        e = ssd.block_norm_backward(norm, x, y, x, y, z=z, post_weight=w1, pre_weight=w2, stream=stream)
        return [a, b, f.o, f.final_state, d.dq, d.dk, d.dv, d.dg, d.dbeta, r, h, e.dx, e.dy, e.dz, e.dscale,
                e.dpost_weight, e.dpre_weight]

    return run


def test_two_streams_at_once():
    one, two = calls(1), calls(2)
    want = [t.clone() for t in one() + two()]
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        got = []
        for s, f in zip(streams, (one, two)):
            got += f(s)
        torch.cuda.synchronize()
        for w, t in zip(want, got):
            assert torch.equal(w, t)


def test_captured_beside_eager_calls():
    one, two = calls(3), calls(4)
    want, other = [t.clone() for t in one()], [t.clone() for t in two()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = one()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        eager = two()
        torch.cuda.synchronize()
        for w, t in zip(want + other, got + eager):
            assert torch.equal(w, t)
