"""A layer of the operators as a model runs them: queries and keys made unit length, turned by their
positions, the gated delta rule, and the norms around the block with its gate and the residual
stream; forward and gradients against autograd of the same formulas in float64, then the same layer
token by token.

Tolerances, of norms.  Every stage leaves 2^-20 of its result or less in float32 (the bounds of the
operators' own tests) and passes on an error of its inputs at most a few times enlarged: turning not
at all, the rule by the keys and betas, which enter twice (u_t reads S k_t and S gains u_t k_t^T), the
norms by 1 + the share of a row's mean square.  Five stages forward and as many back, 2^3 each: 80
2^-20 < 2^-13.  In bf16 a rounded tensor is off by 2^-9 of its norm.  Forward four are between the
input and h (two of q and k, turned twice, o, h), the keys' doubly; 8 2^-9 = 2^-6.  Backward the
same ones are read again and do, dq and dk rounded twice and dv once: 16 2^-9 = 2^-5.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

ACT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def unit(x):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * x.shape[-1] ** -0.5


def turned(x, angles):
    a, b = x.chunk(2, -1)
    c, s = torch.cos(angles)[:, None], torch.sin(angles)[:, None]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def layer(t, freq, seqs, scale, share):
    """(r, h) of float64 leaves."""
    outs = []
    for at, n in seqs:
        sl = slice(at, at + n)
        angles = torch.arange(n, dtype=torch.float64)[:, None] * freq
        q, k = (turned(unit(t[x][sl]), angles).repeat_interleave(share, 1) for x in "qk")
        v, g, beta = t["v"][sl], t["g"][sl], t["beta"][sl]
        S = torch.zeros(v.shape[1], v.shape[2], k.shape[2], dtype=torch.float64)
        for i in range(n):
            S = torch.exp(g[i])[:, None, None] * S
            u = beta[i][:, None] * (v[i] - (S * k[i][:, None]).sum(-1))
            S = S + u[:, :, None] * k[i][:, None]
            outs.append(scale * (S * q[i][:, None]).sum(-1).flatten())
    y = torch.stack(outs)
    y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * t["post"]
    r = t["x"] + t["scale"] * (y * t["z"] * torch.sigmoid(t["z"]))
    return r, r / torch.sqrt((r * r).mean(-1, keepdim=True) + EPS) * t["pre"]


class Layer:
    """The same by the library: packed sequences of one row."""

    def __init__(self, t, act, lens, H, Hk, Dk, Dv):
        import mamba2_ssd_chunked_amd as ssd
        self.ssd, self.t, self.dims = ssd, t, (H, Hk, Dk, Dv)
        L, C = sum(lens), H * Dv
        self.cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
        self.freq, _ = ssd.rope_frequencies(Dk, device="cuda")
        self.w = torch.full((Dk,), Dk ** -0.5, device="cuda")
        sizes = dict(batch=1, seqlen=L, act=act)
        self.norm = ssd.make_norm(rows=L * Hk, channels=Dk, act=act, mode="none", eps=EPS)
        self.rope = ssd.make_rope(nheads=Hk, nkheads=Hk, headdim=Dk, **sizes)
        self.rule = ssd.make_gdelta(nheads=H, nkheads=Hk, keydim=Dk, valdim=Dv, scale=Dk ** -0.5, **sizes)
        self.block = ssd.make_block_norm(rows=L, channels=C, act=act, res="f32", pre=True, post=True,
                                         gate="silu", eps=EPS)

    def forward(self):
        ssd, t, (H, Hk, Dk, Dv) = self.ssd, self.t, self.dims
        q, k = (ssd.norm_forward(self.norm, t[n].reshape(-1, Dk), self.w).view(1, -1, Hk, Dk) for n in "qk")
        self.q, self.k = ssd.rope_forward(self.rope, q, k, self.freq, cu_seqlens=self.cu, out=(q, k))
        o = ssd.gdelta_forward(self.rule, self.q, self.k, t["v"][None], t["g"][None], t["beta"][None],
                               cu_seqlens=self.cu).o
        self.y = o.view(-1, H * Dv)
        self.r, self.h = ssd.block_norm_forward(self.block, t["x"], self.y, z=t["z"], scale=t["scale"],
                                                post_weight=t["post"], pre_weight=t["pre"])
        return self.r, self.h

    def backward(self, dr, dh):
        ssd, t, (H, Hk, Dk, Dv) = self.ssd, self.t, self.dims
        n = ssd.block_norm_backward(self.block, t["x"], self.y, dr, dh, z=t["z"], scale=t["scale"],
                                    post_weight=t["post"], pre_weight=t["pre"])
        b = ssd.gdelta_backward(self.rule, self.q, self.k, t["v"][None], t["g"][None], t["beta"][None],
                                n.dy.view(1, -1, H, Dv), cu_seqlens=self.cu)
        dq, dk = ssd.rope_backward(self.rope, b.dq, b.dk, self.freq, cu_seqlens=self.cu, out=(b.dq, b.dk))
        norm = lambda x, d: ssd.norm_backward(self.norm, x.reshape(-1, Dk), self.w,  # noqa: E731
                                              d.reshape(-1, Dk)).dx.view(x.shape)
        return dict(q=norm(t["q"], dq), k=norm(t["k"], dk), v=b.dv[0], g=b.dg[0], beta=b.dbeta[0], z=n.dz,
                    x=n.dx, scale=n.dscale, post=n.dpost_weight, pre=n.dpre_weight)


def make(act, lens, H, Hk, Dk, Dv):
    g = torch.Generator(device="cuda").manual_seed(11)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    L, C, dt = sum(lens), H * Dv, ACT[act]
    mixed = rnd(L, 2 * Hk * Dk + 2 * C).to(dt)  # one projection's output; v and z are read in place
    q, k, v, z = mixed.split([Hk * Dk, Hk * Dk, C, C], dim=-1)
    return dict(q=q.unflatten(-1, (Hk, Dk)), k=k.unflatten(-1, (Hk, Dk)), v=v.unflatten(-1, (H, Dv)), z=z,
                g=-torch.exp(rnd(L, H) - 2), beta=torch.sigmoid(rnd(L, H)), x=rnd(L, C), scale=rnd(C),
                post=1 + 0.1 * rnd(C), pre=1 + 0.1 * rnd(C)), (rnd(L, C), rnd(L, C).to(dt))


SIZES = dict(lens=[70, 1, 133], H=4, Hk=2, Dk=64, Dv=64)


def reference(t, lens, H, Hk, Dk, Dv):
    import mamba2_ssd_chunked_amd as ssd
    leaves = {n: x.detach().cpu().double().requires_grad_() for n, x in t.items()}
    seqs = [(sum(lens[:i]), n) for i, n in enumerate(lens)]
    return leaves, layer(leaves, ssd.rope_frequencies(Dk)[0], seqs, Dk ** -0.5, H // Hk)


def off(got, want):
    return float((got.cpu().double() - want.detach()).norm() / want.detach().norm())


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_layer(act):
    t, (dr, dh) = make(act, **SIZES)
    m = Layer(t, act, **SIZES)
    r, h = m.forward()
    grads = m.backward(dr, dh)
    leaves, (r64, h64) = reference(t, **SIZES)
    bound = 2.0 ** -13 if act == "f32" else 2.0 ** -6
    assert off(r, r64) <= bound and off(h, h64) <= bound
    ((r64 * dr.cpu().double()).sum() + (h64 * dh.cpu().double()).sum()).backward()
    for n, got in grads.items():
        assert off(got, leaves[n].grad) <= bound * 2, n


def test_gradients_against_differences():
    """(f(x + e d) - f(x - e d)) / 2e of the float64 formulas along random directions d: central differences
    leave e^2 of f's third derivative and 2^-53 f / e; e = 1e-5 leaves 1e-9 or less of f's scale, while the
    gradients are good to 2^-12 of their norm, which a random direction of N values sees as an error of
    2^-12 |grad| / sqrt(N) |d|, allowed five times."""
    t, (dr, dh) = make("f32", **SIZES)
    m = Layer(t, "f32", **SIZES)
    m.forward()
    grads = m.backward(dr, dh)
    leaves, _ = reference(t, **SIZES)
    seqs = [(sum(SIZES["lens"][:i]), n) for i, n in enumerate(SIZES["lens"])]
    f = lambda y: (lambda o: float((o[0] * dr.cpu().double()).sum() + (o[1] * dh.cpu().double()).sum()))(  # noqa: E731
        layer(y, m.freq.cpu(), seqs, SIZES["Dk"] ** -0.5, 2))
    gen = torch.Generator().manual_seed(5)
    with torch.no_grad():
        for n, got in grads.items():
            d = torch.randn(leaves[n].shape, generator=gen, dtype=torch.float64)
            d, e = d / d.norm(), 1e-5
            step = (f(dict(leaves, **{n: leaves[n] + e * d})) - f(dict(leaves, **{n: leaves[n] - e * d}))) / (2 * e)
            want = float((got.cpu().double() * d).sum())
            size = float(got.norm()) / d.numel() ** 0.5
            assert abs(step - want) <= 5 * 2.0 ** -12 * size + 1e-6, (n, step, want)


def test_layer_token_by_token_in_a_graph():
    """A captured step of three rows, replayed for every token with positions that the graph's own inputs give,
    against the layer over the whole sequences; float32, so that both are within 2^-13 of the same values."""
    import mamba2_ssd_chunked_amd as ssd
    n, H, Hk, Dk, Dv = 40, 4, 2, 64, 64
    sizes = dict(lens=[n] * 3, H=H, Hk=Hk, Dk=Dk, Dv=Dv)
    t, _ = make("f32", **sizes)
    r_all, h_all = Layer(t, "f32", **sizes).forward()
    at = {x: y.unflatten(0, (3, n))[:, 0].clone() for x, y in t.items() if y.shape[0] == 3 * n}
    step = dict(batch=3, seqlen=1, act="f32")
    norm = ssd.make_norm(rows=3 * Hk, channels=Dk, act="f32", mode="none", eps=EPS)
    rope = ssd.make_rope(nheads=Hk, nkheads=Hk, headdim=Dk, **step)
    rule = ssd.make_gdelta(nheads=H, nkheads=Hk, keydim=Dk, valdim=Dv, scale=Dk ** -0.5, **step)
    block = ssd.make_block_norm(rows=3, channels=H * Dv, act="f32", pre=True, post=True, gate="silu", eps=EPS)
    freq, _ = ssd.rope_frequencies(Dk, device="cuda")
    w = torch.full((Dk,), Dk ** -0.5, device="cuda")
    pos = torch.zeros(3, 1, dtype=torch.int32, device="cuda")
    slots = torch.tensor([4, 1, 2], dtype=torch.int32, device="cuda")
    pool = torch.full((5, H, Dv, Dk), 3.0, device="cuda")  # position 0 starts from zero whatever was there

    def run():
        q, k = (ssd.norm_forward(norm, at[x].reshape(-1, Dk), w).view(3, 1, Hk, Dk) for x in "qk")
        q, k = ssd.rope_forward(rope, q, k, freq, positions=pos, out=(q, k))
        o = torch.empty(3, 1, H, Dv, device="cuda")
        ssd.ssd_gdelta_step(rule, q, k, at["v"][:, None], at["g"][:, None], at["beta"][:, None], pool, o,
                            slots=slots, positions=pos[:, 0])
        return ssd.block_norm_forward(block, at["x"], o.view(3, -1), z=at["z"], scale=t["scale"],
                                      post_weight=t["post"], pre_weight=t["pre"])

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, h = run()
    for i in range(n):
        for x in at:
            at[x].copy_(t[x].unflatten(0, (3, n))[:, i])
        pos.fill_(i)
        graph.replay()
        torch.cuda.synchronize()
        for got, whole in ((r, r_all), (h, h_all)):
            want = whole.unflatten(0, (3, n))[:, i]
            assert off(got, want.cpu().double()) <= 2.0 ** -12, i
    assert (pool[[0, 3]] == 3.0).all()
