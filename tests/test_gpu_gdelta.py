"""The gated delta rule on the GPU against the float64 recurrence.

Tolerances.  With keys of length one, decays up to 1 and betas in [0, 1] a step never lengthens an
error of the state, and the entries of the chunks' inverses are at most 1, so that errors are bounded
by what each product leaves out of values of the sizes U (largest |u|) and S (largest state norm):
  bf16 outputs, element by element: 2^-8 of the value (one rounding) and 2^-16 of the terms of each
      product on the way, whose magnitudes sum up to S (states: Cauchy-Schwarz) or to 64 U (a chunk's
      tokens); a chunk forms u from X (S) and T R (64 (U + S) in two parts each), then o from S and P u
  norms: the root mean square of roundings to bf16 is 2^-8 / sqrt(3) of a value at the bottom of a
      binade and half of that at the top, 1.66e-3 over a whole; 2^-9 leaves 17 % for everything else
  float32 outputs: three parts leave out 2^-24 per product, sums of n float32 terms sqrt(n) 2^-25 of
      their size: 5 products and sums of up to 256 terms are 13 steps of 2^-24; 2^-20 are 16.  dg_t is
      a sum over the tokens i from t to the chunk's end of q_i . dq_i - v_i . dv_i, which may cancel:
      its error is that of the terms, 2^-20 of |v_i| |dv_i| each, added as independent ones, besides
      the 2^-19 of its own size (two such sums).
"""
import pytest
import torch

import layer_ref as R
from ssd_testlib import log

pytestmark = pytest.mark.gpu

ACT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(lens, H, Hk, Dk, Dv, act, *, packed=True, before=0, behind=0, init=True, fused=False, seed=0,
         keys="random", gates="model"):
    """Inputs on the GPU: packed sequences with `before` and `behind` tokens outside them, or equal
    rows."""
    g = torch.Generator(device="cuda").manual_seed(500 + seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    if packed:
        b, L, at, seqs = 1, before + sum(lens) + behind, before, []
        for n in lens:
            seqs.append((at, n))
            at += n
        cu = torch.tensor([s for s, _ in seqs] + [at], dtype=torch.int32, device="cuda")
    else:
        b, L, cu = len(lens), lens[0], None
        seqs = [(i * L, L) for i in range(b)]
    dt = ACT[act]
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    q, k, v = unit(rnd(b, L, Hk, Dk)), unit(rnd(b, L, Hk, Dk)), rnd(b, L, H, Dv)
    if keys == "same":  # every key nearly the same: the hardest triangular systems
        k = unit(k[:, :1] + 0.03 * k)
    q, k, v = q.to(dt), k.to(dt), v.to(dt)
    if fused:
        x = torch.cat([t.flatten(2) for t in (q, k, v)] + [rnd(b, L, 16).to(dt)], dim=-1)
        q, k, v, _ = x.split([Hk * Dk, Hk * Dk, H * Dv, 16], dim=-1)
        q, k, v = q.unflatten(-1, (Hk, Dk)), k.unflatten(-1, (Hk, Dk)), v.unflatten(-1, (H, Dv))
    wide = rnd(b, L, 2 * H + 3)  # g and beta as views of wider rows
    ld, beta = wide[..., :H], wide[..., H + 1:2 * H + 1]
    ld.copy_(-torch.exp(2 * ld - 2)), beta.copy_(torch.sigmoid(beta))
    if gates == "edges":
        ld[:, ::5], ld[:, 3::7] = 0.0, -float("inf")
        beta[:, ::4], beta[:, 1::6] = 0.0, 1.0
        beta[:, 2::9] = 1e-30
        ld[:, 4::11] = -200.0
    n = len(lens)
    return dict(q=q, k=k, v=v, g=ld, beta=beta, cu=cu, seqs=seqs, scale=Dk ** -0.5, act=act,
                init=rnd(n, H, Dv, Dk) * Dk ** -0.5 if init else None, do=rnd(b, L, H, Dv).to(dt),
                dfinal=rnd(n, H, Dv, Dk) * Dk ** -0.5 if init else None, dims=(b, L, H, Hk, Dk, Dv))


def problem(x):
    import mamba2_ssd_chunked_amd as ssd
    b, L, H, Hk, Dk, Dv = x["dims"]
    return ssd.make_gdelta(batch=b, seqlen=L, nheads=H, nkheads=Hk, keydim=Dk, valdim=Dv, act=x["act"],
                           scale=x["scale"])


def flat(x, *names):
    return [x[n].flatten(0, 1) for n in names]


def live_rows(x):
    rows = torch.zeros(x["dims"][0] * x["dims"][1], dtype=torch.bool)
    for at, n in x["seqs"]:
        rows[at:at + n] = True
    return rows


def summed_terms(x, dv):
    """Norm of what dg sums: root of the summed squares of |v_i| |dv_i| from t to the chunk's end."""
    size = f64_norm(x["v"].flatten(0, 1)) * dv.norm(dim=-1)
    total = 0.0
    for at, n in x["seqs"]:
        for c in range(at, at + n, 64):
            part = size[c:min(c + 64, at + n)] ** 2
            total += float(part.flip(0).cumsum(0).sum())
    return total ** 0.5


def f64_norm(t):
    return R.f64(t).norm(dim=-1)


def near(name, got, want, act, rel32=2.0 ** -20, terms=0.0):
    got, norm = got.cpu().double(), float(want.norm())
    off = float((got - want).norm())
    bound = 2.0 ** -9 if act == "bf16" else rel32
    log(f"{name}: {off / max(norm, 1e-300):.3g} (bound {bound:.3g})")
    assert torch.isfinite(got).all() and off <= bound * norm + 2.0 ** -20 * terms + 1e-30, name


def check_forward(x, want_final=True):
    import mamba2_ssd_chunked_amd as ssd
    p, rows = problem(x), live_rows(x)
    bufs = ssd.GatedDeltaForwardBuffers.allocate(p, len(x["seqs"]), "cuda", final=want_final)
    bufs.o.fill_(7.0)
    ssd.gdelta_forward(p, x["q"], x["k"], x["v"], x["g"], x["beta"], cu_seqlens=x["cu"], init=x["init"],
                       bufs=bufs, want_final=want_final)
    o, fin, U, S = R.gdelta_fwd(*flat(x, "q", "k", "v", "g", "beta"), x["scale"], x["seqs"], x["init"])
    got = bufs.o.flatten(0, 1).cpu()
    assert (got[~rows] == 7.0).all()
    near("o", got[rows], o[rows], x["act"])
    if x["act"] == "bf16":
        terms = x["scale"] * (S + 2 * 64 * (U + S) + 3 * 64 * U)
        assert ((got.double() - o).abs()[rows] <= 2.0 ** -8 * o.abs()[rows] + 2.0 ** -16 * terms).all()
    if want_final:
        near("final", bufs.final_state, fin, "f32")


def check_backward(x, want_dinit=True):
    import mamba2_ssd_chunked_amd as ssd
    p, rows = problem(x), live_rows(x)
    bufs = ssd.GatedDeltaBackwardBuffers.allocate(p, len(x["seqs"]), "cuda", dinit=want_dinit)
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        getattr(bufs, n).fill_(7.0)
    ssd.gdelta_backward(p, x["q"], x["k"], x["v"], x["g"], x["beta"], x["do"], cu_seqlens=x["cu"],
                        init=x["init"], dfinal=x["dfinal"], bufs=bufs, want_dinit=want_dinit)
    want = R.gdelta_bwd(*flat(x, "q", "k", "v", "g", "beta"), x["scale"], x["seqs"],
                        x["do"].flatten(0, 1), x["init"], x["dfinal"])
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        got = getattr(bufs, n).flatten(0, 1).cpu()
        assert (got[~rows] == 7.0).all(), n
        near(n, got[rows], want[n][rows], "f32" if n in ("dg", "dbeta") else x["act"],
             *((2.0 ** -19, summed_terms(x, want["dv"])) if n == "dg" else ()))
    if want_dinit:
        near("dinit", bufs.dinit, want["dinit"], "f32")


CASES = [
    dict(lens=[1], H=1, Hk=1, Dk=64, Dv=64, act="f32"),
    dict(lens=[64], H=2, Hk=1, Dk=128, Dv=64, act="bf16"),
    dict(lens=[65], H=1, Hk=1, Dk=64, Dv=128, act="bf16"),
    dict(lens=[3, 0, 130, 1, 63], H=4, Hk=2, Dk=128, Dv=128, act="bf16", before=5, behind=9, fused=True),
    dict(lens=[3, 0, 130, 1, 63], H=2, Hk=2, Dk=128, Dv=128, act="f32", before=2, behind=70, fused=True),
    dict(lens=[100, 100], H=6, Hk=2, Dk=64, Dv=64, act="bf16", packed=False),
    dict(lens=[127, 127, 127], H=3, Hk=1, Dk=64, Dv=128, act="f32", packed=False, init=False),
    dict(lens=[700], H=2, Hk=1, Dk=128, Dv=128, act="bf16", init=False),
    dict(lens=[33, 200], H=2, Hk=1, Dk=64, Dv=64, act="bf16", gates="edges"),
    dict(lens=[33, 200], H=2, Hk=2, Dk=128, Dv=64, act="f32", gates="edges"),
    dict(lens=[150], H=2, Hk=2, Dk=128, Dv=64, act="bf16", keys="same"),
    dict(lens=[150], H=2, Hk=1, Dk=64, Dv=64, act="f32", keys="same"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c['act']}-{c['Dk']}x{c['Dv']}-{c['lens'][0]}")
def test_forward(case):
    check_forward(make(**case))


def test_forward_without_final_state():
    check_forward(make([77, 190], 4, 2, 128, 128, "bf16"), want_final=False)
    check_forward(make([77, 190], 4, 2, 64, 64, "bf16", init=False), want_final=False)


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c['act']}-{c['Dk']}x{c['Dv']}-{c['lens'][0]}")
def test_backward(case):
    check_backward(make(**case), want_dinit=case.get("init", True))


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_step_continues_a_prompt(act):
    """Prompt of 70 tokens, then single tokens and a call of three, against the whole sequence."""
    import mamba2_ssd_chunked_amd as ssd
    x = make([75, 75, 75], 4, 2, 128, 64, act, packed=False, init=False, fused=True)
    b, L, H, Hk, Dk, Dv = x["dims"]
    o, fin, U, S = R.gdelta_fwd(*flat(x, "q", "k", "v", "g", "beta"), x["scale"], x["seqs"])
    o = o.reshape(b, L, H, Dv)
    cut = lambda n, i, j: x[n][:, i:j].contiguous()  # noqa: E731
    part = lambda i, j: [cut(n, i, j) for n in ("q", "k", "v", "g", "beta")]  # noqa: E731
    sizes = dict(batch=b, nheads=H, nkheads=Hk, keydim=Dk, valdim=Dv, act=act, scale=x["scale"])
    f = ssd.gdelta_forward(ssd.make_gdelta(seqlen=70, **sizes), *part(0, 70), want_final=True)
    pool = torch.full((5, H, Dv, Dk), float("nan"), device="cuda")
    slots = torch.tensor([3, 0, 4], dtype=torch.int32, device="cuda")
    pool[slots.long()] = f.final_state
    for i, j in ((70, 71), (71, 72), (72, 75)):
        out = torch.empty(b, j - i, H, Dv, dtype=ACT[act], device="cuda")
        ssd.ssd_gdelta_step(ssd.make_gdelta(seqlen=j - i, **sizes), *part(i, j), pool, out, slots=slots)
        near(f"step {i}", out, o[:, i:j], act)
    near("state", pool[slots.long()], fin, "f32")
    assert torch.isnan(pool[1]).all() and torch.isnan(pool[2]).all()


def test_step_padding_repeats_and_fresh_rows():
    import mamba2_ssd_chunked_amd as ssd
    x = make([1] * 6, 2, 1, 64, 128, "f32", packed=False)
    b, L, H, Hk, Dk, Dv = x["dims"]
    p = problem(x)
    pool = torch.randn(4, H, Dv, Dk, device="cuda", generator=torch.Generator("cuda").manual_seed(1)) * 0.1
    old = pool.clone()
    slots = torch.tensor([2, -1, 2, 9, 0, 3], dtype=torch.int32, device="cuda")
    pos = torch.tensor([5, 5, 5, 5, 0, -1], dtype=torch.int32, device="cuda")
    out = torch.full((b, 1, H, Dv), 7.0, device="cuda")
    ssd.ssd_gdelta_step(p, x["q"], x["k"], x["v"], x["g"], x["beta"], pool, out, slots=slots, positions=pos)
    init = torch.stack([old[2], torch.zeros_like(old[0])])
    ids = torch.tensor([0, 4], device="cuda")
    o, fin, _, _ = R.gdelta_fwd(*[x[n][ids, 0] for n in ("q", "k", "v", "g", "beta")], x["scale"],
                                [(0, 1), (1, 1)], init)
    near("o", out[ids, 0], o, "f32")
    near("state", pool[[2, 0]], fin, "f32")
    assert (out[[1, 2, 3, 5]] == 7.0).all() and torch.equal(pool[[1, 3]], old[[1, 3]])


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_values_that_are_not_finite(act):
    """They reach no other sequence, no earlier token and, of v, no other channel."""
    import mamba2_ssd_chunked_amd as ssd
    x = make([70, 90, 40], 2, 1, 64, 64, act)
    p = problem(x)
    run = lambda y: ssd.gdelta_forward(p, y["q"], y["k"], y["v"], y["g"], y["beta"], cu_seqlens=y["cu"],  # noqa: E731
                                       init=y["init"], want_final=True)
    good = run(x)
    for name, at, bad in (("v", 100, float("inf")), ("v", 70, float("nan")), ("k", 141, float("nan")),
                          ("beta", 75, float("inf")), ("g", 130, float("nan")), ("q", 99, float("inf"))):
        y = dict(x, **{name: x[name].clone()})
        if name in ("g", "beta"):
            y[name][0, at, 1] = bad
        else:
            y[name][0, at, 0, 5] = bad
        f = run(y)
        same = torch.ones_like(good.o, dtype=torch.bool)
        if name == "q":
            same[0, at] = False
        elif name == "v":
            same[0, at:160, 0, 5] = False
        elif name == "k":
            same[0, at:160] = False
        else:
            same[0, at:160, 1] = False
        assert torch.equal(f.o[same], good.o[same]), (name, at)
        assert not torch.isfinite(f.o[~same]).any(), (name, at)
        keep = torch.ones_like(good.final_state, dtype=torch.bool)
        if name == "v":
            keep[1, 0, 5] = False
        elif name == "k":
            keep[1] = False
        elif name != "q":
            keep[1, 1] = False
        assert torch.equal(f.final_state[keep], good.final_state[keep]), (name, at)
        assert not torch.isfinite(f.final_state[~keep]).any(), (name, at)
        do = x["do"]
        good_b = ssd.gdelta_backward(p, *[x[n] for n in ("q", "k", "v", "g", "beta")], do, cu_seqlens=x["cu"],
                                     init=x["init"])
        bad_b = ssd.gdelta_backward(p, *[y[n] for n in ("q", "k", "v", "g", "beta")], do, cu_seqlens=x["cu"],
                                    init=x["init"])
        for n in ("dq", "dk", "dv", "dg", "dbeta"):
            u, w = getattr(good_b, n), getattr(bad_b, n)
            assert torch.equal(u[0, :70], w[0, :70]) and torch.equal(u[0, 160:], w[0, 160:]), (name, n)


def test_repeats_streams_and_graphs():
    import mamba2_ssd_chunked_amd as ssd
    x = make([70, 0, 190], 4, 2, 128, 64, "bf16")
    p = problem(x)
    ins = [x[n] for n in ("q", "k", "v", "g", "beta")]
    fwd = lambda bufs=None, stream=None: ssd.gdelta_forward(  # noqa: E731
        p, *ins, cu_seqlens=x["cu"], init=x["init"], bufs=bufs, stream=stream, want_final=True)
    bwd = lambda bufs=None, stream=None: ssd.gdelta_backward(  # noqa: E731
        p, *ins, x["do"], cu_seqlens=x["cu"], init=x["init"], dfinal=x["dfinal"], bufs=bufs, stream=stream,
        want_dinit=True)
    names = ("dq", "dk", "dv", "dg", "dbeta", "dinit")
    f, b = fwd(), bwd()
    want = [f.o, f.final_state] + [getattr(b, n) for n in names]
    side = torch.cuda.Stream()
    f2, b2 = fwd(stream=side), bwd(stream=side)
    torch.cuda.synchronize()
    for w, got in zip(want, [f2.o, f2.final_state] + [getattr(b2, n) for n in names]):
        assert torch.equal(w, got)
    want = [w.clone() for w in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fwd(bufs=f)
        bwd(bufs=b)
    got = [f.o, f.final_state] + [getattr(b, n) for n in names]
    for _ in range(3):
        for t in got:
            t.zero_()
        f.ws.fill_(255), b.ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        for w, t in zip(want, got):
            assert torch.equal(w, t)
