"""Linear attention with a decay per head on the GPU against the float64 recurrence.

Tolerances.  With A the result of the same recurrence on absolute values (so A bounds the
sum of the magnitudes of all terms), u half a step of the activation type (2^-8 bf16):
  bf16 outputs  (2 u + 2^-14) A: one rounding of an operand of the last products (the
                scores or the state: each term carries one of them), one of the result
  bf16 states   2^-15 A: the weighted values enter as the sum of two bf16 (2^-16), the
                rest is float32
  float32       (Dk + Dv + 4 nchunks + 160) 2^-24 A: sums of Dk or Dv and up to 64 terms,
                and a decay per chunk
Gradients that sum r heads: A sums them too, and float32 adds r steps of 2^-24.
"""
import pytest
import torch

import mixer_ref as R
from ssd_testlib import log

pytestmark = pytest.mark.gpu

ACT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(lens, H, Hk, Dk, Dv, act, *, packed=True, behind=0, before=0, init=True, fused=False,
         seed=0, decay=None):
    """Inputs on the GPU: packed sequences with `before` and `behind` tokens outside them, or
    equal rows."""
    g = torch.Generator(device="cuda").manual_seed(100 + seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    if packed:
        b, L = 1, before + sum(lens) + behind
        at = before
        seqs = []
        for n in lens:
            seqs.append((at, n))
            at += n
        cu = torch.tensor([s for s, _ in seqs] + [at], dtype=torch.int32, device="cuda")
    else:
        b, L, cu = len(lens), lens[0], None
        seqs = [(i * L, L) for i in range(b)]
    dt = ACT[act]
    if fused:
        x = rnd(b, L, H * Dk + Hk * Dk + Hk * Dv + 16).to(dt)
        q, k, v, _ = x.split([H * Dk, Hk * Dk, Hk * Dv, 16], dim=-1)
        q, k, v = q.unflatten(-1, (H, Dk)), k.unflatten(-1, (Hk, Dk)), v.unflatten(-1, (Hk, Dv))
    else:
        q, k, v = rnd(b, L, H, Dk).to(dt), rnd(b, L, Hk, Dk).to(dt), rnd(b, L, Hk, Dv).to(dt)
    ld = -torch.exp2(-7.0 * torch.arange(1, H + 1, device="cuda") / H) if decay is None else (
        torch.tensor(decay, dtype=torch.float32, device="cuda"))
    n = len(lens)
    return dict(q=q, k=k, v=v, ld=ld, cu=cu, seqs=seqs, scale=Dk ** -0.5,
                init=rnd(n, H, Dv, Dk) if init else None, do=rnd(b, L, H, Dv).to(dt),
                dfinal=rnd(n, H, Dv, Dk) if init else None, act=act,
                dims=(b, L, H, Hk, Dk, Dv))


def problem(x):
    import mamba2_ssd_chunked_amd as ssd
    b, L, H, Hk, Dk, Dv = x["dims"]
    return ssd.make_linattn(batch=b, seqlen=L, nheads=H, nkvheads=Hk, keydim=Dk, valdim=Dv,
                            act=x["act"], scale=x["scale"])


def flat(t):
    return t.reshape(-1, *t.shape[2:])


def tol(x, r=1):
    b, L, H, Hk, Dk, Dv = x["dims"]
    chunks = max(n for _, n in x["seqs"]) // 32 + 1
    f32 = (Dk + Dv + 4 * chunks + 160 + r) * 2.0 ** -24
    return (2 * 2.0 ** -8 + 2.0 ** -14 + f32, 2.0 ** -15 + f32) if x["act"] == "bf16" else (f32, f32)


def check(what, got, want, bound, t):
    got = got.detach().double().cpu().reshape(want.shape)
    bad = (got - want).abs() / (bound + 1e-30)
    worst = float(bad.max()) if bad.numel() else 0.0
    log(f"  {what}: worst |error| / sum of magnitudes {worst:.2e} (tolerance {t:.2e})")
    assert torch.isfinite(got).all(), what
    assert worst <= t, (what, worst, t)


def run_fwd(x, want_final=True, **kw):
    import mamba2_ssd_chunked_amd as ssd
    p = problem(x)
    return ssd.linattn_forward(p, x["q"], x["k"], x["v"], x["ld"], cu_seqlens=x["cu"],
                               init=x["init"], want_final=want_final, **kw)


def run_bwd(x, **kw):
    import mamba2_ssd_chunked_amd as ssd
    p = problem(x)
    return ssd.linattn_backward(p, x["q"], x["k"], x["v"], x["ld"], x["do"], cu_seqlens=x["cu"],
                                init=x["init"], dfinal=x["dfinal"], want_dinit=True, **kw)


def inside(x):
    b, L = x["dims"][:2]
    m = torch.zeros(b * L, dtype=torch.bool)
    for at, n in x["seqs"]:
        m[at:at + n] = True
    return m


def assert_fwd(x):
    import mamba2_ssd_chunked_amd as ssd
    p = problem(x)
    n = len(x["seqs"])
    bufs = ssd.LinAttnForwardBuffers.allocate(p, n, "cuda")
    bufs.o.fill_(7.0)
    run_fwd(x, bufs=bufs)
    torch.cuda.synchronize()
    args = [flat(R.f64(x[c])) for c in "qkv"]
    o, fin = R.linattn_fwd(*args, x["ld"], x["scale"], x["seqs"], x["init"])
    ab = [a.abs() for a in args]
    A, Af = R.linattn_fwd(*ab, x["ld"], abs(x["scale"]), x["seqs"],
                          None if x["init"] is None else x["init"].abs())
    to, ts = tol(x)
    m = inside(x)
    got = flat(bufs.o).cpu()
    check("o", got[m], o[m], A[m], to)
    assert (got[~m] == 7.0).all(), "tokens outside every sequence were written"
    check("final state", bufs.final_state, fin, Af, ts)


def assert_bwd(x):
    import mamba2_ssd_chunked_amd as ssd
    p = problem(x)
    bufs = ssd.LinAttnBackwardBuffers.allocate(p, len(x["seqs"]), "cuda")
    for t in (bufs.dq, bufs.dk, bufs.dv):
        t.fill_(7.0)
    run_bwd(x, bufs=bufs)
    torch.cuda.synchronize()
    args = [flat(R.f64(x[c])) for c in "qkv"]
    do = flat(R.f64(x["do"]))
    want = R.linattn_bwd(*args, x["ld"], x["scale"], x["seqs"], do, x["init"], x["dfinal"])
    ab = lambda t: None if t is None else t.abs()  # noqa: E731
    A = R.linattn_bwd(*[a.abs() for a in args], x["ld"], abs(x["scale"]), x["seqs"], do.abs(),
                      ab(x["init"]), ab(x["dfinal"]))
    to, ts = tol(x, x["dims"][2] // x["dims"][3])
    m = inside(x)
    for name, g, w, b in zip(("dq", "dk", "dv"), (bufs.dq, bufs.dk, bufs.dv), want, A):
        g = flat(g).cpu()
        check(name, g[m], w[m], b[m], to)
        assert (g[~m] == 7.0).all(), f"{name} outside every sequence was written"
    check("dinit", bufs.dinit, want[3], A[3], ts)


LENS = [[1], [2], [15, 1, 16, 17], [31, 32, 33], [63, 64, 65], [0, 5, 0, 0, 130, 0], [257, 300]]


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_forward_lengths(lens, act):
    assert_fwd(make(lens, 4, 2, 64, 64, act, before=3, behind=5))


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_backward_lengths(lens, act):
    assert_bwd(make(lens, 4, 2, 64, 64, act, before=3, behind=5))


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("Dk,Dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("H,Hk", [(3, 3), (4, 1), (6, 2)])
def test_head_layouts(H, Hk, Dk, Dv, act):
    x = make([70, 33], H, Hk, Dk, Dv, act, fused=True)
    assert_fwd(x)
    assert_bwd(x)


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_rows_without_states(act):
    x = make([100, 100, 100], 2, 2, 64, 128, act, packed=False, init=False, fused=True)
    assert_fwd(x)
    assert_bwd(x)


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_long_sequences(act):
    """Long enough that a sequence is walked in several spans."""
    x = make([1500, 1, 2300], 2, 1, 64, 64, act, behind=1)
    assert_fwd(x)
    assert_bwd(x)


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_extreme_decays(act):
    """No decay, nearly full decay (l^2 below the smallest float32) and exactly full decay."""
    x = make([90, 40], 4, 4, 64, 64, act, decay=[0.0, -60.0, -float("inf"), -1e-4])
    assert_fwd(x)
    assert_bwd(x)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_tokens_stay_in_their_future(bad):
    """A non-finite v or k at token t leaves the outputs before t and other sequences alone."""
    x = make([100, 50], 2, 2, 64, 64, "bf16")
    clean = run_fwd(x)
    x["v"][0, 37, 0] = bad
    x["k"][0, 37, 1] = bad
    got = run_fwd(x)
    torch.cuda.synchronize()
    assert torch.equal(got.o[:, :37], clean.o[:, :37])
    assert torch.equal(got.o[:, 100:], clean.o[:, 100:])
    assert torch.equal(got.final_state[1], clean.final_state[1])
    assert not torch.isfinite(got.o[:, 37]).any()


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("Dk,Dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("H,Hk", [(2, 2), (4, 2)])
def test_a_non_finite_channel_stays_in_its_channel(H, Hk, Dk, Dv, act):
    """One channel of v (forward) or of do (backward) that is infinite at one token: NaN in that
    channel from that token on (backwards: up to it), every other value as without it."""
    x = make([150, 70], H, Hk, Dk, Dv, act)
    clean, cg = run_fwd(x), run_bwd(x)
    at, ch, r = 83, Dv - 3, H // Hk
    keep = x["v"][0, at, 1, ch].item()
    x["v"][0, at, 1, ch] = float("inf")
    got = run_fwd(x)
    x["v"][0, at, 1, ch] = keep
    x["do"][0, at, r, ch] = float("-inf")  # a head that reads key/value head 1
    gg = run_bwd(x)
    torch.cuda.synchronize()
    hit = torch.zeros(got.o.shape, dtype=torch.bool, device="cuda")
    hit[0, at:150, r:2 * r, ch] = True
    assert torch.isnan(got.o[hit]).all()
    assert torch.equal(got.o[~hit], clean.o[~hit])
    state = torch.zeros(got.final_state.shape, dtype=torch.bool, device="cuda")
    state[0, r:2 * r, ch] = True
    assert torch.isnan(got.final_state[state]).all()
    assert torch.equal(got.final_state[~state], clean.final_state[~state])
    hit = torch.zeros(gg.dv.shape, dtype=torch.bool, device="cuda")
    hit[0, :at + 1, 1, ch] = True
    assert torch.isnan(gg.dv[hit]).all()
    assert torch.equal(gg.dv[~hit], cg.dv[~hit])
    assert torch.equal(gg.dk[:, at + 1:], cg.dk[:, at + 1:])
    assert torch.equal(gg.dk[:, :, 0], cg.dk[:, :, 0])
    other = [i for i in range(220) if i != at]
    assert torch.equal(gg.dq[:, other], cg.dq[:, other])


def test_sequences_do_not_touch_each_other():
    x = make([64, 40, 96], 2, 1, 64, 64, "bf16")
    a, ga = run_fwd(x), run_bwd(x)
    for c in ("q", "k", "v", "do"):
        x[c][0, 64:104] *= -3.0
    b, gb = run_fwd(x), run_bwd(x)
    torch.cuda.synchronize()
    for s in (slice(0, 64), slice(104, 200)):
        assert torch.equal(a.o[:, s], b.o[:, s])
        for n in ("dq", "dk", "dv"):
            assert torch.equal(getattr(ga, n)[:, s], getattr(gb, n)[:, s])
    assert not torch.equal(a.o[:, 64:104], b.o[:, 64:104])


def test_repeated_runs_are_bitwise_equal():
    x = make([700, 333], 4, 2, 128, 64, "bf16")
    a, ga = run_fwd(x), run_bwd(x)
    b, gb = run_fwd(x), run_bwd(x)
    torch.cuda.synchronize()
    assert torch.equal(a.o, b.o) and torch.equal(a.final_state, b.final_state)
    for n in ("dq", "dk", "dv", "dinit"):
        assert torch.equal(getattr(ga, n), getattr(gb, n))


def test_gradients_by_differences():
    """The float32 backward against central differences of the float32 forward along a random
    direction d.  The outputs are linear in each input alone, so the difference has no error
    but rounding: the loss is a sum of N = 25 000 products of values of up to a few units, each
    off by some 2^-22 independently, so the quotient is off by about 4 sqrt(N) 2^-22 / h =
    0.01 with h = 2^-6; the products grad d that it is compared with have a 2-norm of about
    100 and more.  2^-10 of that norm leaves a factor of ten."""
    import mamba2_ssd_chunked_amd as ssd
    x = make([40, 25], 2, 1, 64, 64, "f32")
    g = run_bwd(x)
    grads = dict(q=g.dq, k=g.dk, v=g.dv, init=g.dinit)
    h = 2.0 ** -6
    for name, grad in grads.items():
        d = torch.randn(x[name].shape, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
        losses = []
        for sign in (1, -1):
            y = dict(x, **{name: x[name] + sign * h * d})
            f = ssd.linattn_forward(problem(y), y["q"], y["k"], y["v"], y["ld"], cu_seqlens=y["cu"],
                                    init=y["init"], want_final=True)
            losses.append(float((f.o.double() * x["do"].double()).sum()
                                + (f.final_state.double() * x["dfinal"].double()).sum()))
        num = (losses[0] - losses[1]) / (2 * h)
        parts = (grad.double() * d.double())
        assert abs(num - float(parts.sum())) <= 2.0 ** -10 * float(parts.square().sum().sqrt())


def test_graph_replay_and_streams():
    """Captured forward and backward replay to the eager result, with eager work of another
    problem between the replays; and a call on a side stream gives the same."""
    x, other = make([300, 130], 4, 2, 64, 128, "bf16"), make([500], 2, 2, 128, 64, "bf16")
    import mamba2_ssd_chunked_amd as ssd
    ef, eb = run_fwd(x), run_bwd(x)
    torch.cuda.synchronize()
    p, n = problem(x), len(x["seqs"])
    fb, bb = (c.allocate(p, n, "cuda") for c in (ssd.LinAttnForwardBuffers,
                                                 ssd.LinAttnBackwardBuffers))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run_fwd(x, bufs=fb, stream=side)
    run_bwd(x, bufs=bb, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    names = ("dq", "dk", "dv", "dinit")

    def same():
        assert torch.equal(fb.o, ef.o) and torch.equal(fb.final_state, ef.final_state)
        for m in names:
            assert torch.equal(getattr(bb, m), getattr(eb, m)), m

    same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_fwd(x, bufs=fb)
        run_bwd(x, bufs=bb)
    for _ in range(3):
        for t in (fb.o, fb.final_state, bb.dq, bb.dk, bb.dv, bb.dinit):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        same()
        run_fwd(other)
        run_bwd(other)
        torch.cuda.synchronize()


def test_buffers_made_for_a_side_stream_survive_their_owner():
    """Buffers made by the call for another stream are not handed out again before it is done."""
    x = make([2000], 4, 4, 128, 128, "bf16", init=False)
    want = run_fwd(x, want_final=False).o.clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        o = run_fwd(x, want_final=False, stream=side).o  # its workspace is dropped here
        junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(16)]
        side.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(o, want)
        del junk


# ------------------------------------------------------------------------ single tokens


def step_inputs(rows, T, H, Hk, Dk, Dv, act, slots, seed=0):
    g = torch.Generator(device="cuda").manual_seed(50 + seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    dt = ACT[act]
    return dict(q=rnd(rows, T, H, Dk).to(dt), k=rnd(rows, T, Hk, Dk).to(dt),
                v=rnd(rows, T, Hk, Dv).to(dt),
                ld=-torch.exp2(-7.0 * torch.arange(1, H + 1, device="cuda") / H),
                state=rnd(slots, H, Dv, Dk), scale=Dk ** -0.5, act=act,
                dims=(rows, T, H, Hk, Dk, Dv))


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("Dk,Dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("rows,T,H,Hk", [(1, 1, 4, 4), (5, 1, 6, 2), (3, 7, 2, 1)])
def test_step(rows, T, H, Hk, Dk, Dv, act):
    """float32 throughout, so also a bf16 state is good to (Dk + 8) 2^-24 of A per token; the
    outputs are rounded once."""
    import mamba2_ssd_chunked_amd as ssd
    slots = rows + 2
    x = step_inputs(rows, T, H, Hk, Dk, Dv, act, slots)
    ids = list(range(slots))[::-1][:rows]
    pos = [9] * rows
    if rows > 1:
        pos[1] = 0        # starts from zero
    if rows > 2:
        ids[2] = -1       # padding
    if rows > 4:
        ids[3] = ids[0]   # the same slot again: skipped
        pos[4] = -1       # skipped
    S0 = R.f64(x["state"])
    o = torch.full((rows, T, H, Dv), 7.0, dtype=ACT[act], device="cuda")
    t32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    ssd.ssd_linattn_step(problem(x), x["q"], x["k"], x["v"], x["ld"], x["state"], o,
                         slots=t32(ids), positions=t32(pos))
    torch.cuda.synchronize()
    want, f = S0.clone(), (Dk + 8 * T + 8) * 2.0 ** -24
    for r in range(rows):
        if ids[r] < 0 or pos[r] < 0 or ids[r] in ids[:r]:
            assert (o[r] == 7.0).all()
            continue
        init = S0[ids[r]] * (pos[r] > 0)
        a = [R.f64(x[c][r]) for c in "qkv"]
        yo, S = R.linattn_fwd(*a, x["ld"], x["scale"], [(0, T)], init[None])
        A, AS = R.linattn_fwd(*[t.abs() for t in a], x["ld"], x["scale"], [(0, T)],
                              init[None].abs())
        want[ids[r]] = S[0]
        check(f"o[{r}]", o[r], yo, A, f + (2.0 ** -8 if act == "bf16" else 0))
        check(f"state[{r}]", x["state"][ids[r]], S[0], AS[0], f)
    used = [i for r, i in enumerate(ids) if i >= 0 and pos[r] >= 0]
    for i in range(slots):
        if i not in used:
            assert torch.equal(x["state"][i].double().cpu(), S0[i])


def test_step_without_slots_continues_a_prompt():
    """A prompt, then its next tokens one by one and three at once, against the whole prompt."""
    import mamba2_ssd_chunked_amd as ssd
    x = make([90, 90], 4, 2, 64, 64, "f32", packed=False)
    whole = run_fwd(x)
    cut = dict(x, **{c: x[c][:, :80].contiguous() for c in "qkv"})
    cut["dims"] = (2, 80) + x["dims"][2:]
    f = run_fwd(cut)
    state, got = f.final_state, []
    for at, n in [(80, 1), (81, 1), (82, 3), (85, 5)]:
        p = ssd.make_linattn(batch=2, seqlen=n, nheads=4, nkvheads=2, keydim=64, valdim=64,
                             act="f32", scale=x["scale"])
        o = torch.empty(2, n, 4, 64, device="cuda")
        part = [x[c][:, at:at + n].contiguous() for c in "qkv"]
        ssd.ssd_linattn_step(p, *part, x["ld"], state, o)
        got.append(o)
    torch.cuda.synchronize()
    args = [flat(R.f64(x[c])).abs() for c in "qkv"]
    A, Af = R.linattn_fwd(*args, x["ld"], x["scale"], x["seqs"], x["init"].abs())
    t = 2 * tol(x)[0]
    check("o", torch.cat(got, 1), whole.o[:, 80:].double().cpu(),
          A.reshape(2, 90, 4, 64)[:, 80:], t)
    check("state", state, whole.final_state.double().cpu(), Af, t)


# ------------------------------------------------------------------- beyond 2^31 elements


def test_tokens_far_apart():
    """q, o, do and dq in rows that reach beyond 2^32 bytes give what packed ones give."""
    import mamba2_ssd_chunked_amd as ssd
    x = make([210, 90], 2, 1, 64, 128, "bf16")
    step = (1 << 23) - 8

    def far(like):
        _, L, H, D = like.shape
        t = torch.empty(L * step, dtype=like.dtype, device="cuda")
        return t.as_strided(like.shape, (L * step, step, D, 1)).copy_(like)

    p, want, wg = problem(x), run_fwd(x), run_bwd(x)
    bufs = ssd.LinAttnForwardBuffers.allocate(p, 2, "cuda")
    grads = ssd.LinAttnBackwardBuffers.allocate(p, 2, "cuda")
    bufs.o, grads.dq = far(bufs.o), far(grads.dq)
    x["q"] = far(x["q"])
    run_fwd(x, bufs=bufs)
    # do has o's stride
    do = bufs.o
    got = do.clone()
    do.copy_(x["do"])
    x["do"] = do
    run_bwd(x, bufs=grads)
    torch.cuda.synchronize()
    assert torch.equal(got, want.o)
    for n in ("dq", "dk", "dv", "dinit"):
        assert torch.equal(getattr(grads, n), getattr(wg, n)), n


def test_step_in_a_large_pool():
    """The last slot of a pool of more than 2^31 state elements gives what a small pool gives."""
    import mamba2_ssd_chunked_amd as ssd
    x = step_inputs(1, 2, 16, 16, 128, 128, "bf16", 1)
    n = (1 << 31) // (16 * 128 * 128) + 2
    pool = torch.empty(n, 16, 128, 128, dtype=torch.float32, device="cuda")
    pool[n - 1] = x["state"][0]
    y = [torch.empty(1, 2, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ssd.ssd_linattn_step(problem(x), x["q"], x["k"], x["v"], x["ld"], x["state"], y[0])
    ssd.ssd_linattn_step(problem(x), x["q"], x["k"], x["v"], x["ld"], pool, y[1],
                         slots=torch.tensor([n - 1], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(*y) and torch.equal(pool[n - 1], x["state"][0])
