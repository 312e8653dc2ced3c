"""The conv1d + SSD path token by token on the GPU, against the float64 recurrence and
against the prompt path.

Tolerances.  Everything between the inputs and the outputs is float32, with exp and the
reciprocal of the SiLU good to a few 2^-23.  With A the recurrence's sum of magnitudes
(|u| of every convolved channel taken from its taps' magnitudes), each of the N products
and W taps and the decays adds a few 2^-24: (N + 4 W + 64) 2^-23 A for the state and the
outputs, doubled once; bf16 outputs are then rounded once (2^-8).
"""
import numpy as np
import pytest
import torch

import mixer_ref as R
import ssd_workloads as W
from ssd_testlib import device_inputs, log, problem_of

pytestmark = pytest.mark.gpu
ACT = {"bf16": torch.bfloat16, "f32": torch.float32}
SHAPES = [("f32", 16, 16), ("f32", 32, 32), ("f32", 64, 64), ("f32", 64, 128), ("bf16", 32, 64),
          ("bf16", 64, 64), ("bf16", 64, 128)]


def draws(rows, T, H, G, P, N, Wc, act, slots, ring, seed=0):
    g = torch.Generator(device="cuda").manual_seed(70 + seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    C, dt = H * P + 2 * G * N, ACT[act]
    return dict(xBC=rnd(rows, T, C).to(dt), conv_w=0.5 * rnd(C, Wc), dt_raw=rnd(rows, T, H).to(dt),
                dt_bias=rnd(H) - 3.0, A_log=torch.rand(H, generator=g, device="cuda") * 2.5,
                D=rnd(H), conv_ring=rnd(slots, ring, C).to(dt), state=rnd(slots, H, P, N))


def magnitudes(x, r, hist, S, pos, G):
    """Sum of magnitudes: |conv| from absolute taps (SiLU(u) <= |u|), then the recurrence on
    absolute values with the same decays."""
    f = {k: R.f64(v) for k, v in x.items()}
    H, P, N = S.shape
    rows = torch.cat([hist, f["xBC"][r]]).abs()
    Wc, n = f["conv_w"].shape[1], f["xBC"].shape[1]
    w, S = f["conv_w"].abs(), S.abs() * (pos > 0)
    ys = []
    for i in range(n):
        at = len(hist) + i
        u = sum(w[:, Wc - 1 - k] * rows[at - k] for k in range(Wc) if at - k >= 0 and pos + i - k >= 0)
        xx = u[:H * P].reshape(H, P)
        B, C = (u[H * P + o * G * N:H * P + (o + 1) * G * N].reshape(G, N)
                .repeat_interleave(H // G, 0) for o in (0, 1))
        dt = torch.log1p(torch.exp(f["dt_raw"][r, i] + f["dt_bias"])).clamp(1e-3, 0.1)
        S = (torch.exp(-dt * torch.exp(f["A_log"]))[:, None, None] * S
             + dt[:, None, None] * xx[:, :, None] * B[:, None, :])
        ys.append((S * C[:, None, :]).sum(-1) + f["D"].abs()[:, None] * xx)
    return torch.stack(ys), S


def check(what, got, want, bound, t):
    worst = float(((got.double().cpu() - want).abs() / (bound + 1e-30)).max())
    log(f"  {what}: worst |error| / sum of magnitudes {worst:.2e} (tolerance {t:.2e})")
    assert worst <= t, (what, worst, t)


@pytest.mark.parametrize("act,P,N", SHAPES)
@pytest.mark.parametrize("Wc,T,extra", [(4, 1, 0), (1, 1, 0), (8, 3, 2), (2, 5, 0)])
def test_step(act, P, N, Wc, T, extra):
    import mamba2_ssd_chunked_amd as ssd
    rows, H, G, slots = 6, 4, 2, 8
    ring = Wc - 1 + T + extra
    x = draws(rows, T, H, G, P, N, Wc, act, slots, ring, seed=P + N + Wc)
    ids, pos = [7, 2, -1, 7, 0, 5], [1000003, 0, 4, 4, 2, -1]
    ids[5] = 5
    ring0, S0 = x["conv_ring"].clone(), R.f64(x["state"])
    y = torch.full((rows, T, H, P), 7.0, dtype=ACT[act], device="cuda")
    p = ssd.make_problem(batch=rows, seqlen=T, nheads=H, headdim=P, dstate=N, ngroups=G, chunk=64,
                         conv_width=Wc, act=act)
    t32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    ssd.ssd_token_step(p, x["xBC"], x["conv_w"], x["dt_raw"], x["dt_bias"], x["A_log"], x["D"],
                       x["conv_ring"], x["state"], t32(pos), y, slots=t32(ids))
    torch.cuda.synchronize()
    tol = 2 * (N + 4 * Wc + 64) * 2.0 ** -23
    want_ring = ring0.clone()
    for r in range(rows):
        if r in (2, 3, 5):  # padding, a slot taken by an earlier row, a negative position
            assert (y[r] == 7.0).all()
            continue
        back = min(pos[r], Wc - 1)
        hist = R.f64(torch.stack([ring0[ids[r], (pos[r] - back + i) % ring] for i in range(back)])
                     if back else x["xBC"][r, :0])
        yo, S = R.token_step(x["xBC"][r], x["conv_w"], x["dt_raw"][r], x["dt_bias"], x["A_log"],
                             x["D"], hist, S0[ids[r]], pos[r], G, p.dt_min, p.dt_max)
        A, AS = magnitudes(x, r, hist, S0[ids[r]], pos[r], G)
        check(f"y[{r}]", y[r], yo, A, tol + (2.0 ** -8 if act == "bf16" else 0))
        check(f"state[{r}]", x["state"][ids[r]], S, AS, tol)
        for i in range(T):
            want_ring[ids[r], (pos[r] + i) % ring] = x["xBC"][r, i]
    assert torch.equal(x["conv_ring"], want_ring)
    for i in (1, 3, 4, 5, 6):
        assert torch.equal(R.f64(x["state"][i]), S0[i])


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_prompt_then_tokens_then_norm(act):
    """forward() on whole chunks, its rows handed over to a StepState, then the remaining
    tokens (several at once, then one by one) and the output norm: the same as one longer
    forward() and its norm.  float32: 1e-4 of the larger of the value and the RMS, bf16:
    2e-2 of the RMS, the tolerances of the prompt path itself."""
    import mamba2_ssd_chunked_amd as ssd
    from ssd_testlib import assert_close
    wl = W.make_workload("handover", batch=2, seqlen=256, nheads=4, headdim=64, dstate=64,
                         ngroups=2, chunk=64, act=act, seed=31)
    x = device_inputs(wl)
    par = (x["dt_bias"], x["A_log"], x["D"])
    full = ssd.forward(problem_of(wl), [(0, 256)], x["xBC"], x["conv_w"], x["dt_raw"], *par,
                       want_final=True)
    cut = 192
    p = ssd.make_problem(batch=2, seqlen=cut, nheads=4, headdim=64, dstate=64, ngroups=2, chunk=64,
                         conv_width=4, act=act)
    head = x["xBC"][:, :cut].contiguous()
    f = ssd.forward(p, [(0, cut)], head, x["conv_w"], x["dt_raw"][:, :cut].contiguous(), *par,
                    want_final=True)
    pool = ssd.StepState.allocate(p, 5, "cuda", tokens=40)
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    pos = pool.load(p, head, f.final_state, slots)
    assert pos.tolist() == [cut, cut]
    z = torch.randn(2, 256, 512, device="cuda").to(ACT[act])[..., :256]
    w = torch.randn(256, device="cuda")
    at, ys, ns = cut, [], []
    for n in [40] + [1] * 24:
        q = ssd.make_problem(batch=2, seqlen=n, nheads=4, headdim=64, dstate=64, ngroups=2,
                             chunk=64, conv_width=4, act=act)
        y = torch.empty(2, n, 4, 64, dtype=ACT[act], device="cuda")
        ssd.ssd_token_step(q, x["xBC"][:, at:at + n].contiguous(), x["conv_w"],
                           x["dt_raw"][:, at:at + n].contiguous(), *par, pool.conv_ring,
                           pool.state, pos, y, slots=slots)
        pn = ssd.make_norm(rows=2 * n, channels=256, ngroups=2, act=act, mode="before")
        ns.append(ssd.norm_forward(pn, y.reshape(2 * n, 256), w,
                                   z=z[:, at:at + n].reshape(2 * n, 256)).reshape(2, n, 256))
        ys.append(y)
        pos += n
        at += n
    pn = ssd.make_norm(rows=512, channels=256, ngroups=2, act=act, mode="before")
    nf = ssd.norm_forward(pn, full.y.reshape(512, 256), w, z=z.reshape(512, 256)).reshape(2, 256, 256)
    torch.cuda.synchronize()
    d = lambda t: t.double().cpu().numpy()  # noqa: E731
    assert_close(d(torch.cat(ys, 1)), d(full.y[:, cut:]), act, "y")
    assert_close(d(pool.state[slots.long()]), d(full.final_state), act, "state")
    assert_close(d(torch.cat(ns, 1)), d(nf[:, cut:]), act, "norm")
    assert np.isfinite(d(torch.cat(ns, 1))).all()


def test_captured_steps_follow_their_inputs():
    """A captured step replayed with new tokens and positions equals the same steps run
    eagerly on another pool, eager work standing between the replays."""
    import mamba2_ssd_chunked_amd as ssd
    rows, H, G, P, N = 4, 4, 1, 64, 128
    steps = [draws(rows, 1, H, G, P, N, 4, "bf16", 6, 4, seed=s) for s in range(5)]
    par = steps[0]
    p = ssd.make_problem(batch=rows, seqlen=1, nheads=H, headdim=P, dstate=N, ngroups=G, chunk=64,
                         conv_width=4, act="bf16")
    slots = torch.tensor([5, 0, -1, 2], dtype=torch.int32, device="cuda")

    def pool():
        return dict(xBC=torch.zeros_like(par["xBC"]), dt=torch.zeros_like(par["dt_raw"]),
                    ring=par["conv_ring"].clone(), state=par["state"].clone(),
                    pos=torch.zeros(rows, dtype=torch.int32, device="cuda"),
                    y=torch.zeros(rows, 1, H, P, dtype=torch.bfloat16, device="cuda"))

    def step(o):
        ssd.ssd_token_step(p, o["xBC"], par["conv_w"], o["dt"], par["dt_bias"], par["A_log"],
                           par["D"], o["ring"], o["state"], o["pos"], o["y"], slots=slots)

    e, c, warm = pool(), pool(), pool()
    step(warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(c)
    for i, s in enumerate(steps):
        for o in (e, c):
            o["xBC"].copy_(s["xBC"])
            o["dt"].copy_(s["dt_raw"])
            o["pos"].fill_(i)
        step(e)
        graph.replay()
        torch.cuda.synchronize()
        for n in ("y", "ring", "state"):
            assert torch.equal(e[n], c[n]), (i, n)


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_many_rows_equal_few(act):
    """A batch large enough to put two heads into one workgroup gives each row what a call
    with that row alone gives, bit for bit."""
    import mamba2_ssd_chunked_amd as ssd
    rows, H, G, P, N = 300, 8, 2, 64, 64
    x = draws(rows, 1, H, G, P, N, 4, act, rows, 4, seed=9)
    pos = torch.arange(rows, dtype=torch.int32, device="cuda") % 7
    want = {n: x[n].clone() for n in ("conv_ring", "state")}

    def step(r, n, ring, state, y):
        p = ssd.make_problem(batch=n, seqlen=1, nheads=H, headdim=P, dstate=N, ngroups=G, chunk=64,
                             conv_width=4, act=act)
        ssd.ssd_token_step(p, x["xBC"][r:r + n], x["conv_w"], x["dt_raw"][r:r + n], x["dt_bias"],
                           x["A_log"], x["D"], ring, state, pos[r:r + n].clone(), y)

    y = torch.empty(rows, 1, H, P, dtype=ACT[act], device="cuda")
    step(0, rows, x["conv_ring"], x["state"], y)
    for r in (0, 1, 77, 151, 299):
        yr = torch.empty(1, 1, H, P, dtype=ACT[act], device="cuda")
        step(r, 1, want["conv_ring"][r:r + 1], want["state"][r:r + 1], yr)
        torch.cuda.synchronize()
        assert torch.equal(yr[0], y[r])
        for n in want:
            assert torch.equal(want[n][r], x[n][r]), (r, n)


def test_last_slot_of_a_large_pool():
    """States and rings of more than 2^31 elements: the last slot gives what a small pool gives."""
    import mamba2_ssd_chunked_amd as ssd
    H, G, P, N = 64, 1, 64, 128
    x = draws(1, 1, H, G, P, N, 4, "bf16", 1, 4, seed=11)
    C = x["xBC"].shape[-1]
    n = (1 << 31) // (H * P * N) + 2
    R = (1 << 31) // (n * C) + 2
    state = torch.empty(n, H, P, N, dtype=torch.float32, device="cuda")
    ring = torch.empty(n, R, C, dtype=torch.bfloat16, device="cuda")
    state[n - 1] = x["state"][0]
    for t in range(3, 6):  # the tokens before place 6
        ring[n - 1, t % R] = x["conv_ring"][0, t % 4]
    p = ssd.make_problem(batch=1, seqlen=1, nheads=H, headdim=P, dstate=N, ngroups=G, chunk=64,
                         conv_width=4, act="bf16")
    pos = torch.tensor([6], dtype=torch.int32, device="cuda")
    y = [torch.empty(1, 1, H, P, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    rest = [x[k] for k in ("xBC", "conv_w", "dt_raw", "dt_bias", "A_log", "D")]
    ssd.ssd_token_step(p, *rest, x["conv_ring"], x["state"], pos, y[0])
    ssd.ssd_token_step(p, *rest, ring, state, pos, y[1],
                       slots=torch.tensor([n - 1], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(*y)
    assert torch.equal(state[n - 1], x["state"][0])
    for t in range(3, 7):
        assert torch.equal(ring[n - 1, t % R], x["conv_ring"][0, t % 4])
