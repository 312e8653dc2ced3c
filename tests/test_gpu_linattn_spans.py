"""Linear attention over sequences that are walked in several spans, against the float64
recurrence: every state size, rows and packed sequences, with and without states, decays of
any size, values that are not finite.  Spans have 256 tokens at these sizes.

Tolerances: those of test_gpu_linattn_rounding, whose terms also hold over spans: a state that
is handed to the next span has its values in two or three parts as every other has, and its
decay over a span is one power more for 256 tokens, inside the 4 that f has for each 32.
"""
import pytest
import torch

import mixer_ref as R
import test_gpu_linattn as LA
from test_gpu_linattn_rounding import assert_rounded_once

pytestmark = pytest.mark.gpu
DIMS = [(64, 64), (64, 128), (128, 64), (128, 128)]


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("Dk,Dv", DIMS)
@pytest.mark.parametrize("H,Hk,init", [(2, 2, False), (2, 1, True)])
def test_rows_in_spans(H, Hk, init, Dk, Dv, act):
    """Rows of 1300 tokens: five whole spans and one of 20 tokens."""
    assert_rounded_once(LA.make([1300, 1300], H, Hk, Dk, Dv, act, packed=False, init=init,
                                fused=init))


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("Dk,Dv", DIMS)
@pytest.mark.parametrize("H,Hk,init", [(2, 2, True), (2, 1, False)])
def test_packed_in_spans(H, Hk, init, Dk, Dv, act):
    assert_rounded_once(LA.make([700, 3, 600], H, Hk, Dk, Dv, act, init=init, before=5, behind=2))


LAYOUTS = [
    [1] * 300 + [1024] + [1] * 40,                       # one long one among many of a token
    [257, 255, 1, 256, 257, 512, 0, 513, 257, 0, 0, 300],  # ends on and beside every border
    [258] * 8,                                           # two spans each, the second of two tokens
    [2, 767, 1, 769, 0, 513],
]


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("lens", LAYOUTS, ids=lambda v: f"{len(v)}x{max(v)}")
@pytest.mark.parametrize("before", [0, 130])
def test_layouts_of_sequences(lens, before, act):
    """States of neighbouring sequences stay apart wherever their spans begin."""
    assert_rounded_once(LA.make(lens, 2, 1, 64, 64, act, before=before, behind=1))


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("packed", [True, False])
def test_decays_over_spans(packed, act):
    """No decay, nearly full, exactly full and a slow one."""
    assert_rounded_once(LA.make([1100, 1100] if packed else [1100], 4, 4, 64, 64, act,
                                packed=packed, decay=[0.0, -60.0, -float("inf"), -1e-3]))


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("-inf")])
@pytest.mark.parametrize("at", [100, 700, 1298])
@pytest.mark.parametrize("Dk,Dv", [(64, 128), (128, 64)])
def test_a_non_finite_channel_in_a_span(Dk, Dv, at, bad, act):
    """One channel of v (backwards: of do) that is not finite at a token of the first span, a
    middle one or the last: from there on that channel and its state are not finite, every other
    value is as without it."""
    x = LA.make([1300, 400], 2, 2, Dk, Dv, act)
    clean, cg = LA.run_fwd(x), LA.run_bwd(x)
    ch = Dv - 5
    keep = x["v"][0, at, 1, ch].item()
    x["v"][0, at, 1, ch] = bad
    got = LA.run_fwd(x)
    x["v"][0, at, 1, ch] = keep
    x["do"][0, at, 1, ch] = bad
    gg = LA.run_bwd(x)
    torch.cuda.synchronize()

    def only(a, b, hit):
        assert not torch.isfinite(a[hit]).any()
        assert torch.equal(a[~hit], b[~hit])

    def at_of(t):
        return torch.zeros(t.shape, dtype=torch.bool, device="cuda")

    hit = at_of(got.o)
    hit[0, at:1300, 1, ch] = True
    only(got.o, clean.o, hit)
    hit = at_of(got.final_state)
    hit[0, 1, ch] = True
    only(got.final_state, clean.final_state, hit)
    hit = at_of(gg.dv)
    hit[0, :at + 1, 1, ch] = True
    only(gg.dv, cg.dv, hit)
    hit = at_of(gg.dinit)
    hit[0, 1, ch] = True
    only(gg.dinit, cg.dinit, hit)
    assert torch.equal(gg.dk[:, at + 1:], cg.dk[:, at + 1:])
    assert torch.equal(gg.dk[:, :, 0], cg.dk[:, :, 0])
    other = [i for i in range(1700) if i != at]
    assert torch.equal(gg.dq[:, other], cg.dq[:, other])


def test_a_non_finite_key_over_spans():
    """A key that is not finite reaches no earlier output and no other sequence or head."""
    x = LA.make([1300, 300], 2, 2, 64, 64, "bf16")
    clean = LA.run_fwd(x)
    x["k"][0, 600, 1, 7] = float("inf")
    got = LA.run_fwd(x)
    torch.cuda.synchronize()
    assert torch.equal(got.o[:, :600], clean.o[:, :600])
    assert torch.equal(got.o[:, 1300:], clean.o[:, 1300:])
    assert torch.equal(got.o[:, :, 0], clean.o[:, :, 0])
    assert torch.equal(got.final_state[1], clean.final_state[1])
    assert not torch.isfinite(got.o[:, 600:1300, 1]).any()


def test_workspace_is_not_overrun():
    """Exactly the bytes that are asked for, between guards that stay as they were."""
    import mamba2_ssd_chunked_amd as ssd
    x = LA.make([1] * 300 + [1024] + [1] * 40 + [1500], 2, 1, 64, 64, "bf16")
    p, n = LA.problem(x), len(x["seqs"])
    want, wg = LA.run_fwd(x), LA.run_bwd(x)
    for kind, run, make_, ref in (
            (ssd.SSD_WS_FORWARD, LA.run_fwd, ssd.LinAttnForwardBuffers, want),
            (ssd.SSD_WS_BACKWARD, LA.run_bwd, ssd.LinAttnBackwardBuffers, wg)):
        need = ssd.ssd_linattn_workspace_bytes(p, n, kind)
        room = torch.full((need + 2 * 65536,), 0x5a, dtype=torch.uint8, device="cuda")
        bufs = make_.allocate(p, n, "cuda")
        bufs.ws = room[65536:65536 + need]
        run(x, bufs=bufs)
        torch.cuda.synchronize()
        assert (room[:65536] == 0x5a).all() and (room[65536 + need:] == 0x5a).all()
        for name in ("o", "final_state") if kind == ssd.SSD_WS_FORWARD else ("dq", "dk", "dv", "dinit"):
            assert torch.equal(getattr(bufs, name), getattr(ref, name)), name


def test_reference_of_absolute_values():
    """The float64 recurrence itself, on a short case, against the sum over pairs of tokens."""
    x = LA.make([6], 1, 1, 64, 64, "f32", decay=[-0.5])
    args = [LA.flat(R.f64(x[c])) for c in "qkv"]
    o, _ = R.linattn_fwd(*args, x["ld"], x["scale"], x["seqs"], x["init"])
    q, k, v = (a[:, 0] for a in args)
    for t in range(6):
        want = sum(torch.exp(torch.tensor(-0.5 * (t - j), dtype=torch.float64)) * (q[t] @ k[j]) * v[j]
                   for j in range(t + 1))
        want = want + torch.exp(torch.tensor(-0.5 * (t + 1), dtype=torch.float64)) * (R.f64(x["init"])[0, 0] @ q[t])
        assert torch.allclose(o[t, 0], x["scale"] * want, rtol=1e-12, atol=1e-12)
