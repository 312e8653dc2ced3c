"""Linear attention with a decay per head: what of the results' types a caller gets.

Tolerances.  With A the recurrence's result on absolute values and f = (Dk + Dv + 4 nchunks +
160 + r) 2^-24 the float32 sums' share (nchunks of 32 tokens, r heads that share keys and
values), in multiples of A:
  bf16 outputs  2^-8 |value| for the one rounding of the result, and 1.5 2^-16 + f: what is
                not bf16 already enters its products as a sum of two bf16.  Weighted values,
                rounded twice, leave out 2^-17 (the rest after the first rounding is at most
                2^-8 and its rounding 2^-17 of a value of 1 to 2); scores and entering states,
                cut off and then rounded, 2^-16; a term has at most one of each
  short states  sums of two products, 2^-24 each: the split in three bf16 leaves 2^-26, a
                power of the decay is the product of two, each off by 2^-23 and by 2^-24 of
                its exponent (below 2 here), and the six additions lose 2^-23 each; in all
                below 24 2^-24.  A value split in two leaves 2^-17, five times that.
"""
import pytest
import torch

import mixer_ref as R
import test_gpu_linattn as LA

pytestmark = pytest.mark.gpu


def float32_share(x):
    b, L, H, Hk, Dk, Dv = x["dims"]
    chunks = max(n for _, n in x["seqs"]) // 32 + 1
    return (Dk + Dv + 4 * chunks + 160 + H // Hk) * 2.0 ** -24


def assert_rounded_once(x, more=0.0):
    """o, dq, dk and dv within the float32 share, and for bf16 one rounding, of float64; states
    and dinit within the float32 share.  `more`: allowed beyond, of the sum of magnitudes."""
    f = LA.run_fwd(x)
    g = LA.run_bwd(x)
    torch.cuda.synchronize()
    args = [LA.flat(R.f64(x[c])) for c in "qkv"]
    do = LA.flat(R.f64(x["do"]))
    ab = lambda t: None if t is None else t.abs()  # noqa: E731
    aa = [a.abs() for a in args]
    o, fin = R.linattn_fwd(*args, x["ld"], x["scale"], x["seqs"], x["init"])
    Ao, Afin = R.linattn_fwd(*aa, x["ld"], x["scale"], x["seqs"], ab(x["init"]))
    want = R.linattn_bwd(*args, x["ld"], x["scale"], x["seqs"], do, x["init"], x["dfinal"])
    A = R.linattn_bwd(*aa, x["ld"], x["scale"], x["seqs"], do.abs(), ab(x["init"]), ab(x["dfinal"]))
    share = float32_share(x) + more
    m = LA.inside(x)
    outs = [("o", f.o, o, Ao), ("dq", g.dq, want[0], A[0]), ("dk", g.dk, want[1], A[1]),
            ("dv", g.dv, want[2], A[2])]
    for name, got, w, a in outs:
        bound = share * a[m]
        if x["act"] == "bf16":
            bound = 2.0 ** -8 * w[m].abs() + (1.5 * 2.0 ** -16 + share) * a[m]
        LA.check(name, LA.flat(got).cpu()[m], w[m], bound, 1.0)
    # the values that enter these states are sums of three bf16
    ts = share + (2.0 ** -24 if x["act"] == "bf16" else 0.0)
    LA.check("final state", f.final_state, fin, Afin, ts)
    LA.check("dinit", g.dinit, want[3], A[3], ts)


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("H,Hk", [(2, 2), (4, 2)])
def test_bf16_outputs_are_rounded_once(H, Hk, Dk, Dv):
    assert_rounded_once(LA.make([200, 64, 1, 35], H, Hk, Dk, Dv, "bf16", behind=3))


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
def test_bf16_states_of_two_tokens(Dk, Dv):
    """A state of two tokens is good to float32's rounding, which no value in fewer than three
    bf16 is; its gradient's sum likewise."""
    x = LA.make([2, 2, 2], 4, 2, Dk, Dv, "bf16", init=False, decay=[-0.3, -1.1, -0.05, -0.7])
    x["do"][:, ::2] *= 0.125  # the older term has the larger share in one of the two directions
    f, g = LA.run_fwd(x), LA.run_bwd(x)
    torch.cuda.synchronize()
    args = [LA.flat(R.f64(x[c])) for c in "qkv"]
    do = LA.flat(R.f64(x["do"]))
    aa = [a.abs() for a in args]
    _, fin = R.linattn_fwd(*args, x["ld"], x["scale"], x["seqs"])
    _, A = R.linattn_fwd(*aa, x["ld"], x["scale"], x["seqs"])
    dinit = R.linattn_bwd(*args, x["ld"], x["scale"], x["seqs"], do)[3]
    Ad = R.linattn_bwd(*aa, x["ld"], x["scale"], x["seqs"], do.abs())[3]
    t = 24 * 2.0 ** -24
    LA.check("final state", f.final_state, fin, A, t)
    # scale and the last decay: two more powers and products
    LA.check("dinit", g.dinit, dinit, Ad, t + 8 * 2.0 ** -24)
