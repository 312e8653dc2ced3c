"""Single tokens of the gated delta rule with values that are not finite, and with decays beyond float32.

What such a value reaches is the same as in a prompt: of q the outputs of its key head's heads, of k, g and
beta all of its heads' outputs and states, of v its channel; everything else keeps its bits.
"""
import pytest
import torch

import layer_ref as R

pytestmark = pytest.mark.gpu

ACT = {"bf16": torch.bfloat16, "f32": torch.float32}
ROWS, H, HK = 3, 4, 2


def make(act, Dk, Dv, tokens=1, seed=0):
    g = torch.Generator(device="cuda").manual_seed(70 + seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(ACT[act])  # noqa: E731
    return dict(q=unit(rnd(ROWS, tokens, HK, Dk)), k=unit(rnd(ROWS, tokens, HK, Dk)),
                v=rnd(ROWS, tokens, H, Dv).to(ACT[act]), g=-rnd(ROWS, tokens, H).abs(),
                beta=torch.sigmoid(rnd(ROWS, tokens, H)), state=rnd(ROWS, H, Dv, Dk) * Dk ** -0.5)


def run(x, positions=None):
    import mamba2_ssd_chunked_amd as ssd
    b, L, Hk, Dk = x["q"].shape
    Dv, act = x["v"].shape[3], "bf16" if x["q"].dtype == torch.bfloat16 else "f32"
    p = ssd.make_gdelta(batch=b, seqlen=L, nheads=H, nkheads=Hk, keydim=Dk, valdim=Dv, act=act)
    state, o = x["state"].clone(), torch.full_like(x["v"], 7.0)
    ssd.ssd_gdelta_step(p, *(x[n] for n in ("q", "k", "v", "g", "beta")), state, o, positions=positions)
    return o, state


# a decay of minus infinity is a value like others
BAD = [(n, b) for n in ("q", "k", "v", "g", "beta") for b in (float("inf"), float("-inf"), float("nan"))
       if (n, b) != ("g", float("-inf"))]


@pytest.mark.parametrize("name,bad", BAD)
@pytest.mark.parametrize("act,Dk,Dv", [("bf16", 128, 64), ("f32", 64, 128)])
def test_a_value_that_is_not_finite(act, Dk, Dv, name, bad):
    x = make(act, Dk, Dv, tokens=2)
    o, state = run(x)
    y = dict(x, **{name: x[name].clone()})
    # row 1, second token; head 1 of the key heads (heads 2 and 3), or head 2
    heads = [2, 3] if name in ("q", "k") else [2]
    if name in ("g", "beta"):
        y[name][1, 1, 2] = bad
    else:
        y[name][1, 1, 1 if name in ("q", "k") else 2, 5] = bad
    o2, state2 = run(y)
    hit, kept = torch.zeros_like(o, dtype=torch.bool), torch.ones_like(state, dtype=torch.bool)
    if name == "v":
        hit[1, 1, 2, 5], kept[1, 2, 5] = True, False
    else:
        hit[1, 1, heads] = True
        if name != "q":
            kept[1, heads] = False
    assert torch.equal(o[~hit], o2[~hit]) and torch.equal(state[kept], state2[kept])
    assert not torch.isfinite(o2[hit]).any()
    assert not torch.isfinite(state2[~kept]).any()


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_decay_of_plus_infinity_is_what_it_is_in_a_prompt(act):
    """Also where the state is zero, of a row that begins."""
    import mamba2_ssd_chunked_amd as ssd
    x = make(act, 64, 64)
    x["g"][0, 0, 1] = x["g"][2, 0, 3] = float("inf")
    pos = torch.tensor([4, 4, 0], dtype=torch.int32, device="cuda")
    o, state = run(x, positions=pos)
    init = x["state"].clone()
    init[2] = 0
    p = ssd.make_gdelta(batch=ROWS, seqlen=1, nheads=H, nkheads=HK, keydim=64, valdim=64, act=act)
    f = ssd.gdelta_forward(p, *(x[n] for n in ("q", "k", "v", "g", "beta")), init=init, want_final=True)
    assert torch.equal(torch.isnan(o), torch.isnan(f.o)) and torch.equal(torch.isnan(state), torch.isnan(f.final_state))
    assert torch.isnan(o[0, 0, 1]).all() and torch.isnan(o[2, 0, 3]).all()
    assert torch.isfinite(o[1]).all() and torch.isfinite(o[0, 0, 0]).all()


def test_decays_beyond_float32():
    """e^90 is no float32 number, 1e-30 e^90 is: the state is multiplied by its root twice.  Each factor is e^45,
    whose exponent is good to 2^-25 of 45 and whose value to some 2^-23: 2^-18 of the result.  A product that
    float32 cannot hold is infinite, and a state of zeros stays zero."""
    x = make("f32", 64, 64)
    x["g"].fill_(90.0)
    x["beta"].zero_()
    x["state"][0] *= 1e-30
    x["state"][2] = 0.0
    o, state = run(x)
    q = x["q"][:, :1].repeat_interleave(H // HK, 2)
    want = R.f64(x["state"][0]) * torch.exp(torch.tensor(90.0, dtype=torch.float64))
    assert ((R.f64(state[0]) - want).abs() <= 2.0 ** -18 * want.abs()).all()
    got = (want * R.f64(q[0, 0])[:, None, :]).sum(-1) * 64 ** -0.5
    size = (want * R.f64(q[0, 0])[:, None, :]).abs().sum(-1) * 64 ** -0.5
    assert ((R.f64(o[0, 0]) - got).abs() <= 2.0 ** -17 * size).all()
    # e^90 is 1.2e39: elements from 0.28 on are beyond 3.4e38, and what meets them in their row
    big, most = R.f64(x["state"][1]) * want.new_tensor(90.0).exp(), torch.finfo(torch.float32).max
    over = big.abs() > most * (1 + 2.0 ** -18)
    assert over.any() and not torch.isfinite(state[1].cpu()[over]).any()
    rows = big.abs().sum(-1) <= most
    assert ((R.f64(state[1]) - big).abs()[rows] <= 2.0 ** -18 * big.abs()[rows]).all()
    assert (state[2] == 0).all() and (o[2] == 0).all()
