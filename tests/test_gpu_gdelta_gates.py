"""Gradients of the gated delta rule where decays are strong: of tokens that keep nothing, and of heads that forget
beside heads that do not."""
import pytest
import torch

import layer_ref as R
from test_gpu_gdelta import f64_norm, flat, make, problem

pytestmark = pytest.mark.gpu


def backward(x):
    import mamba2_ssd_chunked_amd as ssd
    return ssd.gdelta_backward(problem(x), *[x[n] for n in ("q", "k", "v", "g", "beta")], x["do"], cu_seqlens=x["cu"],
                               init=x["init"], dfinal=x["dfinal"], want_dinit=True)


def dg_terms(x, want):
    """[tokens][heads]: sizes of what dg_t is the sum of, from t to the end of its chunk: q_i . dq_i, v_i . dv_i
    and <G, S> behind the chunk, the first and the last by Cauchy-Schwarz.  Keys are of length one, betas in [0, 1] and
    decays at most 1, so that a step lengthens a state's norm by |v| and a gradient's by scale |do| |q| at most."""
    v, do = f64_norm(x["v"].flatten(0, 1)), f64_norm(x["do"].flatten(0, 1))
    dv = want["dv"].norm(dim=-1)
    out = torch.zeros_like(dv)
    H = out.shape[1]
    for s, (at, n) in enumerate(x["seqs"]):
        S = f64_norm(x["init"][s].flatten(1)) if x["init"] is not None else torch.zeros(H, dtype=torch.float64)
        grow = S + v[at:at + n].cumsum(0)  # of the state behind each token
        G = f64_norm(x["dfinal"][s].flatten(1)) if x["dfinal"] is not None else torch.zeros(H, dtype=torch.float64)
        back = x["scale"] * do[at:at + n]
        behind = G + back.flip(0).cumsum(0).flip(0) - back  # of the gradient behind each token
        for c in range(0, n, 64):
            e = min(c + 64, n)
            part = back[c:e] * grow[c:e] + v[at + c:at + e] * dv[at + c:at + e]
            out[at + c:at + e] = part.flip(0).cumsum(0).flip(0) + (behind[e - 1] * grow[e - 1])
    return out


@pytest.mark.parametrize("act,Dk,Dv,Hk", [("bf16", 128, 128, 2), ("f32", 64, 64, 4), ("bf16", 64, 128, 1)])
def test_dg_of_every_head(act, Dk, Dv, Hk):
    """Head 0 keeps nothing anywhere, head 1 decays by e^-20 a token, the others as models do.  Where nothing is
    kept dg is zero and nothing else; elsewhere it is good to 2^-19 of the terms that it is the sum of."""
    x = make([150, 1, 64], 4, Hk, Dk, Dv, act, seed=3)
    x["g"][..., 0], x["g"][..., 1] = -float("inf"), -20.0
    x["g"][0, ::9, 2], x["g"][0, ::7, 3] = -float("inf"), -150.0
    want = R.gdelta_bwd(*flat(x, "q", "k", "v", "g", "beta"), x["scale"], x["seqs"], x["do"].flatten(0, 1),
                        x["init"], x["dfinal"])
    got = backward(x).dg.flatten(0, 1).cpu().double()
    nothing = (x["g"] <= -150.0).flatten(0, 1).cpu()
    assert nothing[:, 0].all() and (want["dg"][nothing].abs() < 1e-40).all()
    assert (got[nothing] == 0.0).all(), float(got[nothing].abs().max())
    err = (got - want["dg"]).abs()
    assert (err <= 2.0 ** -19 * (dg_terms(x, want) + want["dg"].abs())).all()
    # and in the norm, as test_gpu_gdelta.py derives it, but each head by itself
    size = (f64_norm(x["v"].flatten(0, 1)) * want["dv"].norm(dim=-1)) ** 2
    for h in range(4):
        terms = sum(float(size[c:min(c + 64, at + n), h].flip(0).cumsum(0).sum())
                    for at, n in x["seqs"] for c in range(at, at + n, 64)) ** 0.5
        bound = 2.0 ** -19 * float(want["dg"][:, h].norm()) + 2.0 ** -20 * terms
        assert float(err[:, h].norm()) <= bound, (h, float(err[:, h].norm()) / bound)
