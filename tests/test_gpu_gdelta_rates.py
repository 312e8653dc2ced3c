"""Gradients of the gated delta rule where update rates are zero, or so small that the backward, which divides by
them, counts with a larger one."""
import pytest
import torch

import layer_ref as R
from test_gpu_gdelta import ACT, f64_norm, flat, make
from test_gpu_gdelta_gates import backward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act,Dk,Dv,H,Hk", [("bf16", 128, 64, 2, 2), ("f32", 64, 64, 2, 2), ("f32", 128, 128, 4, 2),
                                            ("bf16", 128, 128, 4, 1)])
def test_rates_below_what_the_backward_counts_with(act, Dk, Dv, H, Hk):
    """dv_t and dk_t have a factor beta_t, and what else is in them does not depend on it: between 2^-40 and 2^-60 they
    lose 2^-20 (dk_t but for what other such tokens add, 2^-40 of it: a step where a rounding tips over), at zero
    they are zero.  The other tokens' dq and dk change by 2^-40, dbeta and dinit not at all."""
    x = make([90, 70], H, Hk, Dk, Dv, act, seed=5)
    rows = slice(3, 150, 7)

    def at(beta):
        y = dict(x, beta=x["beta"].clone())
        y["beta"][0, rows] = beta
        return backward(y)

    floor, small, none = at(2.0 ** -40), at(2.0 ** -60), at(0.0)
    minus = at(-0.0)
    def step(a, b):  # at most a step apart
        return ((a.float() - b.float()).abs() <= torch.finfo(a.dtype).eps * torch.maximum(a.float().abs(), b.float().abs())
                + 2.0 ** -34).all()

    assert torch.equal(floor.dv[0, rows].float() * 2.0 ** -20, small.dv[0, rows].float())
    a, b = floor.dk[0, rows].float() * 2.0 ** -20, small.dk[0, rows].float()
    assert b.abs().max() > 0 and ((a - b).abs() <= torch.finfo(floor.dk.dtype).eps * b.abs() + 2.0 ** -94).all()
    for z in (none, minus):
        assert (z.dv[0, rows] == 0).all() and (z.dk[0, rows] == 0).all()
    for z in (small, none):
        for n in ("dbeta", "dinit"):
            assert torch.equal(getattr(floor, n), getattr(z, n)), n
        keep = torch.ones(160, dtype=torch.bool)
        keep[rows] = False
        assert torch.equal(floor.dv[0, keep], z.dv[0, keep])
        assert step(floor.dk[0, keep], z.dk[0, keep]) and step(floor.dq, z.dq)
    y = dict(x, beta=x["beta"].clone())
    y["beta"][0, rows] = 2.0 ** -60
    want = R.gdelta_bwd(*flat(y, "q", "k", "v", "g", "beta"), x["scale"], x["seqs"], x["do"].flatten(0, 1),
                        x["init"], x["dfinal"])
    # of a bf16 value 2^-8, and 2^-16 of the sizes that meet (du: |G| + scale |do|, at most their sums)
    size = float(f64_norm(x["dfinal"].flatten(2)).max()) + x["scale"] * float(f64_norm(x["do"]).max()) * 90
    got = small.dv[0, rows].cpu().double()
    err = (got - want["dv"][rows]).abs()
    u = 2.0 ** -8 if ACT[act] == torch.bfloat16 else 2.0 ** -23
    assert (err <= u * want["dv"][rows].abs() + 2.0 ** -16 * 2.0 ** -60 * size).all()
