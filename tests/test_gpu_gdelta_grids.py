"""The gated delta rule with enough sequences and heads that a walk's workgroups are of two waves, or
of four (with one or two tiles of channels to a wave), and that heads of a key head are taken in turn;
against the float64 recurrence with the bounds of test_gpu_gdelta.py."""
import pytest
import torch

from test_gpu_gdelta import check_backward, check_forward, make, problem

pytestmark = pytest.mark.gpu

FEW = [70, 0, 1, 64, 129, 5, 40, 33, 66]  # 9 sequences; of 8 heads 288 tiles of 16 channels of 64, 576 of 128
MANY = FEW + [7, 65, 2, 100, 63, 31, 128, 3]  # 17 sequences: 544 tiles of 64, 1088 of 128
CASES = [
    dict(lens=FEW, H=8, Hk=4, Dk=128, Dv=64, before=3, behind=6),
    dict(lens=FEW, H=8, Hk=2, Dk=64, Dv=64, gates="edges"),
    dict(lens=FEW[:5], H=8, Hk=8, Dk=64, Dv=128, fused=True),
    dict(lens=MANY, H=8, Hk=8, Dk=64, Dv=64, fused=True),
    dict(lens=MANY, H=8, Hk=1, Dk=128, Dv=64, behind=80),
    dict(lens=FEW, H=8, Hk=4, Dk=128, Dv=128, gates="edges"),
    dict(lens=FEW, H=9, Hk=3, Dk=64, Dv=128, init=False),
    dict(lens=MANY, H=8, Hk=2, Dk=128, Dv=128, fused=True),
    dict(lens=MANY, H=8, Hk=4, Dk=64, Dv=128, gates="edges"),
    dict(lens=FEW[:5], H=16, Hk=8, Dk=128, Dv=64, before=900, behind=900),  # 32 chunks of 8 key heads or more:
    dict(lens=FEW[:5], H=16, Hk=8, Dk=64, Dv=128, before=70, behind=1720),  # their heads in turn
]
name = lambda c: f"{c['Dk']}x{c['Dv']}-{len(c['lens'])}-{c['H']}"  # noqa: E731


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=name)
def test_forward(case, act):
    check_forward(make(act=act, seed=1, **case))


@pytest.mark.parametrize("case", CASES, ids=name)
def test_forward_without_final_state(case):
    check_forward(make(act="bf16", seed=2, **case), want_final=False)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=name)
def test_backward(case, act):
    check_backward(make(act=act, seed=3, **case), want_dinit=case.get("init", True))


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("case", [CASES[0], CASES[3], CASES[5], CASES[7]], ids=name)
def test_values_that_are_not_finite(case, act):
    """One in the middle of a sequence of more than a chunk reaches no other sequence and, forward, no earlier
    token."""
    import mamba2_ssd_chunked_amd as ssd
    x = make(act=act, seed=4, **case)
    p, (first, n) = problem(x), x["seqs"][4]
    at = first + 66
    ins = lambda y: [y[t] for t in ("q", "k", "v", "g", "beta")]  # noqa: E731
    fwd = lambda y: ssd.gdelta_forward(p, *ins(y), cu_seqlens=x["cu"], init=x["init"], want_final=True)  # noqa: E731
    bwd = lambda y: ssd.gdelta_backward(p, *ins(y), x["do"], cu_seqlens=x["cu"], init=x["init"],  # noqa: E731
                                        dfinal=x["dfinal"])
    rows = torch.zeros(x["dims"][1], dtype=torch.bool)
    for a, m in x["seqs"]:
        rows[a:a + m] = True
    others = [s for s in range(len(x["seqs"])) if s != 4]
    good, good_b = fwd(x), bwd(x)
    for t, bad in (("v", float("inf")), ("k", float("nan")), ("g", float("nan")), ("beta", -float("inf"))):
        y = dict(x, **{t: x[t].clone()})
        y[t][0, at].view(-1)[1] = bad
        f, b = fwd(y), bwd(y)
        same = rows.clone()
        same[at:first + n] = False
        assert torch.equal(f.o[0, same], good.o[0, same]), t
        assert torch.equal(f.final_state[others], good.final_state[others]), t
        assert not torch.isfinite(f.final_state[4]).all() and not torch.isfinite(f.o[0, at]).all(), t
        same[first:at] = False
        for d in ("dq", "dk", "dv", "dg", "dbeta"):
            assert torch.equal(getattr(b, d)[0, same], getattr(good_b, d)[0, same]), (t, d)
