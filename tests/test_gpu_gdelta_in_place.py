"""Prompts of the gated delta rule that continue states where they are: final_state in init's memory, for every kind
of walk.  The same bits as in a tensor of its own, which test_gpu_gdelta.py compares with float64."""
import pytest
import torch

from test_gpu_gdelta import make, problem

pytestmark = pytest.mark.gpu

# column tiles (sequences x heads x valdim / 16): teams, two waves, four of one tile, four of two
CASES = [
    dict(lens=[70, 0, 64, 1], H=4, Hk=2, Dk=128, Dv=64, act="bf16"),
    dict(lens=[130] * 3, H=4, Hk=2, Dk=64, Dv=64, act="f32", packed=False),
    dict(lens=[65] * 10, H=4, Hk=1, Dk=128, Dv=128, act="bf16"),
    dict(lens=[65] * 20, H=4, Hk=4, Dk=64, Dv=128, act="bf16"),
    dict(lens=[66] * 40, H=4, Hk=2, Dk=128, Dv=128, act="bf16"),
    dict(lens=[66] * 40, H=4, Hk=2, Dk=64, Dv=128, act="f32"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c['act']}-{c['Dk']}x{c['Dv']}-{len(c['lens'])}")
def test_states_in_place(case):
    import mamba2_ssd_chunked_amd as ssd
    x = make(**case)
    p = problem(x)
    call = lambda init, bufs=None: ssd.gdelta_forward(  # noqa: E731
        p, *[x[n] for n in ("q", "k", "v", "g", "beta")], cu_seqlens=x["cu"], init=init, bufs=bufs, want_final=True)
    want = call(x["init"])
    bufs = ssd.GatedDeltaForwardBuffers.allocate(p, len(x["seqs"]), "cuda")
    bufs.final_state = x["init"].clone()
    got = call(bufs.final_state, bufs)
    assert torch.equal(got.final_state, want.final_state) and torch.equal(got.o, want.o)
