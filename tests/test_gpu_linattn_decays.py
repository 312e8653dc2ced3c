"""Linear attention with decays above 1 (log_decay > 0): short sequences, whose results float32
holds, come out as the recurrence has them.

Tolerances as in test_gpu_linattn_rounding, and 96 2^-24 of the sum of magnitudes more: a power
l^e is exp2 of a float32 of up to 100, off by 2^-24 of it, so 2^-24 ln 2 100 = 70 2^-24 of the
power, split over at most three factors that add 2^-23 each and two products more.
"""
import pytest
import torch

import test_gpu_linattn as LA
from test_gpu_linattn_rounding import assert_rounded_once

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 64), (64, 128), (128, 128)])
@pytest.mark.parametrize("init", [False, True])
def test_growing_states(Dk, Dv, act, init):
    """e^(17 * 4) is the largest power that a sequence has; the chunk's whole length would need
    e^(63 * 4), far beyond float32."""
    x = LA.make([1, 2, 17, 5], 4, 4, Dk, Dv, act, init=init, decay=[2.0, 4.0, 0.7, -0.1])
    assert_rounded_once(x, more=96 * 2.0 ** -24)


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_single_tokens_of_any_decay(act):
    """One token of a new sequence does not depend on its decay: prompts, and the token step."""
    import mamba2_ssd_chunked_amd as ssd
    x = LA.make([1, 1, 1], 4, 2, 64, 128, act, init=False, decay=[100.0, 7.0, -float("inf"), 0.0])
    y = dict(x, ld=torch.full((4,), -0.25, device="cuda"))
    a, b = LA.run_fwd(x), LA.run_fwd(y)
    ga, gb = LA.run_bwd(x), LA.run_bwd(y)
    p = ssd.make_linattn(batch=3, seqlen=1, nheads=4, nkvheads=2, keydim=64, valdim=128, act=act)
    t = [x[c].transpose(0, 1).contiguous() for c in "qkv"]
    steps = []
    for ld in (x["ld"], y["ld"]):
        state = torch.full((3, 4, 128, 64), 9.0, device="cuda")
        o = torch.empty(3, 1, 4, 128, dtype=LA.ACT[act], device="cuda")
        ssd.ssd_linattn_step(p, *t, ld, state, o,
                             positions=torch.zeros(3, dtype=torch.int32, device="cuda"))
        steps.append((o, state))
    torch.cuda.synchronize()
    assert torch.equal(a.o, b.o) and torch.equal(a.final_state, b.final_state)
    for n in ("dq", "dk", "dv"):
        assert torch.equal(getattr(ga, n), getattr(gb, n)), n
    for u, v in zip(*steps):
        assert torch.equal(u, v)
