"""ssd_token_step with tensors that are aligned to their elements only, as slices of rows are."""
import pytest
import torch

import test_gpu_token_step as TS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act,P,N", [("f32", 16, 16), ("f32", 64, 128), ("bf16", 32, 64), ("bf16", 64, 128)])
@pytest.mark.parametrize("rows", [3, 600])
def test_element_aligned_tensors(rows, act, P, N):
    """One element behind a 16-byte border, the values are those of aligned tensors, and nothing
    beside the tensors is written."""
    import mamba2_ssd_chunked_amd as ssd
    H, G, Wc, T = 4, 2, 4, 2
    x = TS.draws(rows, T, H, G, P, N, Wc, act, rows, Wc - 1 + T, seed=P + rows)
    pos = torch.arange(rows, dtype=torch.int32, device="cuda") % 5
    p = ssd.make_problem(batch=rows, seqlen=T, nheads=H, headdim=P, dstate=N, ngroups=G, chunk=64,
                         conv_width=Wc, act=act)

    def shifted(t):
        room = torch.full((t.numel() + 8,), 3.0, dtype=t.dtype, device="cuda")
        v = room[1:1 + t.numel()].view(t.shape)
        v.copy_(t)
        assert v.data_ptr() % 16 == t.element_size()
        return v, room

    names = ("xBC", "conv_w", "dt_raw", "dt_bias", "A_log", "D", "conv_ring")
    y = torch.full((rows, T, H, P), 7.0, dtype=TS.ACT[act], device="cuda")
    s = {n: shifted(x[n]) for n in names}
    ys, state = shifted(y), x["state"].clone()
    ssd.ssd_token_step(p, *(x[n] for n in names), x["state"], pos, y)
    ssd.ssd_token_step(p, *(s[n][0] for n in names), state, pos, ys[0])
    torch.cuda.synchronize()
    assert torch.equal(ys[0], y) and torch.equal(state, x["state"])
    assert torch.equal(s["conv_ring"][0], x["conv_ring"])
    for v, room in [*s.values(), ys]:
        assert room[0] == 3.0 and (room[1 + v.numel():] == 3.0).all()
