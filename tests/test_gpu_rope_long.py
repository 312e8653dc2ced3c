"""More tokens than the rotation has workgroups (2^22), so that some take a second one."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("packed", [False, True])
def test_more_tokens_than_workgroups(packed):
    import mamba2_ssd_chunked_amd as ssd
    T = (1 << 22) + 9
    f, _ = ssd.rope_frequencies(2, device="cuda")
    q = torch.zeros(1, T, 1, 2, device="cuda")
    q[..., 0] = 1.0
    p = ssd.make_rope(batch=1, seqlen=T, nheads=1, headdim=2, act="f32")
    cu, place = None, torch.arange(T, dtype=torch.float64, device="cuda")
    if packed:  # three tokens before, a sequence across the border, another one, two tokens behind
        cu = torch.tensor([3, (1 << 22) + 2, T - 2], dtype=torch.int32, device="cuda")
        place = torch.cat([place[:3] * 0, place[:cu[1] - 3], place[:T - 2 - int(cu[1])], place[:2] * 0])
    out, _ = ssd.rope_forward(p, q, None, f, cu_seqlens=cu, out=(torch.full_like(q, 7.0), None))
    want = torch.stack([place.cos(), place.sin()], dim=-1)  # radians below 2^23: 2^-30 of a turn in float64
    if packed:
        rows = torch.zeros(T, dtype=torch.bool, device="cuda")
        rows[3:T - 2] = True
        assert (out[0, ~rows] == 7.0).all()
        out, want = out[:, rows], want[rows]
    # seven float32 steps (test_gpu_rope.py): 2^-21
    assert float((out[0, :, 0].double() - want).abs().max()) <= 2.0 ** -21
