"""Rotary positions of tensors that are aligned to 16 bytes and to no more, as slices of a projection are: 8 float32
channels at once are 32 bytes.  The same values in tensors of their own give the same bits, and those are compared
with the definition in test_gpu_rope.py."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_rows_aligned_to_16_bytes(act, style, inverse):
    import mamba2_ssd_chunked_amd as ssd
    b, L, H, K, D, rot = 2, 21, 3, 1, 64, 48
    g = torch.Generator(device="cuda").manual_seed(11)
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[act]
    unit = 16 // dt.itemsize
    odd = lambda n: torch.randn(b, L, n, generator=g, device="cuda").to(dt)  # noqa: E731
    # an odd number of 16-byte pieces to a row, and the queries and keys one such piece from its start
    wide, out = odd((H + K) * D + unit), odd((H + K) * D + unit)
    old = out.clone()
    cut = lambda x: (x[..., unit:unit + H * D].unflatten(-1, (H, D)),  # noqa: E731
                     x[..., unit + H * D:].unflatten(-1, (K, D)))
    q, k = cut(wide)
    assert q.data_ptr() % 32 == 16 and q.stride(1) * dt.itemsize % 32 == 16
    p = ssd.make_rope(batch=b, seqlen=L, nheads=H, nkheads=K, headdim=D, rotdim=rot, act=act, style=style)
    f, _ = ssd.rope_frequencies(rot, device="cuda")
    call = ssd.rope_backward if inverse else ssd.rope_forward
    want = call(p, q.contiguous(), k.contiguous(), f)
    got = call(p, q, k, f, out=cut(out))
    assert all(torch.equal(a, w) for a, w in zip(got, want))
    assert torch.equal(out[..., :unit], old[..., :unit])
    call(p, q, k, f, out=(q, k))  # in place
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
