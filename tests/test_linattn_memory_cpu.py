"""How much memory the linear attention asks for (host queries, no GPU): states of spans are
kept for a row's or a packed batch's tokens, not once more for every sequence."""
import pytest
import torch

import mamba2_ssd_chunked_amd as ssd


def la(tokens, H=32, Hk=32, Dk=128, Dv=128, batch=1):
    return ssd.make_linattn(batch=batch, seqlen=tokens, nheads=H, nkvheads=Hk, keydim=Dk,
                            valdim=Dv, act="bf16")


@pytest.mark.parametrize("tokens,nseqs", [(32768, (1, 11, 512, 4096, 32768)), (1025, (1, 2, 1025)),
                                          (5000, (3, 70, 5000)), (200, (1, 7, 200))])
@pytest.mark.parametrize("H,Hk", [(32, 32), (4, 1)])
@pytest.mark.parametrize("kind,states", [(ssd.SSD_WS_FORWARD, 1), (ssd.SSD_WS_BACKWARD, 3)])
def test_workspace_does_not_grow_with_the_sequences(tokens, nseqs, H, Hk, kind, states):
    """Spans have 256 tokens or more, and a span's entering state is one [H][Dv][Dk] float32 (three
    in the backward, beside dv and dk of every head where heads share keys and values)."""
    p = la(tokens, H, Hk)
    most = states * (tokens // 256) * (H * 128 * 128 * 4)
    if kind == ssd.SSD_WS_BACKWARD and H != Hk:
        most += tokens * H * 256 * 4
    for n in nseqs:
        got = ssd.ssd_linattn_workspace_bytes(p, n, kind)
        if n * H * 16 > (2 ** 32 - 1) // 256:  # 16 workgroups compose a (sequence, head): refused
            assert (n, H) == (32768, 32) and got == 0
            continue
        assert 0 < got <= max(most, 256), (n, got, most)


def test_workspace_of_rows():
    """Rows: the spans of every row but its first."""
    p = la(8192, 32, 32, 128, 64, batch=2)
    for kind, states in ((ssd.SSD_WS_FORWARD, 1), (ssd.SSD_WS_BACKWARD, 3)):
        got = ssd.ssd_linattn_workspace_bytes(p, 2, kind)
        assert 0 < got <= states * 2 * 31 * 32 * 128 * 64 * 4
        # neither rows nor packed sequences
        assert ssd.ssd_linattn_workspace_bytes(p, 3, kind) == 0
        assert ssd.ssd_linattn_workspace_bytes(p, 1, kind) == 0


def test_states_that_nobody_asked_for_are_not_made(monkeypatch):
    from mamba2_ssd_chunked_amd import mixer
    calls = {}
    for n in ("ssd_linattn_fwd", "ssd_linattn_bwd"):
        monkeypatch.setattr(mixer, n, lambda *a, n=n: calls.__setitem__(n, a))
    p = la(64, 2, 1, 64, 64)
    x = torch.zeros(1, 64, 2, 64)
    f = ssd.linattn_forward(p, x, x, x, None)
    g = ssd.linattn_backward(p, x, x, x, None, x)
    assert f.final_state is None and g.dinit is None
    assert calls["ssd_linattn_fwd"][8] is None and calls["ssd_linattn_bwd"][12] is None
    f = ssd.linattn_forward(p, x, x, x, None, want_final=True)
    g = ssd.linattn_backward(p, x, x, x, None, x, want_dinit=True)
    assert f.final_state.shape == g.dinit.shape == (1, 2, 64, 64)
    assert calls["ssd_linattn_fwd"][8] is f.final_state and calls["ssd_linattn_bwd"][12] is g.dinit
    # buffers made beforehand hold both, and a call without them refuses to be asked for them
    b = ssd.LinAttnForwardBuffers.allocate(p, 1, "cpu")
    assert b.final_state is not None and ssd.LinAttnBackwardBuffers.allocate(p, 1, "cpu").dinit is not None
    with pytest.raises(ValueError, match="final_state"):
        ssd.linattn_forward(p, x, x, x, None, want_final=True,
                            bufs=ssd.LinAttnForwardBuffers.allocate(p, 1, "cpu", final=False))
    with pytest.raises(ValueError, match="dinit"):
        ssd.linattn_backward(p, x, x, x, None, x, want_dinit=True,
                             bufs=ssd.LinAttnBackwardBuffers.allocate(p, 1, "cpu", dinit=False))
