"""Alignments that ssd_token_step refuses: host-side validation, every call fails a check."""
import pytest

import mamba2_ssd_chunked_amd as ssd
from test_mixer_abi_cpu import FAKE, token


@pytest.mark.parametrize("act,odd", [("bf16", 1), ("f32", 2)])
def test_elements_have_to_be_aligned(act, odd):
    p = ssd.make_problem(batch=4, seqlen=1, nheads=8, headdim=64, dstate=64, ngroups=2, chunk=64,
                         conv_width=4, act=act)
    for name in ("x", "dt", "y"):
        assert token(p, **{name: FAKE + odd}) == -4, name
    assert token(p, ring=FAKE + odd) == -4
    for name in ("w", "db", "A", "D"):
        assert token(p, **{name: FAKE + 2}) == -4, name
    for name in ("slots", "pos"):
        assert token(p, **{name: FAKE + 2}) == -4, name
    for off in (4, 8):
        assert token(p, state=FAKE + off) == -4
