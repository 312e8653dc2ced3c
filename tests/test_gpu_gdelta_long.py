"""The gated delta rule where elements, states and workspace lie beyond 2^31 elements and 2^32 bytes: the
last packed sequence behind a long one against the same sequence alone.

Both are within the bounds of test_gpu_gdelta.py of the same values (2^-9 of their norm for bf16, and for
float32 2^-19), so that they differ by twice that at most; dg's terms, which may cancel, are of unit size
here, and its bound is taken twice more.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

LONG, LAST, H, HK, D = 560_000, 300, 32, 8, 128  # 2.3e9 elements of v


def off(a, b):
    a, b = a.double(), b.double()
    return float((a - b).norm() / b.norm())


def make():
    g = torch.Generator(device="cuda").manual_seed(3)
    T = LONG + LAST
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    unit = lambda x: x.div_(x.norm(dim=-1, keepdim=True))  # noqa: E731
    gates = torch.rand(1, T, 2 * H, generator=g, device="cuda")
    return dict(q=unit(rnd(1, T, HK, D)), k=unit(rnd(1, T, HK, D)), v=rnd(1, T, H, D), g=gates[..., :H].neg(),
                beta=gates[..., H:])


def problem(tokens):
    import mamba2_ssd_chunked_amd as ssd
    return ssd.make_gdelta(batch=1, seqlen=tokens, nheads=H, nkheads=HK, keydim=D, valdim=D, act="bf16")


@pytest.fixture
def room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 140 << 30:
        pytest.skip("needs 140 GB of free device memory")
    yield
    torch.cuda.empty_cache()


def test_forward_and_backward_behind_a_long_sequence(room):
    import mamba2_ssd_chunked_amd as ssd
    x = make()
    cu = torch.tensor([0, LONG, LONG + LAST], dtype=torch.int32, device="cuda")
    last = {n: t[:, LONG:].contiguous() for n, t in x.items()}
    do = torch.randn(last["v"].shape, device="cuda", generator=torch.Generator("cuda").manual_seed(4)).bfloat16()
    alone = ssd.gdelta_forward(problem(LAST), **last, want_final=True)
    f = ssd.gdelta_forward(problem(LONG + LAST), **x, cu_seqlens=cu, want_final=True)
    assert off(f.o[:, LONG:], alone.o) <= 2 * 2.0 ** -9
    assert off(f.final_state[1], alone.final_state[0]) <= 2 * 2.0 ** -19
    del f
    alone = ssd.gdelta_backward(problem(LAST), **last, do=do)
    whole = torch.zeros_like(x["v"])
    whole[:, LONG:] = do
    b = ssd.gdelta_backward(problem(LONG + LAST), **x, do=whole, cu_seqlens=cu)
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        got = getattr(b, n)
        bound = 2.0 ** -8 if n in ("dq", "dk", "dv") else 2.0 ** (-16 if n == "dg" else -18)
        assert off(got[:, LONG:], getattr(alone, n)) <= bound, n
        assert not bool(got[:, :LONG].any()), n  # no gradient enters the first sequence
