"""The float64 references of layer_ref.py against automatic differentiation and differences (CPU)."""
import torch

import layer_ref as R


def _gd(T=7, H=4, Hk=2, Dk=5, Dv=3, seed=0):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    return dict(q=rnd(T, Hk, Dk), k=rnd(T, Hk, Dk), v=rnd(T, H, Dv), g=-rnd(T, H).abs(),
                beta=torch.rand(T, H, generator=g, dtype=torch.float64), init=rnd(2, H, Dv, Dk))


def test_gdelta_forward_is_the_delta_rule():
    """S_t = a S_(t-1) (1 - beta k k^T) + beta v k^T, as one matrix."""
    x = _gd()
    o, fin, _, _ = R.gdelta_fwd(**{n: x[n] for n in ("q", "k", "v", "g", "beta")}, scale=0.7,
                                sequences=[(1, 4), (5, 0)], init=x["init"])
    for h in range(4):
        S = x["init"][0, h]
        for t in range(1, 5):
            k, b = x["k"][t, h // 2], x["beta"][t, h]
            S = torch.exp(x["g"][t, h]) * S @ (torch.eye(5, dtype=torch.float64) - b * torch.outer(k, k))
            S = S + b * torch.outer(x["v"][t, h], k)
            assert torch.allclose(o[t, h], 0.7 * S @ x["q"][t, h // 2], atol=1e-12)
        assert torch.allclose(fin[0, h], S, atol=1e-12)
    assert torch.equal(fin[1], x["init"][1]) and not o[0].any() and not o[5:].any()


def test_gdelta_backward_against_differences():
    x = _gd()
    seqs, h = [(0, 4), (4, 3)], 1e-6
    w = _gd(seed=1)
    do, df = w["v"], w["init"]

    def value(y):
        o, fin, _, _ = R.gdelta_fwd(y["q"], y["k"], y["v"], y["g"], y["beta"], 0.7, seqs, y["init"])
        return float((o * do).sum() + (fin * df).sum())

    got = R.gdelta_bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], 0.7, seqs, do, x["init"], df)
    for name, t in x.items():
        d = torch.randn(t.shape, generator=torch.Generator().manual_seed(3), dtype=torch.float64)
        step = (value(dict(x, **{name: t + h * d})) - value(dict(x, **{name: t - h * d}))) / (2 * h)
        want = float((got["d" + name] * d).sum())
        # central differences: h^2 of a third derivative, and 2^-52 / h of the values
        assert abs(step - want) < 1e-7 * max(1.0, abs(want)), name


def test_block_norm_of_one_row():
    x, y = torch.tensor([[1.0, -2.0, 3.0]]).double(), torch.tensor([[3.0, 0.0, -4.0]]).double()
    one = torch.ones(3).double()
    r, h = R.block_norm(dict(x=x, y=y, z=2 * one[None], scale=0.5 * one, post_weight=one, pre_weight=2 * one),
                        gate="linear", center=False, alpha=2.0, eps=0.0)
    n = (25 / 3) ** 0.5
    want = 2 * x + torch.tensor([[3.0, 0.0, -4.0]]).double() / n
    assert torch.allclose(r, want) and torch.allclose(h, 2 * want / want.square().mean().sqrt())


def test_rope_turns_pairs():
    x = torch.tensor([[[1.0, 2.0, 3.0, 4.0, 9.0]]]).double()
    quarter = torch.tensor([[torch.pi / 2, torch.pi]]).double()
    half = R.rope(x, quarter, 2.0, 4, "half", False)
    assert torch.allclose(half, torch.tensor([[[-6.0, -4.0, 2.0, -8.0, 9.0]]]).double())
    inter = R.rope(x, quarter, 1.0, 4, "interleaved", False)
    assert torch.allclose(inter, torch.tensor([[[-2.0, 1.0, -3.0, -4.0, 9.0]]]).double())
    assert torch.allclose(R.rope(inter, quarter, 1.0, 4, "interleaved", True), x)
