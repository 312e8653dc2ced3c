"""Pins of the float64 references in mixer_ref.py (CPU): closed forms and differences."""
import pytest
import torch

import mixer_ref as R

g = torch.Generator().manual_seed(5)


def rand(*shape):
    return torch.randn(*shape, generator=g, dtype=torch.float64)


def test_linattn_without_decay_is_the_masked_product():
    q, k, v = rand(7, 2, 3), rand(7, 2, 3), rand(7, 2, 4)
    o, fin = R.linattn_fwd(q, k, v, torch.zeros(2), 0.5, [(0, 7)])
    P = torch.einsum("thd,shd->hts", q, k).tril()
    assert torch.allclose(o, 0.5 * torch.einsum("hts,shd->thd", P, v))
    assert torch.allclose(fin[0], torch.einsum("thd,the->hde", v, k))


def test_linattn_full_decay_sees_only_itself():
    q, k, v = rand(5, 1, 3), rand(5, 1, 3), rand(5, 1, 2)
    o, fin = R.linattn_fwd(q, k, v, torch.full((1,), -float("inf")), 1.0, [(0, 5)])
    assert torch.allclose(o, (q * k).sum(-1, keepdim=True) * v)
    assert torch.allclose(fin[0, 0], v[4, 0][:, None] * k[4, 0][None])


def test_linattn_gradients_by_differences():
    seqs, ld, scale = [(0, 3), (3, 0), (4, 4)], -torch.rand(4, generator=g, dtype=torch.float64), 0.3
    x = dict(q=rand(9, 4, 3), k=rand(9, 2, 3), v=rand(9, 2, 2), init=rand(3, 4, 2, 3))
    do, dfin = rand(9, 4, 2), rand(3, 4, 2, 3)

    def loss(**c):
        a = dict(x, **c)
        o, fin = R.linattn_fwd(a["q"], a["k"], a["v"], ld, scale, seqs, a["init"])
        return float((o * do).sum() + (fin * dfin).sum())

    got = dict(zip(("q", "k", "v", "init"),
                   R.linattn_bwd(x["q"], x["k"], x["v"], ld, scale, seqs, do, x["init"], dfin)))
    for name, t in x.items():
        d = rand(*t.shape)
        h = 1e-5
        num = (loss(**{name: t + h * d}) - loss(**{name: t - h * d})) / (2 * h)
        assert num == pytest.approx(float((got[name] * d).sum()), rel=1e-7, abs=1e-8)


def test_token_step_agrees_with_the_prompt_oracle():
    import numpy as np

    import oracle
    import ssd_workloads as W
    wl = W.make_workload("pin", batch=1, seqlen=64, nheads=4, headdim=16, dstate=16, ngroups=2,
                         chunk=64, act="f32", seed=7)
    _, u = oracle.conv_silu(wl.xBC, wl.conv_w, None)
    y, fin = oracle.ssd_fwd(u, wl.dt_raw, wl.dt_bias, wl.A_log, wl.D, nheads=4, headdim=16,
                            dstate=16, ngroups=2, dt_min=wl.dt_min, dt_max=wl.dt_max,
                            want_final=True)
    t = lambda a: torch.from_numpy(np.asarray(a))  # noqa: E731
    S, out, at = torch.zeros(4, 16, 16), [], 0
    for n in (1, 5, 58):
        yy, S = R.token_step(t(wl.xBC)[0, at:at + n], t(wl.conv_w), t(wl.dt_raw)[0, at:at + n],
                             t(wl.dt_bias), t(wl.A_log), t(wl.D), t(wl.xBC)[0, :at], S, at, 2,
                             wl.dt_min, wl.dt_max)
        out.append(yy)
        at += n
    assert torch.allclose(torch.cat(out), t(y)[0].double(), rtol=1e-6, atol=1e-7)
    assert torch.allclose(S, t(fin)[0].double(), rtol=1e-6, atol=1e-7)


@pytest.mark.parametrize("mode", ["none", "silu", "before", "after"])
@pytest.mark.parametrize("center", [False, True])
def test_norm_against_torch(mode, center):
    x, w, b, z = rand(5, 12), rand(12), rand(12), rand(5, 12)
    got = R.norm(x, w, b, z if mode in ("before", "after") else None, 3, mode, center, 1e-5)
    F = torch.nn.functional
    u = x * F.silu(z) if mode == "before" else x
    if center:
        want = F.group_norm(u, 3, w, b, 1e-5)
    else:
        v = u.reshape(5, 3, 4)
        want = (v / (v.pow(2).mean(-1, keepdim=True) + 1e-5).sqrt()).reshape(5, 12) * w + b
    want = want * F.silu(z) if mode == "after" else (F.silu(want) if mode == "silu" else want)
    assert torch.allclose(got, want)
