"""StepState.load: which slots of the pool a prompt's rows go to (plain tensor work, on the CPU)."""
import pytest
import torch

import mamba2_ssd_chunked_amd as ssd

B, L, H, P, N = 4, 9, 2, 16, 16
C = H * P + 2 * N


def problem(batch=B, seqlen=L):
    return ssd.make_problem(batch=batch, seqlen=seqlen, nheads=H, headdim=P, dstate=N, ngroups=1,
                            chunk=64, conv_width=4, act="f32")


def filled(nslots):
    pool = ssd.StepState.allocate(problem(), nslots, "cpu", tokens=2)
    pool.conv_ring.uniform_(-1, 1)
    pool.state.uniform_(-1, 1)
    return pool


def prompt(b=B, n=L):
    g = torch.Generator().manual_seed(4)
    return torch.randn(b, n, C, generator=g), torch.randn(b, H, P, N, generator=g)


@pytest.mark.parametrize("slots,owners", [
    ([3, 0, 5, 1], {3: 0, 0: 1, 5: 2, 1: 3}),
    ([3, -1, 0, 6], {3: 0, 0: 2}),          # two rows of padding, one beyond the pool
    ([-1, 2, 2, 2], {2: 1}),                # of several rows with one slot the first
    ([-1, -1, 99, -7], {}),                 # nothing but padding
    (None, {0: 0, 1: 1, 2: 2, 3: 3}),
])
@pytest.mark.parametrize("kind", [torch.int32, torch.int64])
def test_rows_go_to_their_slots_and_nowhere_else(slots, owners, kind):
    pool, (x, fin) = filled(6), prompt()
    ring, state = pool.conv_ring.clone(), pool.state.clone()
    pos = pool.load(problem(), x, fin, None if slots is None else torch.tensor(slots, dtype=kind))
    for s, r in owners.items():
        state[s] = fin[r]
        for t in range(L - 3, L):
            ring[s, t % 5] = x[r, t]
    assert torch.equal(pool.state, state) and torch.equal(pool.conv_ring, ring)
    assert pos.dtype == torch.int32
    assert pos.tolist() == [L if r in owners.values() else -1 for r in range(B)]


def test_a_prompt_shorter_than_the_taps():
    pool, (x, fin) = filled(6), prompt(n=2)
    ring = pool.conv_ring.clone()
    pos = pool.load(problem(seqlen=2), x, fin, torch.tensor([4, 0, 1, 2]))
    for r, s in enumerate([4, 0, 1, 2]):
        ring[s, :2] = x[r]
    assert torch.equal(pool.conv_ring, ring) and pos.tolist() == [2] * B


def test_refusals():
    pool, (x, fin) = filled(3), prompt()
    with pytest.raises(ValueError, match="slots"):
        pool.load(problem(), x, fin)                            # four rows, three slots
    with pytest.raises(ValueError, match="slots"):
        pool.load(problem(), x, fin, torch.tensor([0, 1, 2]))
    with pytest.raises(ValueError, match="slots"):
        pool.load(problem(), x, fin, torch.tensor([0., 1., 2., -1.]))
    with pytest.raises(ValueError, match="xBC"):
        pool.load(problem(), x[:, 1:], fin, torch.tensor([0, 1, 2, -1]))
    with pytest.raises(ValueError, match="final_state"):
        pool.load(problem(), x, fin[:1], torch.tensor([0, 1, 2, -1]))
    with pytest.raises(ValueError, match="xBC"):
        pool.load(problem(), x.bfloat16(), fin, torch.tensor([0, 1, 2, -1]))
