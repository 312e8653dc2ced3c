"""Slots that many rows of a large batch share: the first row that is not skipped runs."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def draw_slots(rows, nslots):
    """Slots with repeats near and far apart, padding, and rows skipped by their position."""
    g = torch.Generator().manual_seed(rows)
    ids = torch.randint(0, nslots, (rows,), generator=g)
    ids[torch.rand(rows, generator=g) < 0.05] = -1
    pos = torch.randint(1, 50, (rows,), generator=g)
    pos[torch.rand(rows, generator=g) < 0.3] = -1
    live, seen = [], set()
    for r in range(rows):
        s = int(ids[r])
        if s >= 0 and int(pos[r]) >= 0 and s not in seen:
            seen.add(s)
            live.append(r)
    t32 = lambda t: t.to(torch.int32).cuda()  # noqa: E731
    return t32(ids), t32(pos), torch.tensor(live, device="cuda")


@pytest.mark.parametrize("rows,nslots", [(70, 9), (1025, 700), (3000, 2500), (2049, 1)])
def test_linattn_step(rows, nslots):
    import mamba2_ssd_chunked_amd as ssd
    g = torch.Generator("cuda").manual_seed(rows)
    q, k, v = (torch.randn(rows, 1, 1, 64, generator=g, device="cuda") for _ in range(3))
    state = torch.randn(nslots, 1, 64, 64, generator=g, device="cuda")
    ld = torch.tensor([-0.2], device="cuda")
    ids, pos, live = draw_slots(rows, nslots)
    want, o = state.clone(), torch.full((rows, 1, 1, 64), 7.0, device="cuda")
    wo = o.clone()
    p = ssd.make_linattn(batch=rows, seqlen=1, nheads=1, keydim=64, valdim=64, act="f32")
    ssd.ssd_linattn_step(p, q, k, v, ld, state, o, slots=ids, positions=pos)
    # the rows that run, alone: no two of them share a slot
    n = len(live)
    pl = ssd.make_linattn(batch=n, seqlen=1, nheads=1, keydim=64, valdim=64, act="f32")
    ol = torch.empty(n, 1, 1, 64, device="cuda")
    ssd.ssd_linattn_step(pl, q[live], k[live], v[live], ld, want, ol, slots=ids[live])
    wo[live] = ol
    torch.cuda.synchronize()
    assert torch.equal(state, want) and torch.equal(o, wo)


@pytest.mark.parametrize("rows,nslots", [(1025, 700), (2500, 2000)])
def test_token_step(rows, nslots):
    import mamba2_ssd_chunked_amd as ssd
    import test_gpu_token_step as TS
    H, G, P, N = 4, 2, 16, 16
    x = TS.draws(rows, 1, H, G, P, N, 4, "f32", nslots, 4, seed=2)
    ids, pos, live = draw_slots(rows, nslots)
    prob = lambda n: ssd.make_problem(batch=n, seqlen=1, nheads=H, headdim=P, dstate=N,  # noqa: E731
                                      ngroups=G, chunk=64, conv_width=4, act="f32")
    par = (x["dt_bias"], x["A_log"], x["D"])
    ring, state = x["conv_ring"].clone(), x["state"].clone()
    y, n = torch.full((rows, 1, H, P), 7.0, device="cuda"), len(live)
    wy, yl = y.clone(), torch.empty(n, 1, H, P, device="cuda")
    ssd.ssd_token_step(prob(rows), x["xBC"], x["conv_w"], x["dt_raw"], *par, x["conv_ring"],
                       x["state"], pos, y, slots=ids)
    ssd.ssd_token_step(prob(n), x["xBC"][live], x["conv_w"], x["dt_raw"][live], *par, ring, state,
                       pos[live], yl, slots=ids[live])
    wy[live] = yl
    torch.cuda.synchronize()
    assert torch.equal(y, wy) and torch.equal(x["state"], state) and torch.equal(x["conv_ring"], ring)
