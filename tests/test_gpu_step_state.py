"""StepState.load on the GPU: padded rows of a batch, other streams, captured graphs."""
import pytest
import torch

pytestmark = pytest.mark.gpu

ROWS, L, H, P, N, G = 5, 64, 4, 64, 64, 2
C = H * P + 2 * G * N


def make(act=torch.bfloat16):
    import mamba2_ssd_chunked_amd as ssd
    g = torch.Generator("cuda").manual_seed(8)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    par = (0.5 * rnd(C, 4), rnd(ROWS, 1, H).to(act), rnd(H) - 3, rnd(H).abs(), rnd(H))
    prob = lambda n: ssd.make_problem(batch=ROWS, seqlen=n, nheads=H, headdim=P, dstate=N,  # noqa: E731
                                      ngroups=G, chunk=64, conv_width=4, act="bf16")
    pool = ssd.StepState.allocate(prob(1), 6, "cuda")
    pool.conv_ring.copy_(rnd(6, 4, C))
    pool.state.copy_(rnd(6, H, P, N))
    return dict(x=rnd(ROWS, L, C).to(act), fin=rnd(ROWS, H, P, N), new=rnd(ROWS, 1, C).to(act),
                par=par, long=prob(L), one=prob(1), pool=pool,
                slots=torch.tensor([4, -1, 0, 4, 17], dtype=torch.int32, device="cuda"))


def handed_over(m, pool, y, stream=None):
    import mamba2_ssd_chunked_amd as ssd
    w, dt, *rest = m["par"]
    pos = pool.load(m["long"], m["x"], m["fin"], m["slots"], stream=stream)
    ssd.ssd_token_step(m["one"], m["new"], w, dt, *rest, pool.conv_ring, pool.state, pos, y,
                       slots=m["slots"], stream=stream)
    return pos


def copy_of(pool):
    import mamba2_ssd_chunked_amd as ssd
    return ssd.StepState(pool.conv_ring.clone(), pool.state.clone())


def test_padded_rows_touch_no_other_sequence():
    """Slots -1 and 17 of 6 and a slot that is taken: the last slot and the others stay as they
    were, and the step that gets the positions skips these rows."""
    m = make()
    pool, y = copy_of(m["pool"]), torch.full((ROWS, 1, H, P), 7.0, dtype=torch.bfloat16, device="cuda")
    pos = handed_over(m, pool, y)
    torch.cuda.synchronize()
    assert pos.tolist() == [L, -1, L, -1, -1]
    for s in (1, 2, 3, 5):
        assert torch.equal(pool.state[s], m["pool"].state[s])
        assert torch.equal(pool.conv_ring[s], m["pool"].conv_ring[s])
    for r in (1, 3, 4):
        assert (y[r] == 7).all()
    for r, s in ((0, 4), (2, 0)):
        assert not (y[r] == 7).all()
        want = torch.stack([m["x"][r, L - 4 + i] if i else m["new"][r, 0] for i in range(4)])
        assert torch.equal(pool.conv_ring[s], want)  # tokens 64 (over 60), 61, 62, 63


def test_load_and_step_on_another_stream():
    m = make()
    a, b = copy_of(m["pool"]), copy_of(m["pool"])
    ya, yb = (torch.zeros(ROWS, 1, H, P, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    handed_over(m, a, ya)
    side = torch.cuda.Stream()
    pos = handed_over(m, b, yb, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(ya, yb) and torch.equal(a.state, b.state)
    assert torch.equal(a.conv_ring, b.conv_ring) and pos.tolist() == [L, -1, L, -1, -1]


def test_captured_load():
    """Replays follow the slots of the moment, all of them padding included."""
    m = make()
    cap, y = copy_of(m["pool"]), torch.zeros(ROWS, 1, H, P, dtype=torch.bfloat16, device="cuda")
    handed_over(m, copy_of(m["pool"]), torch.zeros_like(y))  # warm up
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pos = handed_over(m, cap, y)
    for slots in ([4, -1, 0, 4, 17], [-1] * 5, [0, 1, 2, 3, 5], [-3, -3, 5, 99, 5]):
        m["slots"].copy_(torch.tensor(slots, dtype=torch.int32))
        cap.conv_ring.copy_(m["pool"].conv_ring)
        cap.state.copy_(m["pool"].state)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        eager, ye = copy_of(m["pool"]), torch.zeros_like(y)
        pe = handed_over(m, eager, ye)
        torch.cuda.synchronize()
        assert torch.equal(pos, pe) and torch.equal(y, ye)
        assert torch.equal(cap.state, eager.state) and torch.equal(cap.conv_ring, eager.conv_ring)
