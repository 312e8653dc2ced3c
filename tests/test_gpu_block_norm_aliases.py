"""The backward of the norms around a block in place: dx in x or dr, dy in y or dh, dz in z, as the header allows.
The same bits as in tensors of their own, over rows of every width that a kernel is made for, more of them than
workgroups where that many are cheap."""
import dataclasses

import pytest
import torch

from test_gpu_block_norm import ACT, make

pytestmark = pytest.mark.gpu

CASES = [
    dict(rows=9001, C=96, act="bf16", res="f32", gate="silu"),
    dict(rows=1700, C=1120, act="f32", res="f32", gate="sigmoid", center=True),
    dict(rows=2500, C=651, act="bf16", res="bf16", gate="linear"),
    dict(rows=700, C=4104, act="bf16", res="bf16", gate="silu", alpha=2.0),
    dict(rows=300, C=8200, act="bf16", res="f32", gate="silu"),
    dict(rows=300, C=5001, act="f32", res="f32", gate="silu", center=True),
    dict(rows=600, C=512, act="bf16", res="f32", gate="none", pre=False),
    dict(rows=600, C=520, act="f32", res="f32", gate="linear", post=False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c['act']}-{c['res']}-{c['rows']}x{c['C']}")
def test_backward_in_place(case):
    import mamba2_ssd_chunked_amd as ssd
    x, how, sizes = make(**case)
    x = dict(x, y=x["y"].contiguous(), **({"z": x["z"].contiguous()} if "z" in x else {}))
    p = ssd.make_block_norm(**sizes)
    rows, C = case["rows"], case["C"]
    g = torch.Generator(device="cuda").manual_seed(78)
    dr = torch.randn(rows, C, generator=g, device="cuda").to(ACT[case["res"]])
    dh = torch.randn(rows, C, generator=g, device="cuda").to(ACT[case["act"]]) if case.get("pre", True) else None
    rest = {n: v for n, v in x.items() if n not in ("x", "y", "z")}
    want = ssd.block_norm_backward(p, x["x"], x["y"], dr, dh=dh, z=x.get("z"), **rest)
    for dx_in, dy_in in (("x", "y"), ("dr", "dh"), ("x", "dh"), ("dr", "y")):
        t = {n: None if v is None else v.clone() for n, v in dict(x=x["x"], y=x["y"], z=x.get("z"), dr=dr, dh=dh).items()}
        if t[dy_in] is None:  # no dh without `pre`
            continue
        fresh = ssd.BlockNormBackwardBuffers.allocate(p, "cuda")
        bufs = dataclasses.replace(fresh, dx=t[dx_in], dy=t[dy_in], dz=t["z"])
        got = ssd.block_norm_backward(p, t["x"], t["y"], t["dr"], dh=t["dh"], z=t["z"], **rest, bufs=bufs)
        for f in dataclasses.fields(got):
            a, b = getattr(got, f.name), getattr(want, f.name)
            if f.name != "ws" and b is not None:
                assert torch.equal(a, b), (f.name, dx_in, dy_in)
