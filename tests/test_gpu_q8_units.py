"""Decode steps of many units: the counts around which the one-launch kernel takes another number of CTAs a
unit, or two launches are taken."""
import pytest
import torch

from _q8 import C_TC

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.mark.parametrize("G,d", [(4, 128), (8, 128), (8, 64), (1, 64)])
@pytest.mark.parametrize("units", [1, 76, 77, 121, 122, 152, 153, 202, 203, 304, 305, 608, 609])
def test_units(kvc, units, G, d):
    cap, block = 512, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(units)
    c = kvc.q8_cache(units, 1, cap, d, block)
    K, V = (torch.randn(units, 1, cap - 70, d, generator=g, device="cuda").to(BF) for _ in range(2))
    kvc.kv_compact_q8(K, V, None, None, c)
    ln = torch.randint(0, cap - 70, (units, 1), generator=g, device="cuda", dtype=torch.int32) // block * block
    ln[0] = cap - 70 - (cap - 70) % block + 5  # rows in the unfinished block
    c["len"].copy_(ln)
    acc = torch.rand(units, 1, cap, generator=g, device="cuda")
    c["acc"].copy_(acc)
    q, kn, vn = (torch.randn(units, h, d, generator=g, device="cuda").to(BF) for h in (G, 1, 1))
    o = kvc.h2o_decode_step_q8(q, kn, vn, c, 9 * cap)
    torch.cuda.synchronize()
    assert torch.equal(c["len"], ln + 1)
    rows = {}
    for n, new in (("K", kn), ("V", vn)):
        x = (c[n].double() * c[n + "s"].double().repeat_interleave(block, -1)[..., None])[:, 0]
        t = c[n + "t"][0, 0].double()
        f = int(ln[0]) // block * block
        x[0, f:f + block] = t
        x.scatter_(1, ln.long()[..., None].expand(units, 1, d), new.double())
        rows[n] = x
    seen = torch.arange(cap, device="cuda") <= ln
    logits = (q.double() @ rows["K"].transpose(1, 2) * d ** -0.5).masked_fill(~seen[:, None], float("-inf"))
    p = logits.softmax(-1)
    dl = C_TC * d ** -0.5 * (q.double().abs() @ rows["K"].abs().transpose(1, 2)).amax((1, 2), keepdim=True)
    rel = 2 * dl + 2.0 ** -18
    assert ((o.double() - p @ rows["V"]).abs() <= rel * (p @ rows["V"].abs()) + 1e-37).all()
    old = torch.where(torch.arange(cap, device="cuda") < ln, acc[:, 0], 0.0).double()
    mass = p.sum(1)
    want = torch.where(seen, old + mass, acc[:, 0].double())
    assert ((c["acc"][:, 0] - want).abs() <= rel[:, 0] * mass + 2.0 ** -23 * want).all()
