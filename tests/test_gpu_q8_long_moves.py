"""Eviction of long units: every moved code, scale and unfinished row against the formula, whose float32
operations the GPU's elementwise ones are too (each rounded to nearest)."""
import pytest
import torch

from _q8 import CODES, clone, same_bits

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _source(kvc, B, H, cap, d, block, dtype, fmt, lens, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = kvc.q8_cache(B, H, cap, d, block, dtype, CODES[fmt])
    for n in ("K", "V"):
        for b in range(B):
            x = (torch.randn(H, cap, d, generator=g, device="cuda") * 0.3).clamp_(-1, 1)
            c[n][b] = (x * 127).round_().to(torch.int8) if fmt == "s8" else (x * 448).to(CODES[fmt])
        c[n + "s"].copy_(torch.rand(c[n + "s"].shape, generator=g, device="cuda") * 0.02 + 0.005)
        c[n + "t"].copy_(torch.randn(c[n + "t"].shape, generator=g, device="cuda").to(dtype))
    c["pos"].copy_(torch.arange(cap, device="cuda").expand(B, H, cap))
    c["acc"].copy_(torch.rand(B, H, cap, generator=g, device="cuda"))
    # the first 60 blocks: one that stays whole, two of which half the slots go, and so on, so that whole blocks
    # move between mixed ones; the rest at random
    front = torch.full((20, 3, block), 2.0, device="cuda")
    front[:, 1, ::2] = front[:, 2, 1::2] = -2.0
    c["acc"][:, :, :60 * block] += front.flatten()
    c["len"].copy_(torch.tensor(lens, dtype=torch.int32).view(B, H))
    return c


def _check_unit(src, before, out, b, h, idx, fmt):
    block, n = src["Kt"].shape[2], int(src["len"][b, h])
    full, m = n // block * block, int(out["len"][b, h])
    at = idx[:m].long()
    nf = m // block
    rows = at[:nf * block].view(nf, block)
    whole = (rows[:, 0] % block == 0) & (rows[:, -1] - rows[:, 0] == block - 1) & (rows[:, -1] < full)
    assert whole.any() and not whole.all()
    top = 127.0 if fmt == "s8" else 448.0
    for name in ("K", "V"):
        code, scale, tail = src[name][b, h], src[name + "s"][b, h], src[name + "t"][b, h]
        old = at < full
        x = code[at.clamp_max(full - 1)].float() * scale[at.clamp_max(full - 1) // block][:, None]
        x = torch.where(old[:, None], x, tail[(at - full).clamp(0, block - 1)].float())
        y = x[:nf * block].view(nf, block, -1)
        big = y.abs().amax((1, 2))
        a = torch.maximum(big / torch.full_like(big, top), torch.full_like(big, 2.0 ** -126))
        y = y * (torch.ones_like(a) / a)[:, None, None]
        want = y.round().to(torch.int8) if fmt == "s8" else y.to(CODES[fmt])
        moved = code.view(torch.uint8).view(-1, block, code.shape[-1])[rows[:, 0] // block]
        want = torch.where(whole[:, None, None], moved, want.view(torch.uint8))
        a = torch.where(whole, scale[rows[:, 0] // block], a)
        got = out[name].view(torch.uint8)[b, h]
        assert torch.equal(got[:nf * block].view(want.shape), want), (name, b, h)
        assert same_bits(out[name + "s"][b, h, :nf], a)
        left = before[name + "t"][b, h].clone()
        left[:m - nf * block] = x[nf * block:].to(left.dtype)
        assert same_bits(out[name + "t"][b, h], left)
        assert torch.equal(got[nf * block:], before[name].view(torch.uint8)[b, h, nf * block:])
        assert same_bits(out[name + "s"][b, h, nf:], before[name + "s"][b, h, nf:])


CASES = [
    # B, H, cap, d, block, dtype, keep, shortened by
    (2, 8, 40960, 128, 64, BF, 20011, 0),       # runs of several blocks
    (2, 16, 32768, 128, 128, F32, 17000, 5),
    (1, 32, 16384, 64, 128, BF, 9000, 100),
    (1, 16, 32768, 128, 32, F32, 30001, 3),
    (1, 24, 16384, 64, 32, BF, 8191, 1),
    (1, 1, 300032, 128, 64, BF, 150001, 7),     # one unit over all SMs
    (1, 2, 400000, 128, 128, F32, 200003, 77),  # longer than the cluster selection takes
    (1, 2, 400000, 64, 64, BF, 399000, 63),
]


@pytest.mark.parametrize("fmt", ["s8", "e4m3"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_moved_values(kvc, case, fmt):
    B, H, cap, d, block, dtype, keep, less = case
    lens = [cap - less * u for u in range(1, B * H + 1)]
    src = _source(kvc, B, H, cap, d, block, dtype, fmt, lens, 1)
    room = (keep + block - 1) // block * block
    out = _source(kvc, B, H, room, d, block, dtype, fmt, [0] * (B * H), 2)
    before = clone(out)
    idx = kvc.kv_evict_q8(src, keep, 100, out, sink=4)
    torch.cuda.synchronize()
    for b in range(B):
        for h in range(H):
            n = lens[b * H + h]
            a = src["acc"][b, h, :n].clone()
            a[:4] = a[n - 100:] = float("inf")
            stay = a.sort(stable=True).indices[n - keep:].sort().values  # equal ones: the first go
            assert torch.equal(idx[b, h].long(), stay) and out["len"][b, h] == keep
            assert same_bits(out["acc"][b, h, :keep], src["acc"][b, h][stay])
            assert torch.equal(out["pos"][b, h, :keep].long(), stay)
            _check_unit(src, before, out, b, h, idx[b, h], fmt)
