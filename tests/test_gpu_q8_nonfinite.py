"""NaN and infinities in rows that enter the 8-bit slot cache: a block that holds one stands for
NaN everywhere, and no other block, unit or row changes a bit."""
import pytest
import torch

from _q8 import CODES, clone, filled_cache, same_bits

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")
FORMATS = pytest.mark.parametrize("fmt", ["s8", "e4m3"])
DTYPES = pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])


def _values(c, name):
    """What the codes stand for: [B][H][blocks][block][d]."""
    B, H, cap, d = c[name].shape
    block = c[name + "t"].shape[2]
    return c[name].float().view(B, H, cap // block, block, d) * c[name + "s"][..., None, None]


def _expect(got, clean, name, bad):
    """Blocks where bad [B][H][blocks] are NaN through and through, the others have the clean run's bits."""
    B, H, cap, d = got[name].shape
    nb = cap // got[name + "t"].shape[2]
    assert got[name + "s"][bad].isnan().all() and _values(got, name)[bad].isnan().all()
    code, want = (c[name].view(torch.uint8).view(B, H, nb, -1) for c in (got, clean))
    assert torch.equal(code[~bad], want[~bad]) and same_bits(got[name + "s"][~bad], clean[name + "s"][~bad])


def _rows(*shape, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


@FORMATS
@DTYPES
@pytest.mark.parametrize("d,block", [(64, 32), (128, 64), (128, 128)])
def test_compact(kvc, dtype, fmt, d, block):
    """One element of a block, wherever it stands in it; the unfinished block's rows stay what they were."""
    H, nb = 2, 9
    T = nb * block + block // 2
    K, V = _rows(1, H, T, d, dtype=dtype, seed=1), _rows(1, H, T, d, dtype=dtype, seed=2)
    clean = kvc.kv_compact_q8(K, V, None, None, kvc.q8_cache(1, H, T + block // 2, d, block, dtype, CODES[fmt]))
    K2, V2 = K.clone(), V.clone()
    bad = {n: torch.zeros((1, H, nb + 1), dtype=torch.bool, device="cuda") for n in "KV"}
    at = [(0, 0), (block - 1, d - 1), (block // 2, 17), (3, d // 2), (block - 2, 1)]
    for i, x in enumerate((NAN, -NAN, INF, -INF, NAN)):
        r, e = at[i]
        K2[0, 0, 2 * i * block + r, e] = x
        bad["K"][0, 0, 2 * i] = 2 * i < nb
        if i < 4:
            V2[0, 1, (2 * i + 1) * block + r, e] = x
            bad["V"][0, 1, 2 * i + 1] = True
    K2[0, 1, nb * block + 1, 5] = NAN
    got = kvc.kv_compact_q8(K2, V2, None, None, kvc.q8_cache(1, H, T + block // 2, d, block, dtype, CODES[fmt]))
    torch.cuda.synchronize()
    for n in "KV":
        _expect(got, clean, n, bad[n])
    rows = T - nb * block
    assert same_bits(got["Kt"][:, :, :rows], K2[:, :, nb * block:]) and same_bits(got["Vt"], clean["Vt"])
    assert same_bits(got["pos"], clean["pos"]) and same_bits(got["len"], clean["len"])


def _step(B, Hkv, G, d, dtype, seed):
    return [_rows(B, h, d, dtype=dtype, seed=seed + i) for i, h in enumerate((Hkv * G, Hkv, Hkv))]


@FORMATS
@DTYPES
@pytest.mark.parametrize("cap", [256, 32768])
@pytest.mark.parametrize("where", ["row", "new"])
def test_decode_fills_a_block(kvc, dtype, fmt, cap, where):
    """A non-finite row waits in the unfinished block; when a step fills the block, that is NaN, and so
    are the steps after it.  Both decode paths; the row is an old one or the step's own."""
    H, G, d, block = 4, 2, 128, 64
    n = 2 * block - 1
    before = filled_cache(kvc, 1, H, cap, d, block, dtype, fmt, [n] * H, 3)
    q, kn, vn = _step(1, H, G, d, dtype, 5)
    clean = clone(before)
    o = kvc.h2o_decode_step_q8(q, kn, vn, clean, 9 * cap)
    c = clone(before)
    kn2, vn2 = kn.clone(), vn.clone()
    k, v = (c["Kt"][:, :, 30], c["Vt"][:, :, 30]) if where == "row" else (kn2, vn2)
    k[0, 0, 9], v[0, 1, 127], v[0, 2, 0] = NAN, -INF, NAN
    o2 = kvc.h2o_decode_step_q8(q, kn2, vn2, c, 9 * cap)
    q, kn, vn = _step(1, H, G, d, dtype, 8)
    o3, o4 = kvc.h2o_decode_step_q8(q, kn, vn, c, 9 * cap + 1), kvc.h2o_decode_step_q8(q, kn, vn, clean, 9 * cap + 1)
    torch.cuda.synchronize()
    bad = {x: torch.zeros((1, H, cap // block), dtype=torch.bool, device="cuda") for x in "KV"}
    bad["K"][0, 0, 1] = bad["V"][0, 1, 1] = bad["V"][0, 2, 1] = True
    for x in "KV":
        _expect(c, clean, x, bad[x])
    assert o2[0, :G].isnan().all() and not o2[0, G:2 * G].isfinite().all(-1).any()
    assert not o2[0, 2 * G:3 * G].isfinite().all(-1).any()
    assert o3[0, :3 * G].isnan().all()
    for a, b in ((o, o2), (o4, o3)):  # the other units
        assert same_bits(a[0, 3 * G:], b[0, 3 * G:])
    assert same_bits(c["acc"][0, 1:], clean["acc"][0, 1:])  # a NaN in V takes nothing from the weights


@FORMATS
@DTYPES
@pytest.mark.parametrize("d,block", [(64, 32), (128, 32), (64, 128), (128, 128)])
def test_evict_mixes_blocks(kvc, dtype, fmt, d, block):
    """Rows of a NaN block make the blocks NaN that they are mixed into, moved as a whole it keeps its codes,
    and in the unfinished block they are NaN rows; slots of finite blocks are moved as ever."""
    H, nb = 2, 8
    n = nb * block + 5
    src = filled_cache(kvc, 1, H, (nb + 1) * block, d, block, dtype, fmt, [n] * H, 11)
    acc = torch.full((nb + 1, block), 4.0, device="cuda")
    acc[0, ::2] = acc[3, 1::2] = 1.0                   # half of blocks 0 and 3 go, 1, 2, 4.. are mixed by that
    acc = acc.flatten()
    src["acc"][0].copy_(acc)
    keep = n - block
    recent = 5
    into = filled_cache(kvc, 1, H, (nb + 1) * block, d, block, dtype, fmt, [0] * H, 12)
    clean, got = clone(into), clone(into)
    idx = kvc.kv_evict_q8(src, keep, recent, clean)
    bad_src = clone(src)
    bad_src["Ks"][0, 0, 2] = NAN
    bad_src["Vs"][0, 0, 5] = -NAN
    bad_src["Vs"][0, 1, nb - 1] = NAN
    idx2 = kvc.kv_evict_q8(bad_src, keep, recent, got)
    torch.cuda.synchronize()
    assert same_bits(idx, idx2)
    whole = nb * block
    row = {"K": [(0, 2)], "V": [(0, 5), (1, nb - 1)]}
    nf = keep // block
    for x in "KV":
        nan_row = torch.zeros((1, H, keep), dtype=torch.bool, device="cuda")
        for h, b in row[x]:
            nan_row[0, h] = (idx[0, h] // block == b) & (idx[0, h] < whole)
        bad = torch.zeros((1, H, nb + 1), dtype=torch.bool, device="cuda")
        bad[:, :, :nf] = nan_row[:, :, :nf * block].view(1, H, nf, block).any(-1)
        assert bad.any()
        _expect(got, clean, x, bad)
        rest = nan_row[:, :, nf * block:]
        t, want = got[x + "t"][:, :, :keep - nf * block], clean[x + "t"][:, :, :keep - nf * block]
        assert t[rest].isnan().all() and same_bits(t[~rest], want[~rest])
    assert same_bits(got["acc"], clean["acc"]) and same_bits(got["pos"], clean["pos"])


@FORMATS
def test_evict_whole_block_and_unfinished_rows(kvc, fmt):
    """A NaN block that moves as it is, one whose rows end up in the unfinished block, and a NaN row of the old
    unfinished block that ends up in a full one."""
    H, block, d, cap = 3, 32, 64, 256
    n = 5 * block + 7
    src = filled_cache(kvc, 1, H, cap, d, block, F32, fmt, [n] * H, 21)
    src["acc"].fill_(4.0)
    src["acc"][0, :, 3 * block:3 * block + 9] = 1.0     # nine slots go: the old unfinished rows move forward
    src["Ks"][0, 0, 1] = NAN
    src["Vs"][0, 1, 4] = NAN
    src["Kt"][0, 2, 1, 3] = INF
    out = kvc.q8_cache(1, H, cap, d, block, F32, CODES[fmt])
    idx = kvc.kv_evict_q8(src, n - 9, 7, out)
    torch.cuda.synchronize()
    assert same_bits(out["K"][0, 0, block:2 * block], src["K"][0, 0, block:2 * block]) and out["Ks"][0, 0, 1].isnan()
    assert out["Ks"][0, 0, [0, 2, 3]].isfinite().all()
    nf = (n - 9) // block
    old = idx[0, 1, nf * block:]
    t = out["Vt"][0, 1, :len(old)]
    nan_row = (old >= 4 * block) & (old < 5 * block)
    assert nan_row.any() and not nan_row.all()
    assert t[nan_row].isnan().all() and t[~nan_row].isfinite().all()
    assert out["Vs"][0, 1, 3].isnan() and out["Vs"][0, 1, 4].isnan() == (nf > 4)
    at = int((idx[0, 2] == 5 * block + 1).nonzero())
    assert not out["Kt"][0, 2, at % block, 3].isfinite() if at >= nf * block else out["Ks"][0, 2, at // block].isnan()


@FORMATS
@pytest.mark.parametrize("cap,n", [(1024, 970), (32768, 30000)])
def test_decode_nan_behind_vanishing_weights(kvc, fmt, cap, n):
    """P_g(j) > 0 for every slot, however small: a NaN in V reaches the output where fp32 weights are 0 too.
    The slots of the first half have logits of -1016; both decode paths."""
    H, G, d, block = 2, 2, 64, 64
    c = kvc.q8_cache(1, H, cap, d, block, F32, CODES[fmt])
    c["K"][:, :, :n // 2 // block * block] = torch.tensor(-127.0 if fmt == "s8" else -128.0, device="cuda").to(CODES[fmt])
    c["Ks"].fill_(1.0)
    c["Vs"].fill_(1.0)
    c["Vs"][0, 0, 0] = NAN
    c["len"].fill_(n)
    q = torch.ones(1, H * G, d, device="cuda")
    new = torch.zeros(1, H, d, device="cuda")
    o = kvc.h2o_decode_step_q8(q, new, new, c, 2 * cap)
    torch.cuda.synchronize()
    assert o[0, :G].isnan().all() and (o[0, G:] == 0).all() and c["acc"].isfinite().all()
