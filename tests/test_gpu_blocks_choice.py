"""Which blocks block-sparse attention chooses where float32 bounds do not tell."""
import math

import numpy as np
import pytest
import torch

from _long import BF, F32, rand

pytestmark = pytest.mark.gpu

TYPES = pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])


def _blocks(B, H, nb, block, d, dtype):
    """A cache whose keys are the same within a block, and its view by blocks."""
    K = torch.zeros(B, H, nb * block, d, dtype=dtype, device="cuda")
    return K, K.view(B, H, nb, block, d)


def _chosen(q, dig, seen, block, n_sel, sink, recent):
    """As choose, each block's sum in the same order, so that equal blocks have equal bounds here too."""
    nb = -(-seen // block)
    if nb <= n_sel:
        return list(range(nb))
    q, dig = q.cpu().numpy(), dig[:nb].cpu().numpy()
    with np.errstate(all="ignore"):
        u = np.stack([(np.maximum(x, 0) * dig[:, 1] + np.minimum(x, 0) * dig[:, 0]).sum(-1) for x in q])
    u = np.where(np.isnan(u), np.inf, u).max(0)
    mid = np.arange(sink, nb - recent)
    best = mid[np.lexsort((mid, -u[mid]))][:n_sel - sink - recent]
    return sorted([*range(sink), *best.tolist(), *range(nb - recent, nb)])


def _run(kvc, q, K, ln, block, n_sel, sink=1, recent=1, dig=None):
    V = rand(K.shape, K.dtype, 99)
    if dig is None:
        dig = kvc.kv_block_digest(K, block)
    o, lse, sel = kvc.kv_attn_blocks(q, K, V, ln.cuda(), dig, block, n_sel, sink=sink, recent=recent)
    B, Hkv = K.shape[:2]
    G = q.shape[1] // Hkv
    for b in range(B):
        for h in range(Hkv):
            want = _chosen(q[b, h * G:(h + 1) * G, 0].double(), dig[b, h].double(), int(ln[b, h]), block, n_sel, sink, recent)
            got = sel[b, h, 0].tolist()
            assert got == want + [-1] * (n_sel - len(want)), f"b {b} h {h}: {[j for j in got if j not in want]} for {[j for j in want if j not in got]}"
    return o, lse, sel


def _full(B, H, n):
    return torch.full((B, H), n, dtype=torch.int32)


@TYPES
@pytest.mark.parametrize("qs,ks", [(1e-30, 1e-20), (1e-25, 1e-10), (1e-10, 1e-36)])
def test_bounds_that_underflow(kvc, dtype, qs, ks):
    d, block, nb = 64, 16, 200
    K = (rand((1, 2, nb * block, d), F32, 1) * ks).to(dtype)
    q = (rand((1, 8, 1, d), F32, 2) * qs).to(dtype)
    assert bool((q != 0).any()) and bool((K != 0).any())
    _run(kvc, q, K, _full(1, 2, nb * block - 3), block, 21)
    # and those of one unit alone
    K[0, 0] = rand((nb * block, d), dtype, 3)
    q[0, :4] = rand((4, 1, d), dtype, 4)
    _run(kvc, q, K, _full(1, 2, nb * block), block, 21)


@TYPES
def test_last_places_of_64_bits(kvc, dtype):
    """u = 1 + 2^-25 + i 2^-51, i < 4, exact in 64 bits."""
    d, block, nb = 64, 16, 300
    K, by_block = _blocks(1, 1, nb, block, d, dtype)
    g = torch.Generator().manual_seed(5)
    i = torch.randint(0, 4, (nb,), generator=g).float().cuda()
    by_block[..., 0], by_block[..., 1], by_block[..., 2] = 1.0, 2.0 ** -13, (i * 2.0 ** -26).to(dtype)[:, None]
    q = torch.zeros(1, 2, 1, d, dtype=dtype, device="cuda")
    q[..., 0], q[..., 1], q[..., 2] = 1.0, 2.0 ** -12, 2.0 ** -25
    assert 40 < int((i == 3).sum()) < 110
    for n_sel in (20, 60, 120, 290):
        _run(kvc, q, K, _full(1, 1, nb * block), block, n_sel)


@TYPES
def test_same_terms_in_other_orders(kvc, dtype):
    """Blocks whose bounds are sums of the same terms in other channels are equal: the lower ones are chosen."""
    d, block, nb = 64, 16, 120
    K, by_block = _blocks(1, 1, nb, block, d, dtype)
    terms = torch.tensor([2.0 ** -x for x in (0, 3, 13, 19, 25, 31, 38, 44)] + [0.0] * (d - 8), device="cuda")
    for j in range(nb):
        by_block[0, 0, j] = terms[torch.randperm(d, generator=torch.Generator().manual_seed(j))].to(dtype)
    q = torch.ones(1, 4, 1, d, dtype=dtype, device="cuda")
    sel = _run(kvc, q, K, _full(1, 1, nb * block), block, 30)[2]
    assert sel[0, 0, 0].tolist() == list(range(29)) + [nb - 1]


@TYPES
@pytest.mark.parametrize("nb", [700, 9000])
def test_many_equal_bounds(kvc, dtype, nb):
    d, block = 64, 16
    K, by_block = _blocks(2, 2, nb, block, d, dtype)
    by_block[0, 0] = rand((d,), dtype, 10)                       # one kind
    few = rand((5, d), F32, 11)
    by_block[0, 1] = few[torch.arange(nb, device="cuda") * 7 % 5].to(dtype)[:, None]   # five kinds in turn
    K[1, 0] = 0                                                  # nothing
    by_block[1, 1] = rand((d,), dtype, 12)
    by_block[1, 1, 3::11, :, 5] += 2.0                           # one kind and some above
    q = rand((2, 8, 1, d), dtype, 13)
    for n_sel in (3, 40, 300, nb - 5):
        _run(kvc, q, K, torch.tensor([[nb * block, nb * block - 17], [nb * block - 1, nb * block]], dtype=torch.int32), block, n_sel)


@TYPES
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_bad_keys_in_many_blocks(kvc, dtype, bad):
    """Blocks whose bound is no number are the first chosen, by number, and the others are told apart as ever."""
    d, block, nb = 64, 16, 3000
    K = rand((1, 3, nb * block, d), dtype, 20)
    K[0, 0, 777 * block + 3, 9] = bad
    K[0, 1, 5 * block::37 * block, 1] = bad
    K[0, 2, ::block, 2] = bad
    q = rand((1, 12, 1, d), dtype, 21)
    q[..., 9], q[..., 1] = q[..., 9].abs() + 0.1, -q[..., 1].abs() - 0.1
    for n_sel in (5, 40, 100, 2000):
        _run(kvc, q, K, _full(1, 3, nb * block), block, n_sel)


@TYPES
def test_bad_queries(kvc, dtype):
    d, block, nb = 64, 16, 500
    K, q = rand((1, 2, nb * block, d), dtype, 30), rand((1, 8, 1, d), dtype, 31)
    q[0, 2, 0, 5], q[0, 5, 0, 6] = math.nan, math.inf
    _run(kvc, q, K, _full(1, 2, nb * block), block, 30)


@TYPES
def test_no_terms_at_all(kvc, dtype):
    """Keys of 0, among them some that are no numbers."""
    d, block, nb = 64, 16, 900
    K = torch.zeros(1, 2, nb * block, d, dtype=dtype, device="cuda")
    K[0, 1, 50 * block::30 * block, 3] = math.nan
    q = rand((1, 8, 1, d), dtype, 35)
    for n_sel in (10, 60):
        _run(kvc, q, K, _full(1, 2, nb * block), block, n_sel)


@TYPES
def test_time_of_equal_bounds(kvc, dtype):
    """Equal bounds, and a key that is no number, cost some times an ordinary call, not hundreds of times: near
    bounds are shared out and ranked in linear time."""
    d, block, nb, H = 128, 16, 12000, 8
    q = rand((1, 4 * H, 1, d), dtype, 50)
    K = rand((1, H, nb * block, d), dtype, 51)
    ln = _full(1, H, nb * block).cuda()

    def us(K):
        dig = kvc.kv_block_digest(K, block)
        call = lambda: kvc.kv_attn_blocks(q, K, K, ln, dig, block, 64, sink=1, recent=1)  # noqa: E731
        call()
        best = math.inf
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(4):
                call()
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b) * 250)
        return best

    plain = us(K)
    K[0, 3, 12345, 7] = math.nan
    one_nan = us(K)
    K[0, 3, 12345, 7] = math.inf
    one_inf = us(K)
    K[:] = rand((1, H, 1, d), dtype, 52)
    equal = us(K)
    print(f"ordinary {plain:.1f} us, one NaN {one_nan:.1f}, one infinity {one_inf:.1f}, equal keys {equal:.1f}")
    assert one_nan < 4 * plain and one_inf < 4 * plain and equal < 20 * plain


@TYPES
def test_nan_in_one_query(kvc, dtype):
    """Every bound of its group is +inf: the lowest blocks are chosen, as quickly as ever, and the other rows are untouched."""
    d, block, nb, H = 128, 16, 12000, 8
    q, K = rand((1, 4 * H, 1, d), dtype, 60), rand((1, H, nb * block, d), dtype, 61)
    ln = _full(1, H, nb * block).cuda()
    dig = kvc.kv_block_digest(K, block)
    call = lambda: kvc.kv_attn_blocks(q, K, K, ln, dig, block, 64, sink=1, recent=1)  # noqa: E731

    def us():
        call()
        best = math.inf
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(4):
                call()
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b) * 250)
        return best

    want, plain = call(), us()
    q[0, 9, 0, 100] = math.nan
    got, bad = call(), us()
    assert got[2][0, 2, 0].tolist() == list(range(63)) + [nb - 1]
    assert got[0][0, 9].isnan().all() and got[1][0, 9].isnan().all()
    others = [h for h in range(4 * H) if h // 4 != 2]
    assert all(torch.equal(x[0, others], y[0, others]) for x, y in zip(got[:2], want[:2]))
    assert torch.equal(got[2][0, [0, 1, 3, 4, 5, 6, 7]], want[2][0, [0, 1, 3, 4, 5, 6, 7]]) and got[0][0, 8].isfinite().all()
    print(f"ordinary {plain:.1f} us, NaN in a query {bad:.1f}")
    assert bad < 4.5 * plain
