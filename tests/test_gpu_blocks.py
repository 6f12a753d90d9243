"""Block digests and block-sparse attention on the GPU against float64."""
import pytest
import torch

from _long import BF, F32, check_rows, choose, digests, rand

pytestmark = pytest.mark.gpu


def _lens(B, H, least, most, seed):
    g = torch.Generator().manual_seed(seed)
    ln = torch.randint(least, most + 1, (B, H), generator=g, dtype=torch.int32)
    ln.view(-1)[-1] = most
    return ln


def _keys(B, H, cap, d, dtype, seed):
    """Blocks that differ: a centre for every 48 slots, large channels, noise."""
    x = rand((B, H, cap, d), F32, seed)
    x += rand((B, H, (cap + 47) // 48, d), F32, seed + 1).repeat_interleave(48, 2)[:, :, :cap]
    x[..., ::17] += 5
    return x.to(dtype)


def _check(q, K, V, ln, dig, block, n_sel, sink, recent, o, lse, sel, scale, units=None):
    B, Hq, nq, d = q.shape
    Hkv = K.shape[1]
    G = Hq // Hkv
    for b in range(B):
        for h in range(Hkv):
            if units is not None and (b, h) not in units:
                continue
            n = int(ln[b, h])
            for t in range(nq):
                seen = max(0, n - nq + t + 1)
                what = f"b {b} h {h} t {t} seen {seen}"
                rows = q[b, h * G:(h + 1) * G, t]
                want = choose(rows.double(), dig[b, h].double(), seen, block, n_sel, sink, recent) if seen else []
                got = sel[b, h, t].tolist()
                assert got == want + [-1] * (n_sel - len(want)), f"{what}: {got} {want}"
                at = torch.cat([torch.arange(j * block, min(seen, (j + 1) * block)) for j in want]).cuda() if want else \
                    torch.zeros(0, dtype=torch.long, device="cuda")
                check_rows(o[b, h * G:(h + 1) * G, t], lse[b, h * G:(h + 1) * G, t], rows, K[b, h, at], V[b, h, at], scale,
                           2.0 ** -16 if q.dtype == BF else 2.0 ** -20, what)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("block,cap", [(16, 100), (32, 700), (64, 1500), (128, 129), (64, 64), (16, 1)])
def test_digests(kvc, dtype, d, block, cap):
    B, H = 2, 3
    K = rand((B, H, cap, d), dtype, 1)
    nb = -(-cap // block)
    for n_new in (None, 1, 5, block, block + 1, cap):
        ln = _lens(B, H, 0, cap, cap + (n_new or 0))
        old = rand((B, H, nb, 2, d), dtype, 2)
        K2 = K.clone()
        for b in range(B):
            for h in range(H):
                K2[b, h, int(ln[b, h]):] = float("nan")  # behind the last slot: not looked at
        got = kvc.kv_block_digest(K2, block, ln.cuda(), n_new=n_new, out=old.clone())
        assert torch.equal(got, digests(K2, ln.tolist(), block, old, n_new)), (n_new, ln)
    full = kvc.kv_block_digest(K, block)
    assert torch.equal(full, digests(K, [[cap] * H] * B, block, old))


def test_digest_keeps_nan_and_refuses_lengths(kvc):
    K = rand((1, 2, 256, 64), BF, 3)
    K[0, 0, 70, 5] = float("nan")
    dig = kvc.kv_block_digest(K, 64)
    assert dig[0, 0, 1, :, 5].isnan().all() and int(dig.isnan().sum()) == 2
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    old = dig.clone()
    kvc.kv_block_digest(K, 64, torch.tensor([[257, -1]], dtype=torch.int32, device="cuda"), out=dig, dev_status=st)
    assert int(st) == -1 and torch.equal(dig.nan_to_num(7.0), old.nan_to_num(7.0))


def test_many_digests_at_once(kvc):
    """More blocks than run at once, several per warp."""
    K = rand((3, 8, 9000, 128), BF, 4)
    dig = kvc.kv_block_digest(K, 16)
    x = torch.cat((K, K[:, :, -1:].expand(-1, -1, 8, -1)), 2).view(3, 8, 563, 16, 128)
    assert torch.equal(dig[..., 0, :], x.amin(3)) and torch.equal(dig[..., 1, :], x.amax(3))


CASES = [
    # B, Hq, Hkv, nq, cap, d, block, n_sel, sink, recent, least, most, dtype
    (1, 4, 4, 1, 512, 64, 32, 6, 1, 2, 512, 512, F32),
    (1, 32, 8, 1, 2048, 128, 32, 16, 1, 2, 2001, 2047, BF),
    (1, 1, 1, 1, 1, 128, 16, 1, 0, 1, 1, 1, BF),
    (1, 2, 1, 1, 4000, 128, 16, 20, 2, 1, 3999, 4000, BF),      # one unit: a cluster of 16
    (2, 3, 1, 1, 3001, 64, 64, 7, 0, 1, 2000, 3001, BF),        # cap no multiple of block
    (3, 8, 1, 1, 1000, 128, 128, 4, 1, 1, 0, 1000, BF),         # eight queries a head, empty units
    (2, 10, 2, 1, 900, 128, 64, 3, 1, 2, 0, 900, BF),           # no place left for bounds
    (2, 12, 2, 1, 900, 64, 64, 99, 1, 2, 0, 900, F32),          # every block
    (1, 7, 1, 5, 2000, 128, 32, 9, 1, 1, 3, 2000, BF),          # tokens that see nothing
    (2, 8, 2, 3, 300, 64, 16, 8, 0, 2, 290, 300, F32),
    (2, 4, 4, 7, 1111, 128, 64, 5, 2, 2, 900, 1111, BF),
    (40, 16, 16, 1, 400, 128, 32, 5, 1, 1, 0, 400, BF),         # one CTA a unit
    (9, 16, 8, 1, 1200, 64, 32, 8, 1, 1, 1000, 1200, BF),       # clusters of 8
    (5, 32, 16, 2, 700, 128, 32, 6, 1, 1, 600, 700, F32),
    (1, 8, 2, 20, 800, 128, 32, 6, 1, 1, 15, 799, BF),          # more new tokens than a block
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_attention(kvc, case):
    B, Hq, Hkv, nq, cap, d, block, n_sel, sink, recent, least, most, dtype = case
    K, V = _keys(B, Hkv, cap, d, dtype, 10), rand((B, Hkv, cap, d), dtype, 12)
    ln = _lens(B, Hkv, least, most, 13)
    q = rand((B, Hq, nq, d), dtype, 14)
    dig = kvc.kv_block_digest(K, block, ln.cuda(), out=torch.zeros(B, Hkv, -(-cap // block), 2, d, dtype=dtype, device="cuda"))
    for b in range(B):
        for h in range(Hkv):  # what stands behind the last slot does not matter
            K[b, h, int(ln[b, h]):] = float("nan")
            V[b, h, int(ln[b, h]):] = float("nan")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse, sel = kvc.kv_attn_blocks(q, K, V, ln.cuda(), dig, block, n_sel, sink=sink, recent=recent, dev_status=st)
    assert int(st) == 0
    _check(q, K, V, ln, dig, block, n_sel, sink, recent, o, lse, sel, d ** -0.5)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_equal_and_near_bounds(kvc, dtype):
    """Equal bounds go to the lower block; bounds that differ by less than fp32 sums resolve are told apart."""
    d, block, nb = 128, 16, 300
    K = rand((1, 1, 1, 1, d), F32, 20).expand(1, 1, nb, block, d).reshape(1, 1, nb * block, d).to(dtype).clone()
    q = rand((1, 4, 1, d), dtype, 21)
    V = rand(K.shape, dtype, 22)
    ln = torch.full((1, 1), nb * block, dtype=torch.int32)
    run = lambda: kvc.kv_attn_blocks(q, K, V, ln.cuda(), dig, block, 20, sink=1, recent=1)  # noqa: E731
    dig = kvc.kv_block_digest(K, block)
    o, lse, sel = run()
    assert sel[0, 0, 0].tolist() == list(range(19)) + [nb - 1]
    _check(q, K, V, ln, dig, block, 20, 1, 1, o, lse, sel, d ** -0.5)
    # one large channel hides tiny differences in another from sums of fp32
    q[..., 0], K[..., 0] = 1000.0, 1000.0
    q[..., 1] = 2.0 ** -6
    g = torch.Generator().manual_seed(23)
    K.view(1, 1, nb, block, d)[..., 1] = (torch.randperm(nb, generator=g).float().cuda() / 256).to(dtype)[None, None, :, None]
    dig = kvc.kv_block_digest(K, block)
    o, lse, sel = run()
    _check(q, K, V, ln, dig, block, 20, 1, 1, o, lse, sel, d ** -0.5)
    # no query at all: every bound is 0
    q.zero_()
    assert run()[2][0, 0, 0].tolist() == list(range(19)) + [nb - 1]


def test_nan_and_overflow_in_digests(kvc):
    """A block with a NaN is chosen (and makes its rows NaN); bounds past fp32 are told apart in 64 bits."""
    K, V, q = rand((1, 1, 3200, 64), F32, 30), rand((1, 1, 3200, 64), F32, 31), rand((1, 2, 1, 64), F32, 32)
    ln = torch.full((1, 1), 3200, dtype=torch.int32, device="cuda")
    K[0, 0, 20 * 32 + 3, 7] = float("nan")
    dig = kvc.kv_block_digest(K, 32)
    o, lse, sel = kvc.kv_attn_blocks(q, K, V, ln, dig, 32, 5)
    assert sel[0, 0, 0].tolist() == choose(q[0, :, 0].double(), dig[0, 0].double(), 3200, 32, 5, 0, 1) and 20 in sel[0, 0, 0].tolist()
    assert o.isnan().all() and lse.isnan().all()
    q, K = q.abs() * 1e20, rand((1, 1, 3200, 64), F32, 33).abs() * 1e19
    dig = kvc.kv_block_digest(K, 32)
    sel = kvc.kv_attn_blocks(q, K, V, ln, dig, 32, 5)[2]
    assert sel[0, 0, 0].tolist() == choose(q[0, :, 0].double(), dig[0, 0].double(), 3200, 32, 5, 0, 1)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_many_blocks(kvc, dtype):
    """Thousands of blocks, many of which have the same or nearly the same bounds: bins that overflow, whole
    ranges of equal bounds."""
    d, block, nb = 64, 16, 9000
    g = torch.Generator(device="cuda").manual_seed(24)
    K = torch.zeros(1, 2, nb * block, d, dtype=dtype, device="cuda")
    # head 0: 40 different blocks, each many times; head 1: differences in the last places around a large value
    kinds = rand((40, d), F32, 25)
    K.view(1, 2, nb, block, d)[0, 0] = kinds[torch.randint(0, 40, (nb,), generator=g, device="cuda")].to(dtype)[:, None]
    K[0, 1, :, 0] = 64.0
    K.view(1, 2, nb, block, d)[0, 1, :, :, 1] = (torch.randint(0, 256, (nb,), generator=g, device="cuda").float() / 256).to(dtype)[:, None]
    V, q = rand(K.shape, dtype, 26), rand((1, 4, 1, d), dtype, 27)
    q[..., 0], q[..., 1] = 100.0, 0.01
    ln = torch.full((1, 2), nb * block - 5, dtype=torch.int32)
    dig = kvc.kv_block_digest(K, block, ln.cuda())
    for n_sel in (8, 700, 5000):
        o, lse, sel = kvc.kv_attn_blocks(q, K, V, ln.cuda(), dig, block, n_sel, sink=2, recent=3)
        _check(q, K, V, ln, dig, block, n_sel, 2, 3, o, lse, sel, d ** -0.5)


def test_as_many_blocks_as_there_may_be(kvc):
    nb = 12288
    K, V, q = _keys(1, 2, nb * 16, 128, BF, 80), rand((1, 2, nb * 16, 128), BF, 81), rand((1, 16, 1, 128), BF, 82)
    ln = torch.tensor([[nb * 16, nb * 16 - 40]], dtype=torch.int32)
    dig = kvc.kv_block_digest(K, 16, ln.cuda(), out=torch.zeros(1, 2, nb, 2, 128, dtype=BF, device="cuda"))
    o, lse, sel = kvc.kv_attn_blocks(q, K, V, ln.cuda(), dig, 16, 50, sink=1, recent=2)
    _check(q, K, V, ln, dig, 16, 50, 1, 2, o, lse, sel, 128 ** -0.5)
    K = K.float()
    dig = kvc.kv_block_digest(K, 16, ln.cuda(), out=torch.zeros(1, 2, nb, 2, 128, device="cuda"))
    o, lse, sel = kvc.kv_attn_blocks(q.float(), K, V.float(), ln.cuda(), dig, 16, 50, sink=1, recent=2)
    _check(q.float(), K, V.float(), ln, dig, 16, 50, 1, 2, o, lse, sel, 128 ** -0.5)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_hidden_slots_hold_anything(kvc, dtype):
    """A later new token's value does not reach an earlier one, whatever it is."""
    K, V, q = rand((1, 2, 500, 64), dtype, 90), rand((1, 2, 500, 64), dtype, 91), rand((1, 8, 3, 64), dtype, 92)
    ln = torch.tensor([[490, 481]], dtype=torch.int32)
    dig = kvc.kv_block_digest(K, 16, ln.cuda())
    want = kvc.kv_attn_blocks(q, K, V, ln.cuda(), dig, 16, 6)
    for h in range(2):
        V[0, h, int(ln[0, h]) - 1] = float("inf")
    o, lse, sel = kvc.kv_attn_blocks(q, K, V, ln.cuda(), dig, 16, 6)
    assert torch.equal(o[:, :, :2], want[0][:, :, :2]) and torch.equal(lse, want[1]) and torch.equal(sel, want[2])
    assert not o[:, :, 2].isfinite().any()


def test_output_over_the_queries(kvc):
    K, V, q = rand((2, 2, 900, 128), BF, 93), rand((2, 2, 900, 128), BF, 94), rand((2, 8, 2, 128), BF, 95)
    ln = torch.full((2, 2), 900, dtype=torch.int32, device="cuda")
    dig = kvc.kv_block_digest(K, 32)
    want = kvc.kv_attn_blocks(q, K, V, ln, dig, 32, 6)
    q2 = q.clone()
    kvc.kv_attn_blocks(q2, K, V, ln, dig, 32, 6, out=q2)
    assert torch.equal(q2, want[0])
    want = kvc.kv_attn_shared(q, K[0], V[0], K, V, ln)[0]
    kvc.kv_attn_shared(q, K[0], V[0], K, V, ln, out=q)
    assert torch.equal(q, want)


def test_first_call_of_its_sizes_in_a_capture(kvc):
    """What is asked of the device once (which clusters fit) may be asked while a graph is being captured."""
    K, V, q = rand((1, 3, 1777, 64), BF, 96), rand((1, 3, 1777, 64), BF, 97), rand((1, 6, 1, 64), BF, 98)
    ln = torch.full((1, 3), 1700, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dig = kvc.kv_block_digest(K, 16, ln)
        got = kvc.kv_attn_blocks(q, K, V, ln, dig, 16, 11, sink=1, recent=2)
    g.replay()
    _check(q, K, V, ln.cpu(), dig, 16, 11, 1, 2, *got, 64 ** -0.5)


def test_layouts_scale_and_given_outputs(kvc):
    B, Hq, Hkv, nq, cap, d = 2, 8, 2, 3, 500, 128
    K, V = _keys(B, Hkv, cap, d, BF, 40), rand((B, Hkv, cap, d), BF, 41)
    ln = _lens(B, Hkv, 400, 500, 42)
    fused = rand((B, nq, Hq + 5, d), BF, 43)
    q = fused[:, :, 2:2 + Hq].transpose(1, 2)
    out = torch.zeros(B, nq, Hq, d, dtype=BF, device="cuda").transpose(1, 2)
    lse = torch.zeros(B, Hq, nq, device="cuda")
    sel = torch.zeros(B, Hkv, nq, 6, dtype=torch.int32, device="cuda")
    dig = kvc.kv_block_digest(K, 32, ln.cuda())
    got = kvc.kv_attn_blocks(q, K, V, ln.cuda(), dig, 32, 6, sink=1, recent=2, scale=0.2, out=out, lse_out=lse, sel_out=sel)
    assert got[0] is out and got[1] is lse and got[2] is sel
    _check(q, K, V, ln, dig, 32, 6, 1, 2, out, lse, sel, 0.2)


def test_bad_lengths_leave_their_units(kvc):
    K, V = rand((2, 2, 200, 64), BF, 50), rand((2, 2, 200, 64), BF, 51)
    q = rand((2, 4, 1, 64), BF, 52)
    ln = torch.tensor([[200, 201], [-3, 100]], dtype=torch.int32, device="cuda")
    dig = kvc.kv_block_digest(K, 16)
    out, st = torch.full_like(q, 9.0), torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse, sel = kvc.kv_attn_blocks(q, K, V, ln, dig, 16, 4, out=out, dev_status=st)
    assert int(st) == -1
    assert (o[0, 2:] == 9).all() and (o[1, :2] == 9).all()
    _check(q, K, V, ln.cpu(), dig, 16, 4, 0, 1, o, lse, sel, 64 ** -0.5, units=[(0, 0), (1, 1)])


def test_offsets_past_32_bits(kvc):
    """A cache of more than 2^31 elements: its last unit."""
    H, cap, d = 18, 1000000, 128
    K = torch.empty(1, H, cap, d, dtype=BF, device="cuda")
    V = torch.empty(1, H, cap, d, dtype=BF, device="cuda")
    K[:, -1:], V[:, -1:] = _keys(1, 1, cap, d, BF, 60), rand((1, 1, cap, d), BF, 61)
    ln = torch.zeros(1, H, dtype=torch.int32, device="cuda")
    ln[0, -1] = cap - 3
    q = rand((1, H, 1, d), BF, 62)
    dig = kvc.kv_block_digest(K, 128, ln, out=torch.zeros(1, H, 7813, 2, d, dtype=BF, device="cuda"))
    assert torch.equal(dig[0, -1, :7812, 1], K[0, -1, :7812 * 128].view(7812, 128, d).amax(1))
    o, lse, sel = kvc.kv_attn_blocks(q, K, V, ln, dig, 128, 9, sink=1, recent=2)
    assert (o[0, :-1] == 0).all() and (lse[0, :-1] == -float("inf")).all() and (sel[0, :-1] == -1).all()
    _check(q, K, V, ln.cpu(), dig, 128, 9, 1, 2, o, lse, sel, d ** -0.5, units=[(0, H - 1)])


def test_captured_and_on_another_stream(kvc):
    B, Hq, Hkv, cap, d = 2, 8, 2, 1000, 64
    K, V = _keys(B, Hkv, cap, d, BF, 70), rand((B, Hkv, cap, d), BF, 71)
    ln = torch.full((B, Hkv), 777, dtype=torch.int32, device="cuda")
    q = rand((B, Hq, 1, d), BF, 72)
    dig = torch.zeros(B, Hkv, 32, 2, d, dtype=BF, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kvc.kv_block_digest(K, 32, ln, out=dig)
        want = kvc.kv_attn_blocks(q, K, V, ln, dig, 32, 7)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvc.kv_block_digest(K, 32, ln, n_new=1, out=dig)
        got = kvc.kv_attn_blocks(q, K, V, ln, dig, 32, 7)
    g.replay()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    # new tokens in the replayed buffers
    ln += 1
    K[:, :, 777], q[:] = rand((B, Hkv, d), BF, 73), rand((B, Hq, 1, d), BF, 74)
    g.replay()
    _check(q, K, V, ln.cpu(), digests(K, ln.tolist(), 32, dig), 32, 7, 0, 1, *got, d ** -0.5)
