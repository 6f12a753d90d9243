"""Prompt attention on the GPU against float64."""
import numpy as np
import pytest
import torch

from _q8 import C_CUDA, C_TC, np64, same_bits, within

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def q8():
    from oracle import q8
    return q8


def _rand(shape, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _check(q8, o, lse, q, k, v, scale, what, rows=None):
    """One sequence and query head."""
    bf = q.dtype == BF
    Q, K, V = np64(q), np64(k), np64(v)
    nq, nk = len(Q), len(K)
    pick = np.arange(nq) if rows is None else rows
    for i in pick if rows is not None else [None]:
        if i is None:
            want, wl, mass = q8.attn_prompt(Q, K, V, scale)
            qq, oo, ll = Q, np64(o), np64(lse)
        else:  # one row alone: it sees the keys up to i + nk - nq
            n = min(nk, i + nk - nq + 1)
            want, wl, mass = q8.attn_prompt(Q[i:i + 1], K[:max(n, 0)], V[:max(n, 0)], scale)
            qq, oo, ll = Q[i:i + 1], np64(o[i:i + 1]), np64(lse[i:i + 1])
        big = scale * (np.abs(qq) @ np.abs(K).T).max(-1, initial=0.0)
        dl = (C_TC if bf else C_CUDA) * big
        rel = 2 * dl + 2.0 ** -18 + (2.0 ** -8 if bf else 0.0)
        within(oo, want, rel[:, None] * mass + (2.0 ** -8 if bf else 0.0) * np.abs(want) + 1e-37, f"o {what}")
        empty = np.isneginf(wl)
        assert np.array_equal(np.isneginf(ll), empty)
        within(ll[~empty], wl[~empty], (dl + 2.0 ** -20)[~empty] + 2.0 ** -22 * np.abs(wl[~empty]), f"lse {what}")


DENSE = [
    # B, Hq, Hkv, Tq, Tk, d, dtype
    (1, 4, 4, 512, 512, 64, F32),
    (1, 1, 1, 1, 1, 64, F32),
    (1, 1, 1, 1, 1, 128, BF),
    (2, 6, 2, 130, 130, 128, F32),
    (1, 8, 1, 65, 200, 64, F32),        # a chunk behind cached keys
    (1, 2, 2, 100, 37, 128, F32),       # rows that see no key
    (1, 2, 1, 3, 0, 64, F32),           # no keys at all
    (1, 16, 4, 650, 650, 64, F32),      # tiles of 64 rows
    (2, 16, 16, 333, 400, 128, F32),
    (1, 16, 8, 700, 20, 128, F32),
    (2, 4, 2, 257, 257, 128, BF),
    (1, 3, 1, 300, 300, 64, BF),
    (1, 2, 2, 1, 777, 128, BF),         # one token
    (1, 2, 1, 200, 90, 128, BF),        # rows that see no key
    (1, 2, 1, 300, 40, 64, BF),
    (1, 2, 1, 3, 0, 128, BF),
    (1, 4, 1, 129, 1000, 128, BF),
    (1, 1, 1, 513, 513, 128, BF),
    (1, 2, 2, 256, 256, 128, BF),
    (1, 2, 2, 384, 640, 64, BF),
    # few rows, many keys: the keys in shares that are joined
    (1, 4, 2, 130, 5000, 128, BF),
    (1, 3, 1, 5, 3003, 64, BF),
    (2, 8, 2, 1, 2500, 128, BF),
    (1, 2, 1, 600, 1300, 128, BF),
    (1, 1, 1, 700, 1200, 64, BF),
    (1, 64, 32, 700, 2100, 64, BF),     # the last, partial round of tiles in shares
    (2, 40, 8, 300, 1900, 128, BF),
    (1, 35, 7, 1100, 3000, 64, BF),
]


@pytest.mark.parametrize("case", DENSE, ids=str)
def test_dense(kvc, q8, case):
    B, Hq, Hkv, Tq, Tk, d, dtype = case
    Q, K, V = _rand((B, Hq, Tq, d), dtype, 1), _rand((B, Hkv, Tk, d), dtype, 2), _rand((B, Hkv, Tk, d), dtype, 3)
    K[:, :, :2] *= 3
    o, lse = kvc.kv_attn_prompt(Q, K, V)
    torch.cuda.synchronize()
    G = Hq // Hkv
    for b in range(B):
        for h in range(Hq):
            _check(q8, o[b, h], lse[b, h], Q[b, h], K[b, h // G], V[b, h // G], d ** -0.5, (b, h))
    o2, lse2 = kvc.kv_attn_prompt(Q, K, V)
    assert same_bits(o, o2) and same_bits(lse, lse2)


PACKED = [
    # Hq, Hkv, d, dtype, query lengths, keys in front of them
    (4, 2, 64, F32, [5, 0, 130, 1], [0, 0, 20, 3]),
    (2, 2, 128, F32, [64, 65, 63], [0, 0, 0]),
    (4, 1, 128, BF, [1, 0, 0, 300, 129, 77, 0], [0, 0, 5, 0, 33, 200, 0]),
    (2, 1, 64, BF, [256, 255, 257, 2], [0, 1, 0, 400]),
    (1, 1, 128, BF, [3] * 40, [0] * 40),
    (2, 1, 128, BF, [7, 0, 200, 1], [3000, 5, 0, 1100]),   # in shares, some of them without a key
    (3, 1, 64, BF, [300, 2], [0, 4000]),
]


def _packed(case, layout):
    Hq, Hkv, d, dtype, lens, front = case
    keys = [a + f for a, f in zip(lens, front)]
    tq, tk = sum(lens), sum(keys)

    def make(H, T, seed):
        if layout == "token":
            return _rand((T, H, d), dtype, seed).transpose(0, 1).unsqueeze(0)
        if layout == "fused":  # a slice of a wider projection
            return _rand((T, H + 3, 2 * d), dtype, seed)[:, 1:H + 1, d:].transpose(0, 1).unsqueeze(0)
        return _rand((1, H, T, d), dtype, seed)

    q, k, v = make(Hq, tq, 1), make(Hkv, tk, 2), make(Hkv, tk, 3)
    sq = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    sk = torch.tensor(np.cumsum([0] + keys), dtype=torch.int32, device="cuda")
    return q, k, v, sq, sk


@pytest.mark.parametrize("layout", ["head", "token", "fused"])
@pytest.mark.parametrize("case", PACKED, ids=str)
def test_packed(kvc, q8, case, layout):
    Hq, Hkv, d, dtype, lens, front = case
    q, k, v, sq, sk = _packed(case, layout)
    o, lse = kvc.kv_attn_prompt(q, k, v, scale=0.15, seq_q=sq, seq_k=sk, packed=True)
    torch.cuda.synchronize()
    assert layout != "token" or o.stride() == q.stride()
    a, b = sq.tolist(), sk.tolist()
    for i in range(len(lens)):
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            _check(q8, o[0, h, a[i]:a[i + 1]], lse[0, h, a[i]:a[i + 1]], q[0, h, a[i]:a[i + 1]],
                   k[0, hk, b[i]:b[i + 1]], v[0, hk, b[i]:b[i + 1]], 0.15, (i, h))


@pytest.mark.parametrize("dtype,d", [(F32, 64), (BF, 128), (BF, 64)])
def test_many_packed_sequences(kvc, q8, dtype, d):
    """More sequences than one look at the offsets covers, empty ones among them."""
    r = np.random.default_rng(8)
    lens = [int(x) for x in r.integers(0, 40, 700)]
    lens[3] = lens[600] = 300
    case = (4, 2, d, dtype, lens, [int(x) for x in r.integers(0, 3, 700)])
    q, k, v, sq, sk = _packed(case, "token")
    o, lse = kvc.kv_attn_prompt(q, k, v, seq_q=sq, seq_k=sk, packed=True)
    torch.cuda.synchronize()
    a, b = sq.tolist(), sk.tolist()
    for i in (0, 3, 31, 32, 127, 128, 129, 255, 256, 511, 512, 600, 640, 698, 699):
        for h in range(4):
            _check(q8, o[0, h, a[i]:a[i + 1]], lse[0, h, a[i]:a[i + 1]], q[0, h, a[i]:a[i + 1]],
                   k[0, h // 2, b[i]:b[i + 1]], v[0, h // 2, b[i]:b[i + 1]], d ** -0.5, (i, h))
    # every row is some sequence's
    one, _ = kvc.kv_attn_prompt(q, k, v, seq_q=sq, seq_k=sk, packed=True, out=torch.full_like(q, float("nan")))
    assert not one.isnan().any() and same_bits(one, o)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_padded_batch_and_garbage_behind_it(kvc, q8, dtype):
    """Rows of different lengths; NaN and infinities behind them change nothing and stay unread."""
    B, Hq, Hkv, T, d = 4, 4, 2, 300, 128
    Q, K, V = (_rand((B, h, T, d), dtype, s) for s, h in ((1, Hq), (2, Hkv), (3, Hkv)))
    lens = [300, 1, 0, 155]
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for b, n in enumerate(lens):
        K[b, :, n:] = float("nan")
        V[b, :, n:] = float("inf")
        Q[b, :, n:] = float("nan")
    out = torch.full_like(Q, 5.0)
    lse = torch.full((B, Hq, T), 5.0, device="cuda")
    kvc.kv_attn_prompt(Q, K, V, seq_q=ln, seq_k=ln, out=out, lse_out=lse)
    torch.cuda.synchronize()
    for b, n in enumerate(lens):
        assert (out[b, :, n:] == 5).all() and (lse[b, :, n:] == 5).all()
        for h in range(Hq):
            _check(q8, out[b, h, :n], lse[b, h, :n], Q[b, h, :n], K[b, h // 2, :n], V[b, h // 2, :n], d ** -0.5, (b, h))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_garbage_between_packed_sequences(kvc, dtype):
    """A sequence's result does not change with its neighbours, NaN among them."""
    case = (2, 1, 128, dtype, [70, 200, 90], [10, 0, 300])
    q, k, v, sq, sk = _packed(case, "head")
    o, lse = kvc.kv_attn_prompt(q, k, v, seq_q=sq, seq_k=sk, packed=True)
    a, b = sq.tolist(), sk.tolist()
    keep = slice(a[1], a[2])
    for t, off in ((q, a), (k, b), (v, b)):
        t[:, :, :off[1]] = float("nan")
        t[:, :, off[2]:] = float("inf")
    o2, lse2 = kvc.kv_attn_prompt(q, k, v, seq_q=sq, seq_k=sk, packed=True)
    torch.cuda.synchronize()
    assert same_bits(o[:, :, keep], o2[:, :, keep]) and same_bits(lse[:, :, keep], lse2[:, :, keep])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("shape", [(2, 1, 40, 40, 128), (4, 2, 600, 600, 64), (32, 8, 500, 500, 128), (2, 1, 7, 5000, 128),
                                   (3, 1, 300, 300, 128)], ids=str)
def test_nan_reaches_the_rows_that_see_it_and_no_others(kvc, dtype, shape):
    """A NaN query makes its row NaN, a NaN key the rows from its own on; the others keep their bits."""
    Hq, Hkv, Tq, Tk, d = shape
    Q, K, V = _rand((1, Hq, Tq, d), dtype, 1), _rand((1, Hkv, Tk, d), dtype, 2), _rand((1, Hkv, Tk, d), dtype, 3)
    o, lse = kvc.kv_attn_prompt(Q, K, V)
    Q2, K2 = Q.clone(), K.clone()
    Q2[:, 1, 3] = float("nan")
    K2[:, :, Tk - 2, 5] = float("nan")   # seen by the last two rows
    o2, lse2 = kvc.kv_attn_prompt(Q2, K2, V)
    torch.cuda.synchronize()
    bad = torch.zeros((1, Hq, Tq), dtype=torch.bool, device="cuda")
    bad[:, 1, 3] = True
    bad[:, :, -2:] = True
    assert o2[bad].isnan().all() and lse2[bad].isnan().all()
    assert same_bits(o2[~bad], o[~bad]) and same_bits(lse2[~bad], lse[~bad])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_bad_offsets_are_reported(kvc, dtype):
    q, k, v = (_rand((1, 2, 100, 64), dtype, s) for s in (1, 2, 3))
    out = torch.full_like(q, 5.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    sq = torch.tensor([0, 40, 30, 100], dtype=torch.int32, device="cuda")   # the second decreases
    sk = torch.tensor([0, 40, 40, 101], dtype=torch.int32, device="cuda")   # the third passes the end
    kvc.kv_attn_prompt(q, k, v, seq_q=sq, seq_k=sk, packed=True, out=out, dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == kvc.KV_ERR_INVALID_ARG
    assert (out[:, :, 40:] == 5).all() and not (out[:, :, :40] == 5).any()
    status.zero_()
    out.fill_(5.0)
    kvc.kv_attn_prompt(q, k, v, seq_q=torch.tensor([-1], dtype=torch.int32, device="cuda"), out=out, dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == kvc.KV_ERR_INVALID_ARG and (out == 5).all()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_large_logits_and_descending_maxima(kvc, q8, dtype):
    """Running maxima that climb a long way, that never change, and rows of equal logits."""
    T, d = 700, 128
    Q, K, V = (_rand((1, 3, T, d), dtype, s) for s in (4, 5, 6))
    K[:, 0] *= torch.linspace(0.01, 20, T, device="cuda")[:, None].to(dtype)
    K[:, 1] *= torch.linspace(20, 0.01, T, device="cuda")[:, None].to(dtype)
    K[:, 2] = K[:, 2, :1].clone()
    o, lse = kvc.kv_attn_prompt(Q, K, V)
    torch.cuda.synchronize()
    for h in range(3):
        _check(q8, o[0, h], lse[0, h], Q[0, h], K[0, h], V[0, h], d ** -0.5, h)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("scale", [0.0, -0.2])
@pytest.mark.parametrize("shape", [(2, 1, 90, 130, 128), (8, 4, 700, 700, 64)], ids=str)
def test_odd_scales(kvc, q8, dtype, scale, shape):
    """Scales that turn the order of the logits round, or make them all equal."""
    Hq, Hkv, Tq, Tk, d = shape
    Q, K, V = _rand((1, Hq, Tq, d), dtype, 1), _rand((1, Hkv, Tk, d), dtype, 2), _rand((1, Hkv, Tk, d), dtype, 3)
    o, lse = kvc.kv_attn_prompt(Q, K, V, scale=scale)
    torch.cuda.synchronize()
    for h in range(Hq):
        hk = h // (Hq // Hkv)
        want, wl, mass = q8.attn_prompt(np64(Q[0, h]), np64(K[0, hk]), np64(V[0, hk]), scale)
        dl = C_CUDA * abs(scale) * (np.abs(np64(Q[0, h])) @ np.abs(np64(K[0, hk])).T).max(-1)
        half = 2.0 ** -8 if dtype == BF else 0.0
        within(np64(o[0, h]), want, (2 * dl + 2.0 ** -18)[:, None] * mass + half * np.abs(want) + 1e-37, f"o {h}")
        within(np64(lse[0, h]), wl, dl + 2.0 ** -20 + 2.0 ** -22 * np.abs(wl), f"lse {h}")


@pytest.mark.parametrize("shape", [(4, 512, 512, 64), (2, 4000, 4000, 128), (2, 500, 20000, 128)], ids=str)
def test_fp32_error_of_the_whole_output(kvc, shape):
    """The error in norm stays that of fp32 sums.  A logit of unit size gathers at most d / 8 = 16 cut
    sums of 2^-23 (half of that on average, of partial sums that are smaller): 2^-20.  A tile's share
    of O has four such steps, and the shares are added with roundings that average out.  Sums cut
    at every step over all keys would be off by (keys / 8) 2^-24, 2^-17 at 1000 keys already."""
    H, Tq, Tk, d = shape
    Q, K, V = _rand((1, H, Tq, d), F32, 1), _rand((1, H, Tk, d), F32, 2), _rand((1, H, Tk, d), F32, 3)
    o, _ = kvc.kv_attn_prompt(Q, K, V)
    hidden = ~torch.ones((Tq, Tk), dtype=torch.bool, device="cuda").tril(Tk - Tq)
    for h in range(H):
        w = (Q[0, h].double() @ K[0, h].double().T * d ** -0.5).masked_fill(hidden, float("-inf")).softmax(-1)
        want = w @ V[0, h].double()
        assert (o[0, h].double() - want).norm() <= 2.0 ** -20 * want.norm()


def test_long_rows(kvc, q8):
    """A long sequence, some rows of it (the first, the last, around tile borders)."""
    T, d = 9001, 128
    Q, K, V = _rand((1, 2, T, d), BF, 7), _rand((1, 1, T, d), BF, 8), _rand((1, 1, T, d), BF, 9)
    o, lse = kvc.kv_attn_prompt(Q, K, V)
    torch.cuda.synchronize()
    for h in range(2):
        _check(q8, o[0, h], lse[0, h], Q[0, h], K[0, 0], V[0, 0], d ** -0.5, h,
               rows=[0, 1, 127, 128, 255, 256, 4096, 8191, 8192, 8959, 8960, 9000])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_captured_and_on_another_stream(kvc, dtype):
    case = (4, 2, 64, dtype, [33, 300], [0, 40])
    q, k, v, sq, sk = _packed(case, "token")
    o, lse = kvc.kv_attn_prompt(q, k, v, seq_q=sq, seq_k=sk, packed=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o2, lse2 = kvc.kv_attn_prompt(q, k, v, seq_q=sq, seq_k=sk, packed=True, stream=side)
    side.synchronize()
    assert same_bits(o, o2) and same_bits(lse, lse2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, lse3 = kvc.kv_attn_prompt(q, k, v, seq_q=sq, seq_k=sk, packed=True)
    graph.replay()
    torch.cuda.synchronize()
    assert same_bits(o, o3) and same_bits(lse, lse3)
    # other lengths of the same total: the captured call reads them from the device
    sq.copy_(torch.tensor([0, 133, 333], dtype=torch.int32))
    sk.copy_(torch.tensor([0, 173, 373], dtype=torch.int32))
    graph.replay()
    o4, lse4 = kvc.kv_attn_prompt(q, k, v, seq_q=sq, seq_k=sk, packed=True)
    torch.cuda.synchronize()
    assert same_bits(o3, o4) and same_bits(lse3, lse4)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_offsets_past_32_bits(kvc, q8, dtype):
    """A sequence at the end of tensors of more than 2^32 bytes."""
    T, n, d, Hq = 2 ** 24, 300, 128, 2
    q, k, v = _rand((1, Hq, n, d), dtype, 1), _rand((1, 1, n, d), dtype, 2), _rand((1, 1, n, d), dtype, 3)
    Q, K, V = (torch.zeros((1, x.shape[1], T, d), dtype=dtype, device="cuda") for x in (q, k, v))
    for x, y in ((Q, q), (K, k), (V, v)):
        x[:, :, -n:] = y
    off = torch.tensor([T - n, T], dtype=torch.int32, device="cuda")
    out = torch.zeros_like(Q)
    lse = torch.full((1, Hq, T), 5.0, device="cuda")
    kvc.kv_attn_prompt(Q, K, V, seq_q=off, seq_k=off, packed=True, out=out, lse_out=lse)
    torch.cuda.synchronize()
    for h in range(Hq):
        _check(q8, out[0, h, -n:], lse[0, h, -n:], q[0, h], k[0, 0], v[0, 0], d ** -0.5, h)
    assert not out[:, :, :-n].any() and (lse[:, :, :-n] == 5).all()
