"""Attention over a common prefix and own slots on the GPU against float64."""
import pytest
import torch

from _long import BF, F32, check_rows, rand

pytestmark = pytest.mark.gpu


def _lens(B, H, least, most, seed):
    g = torch.Generator().manual_seed(seed)
    ln = torch.randint(least, most + 1, (B, H), generator=g, dtype=torch.int32)
    ln.view(-1)[-1] = most
    return ln


def _check(q, Kp, Vp, K, V, ln, o, lse, scale, units=None):
    B, Hq, nq, d = q.shape
    Hkv = K.shape[1] if K is not None else Kp.shape[0]
    G = Hq // Hkv
    none = q.new_zeros(0, d)
    w = 2.0 ** -8 if q.dtype == BF else 2.0 ** -20
    for b in range(B):
        for h in range(Hkv):
            if units is not None and (b, h) not in units:
                continue
            for t in range(nq):
                n = max(0, int(ln[b, h]) - nq + t + 1) if K is not None else 0
                k, v = (none, none) if Kp is None else (Kp[h], Vp[h])
                if n:
                    k, v = torch.cat((k, K[b, h, :n])), torch.cat((v, V[b, h, :n]))
                hs = slice(h * G, (h + 1) * G)
                check_rows(o[b, hs, t], lse[b, hs, t], q[b, hs, t], k, v, scale, w, f"b {b} h {h} t {t} own {n}")


CASES = [
    # B, Hq, Hkv, nq, P, cap, d, least, most, dtype
    (1, 4, 4, 1, 512, 64, 64, 1, 64, F32),
    (1, 1, 1, 1, 1, 1, 128, 1, 1, BF),
    (4, 32, 8, 1, 1000, 200, 128, 0, 200, BF),
    (3, 8, 1, 2, 777, 100, 64, 0, 100, BF),
    (2, 12, 4, 1, 128, 40, 128, 40, 40, BF),        # one key tile: the second softmax has none
    (2, 12, 4, 1, 129, 40, 128, 0, 3, BF),
    (5, 6, 2, 4, 300, 50, 128, 2, 50, BF),          # tokens that see no own slot
    (40, 8, 2, 1, 2000, 300, 128, 100, 300, BF),    # 160 rows: two tiles
    (33, 8, 1, 1, 700, 130, 64, 0, 130, BF),        # 264 rows: two pairs, the last with 8 rows
    (70, 16, 2, 1, 5000, 64, 128, 10, 64, BF),      # 560 rows
    (2, 16, 1, 9, 333, 40, 64, 5, 40, BF),          # 18 groups of rows
    (3, 5, 5, 1, 4097, 0, 128, 0, 0, BF),           # no own slots
    (3, 10, 5, 2, 0, 700, 128, 0, 700, BF),         # no prefix
    (2, 6, 3, 3, 0, 90, 64, 0, 90, F32),
    (2, 6, 3, 1, 900, 0, 128, 0, 0, F32),
    (9, 8, 2, 3, 501, 90, 128, 0, 90, F32),
    (1, 4, 1, 1, 20000, 3000, 128, 2999, 2999, BF),
    (130, 1, 1, 1, 260, 20, 64, 0, 20, BF),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_attention(kvc, case):
    B, Hq, Hkv, nq, P, cap, d, least, most, dtype = case
    Kp, Vp = (rand((Hkv, P, d), dtype, 1), rand((Hkv, P, d), dtype, 2)) if P else (None, None)
    q = rand((B, Hq, nq, d), dtype, 3)
    K = V = ln = None
    if cap:
        K, V = rand((B, Hkv, cap, d), dtype, 4), rand((B, Hkv, cap, d), dtype, 5)
        ln = _lens(B, Hkv, least, most, 6)
        for b in range(B):
            for h in range(Hkv):  # what stands behind the last slot does not matter
                K[b, h, int(ln[b, h]):] = float("nan")
                V[b, h, int(ln[b, h]):] = float("nan")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = kvc.kv_attn_shared(q, Kp, Vp, K, V, None if ln is None else ln.cuda(), dev_status=st)
    assert int(st) == 0
    _check(q, Kp, Vp, K, V, ln, o, lse, d ** -0.5)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_layouts_scale_and_given_outputs(kvc, dtype):
    B, Hq, Hkv, nq, P, cap, d = 6, 8, 2, 3, 300, 80, 128
    fused = rand((P, 2 * Hkv + 1, d), dtype, 10)  # the prefix as a projection lays it out
    Kp, Vp = fused[:, :Hkv].transpose(0, 1), fused[:, Hkv:2 * Hkv].transpose(0, 1)
    q = rand((B, nq, Hq + 3, d), dtype, 11)[:, :, 1:1 + Hq].transpose(1, 2)
    K, V = rand((B, Hkv, cap, d), dtype, 12), rand((B, Hkv, cap, d), dtype, 13)
    ln = _lens(B, Hkv, 3, 80, 14)
    out = torch.zeros(B, nq, Hq, d, dtype=dtype, device="cuda").transpose(1, 2)
    lse = torch.zeros(B, Hq, nq, device="cuda")
    got = kvc.kv_attn_shared(q, Kp, Vp, K, V, ln.cuda(), scale=0.2, out=out, lse_out=lse)
    assert got[0] is out and got[1] is lse
    _check(q, Kp, Vp, K, V, ln, out, lse, 0.2)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_rising_logits_and_large_values(kvc, dtype):
    """References that move at nearly every tile, in the prefix and across the join."""
    P, cap, d = 3000, 400, 64
    q = torch.ones(2, 2, 1, d, dtype=dtype, device="cuda")
    ramp = torch.linspace(-3, 12, P, device="cuda")[:, None].expand(P, d)
    Kp = (ramp + 0.1 * rand((1, P, d), F32, 20)).to(dtype)
    Vp = rand((1, P, d), dtype, 21)
    K = (torch.linspace(11, 13, cap, device="cuda")[:, None].expand(cap, d) + 0.1 * rand((2, 1, cap, d), F32, 22)).to(dtype)
    V = rand((2, 1, cap, d), dtype, 23)
    ln = torch.tensor([[cap], [7]], dtype=torch.int32)
    o, lse = kvc.kv_attn_shared(q, Kp, Vp, K, V, ln.cuda())
    _check(q, Kp, Vp, K, V, ln, o, lse, d ** -0.5)
    o, lse = kvc.kv_attn_shared(q, Kp.flip(1).contiguous(), Vp, K, V, ln.cuda())
    _check(q, Kp.flip(1), Vp, K, V, ln, o, lse, d ** -0.5)


@pytest.mark.parametrize("case", [
    # B, Hq, Hkv, nq, P, cap, d, dtype, lens: many rows of little; more heads than lengths are kept on chip
    (300, 16, 8, 1, 40, 64, 64, BF, "some empty"),
    (600, 8, 4, 1, 17, 40, 64, F32, "some empty"),
    (3, 4, 4, 1, 200, 5000, 128, BF, "one long"),
    (64, 2, 2, 1, 100, 3000, 128, BF, "one long"),
    (2, 2, 1, 1, 100, 50, 64, BF, "none"),
], ids=str)
def test_uneven_lengths(kvc, case):
    B, Hq, Hkv, nq, P, cap, d, dtype, how = case
    Kp, Vp, q = rand((Hkv, P, d), dtype, 60), rand((Hkv, P, d), dtype, 61), rand((B, Hq, nq, d), dtype, 62)
    K, V = rand((B, Hkv, cap, d), dtype, 63), rand((B, Hkv, cap, d), dtype, 64)
    ln = _lens(B, Hkv, 0, cap, 65) * (_lens(B, Hkv, 0, 3, 66) > 1) if how == "some empty" else torch.zeros(B, Hkv, dtype=torch.int32)
    if how == "one long":
        ln[B // 2, 1], ln[0, 0], ln[-1, -1] = cap, 1, 33
    o, lse = kvc.kv_attn_shared(q, Kp, Vp, K, V, ln.to(torch.int32).cuda())
    g = torch.Generator().manual_seed(67)
    units = {(int(torch.randint(0, B, (1,), generator=g)), int(torch.randint(0, Hkv, (1,), generator=g))) for _ in range(150)}
    _check(q, Kp, Vp, K, V, ln, o, lse, d ** -0.5, units=units | {(0, 0), (B // 2, Hkv - 1), (B - 1, Hkv - 1)})


def test_offsets_past_32_bits(kvc):
    """Own slots of more than 2^31 elements: the last rows'."""
    B, Hkv, cap, d = 17, 1, 1000000, 128
    K = torch.empty(B, Hkv, cap, d, dtype=BF, device="cuda")
    V = torch.empty(B, Hkv, cap, d, dtype=BF, device="cuda")
    K[-1, :, :5000], V[-1, :, :5000] = rand((Hkv, 5000, d), BF, 70), rand((Hkv, 5000, d), BF, 71)
    K[-1, :, -300:], V[-1, :, -300:] = rand((Hkv, 300, d), BF, 72), rand((Hkv, 300, d), BF, 73)
    q, Kp, Vp = rand((B, 2, 1, d), BF, 74), rand((Hkv, 64, d), BF, 75), rand((Hkv, 64, d), BF, 76)
    ln = torch.zeros(B, Hkv, dtype=torch.int32)
    ln[-1] = 5000
    o, lse = kvc.kv_attn_shared(q, Kp, Vp, K, V, ln.cuda())
    _check(q, Kp, Vp, K, V, ln, o, lse, d ** -0.5)
    K[-1, :, 5000:-300], V[-1, :, 5000:-300] = 0, 0
    ln[-1] = cap
    o, lse = kvc.kv_attn_shared(q, Kp, Vp, K, V, ln.cuda())
    _check(q, Kp, Vp, K, V, ln, o, lse, d ** -0.5, units=[(B - 1, 0)])


def test_nan_reaches_the_rows_that_see_it(kvc):
    B, Hq, Hkv, P, cap, d = 3, 4, 2, 500, 100, 128
    q, Kp, Vp = rand((B, Hq, 1, d), BF, 30), rand((Hkv, P, d), BF, 31), rand((Hkv, P, d), BF, 32)
    K, V = rand((B, Hkv, cap, d), BF, 33), rand((B, Hkv, cap, d), BF, 34)
    ln = torch.full((B, Hkv), cap, dtype=torch.int32)
    K[1, 0, 50, 3] = float("nan")
    o, lse = kvc.kv_attn_shared(q, Kp, Vp, K, V, ln.cuda())
    assert o[1, :2].isnan().all() and lse[1, :2].isnan().all() and int(lse.isnan().sum()) == 2
    _check(q, Kp, Vp, K, V, ln, o, lse, d ** -0.5, units=[(0, 0), (0, 1), (1, 1), (2, 0), (2, 1)])
    Kp[1, 300, 0] = float("nan")
    o, lse = kvc.kv_attn_shared(q, Kp, Vp, K, V, ln.cuda())
    assert o[:, 2:].isnan().all() and lse[:, 2:].isnan().all() and not lse[0, :2].isnan().any()


def test_bad_lengths_leave_their_units(kvc):
    q, Kp, Vp = rand((2, 4, 1, 64), BF, 40), rand((2, 300, 64), BF, 41), rand((2, 300, 64), BF, 42)
    K, V = rand((2, 2, 50, 64), BF, 43), rand((2, 2, 50, 64), BF, 44)
    ln = torch.tensor([[50, 51], [-1, 0]], dtype=torch.int32)
    out, st = torch.full_like(q, 9.0), torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = kvc.kv_attn_shared(q, Kp, Vp, K, V, ln.cuda(), out=out, dev_status=st)
    assert int(st) == -1 and (o[0, 2:] == 9).all() and (o[1, :2] == 9).all()
    _check(q, Kp, Vp, K, V, ln, o, lse, 64 ** -0.5, units=[(0, 0), (1, 1)])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_captured_and_on_two_streams(kvc, dtype):
    B, Hq, Hkv, P, cap, d = 5, 8, 2, 2100, 300, 128
    Kp, Vp = rand((Hkv, P, d), dtype, 50), rand((Hkv, P, d), dtype, 51)
    K, V = rand((B, Hkv, cap, d), dtype, 52), rand((B, Hkv, cap, d), dtype, 53)
    q = [rand((B, Hq, 1, d), dtype, 54 + i) for i in range(2)]
    ln = _lens(B, Hkv, 100, 250, 56).cuda()
    want = [kvc.kv_attn_shared(x, Kp, Vp, K, V, ln) for x in q]
    streams = [torch.cuda.Stream() for _ in q]
    got = [None, None]
    for _ in range(10):
        for i, s in enumerate(streams):
            s.wait_stream(torch.cuda.current_stream())
            got[i] = kvc.kv_attn_shared(q[i], Kp, Vp, K, V, ln, stream=s)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    g = torch.cuda.CUDAGraph()
    x = q[0].clone()
    with torch.cuda.graph(g):
        o, lse = kvc.kv_attn_shared(x, Kp, Vp, K, V, ln)
        ln += 1  # the next step's length: the call before has to have read it
    for i in (0, 1):
        x.copy_(q[i])
        n = ln.clone()
        g.replay()
        _check(x, Kp, Vp, K, V, n.cpu(), o, lse, d ** -0.5)
