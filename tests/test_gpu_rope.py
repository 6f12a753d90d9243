"""Norm, rotary positions and the cache's rows on the GPU against float64."""
import math

import pytest
import torch

from _long import BF, F32, HALF, rand

pytestmark = pytest.mark.gpu

EPS = 1e-5


def _want(x, w, f, pos, interleaved, eps, one_plus, scale):
    """x [B][H][T][d], pos [B][T] -> values and bounds, float64."""
    y = x.double()
    d = x.shape[-1]
    if eps is not None:
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps)
        if w is not None:
            y = y * (w.double() + (1.0 if one_plus else 0.0))
    m = 0 if f is None else f.numel()
    i = torch.arange(m, device=x.device)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + m)
    out, size = y.clone(), y.abs()
    if m:
        ang = pos.double()[:, None, :, None] * f
        a, b = y[..., ia], y[..., ib]
        out[..., ia], out[..., ib] = (a * ang.cos() - b * ang.sin()) * scale, (b * ang.cos() + a * ang.sin()) * scale
        size[..., ia] = size[..., ib] = (a.abs() + b.abs()) * scale
    return out, 2.0 ** -19 * size + HALF[x.dtype] * out.abs() + 1e-37


def _near(got, want, what):
    err = (got.double() - want[0]).abs()
    assert bool((err <= want[1]).all()), f"{what}: {float((err / want[1]).max()):.2f} of its bound"


CASES = [
    # B, T, Hq, Hkv, d, rot, interleaved, norm, dtype
    (1, 1, 32, 8, 128, 128, False, True, BF),
    (64, 1, 32, 8, 128, 128, False, True, BF),
    (2, 37, 4, 4, 64, 32, True, True, F32),
    (1, 100, 6, 2, 64, 24, False, True, BF),      # 12 pairs: element by element
    (1, 33, 3, 1, 128, 24, False, False, F32),
    (2, 9, 5, 5, 128, 64, False, True, F32),
    (3, 17, 1, 1, 64, 64, True, False, BF),
    (1, 5, 7, 3, 128, 2, False, True, BF),
    (1, 5, 7, 3, 128, 2, True, True, BF),
    (1, 11, 2, 2, 64, 0, False, True, BF),        # norm alone
    (4, 700, 9, 2, 128, 128, True, True, BF),
    (1, 3000, 32, 8, 64, 64, False, True, F32),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_heads(kvc, case):
    B, T, Hq, Hkv, d, rot, inter, norm, dtype = case
    x = rand((B, T, Hq + 2 * Hkv, d), dtype, 1, 2.0).transpose(1, 2)
    q, k, v = x.split([Hq, Hkv, Hkv], 1)
    wq, wk = ((1 + 0.3 * rand((d,), F32, 2)).to(dtype), rand((d,), dtype, 3)) if norm else (None, None)
    f, scale = kvc.kv_rope_freqs(rot, 500000.0, "yarn", factor=8.0, context=4096) if rot else (None, 1.0)
    g = torch.Generator().manual_seed(4)
    pos = (torch.randint(0, 1000000, (B, 1), generator=g) + torch.arange(T)).int().cuda()
    cap = T + 7
    slot = torch.randint(0, 8, (B, Hkv), generator=g, dtype=torch.int32)
    K, V = torch.full((B, Hkv, cap, d), 3.0, dtype=dtype, device="cuda"), torch.full((B, Hkv, cap, d), 4.0, dtype=dtype, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo, ko, vo = kvc.kv_qk_norm_rope(q, k, v, f, pos, q_weight=wq, k_weight=wk, eps=EPS if norm else None, interleaved=inter,
                                     rot_scale=scale, slot=slot.cuda(), k_out=K, v_out=V, dev_status=st)
    assert int(st) == 0 and ko is K and vo is V and qo.is_contiguous()
    _near(qo, _want(q, wq, f, pos, inter, EPS if norm else None, False, scale), "q")
    want = _want(k, wk, f, pos, inter, EPS if norm else None, False, scale)
    for b in range(B):
        for h in range(Hkv):
            s = int(slot[b, h])
            _near(K[b, h, s:s + T], (want[0][b, h], want[1][b, h]), f"k {b} {h}")
            assert torch.equal(V[b, h, s:s + T], v[b, h])
            rest = torch.cat((torch.arange(s), torch.arange(s + T, cap))).cuda()
            assert (K[b, h, rest] == 3).all() and (V[b, h, rest] == 4).all()


@pytest.mark.parametrize("pos", [2147483647, -2147483648, -1, 0, 1 << 24])
def test_angles_at_any_position(kvc, pos):
    """The angle at far positions is that of position times frequency in 64 bits: there the reference's own
    product is rounded at 2^-53 of up to 2^31 rad, and the frequency's fraction of a turn at 2^-55 turns."""
    d, T = 64, 3
    k = rand((1, 2, T, d), F32, 5)
    f, _ = kvc.kv_rope_freqs(d, 10000.0)
    p = torch.full((1, T), pos, dtype=torch.int32, device="cuda")
    got = kvc.kv_qk_norm_rope(None, k, None, f, p)[1]
    want, bound = _want(k, None, f, p, False, None, False, 1.0)
    extra = abs(pos) * (2.0 ** -53 + 2 * math.pi * 2.0 ** -55 + 2.0 ** -53)
    a = k.double().abs()
    size = torch.cat((a[..., :32] + a[..., 32:],) * 2, -1)
    _near(got, (want, bound + extra * size), str(pos))


def test_parts_of_a_call(kvc):
    q, k, v = (rand((2, 3, 20, 64), BF, 10 + i) for i in range(3))
    f, _ = kvc.kv_rope_freqs(64)
    pos = torch.arange(20, dtype=torch.int32, device="cuda").expand(2, 20).contiguous()
    qo, ko, vo = kvc.kv_qk_norm_rope(q, k, v, f)           # positions 0 .. T - 1
    full = kvc.kv_qk_norm_rope(q, k, v, f, pos)
    assert torch.equal(qo, full[0]) and torch.equal(ko, full[1]) and torch.equal(vo, v)
    alone = kvc.kv_qk_norm_rope(None, k, None, f, pos)
    assert alone[0] is None and alone[2] is None and torch.equal(alone[1], ko)
    assert torch.equal(kvc.kv_qk_norm_rope(q, None, None, f, pos)[0], qo)
    # in place
    q2, k2 = q.clone(), k.clone()
    kvc.kv_qk_norm_rope(q2, k2, None, f, pos, q_out=q2, k_out=k2)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)
    # weights of 1 + w, and none
    w = rand((64,), BF, 14, 0.1)
    got = kvc.kv_qk_norm_rope(q, k, None, f, pos, q_weight=w, eps=EPS, one_plus=True)
    _near(got[0], _want(q, w, f, pos, False, EPS, True, 1.0), "1 + w")
    _near(got[1], _want(k, None, f, pos, False, EPS, False, 1.0), "no weight")


def test_moved_keys(kvc):
    """Rotated keys moved to other positions by their differences."""
    k = rand((1, 2, 50, 128), F32, 20)
    f, _ = kvc.kv_rope_freqs(128)
    at = torch.arange(50, dtype=torch.int32, device="cuda")[None] * 7
    to = torch.arange(50, dtype=torch.int32, device="cuda")[None]
    first = kvc.kv_qk_norm_rope(None, k, None, f, at)[1]
    moved = kvc.kv_qk_norm_rope(None, first, None, f, to - at)[1]
    want, bound = _want(k, None, f, to, False, None, False, 1.0)
    _near(moved, (want, 4 * bound), "moved")  # two turns, the second of a turned pair (at most 2^0.5 longer)


def test_lengths_and_slots_out_of_range(kvc):
    B, T, H, d = 3, 6, 2, 64
    q, k, v = (rand((B, H, T, d), BF, 30 + i) for i in range(3))
    f, _ = kvc.kv_rope_freqs(d)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    seq = torch.tensor([0, 4, 6], dtype=torch.int32, device="cuda")
    new = lambda: [torch.full((B, H, T, d), 5.0, dtype=BF, device="cuda") for _ in range(3)]  # noqa: E731
    outs = new()
    kvc.kv_qk_norm_rope(q, k, v, f, seq=seq, q_out=outs[0], k_out=outs[1], v_out=outs[2], dev_status=st)
    want = kvc.kv_qk_norm_rope(q, k, v, f)
    assert int(st) == 0
    for o, w in zip(outs, want):
        for b, n in enumerate(seq.tolist()):
            assert torch.equal(o[b, :, :n], w[b, :, :n]) and (o[b, :, n:] == 5).all()
    outs = new()
    kvc.kv_qk_norm_rope(q, k, v, f, seq=torch.tensor([7, -1, 6], dtype=torch.int32, device="cuda"), q_out=outs[0], k_out=outs[1],
                        v_out=outs[2], dev_status=st)
    assert int(st) == -1
    for o, w in zip(outs, want):
        assert (o[:2] == 5).all() and torch.equal(o[2], w[2])
    st.zero_()
    outs = new()
    slot = torch.tensor([[0, 2], [-3, 0], [6, 0]], dtype=torch.int32, device="cuda")
    kvc.kv_qk_norm_rope(q, k, v, f, slot=slot, q_out=outs[0], k_out=outs[1], v_out=outs[2], dev_status=st)
    assert int(st) == -1 and torch.equal(outs[0], want[0])
    for o, w in zip(outs[1:], want[1:]):
        assert torch.equal(o[0, 0], w[0, 0]) and torch.equal(o[0, 1, 2:], w[0, 1, :4]) and (o[0, 1, :2] == 5).all()
        assert torch.equal(o[1, 0, :3], w[1, 0, 3:]) and (o[1, 0, 3:] == 5).all() and (o[2, 0] == 5).all()


@pytest.mark.parametrize("case", [
    # B, T, Hq, Hkv, d, rot, interleaved, dtype, keys and values only: thousands of tokens through the ring
    (1, 9001, 32, 8, 128, 128, False, BF, False),
    (3, 2000, 5, 3, 64, 32, True, F32, False),
    (2, 5003, 9, 9, 128, 64, False, BF, False),
    (1, 9001, 32, 8, 128, 128, True, BF, True),
    (1, 6000, 1, 40, 64, 24, False, BF, False),
], ids=str)
def test_many_tokens(kvc, case):
    B, T, Hq, Hkv, d, rot, inter, dtype, only = case
    q, k, v = rand((B, T, Hq + 2 * Hkv, d), dtype, 60).transpose(1, 2).split([Hq, Hkv, Hkv], 1)
    f, _ = kvc.kv_rope_freqs(rot)
    pos = (torch.arange(B * T, device="cuda") * 17 % 100003).int().view(B, T)
    wk = (1 + 0.3 * rand((d,), F32, 61)).to(dtype)
    slot = torch.arange(B * Hkv, dtype=torch.int32, device="cuda").view(B, Hkv) % 5 - 1  # token 0 of some heads has no row
    K, V = torch.full((B, Hkv, T, d), 3.0, dtype=dtype, device="cuda"), torch.full((B, Hkv, T, d), 4.0, dtype=dtype, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo = kvc.kv_qk_norm_rope(None if only else q, k, v, f, pos, k_weight=wk, eps=EPS, interleaved=inter, slot=slot, k_out=K, v_out=V,
                             dev_status=st)[0]
    assert int(st) == -1
    if not only:
        _near(qo, _want(q, None, f, pos, inter, EPS, False, 1.0), "q")
    want = _want(k, wk, f, pos, inter, EPS, False, 1.0)
    for b in range(B):
        for h in range(Hkv):
            s = int(slot[b, h])
            lo, hi = max(0, s), min(T, T + s)
            _near(K[b, h, lo:hi], (want[0][b, h, lo - s:hi - s], want[1][b, h, lo - s:hi - s]), f"k {b} {h}")
            assert torch.equal(V[b, h, lo:hi], v[b, h, lo - s:hi - s])
            assert (K[b, h, :lo] == 3).all() and (V[b, h, :lo] == 4).all() and (K[b, h, hi:] == 3).all()


def test_many_tokens_of_padded_rows(kvc):
    B, T, H, d = 3, 4000, 4, 128
    q, k, v = (rand((B, H, T, d), BF, 70 + i) for i in range(3))
    f, _ = kvc.kv_rope_freqs(d)
    want = kvc.kv_qk_norm_rope(q, k, v, f, eps=EPS)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for lens, status in (((4000, 0, 1777), 0), ((4001, 3, -1), -1)):
        outs = [torch.full((B, H, T, d), 5.0, dtype=BF, device="cuda") for _ in range(3)]
        kvc.kv_qk_norm_rope(q, k, v, f, eps=EPS, seq=torch.tensor(lens, dtype=torch.int32, device="cuda"), q_out=outs[0], k_out=outs[1],
                            v_out=outs[2], dev_status=st)
        assert int(st) == status
        for o, w in zip(outs, want):
            for b, n in enumerate(lens):
                n = n if 0 <= n <= T else 0
                assert torch.equal(o[b, :, :n], w[b, :, :n]) and (o[b, :, n:] == 5).all()
    # in place
    kvc.kv_qk_norm_rope(q, k, v, f, eps=EPS, q_out=q, k_out=k, v_out=v)
    assert all(torch.equal(a, b) for a, b in zip((q, k, v), want))


def test_captured(kvc):
    """A decode step's call, replayed with other positions and slots in the same tensors."""
    B, Hq, Hkv, d, cap = 4, 8, 2, 128, 16
    q, k, v = rand((B, Hq, 1, d), BF, 40), rand((B, Hkv, 1, d), BF, 41), rand((B, Hkv, 1, d), BF, 42)
    f, _ = kvc.kv_rope_freqs(d)
    pos = torch.zeros(B, 1, dtype=torch.int32, device="cuda")
    ln = torch.zeros(B, Hkv, dtype=torch.int32, device="cuda")
    K, V = torch.zeros(B, Hkv, cap, d, dtype=BF, device="cuda"), torch.zeros(B, Hkv, cap, d, dtype=BF, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qo = kvc.kv_qk_norm_rope(q, k, v, f, pos, eps=EPS, slot=ln, k_out=K, v_out=V)[0]
        pos += 1
        ln += 1
    for t in range(5):
        g.replay()
        want = kvc.kv_qk_norm_rope(q, k, v, f, torch.full_like(pos, t), eps=EPS)
        assert torch.equal(qo, want[0]) and torch.equal(K[:, :, t:t + 1], want[1]) and torch.equal(V[:, :, t:t + 1], v)
    assert (K[:, :, 5:] == 0).all()
