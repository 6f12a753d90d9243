"""The 8-bit slot cache on the GPU against float64: compaction, decode steps, eviction."""
import numpy as np
import pytest
import torch

from _q8 import (C_TC, CODES, check_written, clone, filled_cache, np64, same_bits, unit_rows, within)

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def q8():
    from oracle import q8
    return q8


# ---- compaction -------------------------------------------------------------------

COMPACT = [
    # B, H, T, k, cap, d, block, dtype, fmt
    (1, 4, 512, 102, 128, 64, 32, F32, "s8"),
    (2, 3, 300, 300, 320, 128, 64, BF, "s8"),
    (1, 1, 1, 1, 32, 64, 32, BF, "e4m3"),
    (2, 2, 200, 128, 256, 128, 128, BF, "e4m3"),
    (1, 2, 500, 127, 128, 128, 128, F32, "e4m3"),
    (3, 1, 97, 65, 64 * 3, 64, 64, F32, "s8"),
    (1, 2, 90, 31, 32, 128, 32, BF, "s8"),
]


def _prompt(B, H, T, d, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    K, V = (torch.randn(B, H, T, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    return K, V, torch.rand(B, H, T, generator=g, device="cuda")


def _indices(B, H, T, k, seed):
    r = np.random.default_rng(seed)
    a = np.stack([np.sort(r.choice(T, k, replace=False)) for _ in range(B * H)]).reshape(B, H, k)
    return torch.from_numpy(a.astype(np.int32)).cuda()


@pytest.mark.parametrize("case", COMPACT, ids=str)
def test_compact(kvc, q8, case):
    B, H, T, k, cap, d, block, dtype, fmt = case
    K, V, s = _prompt(B, H, T, d, dtype, 3)
    idx = None if k == T else _indices(B, H, T, k, 4)
    before = filled_cache(kvc, B, H, cap, d, block, dtype, fmt, np.zeros(B * H), 5)
    c = clone(before)
    assert kvc.kv_compact_q8(K, V, s, idx, c) is c
    torch.cuda.synchronize()
    at = np.arange(T)[None, None].repeat(B, 0).repeat(H, 1) if idx is None else idx.cpu().numpy()
    for b in range(B):
        for h in range(H):
            for name, src in (("K", K), ("V", V)):
                check_written(q8, before, c, name, (b, h), np64(src[b, h])[at[b, h]], k, fmt)
            np.testing.assert_array_equal(c["pos"][b, h, :k].cpu().numpy(), at[b, h])
            np.testing.assert_array_equal(c["acc"][b, h, :k].cpu().numpy(), s[b, h].cpu().numpy()[at[b, h]])
    assert same_bits(c["pos"][..., k:], before["pos"][..., k:])
    assert same_bits(c["acc"][..., k:], before["acc"][..., k:])
    assert (c["len"] == k).all()


@pytest.mark.parametrize("fmt", ["s8", "e4m3"])
def test_compact_extreme_blocks(kvc, q8, fmt):
    """Blocks of zeros, of subnormals, of one huge value, and exact ties between codes."""
    T, d, block = 128, 64, 32
    K, V, _ = _prompt(1, 1, T, d, F32, 7)
    K[0, 0, :32] = 0
    K[0, 0, 32:64] *= 1e-41
    K[0, 0, 64:96] *= 1e-3
    K[0, 0, 70, 5] = 3e38
    half = torch.arange(32 * 64, device="cuda").reshape(32, 64).float() % 254 / 2 - 63.25 - 0.25
    K[0, 0, 96:] = half * 2
    K[0, 0, 96, 0] = 127.0
    before = filled_cache(kvc, 1, 1, T, d, block, F32, fmt, [0], 5)
    c = clone(before)
    kvc.kv_compact_q8(K, V, None, None, c)
    torch.cuda.synchronize()
    check_written(q8, before, c, "K", (0, 0), np64(K[0, 0]), T, fmt)
    check_written(q8, before, c, "V", (0, 0), np64(V[0, 0]), T, fmt)
    assert (c["acc"][..., :T] == 0).all()


def test_compact_pinned_host_and_bad_index(kvc, q8):
    B, H, T, k, d = 1, 2, 200, 70, 128
    K, V, s = _prompt(B, H, T, d, BF, 9)
    idx = _indices(B, H, T, k, 10)
    a = kvc.kv_compact_q8(K, V, s, idx, kvc.q8_cache(B, H, 128, d))
    b = kvc.kv_compact_q8(K.cpu().pin_memory(), V.cpu().pin_memory(), s, idx, kvc.q8_cache(B, H, 128, d))
    torch.cuda.synchronize()
    assert all(same_bits(a[n], b[n]) for n in a)
    idx[0, 1, 3], idx[0, 1, 66] = T, -5
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c = kvc.kv_compact_q8(K, V, s, idx, kvc.q8_cache(B, H, 128, d), dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == kvc.KV_ERR_INVALID_ARG
    assert c["pos"][0, 1, 3] == -1 and c["acc"][0, 1, 66] == 0
    assert (np64(c["K"][0, 1, 3]) == 0).all() and (c["Vt"][0, 1, 2] == 0).all()
    assert same_bits(c["K"][0, 0], a["K"][0, 0])


# ---- decode -----------------------------------------------------------------------

DECODE = [
    # B, Hkv, G, cap, d, block, dtype, fmt, lens
    (1, 1, 1, 64, 64, 32, BF, "s8", [0]),
    (1, 3, 1, 64, 128, 64, BF, "e4m3", [0, 1, 63]),
    (1, 4, 2, 128, 128, 32, F32, "s8", [31, 32, 33, 127]),
    (2, 2, 4, 704, 128, 64, BF, "s8", [640, 65, 700, 703]),
    (1, 2, 8, 1024, 128, 128, BF, "e4m3", [1000, 127]),
    (1, 2, 5, 640, 64, 64, F32, "e4m3", [575, 200]),
    (2, 1, 3, 4096, 128, 64, BF, "s8", [4095, 1]),
    (1, 2, 7, 320, 128, 64, BF, "s8", [256, 319]),
    (1, 1, 6, 5120, 64, 128, F32, "s8", [5000]),
    # past the one-launch kernel's caches
    (1, 2, 8, 16384, 64, 64, BF, "s8", [16000, 130]),
    (1, 3, 4, 20480, 128, 64, BF, "e4m3", [20479, 9000, 0]),
    (1, 2, 1, 65536, 64, 128, BF, "s8", [65535, 40001]),
    (1, 2, 3, 24576, 128, 32, F32, "s8", [24000, 31]),
    (1, 2, 2, 32768, 128, 64, BF, "e4m3", [32703, 20000]),
]


def _step_inputs(B, Hkv, G, d, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [torch.randn(B, h, d, generator=g, device="cuda").to(dtype) for h in (Hkv * G, Hkv, Hkv)]


def _check_step(q8, before, after, o, q, kn, vn, new_pos, fmt, scale=None, len_out=None):
    B, Hkv, cap, d = before["K"].shape
    G, block = q.shape[1] // Hkv, before["Kt"].shape[2]
    scale = d ** -0.5 if scale is None else scale
    for b in range(B):
        for h in range(Hkv):
            n = int(before["len"][b, h])
            k = np.concatenate([unit_rows(q8, before, "K", b, h, n), np64(kn[b, h])[None]])
            v = np.concatenate([unit_rows(q8, before, "V", b, h, n), np64(vn[b, h])[None]])
            qq = np64(q[b, h * G:(h + 1) * G])
            want, p, mass = q8.decode(qq, k, v, scale)
            dl = C_TC * scale * (np.abs(qq) @ np.abs(k).T).max()
            rel = 2 * dl + 2.0 ** -18
            within(o[b, h * G:(h + 1) * G].cpu().numpy(), want, rel * mass + 1e-37, f"o {b, h}")
            if before["acc"] is not None:
                old = np.append(np64(before["acc"][b, h, :n]), 0.0)
                mine = p.sum(0) + old
                within(after["acc"][b, h, :n + 1].cpu().numpy(), mine, rel * p.sum(0) + 2.0 ** -23 * np.abs(mine) + 1e-37,
                       f"acc {b, h}")
                assert same_bits(after["acc"][b, h, n + 1:], before["acc"][b, h, n + 1:])
            assert (len_out if len_out is not None else after["len"])[b, h] == n + 1
            want_pos = before["pos"][b, h].clone()
            want_pos[n] = new_pos[b] if hasattr(new_pos, "__len__") else new_pos
            assert torch.equal(after["pos"][b, h], want_pos)
            f = n // block
            for name, new in (("K", kn), ("V", vn)):
                tail = before[name + "t"][b, h].clone()
                tail[n % block] = new[b, h]
                assert same_bits(after[name + "t"][b, h], tail)
                code, sc = before[name][b, h].clone(), before[name + "s"][b, h].clone()
                if (n + 1) % block == 0:
                    c, a = q8.quantise(tail.float().cpu().numpy(), fmt)
                    code[f * block:(f + 1) * block] = torch.from_numpy(c).to(torch.float32).to(code.dtype)
                    sc[f] = float(a)
                assert same_bits(after[name][b, h], code), (b, h, name)
                assert same_bits(after[name + "s"][b, h], sc)


@pytest.mark.parametrize("case", DECODE, ids=str)
def test_decode_step(kvc, q8, case):
    B, Hkv, G, cap, d, block, dtype, fmt, lens = case
    before = filled_cache(kvc, B, Hkv, cap, d, block, dtype, fmt, lens, 21)
    c = clone(before)
    q, kn, vn = _step_inputs(B, Hkv, G, d, dtype, 22)
    o = kvc.h2o_decode_step_q8(q, kn, vn, c, 9 * cap)
    torch.cuda.synchronize()
    _check_step(q8, before, c, o, q, kn, vn, 9 * cap, fmt)
    # the same bits from the same state
    c2 = clone(before)
    o2 = kvc.h2o_decode_step_q8(q, kn, vn, c2, 9 * cap)
    assert same_bits(o, o2) and all(same_bits(c[n], c2[n]) for n in c)


def test_decode_without_scores_row_positions_and_len_out(kvc, q8):
    B, Hkv, G, cap, d = 2, 2, 4, 256, 128
    before = filled_cache(kvc, B, Hkv, cap, d, 64, BF, "s8", [100, 64, 0, 255], 31, acc=False)
    c = clone(before)
    q, kn, vn = _step_inputs(B, Hkv, G, d, BF, 32)
    pos = torch.tensor([5000, 7000], dtype=torch.int32, device="cuda")
    ln = torch.zeros_like(c["len"])
    o = kvc.h2o_decode_step_q8(q, kn, vn, c, pos, scale=0.2, len_out=ln)
    torch.cuda.synchronize()
    assert torch.equal(c["len"], before["len"])
    _check_step(q8, before, c, o, q, kn, vn, pos.tolist(), "s8", scale=0.2, len_out=ln)


@pytest.mark.parametrize("G", [1, 4, 5])
def test_decode_without_scores_in_a_long_cache(kvc, q8, G):
    """The two-launch path without accumulators, a block that becomes full among the units."""
    before = filled_cache(kvc, 1, 3, 32768, 64, 64, BF, "s8", [32767, 20000, 64 * 300 - 1], 33, acc=False)
    c = clone(before)
    q, kn, vn = _step_inputs(1, 3, G, 64, BF, 34)
    o = kvc.h2o_decode_step_q8(q, kn, vn, c, 10 ** 6)
    torch.cuda.synchronize()
    _check_step(q8, before, c, o, q, kn, vn, 10 ** 6, "s8")


@pytest.mark.parametrize("fmt", ["s8", "e4m3"])
def test_decode_wide_ranges(kvc, q8, fmt):
    """Block scales over many powers of two, large logits, queries of very different sizes, one of zeros."""
    before = filled_cache(kvc, 1, 2, 1024, 128, 64, F32, fmt, [1000, 900], 41)
    r = torch.arange(16, device="cuda").float()
    before["Vs"].mul_(torch.exp2((r * 5) % 37 - 18))
    before["Ks"].mul_(torch.exp2((r * 3) % 7 - 3))
    before["Vs"][0, 1, 3] = 2.0 ** -126
    q, kn, vn = _step_inputs(1, 2, 4, 128, F32, 42)
    q *= torch.tensor([1e-6, 1.0, 4.0, 0.0, 1e-20, 3.0, 0.5, 1e-3], device="cuda")[None, :, None]
    c = clone(before)
    o = kvc.h2o_decode_step_q8(q, kn, vn, c, 10 ** 6)
    torch.cuda.synchronize()
    _check_step(q8, before, c, o, q, kn, vn, 10 ** 6, fmt)


def test_decode_ignores_what_is_behind_the_last_slot(kvc):
    before = filled_cache(kvc, 1, 2, 256, 64, 32, BF, "e4m3", [70, 128], 51)
    q, kn, vn = _step_inputs(1, 2, 4, 64, BF, 52)
    c = clone(before)
    o = kvc.h2o_decode_step_q8(q, kn, vn, c, 999)
    for n in ("K", "V"):
        before[n].view(torch.uint8)[0, 0, 64:] = 0x7F   # NaN in e4m3
        before[n].view(torch.uint8)[0, 1, 128:] = 0xFF
        before[n + "s"][0, 0, 2:] = float("nan")
        before[n + "s"][0, 1, 4:] = float("inf")
        before[n + "t"][0, 0, 6:] = float("nan")
        before[n + "t"][0, 1] = float("inf")
    before["acc"][0, 0, 71:] = float("nan")
    c2 = clone(before)
    o2 = kvc.h2o_decode_step_q8(q, kn, vn, c2, 999)
    torch.cuda.synchronize()
    assert same_bits(o, o2) and same_bits(c["acc"][0, 0, :71], c2["acc"][0, 0, :71])
    assert same_bits(c["acc"][0, 1, :129], c2["acc"][0, 1, :129])


def test_decode_reports_units_without_room(kvc):
    before = filled_cache(kvc, 1, 3, 64, 64, 32, BF, "s8", [64, 10, -1], 61)
    q, kn, vn = _step_inputs(1, 3, 2, 64, BF, 62)
    c = clone(before)
    o = torch.full((1, 6, 64), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvc.h2o_decode_step_q8(q, kn, vn, c, 999, o_out=o, dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == kvc.KV_ERR_INVALID_ARG
    for u in (0, 2):
        assert all(same_bits(c[n][0, u], before[n][0, u]) for n in c)
        assert (o[0, 2 * u:2 * u + 2] == 7).all()
    assert c["len"][0, 1] == 11 and not (o[0, 2:4] == 7).any()


def test_decode_captured_and_on_another_stream(kvc):
    """Steps replayed from a graph, and steps on a side stream, give the eager steps' bits."""
    before = filled_cache(kvc, 2, 2, 256, 128, 64, BF, "s8", [60, 61, 125, 3], 71)
    ins = [_step_inputs(2, 2, 4, 128, BF, 72 + i) for i in range(6)]
    c = clone(before)
    eager = [kvc.h2o_decode_step_q8(*x, c, 500 + i).clone() for i, x in enumerate(ins)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    c2 = clone(before)
    torch.cuda.synchronize()
    outs = [kvc.h2o_decode_step_q8(*x, c2, 500 + i, stream=side) for i, x in enumerate(ins)]
    side.synchronize()
    assert all(same_bits(a, b) for a, b in zip(eager, outs)) and all(same_bits(c[n], c2[n]) for n in c)
    c3 = clone(before)
    q, kn, vn = (t.clone() for t in ins[0])
    pos = torch.full((2,), 500, dtype=torch.int32, device="cuda")
    warm = clone(before)
    kvc.h2o_decode_step_q8(q, kn, vn, warm, pos)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = kvc.h2o_decode_step_q8(q, kn, vn, c3, pos)
        pos += 1
    for a, x in zip(eager, ins):
        for dst, src in zip((q, kn, vn), x):
            dst.copy_(src)
        graph.replay()
        assert same_bits(o, a)
    assert all(same_bits(c[n], c3[n]) for n in c)


# ---- eviction ---------------------------------------------------------------------

EVICT = [
    # B, H, cap, cap_out, d, block, dtype, fmt, lens, keep, recent, sink
    (1, 3, 128, 64, 64, 32, BF, "s8", [128, 100, 64], 60, 20, 0),
    (2, 2, 320, 192, 128, 64, BF, "e4m3", [320, 250, 10, 0], 150, 30, 5),
    (1, 2, 512, 256, 128, 128, F32, "s8", [511, 300], 256, 0, 3),
    (1, 2, 64, 64, 64, 32, F32, "e4m3", [64, 63], 2, 1, 0),
    (1, 1, 64, 32, 128, 32, BF, "s8", [64], 1, 0, 0),
    (1, 2, 2048, 2048, 128, 64, BF, "s8", [2048, 2000], 1999, 64, 4),
    (1, 1, 4096, 4096, 64, 64, BF, "s8", [4095], 4094, 2000, 2000),
    (1, 3, 64, 128, 64, 32, BF, "s8", [64, 33, 0], 100, 10, 2),          # keep past the capacity
    (2, 8, 1024, 512, 128, 128, F32, "s8", [1024, 1000, 900, 513] * 4, 500, 17, 1),
]


def _check_evicted(q8, src, before, out, idx, keep, recent, sink, fmt):
    B, H, cap, d = src["K"].shape
    block = src["Kt"].shape[2]
    for b in range(B):
        for h in range(H):
            n = int(src["len"][b, h])
            stay = q8.evict(np64(src["acc"][b, h]), src["pos"][b, h].cpu().numpy(), n, keep, recent, sink)
            nn = len(stay)
            got = idx[b, h].cpu().numpy()
            np.testing.assert_array_equal(got[:nn], stay)
            assert (got[nn:] == -1).all() and out["len"][b, h] == nn
            at = torch.from_numpy(stay).cuda()
            for name in ("pos", "acc"):
                assert same_bits(out[name][b, h, :nn], src[name][b, h][at])
                assert same_bits(out[name][b, h, nn:], before[name][b, h, nn:])
            for name in ("K", "V"):
                x = unit_rows(q8, src, name, b, h, n)[stay].astype(np.float32).astype(np.float64)
                f, whole = nn // block, n // block * block
                code, sc = np64(out[name][b, h]), out[name + "s"][b, h].cpu().numpy()
                for i in range(f):
                    rows = stay[i * block:(i + 1) * block]
                    if rows[0] % block == 0 and rows[-1] == rows[0] + block - 1 < whole:
                        want, a = np64(src[name][b, h, rows[0]:rows[0] + block]), src[name + "s"][b, h, rows[0] // block].item()
                    else:
                        want, a = q8.quantise(x[i * block:(i + 1) * block], fmt)
                    assert sc[i] == a, (b, h, name, i)
                    np.testing.assert_array_equal(code[i * block:(i + 1) * block], want)
                tail = before[name + "t"][b, h].clone()
                tail[:nn - f * block] = torch.from_numpy(x[f * block:].astype(np.float32)).cuda().to(tail.dtype)
                assert same_bits(out[name + "t"][b, h], tail)
                assert same_bits(out[name][b, h, f * block:], before[name][b, h, f * block:])
                assert same_bits(out[name + "s"][b, h, f:], before[name + "s"][b, h, f:])


@pytest.mark.parametrize("case", EVICT, ids=str)
def test_evict(kvc, q8, case):
    B, H, cap, cap_out, d, block, dtype, fmt, lens, keep, recent, sink = case
    src = filled_cache(kvc, B, H, cap, d, block, dtype, fmt, lens, 81)
    before = filled_cache(kvc, B, H, cap_out, d, block, dtype, fmt, np.zeros(B * H), 82)
    kept, out = clone(src), clone(before)
    idx = kvc.kv_evict_q8(src, keep, recent, out, sink=sink)
    torch.cuda.synchronize()
    assert all(same_bits(src[n], kept[n]) for n in src)
    _check_evicted(q8, src, before, out, idx, keep, recent, sink, fmt)


@pytest.mark.parametrize("acc", ["equal", "signs", "huge"])
def test_evict_orders(kvc, q8, acc):
    src = filled_cache(kvc, 1, 2, 640, 64, 64, BF, "s8", [640, 600], 91)
    if acc == "equal":
        src["acc"].fill_(0.5)
    elif acc == "signs":
        src["acc"].sub_(2.0)
        src["acc"][..., ::7] = -0.0
        src["acc"][..., 3::7] = 0.0
    else:
        src["acc"][..., ::3] = 3e38
        src["acc"][..., 1::3] = 1e-44
    before = filled_cache(kvc, 1, 2, 640, 64, 64, BF, "s8", [0, 0], 92)
    out = clone(before)
    idx = kvc.kv_evict_q8(src, 333, 10, out, sink=2)
    torch.cuda.synchronize()
    _check_evicted(q8, src, before, out, idx, 333, 10, 2, "s8")


def test_evict_whole_blocks_between_mixed_ones(kvc, q8):
    """Long runs in which every other destination block is a source block moved as it is: half of
    blocks 0 and 1 mod 3 go, blocks 2 mod 3 stay whole."""
    B, H, block, d, nb = 1, 4, 32, 64, 3 * 700
    cap = nb * block
    src = filled_cache(kvc, B, H, cap, d, block, BF, "s8", [cap] * H, 93)
    acc = torch.full((nb, block), 4.0, device="cuda")
    acc[0::3, ::2] = 1.0
    acc[1::3, 1::2] = 1.0
    src["acc"].copy_(acc.flatten())
    keep = cap // 3 * 2
    before = filled_cache(kvc, B, H, keep, d, block, BF, "s8", [0] * H, 94)
    out = clone(before)
    idx = kvc.kv_evict_q8(src, keep, 0, out, sink=0)
    torch.cuda.synchronize()
    stay = torch.arange(cap, device="cuda")[acc.flatten() > 2]
    assert torch.equal(idx.long(), stay.expand(B, H, -1)) and (out["len"] == keep).all()
    rows = stay.view(-1, block)
    whole = rows[:, -1] - rows[:, 0] == block - 1
    assert whole[1::2].all() and not whole[0::2].any()
    for name in ("K", "V"):
        code, scale = src[name][0].view(H, nb, block, d), src[name + "s"][0]
        got, gs = out[name][0].view(H, -1, block, d), out[name + "s"][0]
        assert torch.equal(got[:, 1::2], code[:, 2::3]) and torch.equal(gs[:, 1::2], scale[:, 2::3])
        x = (src[name][0].float() * scale.repeat_interleave(block, 1)[..., None])[:, stay].view(H, -1, block, d)
        for h in range(H):
            for i in range(0, rows.shape[0], 2):
                want, a = q8.quantise(np64(x[h, i]), "s8") if i % 64 == 0 else (None, None)
                if want is not None:
                    assert gs[h, i].item() == a
                    np.testing.assert_array_equal(np64(got[h, i]), want)
        # every mixed block's largest code is 127 by its own scale: no other block's scale was used
        assert (got[:, 0::2].int().abs().amax((-1, -2)) == 127).all()
        top = x[:, 0::2].abs().amax((-1, -2)) / 127
        assert ((gs[:, 0::2] - top).abs() <= top * 2.0 ** -23).all()


def test_evict_long_unit(kvc, q8):
    """A unit longer than any on-chip buffer: the kept slots against a sort."""
    cap, keep, recent = 300032, 100001, 77
    src = kvc.q8_cache(1, 1, cap, 64, 64)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    src["acc"].copy_((torch.rand(1, 1, cap, generator=g, device="cuda") * 5000).floor())
    src["pos"].copy_(torch.arange(cap, device="cuda"))
    src["K"].copy_(torch.randint(-127, 128, src["K"].shape, generator=g, device="cuda", dtype=torch.int8))
    src["Ks"].fill_(1.0)
    src["len"].fill_(cap - 5)
    out = kvc.q8_cache(1, 1, 100032, 64, 64)
    idx = kvc.kv_evict_q8(src, keep, recent, out, sink=4)
    a = src["acc"][0, 0].cpu().numpy()
    free = np.arange(4, cap - 5 - recent)
    gone = free[np.lexsort((free, a[free]))[:cap - 5 - keep]]
    stay = np.setdiff1d(np.arange(cap - 5), gone)
    np.testing.assert_array_equal(idx[0, 0].cpu().numpy(), stay)
    assert out["len"].item() == keep
    np.testing.assert_array_equal(out["pos"][0, 0, :keep].cpu().numpy(), stay)


@pytest.mark.parametrize("cap", [640, 400000])
def test_evict_keeps_protected_slots_among_nan_scores(kvc, q8, cap):
    """More slots of NaN score than stay: sinks and recent slots stay all the same."""
    block, d, keep, recent, sink = 32, 64, 200, 10, 3
    src = kvc.q8_cache(1, 2, cap, d, block)
    src["pos"].copy_(torch.arange(cap, device="cuda").expand(1, 2, cap))
    src["acc"].copy_(torch.rand(1, 2, cap, device="cuda"))
    src["acc"][..., ::2] = float("nan")
    src["len"].fill_(cap - 1)
    out = kvc.q8_cache(1, 2, 224, d, block)
    idx = kvc.kv_evict_q8(src, keep, recent, out, sink=sink)
    torch.cuda.synchronize()
    for h in range(2):
        got = idx[0, h].cpu().numpy()
        assert (np.diff(got) > 0).all() and (out["len"] == keep).all()
        np.testing.assert_array_equal(got[:sink], np.arange(sink))
        np.testing.assert_array_equal(got[-recent:], np.arange(cap - 1 - recent, cap - 1))


@pytest.mark.parametrize("levels", [1, 5000, 10 ** 9])
def test_evict_unit_past_the_cluster(kvc, q8, levels):
    """Units whose scores no cluster holds, with equal slots at the threshold and without."""
    cap, keep, recent, sink = 400000, 150001, 1001, 4
    src = kvc.q8_cache(1, 2, cap, 64, 64)
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    src["acc"].copy_((torch.rand(1, 2, cap, generator=g, device="cuda") * levels).floor())
    src["pos"].copy_(torch.arange(cap, device="cuda").expand(1, 2, cap))
    src["len"].copy_(torch.tensor([[cap, cap - 77]]))
    out = kvc.q8_cache(1, 2, 150016, 64, 64)
    idx = kvc.kv_evict_q8(src, keep, recent, out, sink=sink)
    for h in range(2):
        n = int(src["len"][0, h])
        a, free = src["acc"][0, h].cpu().numpy(), np.arange(sink, n - recent)
        stay = np.setdiff1d(np.arange(n), free[np.lexsort((free, a[free]))[:n - keep]])
        np.testing.assert_array_equal(idx[0, h].cpu().numpy(), stay)
        np.testing.assert_array_equal(out["pos"][0, h, :keep].cpu().numpy(), stay)
    assert (out["len"] == keep).all()


def test_evict_reports_bad_lengths(kvc):
    src = filled_cache(kvc, 1, 3, 64, 64, 32, BF, "s8", [65, 40, -3], 95)
    before = filled_cache(kvc, 1, 3, 32, 64, 32, BF, "s8", [1, 2, 3], 96)
    out = clone(before)
    idx = torch.full((1, 3, 20), 77, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvc.kv_evict_q8(src, 20, 5, out, idx_out=idx, dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == kvc.KV_ERR_INVALID_ARG
    for u in (0, 2):
        assert all(same_bits(out[n][0, u], before[n][0, u]) for n in out) and (idx[0, u] == 77).all()
    assert out["len"][0, 1] == 20


# ---- together -----------------------------------------------------------------------


@pytest.mark.parametrize("fmt", ["s8", "e4m3"])
def test_prompt_compress_decode_evict_together(kvc, q8, fmt):
    """A prompt attended and compressed, decode steps until the cache is full, an eviction, more steps."""
    B, Hq, Hkv, T, d, block = 2, 8, 2, 700, 128, 32
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    Q, K, V = (torch.randn(B, h, T, d, generator=g, device="cuda").to(BF) for h in (Hq, Hkv, Hkv))
    o, lse, c = kvc.compress_prefill_q8(Q, K, V, W=16, k=100, recent=16, r=0.2, cap=128, block=block, codes=CODES[fmt])
    assert o.shape == Q.shape and lse.shape == (B, Hq, T) and (c["len"] == 100).all()
    spare = kvc.q8_cache(B, Hkv, 128, d, block, BF, CODES[fmt])
    pos = T
    for rounds in range(2):
        while int(c["len"].max()) < 128:
            before = clone(c)
            q, kn, vn = _step_inputs(B, Hkv, Hq // Hkv, d, BF, pos)
            y = kvc.h2o_decode_step_q8(q, kn, vn, c, pos)
            _check_step(q8, before, c, y, q, kn, vn, pos, fmt)
            pos += 1
        before = clone(spare)
        idx = kvc.kv_evict_q8(c, 90, 20, spare, sink=1)
        _check_evicted(q8, c, before, spare, idx, 90, 20, 1, fmt)
        c, spare = spare, c
    assert (c["len"] == 90).all()


def _chain(kvc, K, V, s, idx, rows, c, spare, pos0, stream=None):
    """Compaction, steps until a block has filled, eviction, one more step; returns the outputs."""
    kvc.kv_compact_q8(K, V, s, idx, c, stream=stream)
    out = [kvc.h2o_decode_step_q8(q, kn, vn, c, pos0 + i, stream=stream) for i, (q, kn, vn) in enumerate(rows[:-1])]
    back = kvc.kv_evict_q8(c, 90, 20, spare, sink=1, stream=stream)
    out.append(kvc.h2o_decode_step_q8(*rows[-1], spare, pos0 + len(rows), stream=stream))
    return out + [back]


@pytest.mark.parametrize("cap", [128, 32768])
def test_chain_captured_and_on_two_streams(kvc, cap):
    """The operators in one graph, replayed with other inputs, and two chains at once on streams of
    their own: the bits of the eager calls.  Both decode paths (one launch, two launches)."""
    B, Hkv, G, T, d, k = 1, 2, 4, 500, 64, 122
    g = torch.Generator(device="cuda")

    def inputs(seed):
        g.manual_seed(seed)
        K, V = (torch.randn(B, Hkv, T, d, generator=g, device="cuda").to(BF) for _ in range(2))
        s = torch.rand(B, Hkv, T, generator=g, device="cuda")
        idx = torch.rand(B, Hkv, T, generator=g, device="cuda").argsort(-1)[..., :k].sort(-1).values.int().contiguous()
        return K, V, s, idx, [_step_inputs(B, Hkv, G, d, BF, 10 * seed + i) for i in range(7)]

    def caches():
        return [kvc.q8_cache(B, Hkv, cap, d, 64) for _ in range(2)]

    want = []
    for seed in (1, 2):
        c = caches()
        want.append((_chain(kvc, *inputs(seed), *c, T), c))
    torch.cuda.synchronize()

    def same(got, c, i):
        torch.cuda.synchronize()
        assert all(same_bits(a, b) for a, b in zip(got, want[i][0]))
        assert all(same_bits(x[n], y[n]) for x, y in zip(c, want[i][1]) for n in x)

    streams = [torch.cuda.Stream() for _ in range(2)]
    both = [(inputs(seed), caches()) for seed in (1, 2)]
    torch.cuda.synchronize()
    got = [_chain(kvc, *x, *c, T, stream=st) for (x, c), st in zip(both, streams)]
    for i in range(2):
        same(got[i], both[i][1], i)

    x, c = inputs(1), caches()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = _chain(kvc, *x, *c, T)
    for i, seed in ((0, 1), (1, 2)):
        new = inputs(seed)
        for a, b in zip((*x[:4], *sum(x[4], [])), (*new[:4], *sum(new[4], []))):
            a.copy_(b)
        for z in c:
            for t in z.values():
                t.view(torch.uint8).zero_()
        graph.replay()
        same(y, c, i)


def test_offsets_past_32_bits(kvc):
    """Rows and slots whose byte and element offsets pass 2^32: a prompt's last rows into a cache, a
    step that looks at a slot near the end of the last unit, whole blocks from there moved."""
    H, T, d, block = 3, 2 ** 24, 128, 128
    K = torch.zeros((1, H, T, d), dtype=BF, device="cuda")
    V = torch.zeros((1, H, T, d), dtype=BF, device="cuda")
    r = torch.randn(2, H, 200, d, device="cuda").to(BF)
    K[0, :, -200:] = r[0]
    V[0, :, -200:] = r[1]
    small = kvc.q8_cache(1, H, 256, d, block)
    idx = torch.arange(T - 200, T, dtype=torch.int32, device="cuda").expand(1, H, 200).contiguous()
    kvc.kv_compact_q8(K, V, None, idx, small)
    near = kvc.q8_cache(1, H, 256, d, block)
    kvc.kv_compact_q8(r[0][None], r[1][None], None, None, near)
    torch.cuda.synchronize()
    assert all(same_bits(small[n], near[n]) for n in ("K", "V", "Ks", "Vs", "Kt", "Vt", "len"))
    del K, V

    c = kvc.q8_cache(1, H, T, d, block)
    c["pos"].copy_(torch.arange(T, dtype=torch.int32, device="cuda").expand(1, H, T))
    c["Ks"].fill_(1.0)
    c["Vs"].fill_(1.0)
    c["len"].fill_(T - 1)
    at = T - 2 * block + 5
    code = torch.randint(-127, 128, (H, d), device="cuda").to(torch.int8)
    c["K"][0, :, at] = 1                     # <q, k> = 128 with q of ones: the other logits are 0
    c["V"][0, :, at] = code
    kt = torch.zeros(1, H, d, device="cuda", dtype=BF)
    o = kvc.h2o_decode_step_q8(torch.ones(1, H, d, device="cuda", dtype=BF), kt, kt, c, T, scale=0.5)
    torch.cuda.synchronize()
    # its weight is 1 / (1 + 2^24 e^-64) = 1 to 2^-68; the error is that of a weight, 2 dl + 2^-18 with
    # dl = 2^-18 64
    assert ((o[0] - code).abs() <= code.abs() * (2.0 ** -11 + 2.0 ** -18)).all()
    assert (c["len"] == T).all() and ((c["acc"][0, :, at] - 1).abs() <= 2.0 ** -10).all()

    # the last four blocks and nothing else among the recent slots: whole blocks, moved as they are
    c["acc"].zero_()
    c["acc"][0, :, -4 * block:-2 * block] = 1.0
    c["K"][0, :, -4 * block:] = torch.randint(-127, 128, (H, 4 * block, d), device="cuda").to(torch.int8)
    out = kvc.q8_cache(1, H, 4 * block, d, block)
    back = kvc.kv_evict_q8(c, 4 * block, 2 * block, out)
    torch.cuda.synchronize()
    assert torch.equal(back[0], torch.arange(T - 4 * block, T, dtype=torch.int32, device="cuda").expand(H, -1))
    for n in ("K", "V"):
        assert same_bits(out[n][0], c[n][0, :, -4 * block:]) and same_bits(out[n + "s"][0], c[n + "s"][0, :, -4:])
