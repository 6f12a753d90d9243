"""Infinities, NaN and the largest finite values in the keys and values of block-sparse and shared-prefix attention:
what a token sees has the formula's effect, what it does not see has none."""
import math

import pytest
import torch

from _long import BF, F32, attend, check_rows, rand

pytestmark = pytest.mark.gpu

TYPES = pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
INF, NAN = math.inf, math.nan


def _check(o, lse, q, k, v, scale, w, what):
    """As check_rows, with the formula's infinities and NaN where it has them."""
    want, wl, _, _ = attend(q.double(), k.double(), v.double(), scale)
    got = o.double()
    assert torch.equal(got.isnan(), want.isnan()), f"{what}: NaN in other places"
    assert torch.equal(got.isinf(), want.isinf()) and torch.equal(got[want.isinf()], want[want.isinf()]), f"{what}: infinities"
    clean = v.masked_fill(~v.isfinite().all(0), 0.0)  # whole channels
    ok = want.isfinite()
    rows = ok.any(-1)
    if bool(rows.any()):
        near = torch.where(v.isfinite().all(0), o, torch.zeros_like(o))
        kept = (k.abs() < 1e30).all(-1)  # the others weigh nothing here
        check_rows(near[rows], lse[rows], q[rows], k[kept], clean[kept], scale, w, what)


def _shared(kvc, dtype, P, d=128, nq=1, seed=1, n=200):
    q, K, V = rand((2, 8, nq, d), dtype, seed), rand((2, 2, n, d), dtype, seed + 1), rand((2, 2, n, d), dtype, seed + 2)
    Kp, Vp = rand((2, max(P, 1), d), dtype, seed + 3)[:, :P], rand((2, max(P, 1), d), dtype, seed + 4)[:, :P]
    return q, Kp, Vp, K, V, torch.full((2, 2), n, dtype=torch.int32, device="cuda")


def _run_shared(kvc, q, Kp, Vp, K, V, ln, what, units=None):
    P, nq, d = Kp.shape[1], q.shape[2], q.shape[3]
    o, lse = kvc.kv_attn_shared(q, Kp if P else None, Vp if P else None, K, V, ln)
    w = (2.0 ** -8 if P else 2.0 ** -16) if q.dtype == BF else 2.0 ** -20
    for b in range(2):
        for h in range(2):
            for t in range(nq):
                s, hs = int(ln[b, h]) - nq + t + 1, slice(4 * h, 4 * h + 4)
                _check(o[b, hs, t], lse[b, hs, t], q[b, hs, t], torch.cat((Kp[h], K[b, h, :s])), torch.cat((Vp[h], V[b, h, :s])), d ** -0.5,
                       w, f"{what} b {b} h {h} t {t}")
    return o, lse


@TYPES
@pytest.mark.parametrize("bad", [INF, -INF, NAN])
@pytest.mark.parametrize("P", [0, 300])
def test_shared_values(kvc, dtype, bad, P):
    q, Kp, Vp, K, V, ln = _shared(kvc, dtype, P)
    V[0, 0, 17, 5], V[0, 1, 199, 127], V[1, 1, 0, 0], V[1, 1, 3, 0] = bad, bad, bad, 1.0
    _run_shared(kvc, q, Kp, Vp, K, V, ln, "own values")
    if P:
        Vp[0, 280, 64], Vp[1, 0, 3] = bad, bad
        _run_shared(kvc, q, Kp, Vp, K, V, ln, "prefix values")


@TYPES
def test_shared_infinities_of_both_signs(kvc, dtype):
    q, Kp, Vp, K, V, ln = _shared(kvc, dtype, 0)
    V[0, 0, 17, 5], V[0, 0, 90, 5], V[0, 0, 91, 6] = INF, -INF, -INF
    o, _ = _run_shared(kvc, q, Kp, Vp, K, V, ln, "both signs")
    assert o[0, :4, 0, 5].isnan().all() and (o[0, :4, 0, 6] == -INF).all()


@TYPES
@pytest.mark.parametrize("P", [0, 300])
def test_shared_keys(kvc, dtype, P):
    """A key that makes a logit -inf weighs nothing; one that makes it +inf makes the row NaN."""
    q, Kp, Vp, K, V, ln = _shared(kvc, dtype, P)
    q[..., 7] = q[..., 7].abs() + 0.5
    K[0, 0, 33, 7] = -INF
    K[1, 1, 199, 7] = -INF
    if P:
        Kp[1, 100, 7] = -INF
    _run_shared(kvc, q, Kp, Vp, K, V, ln, "-inf")
    K[0, 1, 5, 7] = INF
    o, lse = kvc.kv_attn_shared(q, Kp if P else None, Vp if P else None, K, V, ln)
    assert o[0, 4:].isnan().all() and lse[0, 4:].isnan().all() and o[0, :4].isfinite().all() and o[1].isfinite().all()


@TYPES
@pytest.mark.parametrize("bad", [INF, -INF, NAN])
@pytest.mark.parametrize("P", [0, 300])
def test_shared_later_tokens(kvc, dtype, bad, P):
    """A later new token's key and value do not reach an earlier one."""
    q, Kp, Vp, K, V, ln = _shared(kvc, dtype, P, nq=3)
    ln[1, 0] = 177
    for b in range(2):
        for h in range(2):
            n = int(ln[b, h])
            V[b, h, n - 1, ::2], V[b, h, n - 2, 1], K[b, h, n - 1, 4] = bad, bad, NAN
    o, lse = kvc.kv_attn_shared(q, Kp if P else None, Vp if P else None, K, V, ln)
    w = (2.0 ** -8 if P else 2.0 ** -16) if dtype == BF else 2.0 ** -20
    for b in range(2):
        for h in range(2):
            hs, n = slice(4 * h, 4 * h + 4), int(ln[b, h])
            for t in range(2):
                _check(o[b, hs, t], lse[b, hs, t], q[b, hs, t], torch.cat((Kp[h], K[b, h, :n - 2 + t])),
                       torch.cat((Vp[h], V[b, h, :n - 2 + t])), 128 ** -0.5, w, f"b {b} h {h} t {t}")
            assert o[b, hs, 2].isnan().all() and lse[b, hs, 2].isnan().all()


@TYPES
def test_shared_largest_own_values(kvc, dtype):
    """The largest finite values, among them float32 ones that no sum of two tf32 parts holds."""
    q, Kp, Vp, K, V, ln = _shared(kvc, dtype, 0, d=64)
    K[:, :, :, 3] += torch.linspace(0, 20, 200, device="cuda").to(dtype)  # references that move
    q[..., 3] = q[..., 3].abs()
    top = torch.finfo(dtype).max
    V[0, 0, 199, 5], V[0, 1, 0, 9], V[1, 1, 44, 2] = top, top, -top
    _run_shared(kvc, q, Kp, Vp, K, V, ln, "values")


def test_shared_largest_values_of_float32(kvc):
    q, Kp, Vp, K, V, ln = _shared(kvc, F32, 300, d=64)
    top = torch.finfo(F32).max
    Vp[0, 3, 9], V[1, 1, 44, 2] = top, -top
    _run_shared(kvc, q, Kp, Vp, K, V, ln, "values")
    K[1, 0, 7, 11] = top
    q[1, :, :, 11] = -q[1, :, :, 11].abs() - 0.5
    _run_shared(kvc, q, Kp, Vp, K, V, ln, "keys")


@TYPES
@pytest.mark.parametrize("G", [1, 4, 8])
def test_blocks(kvc, dtype, G):
    d, cap, block = 64, 700, 32
    K, V, q = rand((2, 2, cap, d), dtype, 11), rand((2, 2, cap, d), dtype, 12), rand((2, 2 * G, 2, d), dtype, 13)
    ln = torch.tensor([[700, 650], [333, 31]], dtype=torch.int32, device="cuda")
    q[..., 7] = q[..., 7].abs() + 0.5
    V[0, 0, 17, 5], V[0, 0, 699, 6], V[0, 1, 640, 63], V[1, 1, 0, 0] = INF, -INF, NAN, INF
    K[1, 0, 100, 7] = -INF
    if dtype == F32:
        V[1, 0, 5, 1], K[1, 1, 3, 7] = torch.finfo(F32).max, -torch.finfo(F32).max
    dig = kvc.kv_block_digest(K, block, ln)
    for n_sel in (99, 6):
        o, lse, sel = kvc.kv_attn_blocks(q, K, V, ln, dig, block, n_sel, sink=1, recent=2)
        for b in range(2):
            for h in range(2):
                for t in range(2):
                    hs, seen = slice(G * h, G * h + G), int(ln[b, h]) - 1 + t
                    at = torch.cat([torch.arange(j * block, min(seen, (j + 1) * block)) for j in sel[b, h, t].tolist() if j >= 0]).cuda()
                    _check(o[b, hs, t], lse[b, hs, t], q[b, hs, t], K[b, h, at], V[b, h, at], d ** -0.5,
                           2.0 ** -16 if dtype == BF else 2.0 ** -20, f"n_sel {n_sel} b {b} h {h} t {t}")
