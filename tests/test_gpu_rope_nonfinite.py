"""Norm and rotary positions of heads with an infinity or a NaN in them: an element that does not turn
reaches no other one."""
import math

import pytest
import torch

from _long import BF, F32, HALF, rand

pytestmark = pytest.mark.gpu

EPS = 1e-5
BAD = (math.inf, -math.inf, math.nan)


def _want(x, f, pos, interleaved, eps):
    """x [B][H][T][d], pos [B][T] -> values and bounds, float64."""
    y = x.double()
    if eps is not None:
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps)
    m = 0 if f is None else f.numel()
    i = torch.arange(m, device=x.device)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + m)
    out, size = y.clone(), y.abs()
    if m:
        ang = pos.double()[:, None, :, None] * f
        a, b = y[..., ia], y[..., ib]
        out[..., ia], out[..., ib] = a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()
        size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return out, 2.0 ** -19 * size + HALF[x.dtype] * out.abs() + 1e-37


def _check(got, want, what):
    ref, bound = want
    got, fin = got.double(), ref.isfinite()
    assert torch.equal(got.isnan(), ref.isnan()), f"{what}: NaN in other places"
    assert torch.equal(got.isinf(), ref.isinf()) and torch.equal(got[ref.isinf()], ref[ref.isinf()]), f"{what}: infinities"
    assert bool(((got - ref).abs()[fin] <= bound[fin]).all()), what


# 200 tokens: a warp has some rows of a token; 2600: a token, or several groups of its rows (64/8 heads)
@pytest.mark.parametrize("T,Hq,Hkv", [(200, 3, 2), (2600, 3, 2), (2600, 64, 8)])
@pytest.mark.parametrize("d,rot", [(64, 0), (64, 32), (64, 24), (64, 64), (128, 32), (128, 2), (128, 104), (128, 128)])
@pytest.mark.parametrize("inter", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_one_bad_element(kvc, T, Hq, Hkv, d, rot, inter, dtype):
    """Token t has a bad element at place t of each head."""
    t = torch.arange(T, device="cuda")
    pos = (7 + 3 * t % 1009).int()[None]
    f = kvc.kv_rope_freqs(rot, 10000.0)[0] if rot else None
    for bad in BAD:
        q, k, v = (rand((1, h, T, d), dtype, 1 + i) for i, h in enumerate((Hq, Hkv, Hkv)))
        for x in (q, k, v):
            x[0, :, t, t % d] = bad
        for eps in (None, EPS):
            qo, ko, vo = kvc.kv_qk_norm_rope(q, k, v, f, pos, eps=eps, interleaved=inter)
            _check(qo, _want(q, f, pos, inter, eps), f"q {bad} {eps}")
            _check(ko, _want(k, f, pos, inter, eps), f"k {bad} {eps}")
            assert torch.equal(vo.isnan(), v.isnan()) and torch.equal(vo.nan_to_num(7.0), v.nan_to_num(7.0))


@pytest.mark.parametrize("inter", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rot", [0, 16, 20])
def test_what_does_not_turn_is_copied(kvc, dtype, rot, inter):
    """Without the norm, zeros keep their sign and the least and the largest values are what they were."""
    d, T = 64, 64
    k = torch.zeros(1, 2, T, d, dtype=dtype, device="cuda")
    k[0, 0] = -0.0
    k[0, 1, :, ::3], k[0, 1, :, 1::3] = torch.finfo(dtype).max, -torch.finfo(dtype).tiny
    f = kvc.kv_rope_freqs(rot)[0] if rot else None
    got = kvc.kv_qk_norm_rope(None, k, None, f, interleaved=inter)[1]
    word = torch.int16 if dtype == BF else torch.int32
    assert torch.equal(got[..., rot:].contiguous().view(word), k[..., rot:].contiguous().view(word))
