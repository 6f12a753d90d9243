"""Pins of the float64 forms that the 8-bit cache and prompt attention are held to (CPU)."""
import math

import numpy as np
import pytest
import torch

from oracle import alg1, q8  # noqa: F401


def test_codes_are_the_nearest_values():
    r = np.random.default_rng(0)
    x = r.standard_normal((32, 64)).astype(np.float32)
    for fmt, values in (("s8", np.arange(-127, 128.0)),
                        ("e4m3", torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy())):
        values = np.sort(values[np.isfinite(values)].astype(np.float64))
        c, a = q8.quantise(x, fmt)
        assert a == np.float32(np.abs(x).max()) / np.float32(q8.TOP[fmt])
        assert np.isin(c, values).all() and np.abs(c).max() == q8.TOP[fmt]
        y = x.astype(np.float64) / np.float64(a)
        best = np.abs(y[..., None] - values).min(-1)
        assert (np.abs(y - c) <= best + 1e-4).all()


def test_e4m3_matches_the_type():
    y = torch.cat([torch.randn(4000) * 100, torch.randn(4000) * 0.01, torch.arange(-448, 449).float(),
                   torch.tensor([0.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 447.9, 0.0175])])
    y = y.clamp(-448, 448)
    np.testing.assert_array_equal(q8.to_e4m3(y.numpy()), y.to(torch.float8_e4m3fn).double().numpy())


def test_blocks_of_zeros_and_subnormals_have_a_scale():
    for x in (np.zeros((4, 4)), np.full((4, 4), 1e-44)):
        c, a = q8.quantise(x.astype(np.float32), "s8")
        assert a == np.float32(2.0 ** -126) and np.isfinite(c).all()


def test_attention_rows_by_hand():
    q = np.array([[1.0, 0.0], [0.0, 2.0], [1.0, 1.0]])
    k, v = np.array([[1.0, 0.0], [0.0, 1.0]]), np.array([[3.0, 0.0], [0.0, 5.0]])
    o, lse, _ = q8.attn_prompt(q, k, v, 1.0)
    assert (o[0] == 0).all() and lse[0] == -np.inf            # one key fewer than rows: the first sees none
    np.testing.assert_allclose(o[1], [3, 0])
    np.testing.assert_allclose(lse[1], 0)
    np.testing.assert_allclose(o[2], [1.5, 2.5])
    np.testing.assert_allclose(lse[2], 1 + math.log(2))


def test_decode_is_the_last_row_of_prompt_attention():
    r = np.random.default_rng(1)
    q, k, v = r.standard_normal((3, 8)), r.standard_normal((9, 8)), r.standard_normal((9, 8))
    o, p, _ = q8.decode(q, k, v, 0.3)
    np.testing.assert_allclose(p.sum(-1), 1)
    for g in range(3):
        np.testing.assert_allclose(o[g], q8.attn_prompt(q[g:g + 1], k, v, 0.3)[0][0])


@pytest.mark.parametrize("recent,sink", [(0, 0), (3, 0), (2, 4)])
def test_bulk_eviction_is_the_single_victims_in_turn(recent, sink):
    r = np.random.default_rng(2)
    acc, pos = np.floor(r.random(30) * 8), np.cumsum(r.integers(1, 3, 30)) - 1
    stay = q8.evict(acc, pos, 30, 12, recent, sink)
    free = [i for i in range(30) if i < 30 - recent and pos[i] >= sink]
    gone = sorted(free, key=lambda i: (acc[i], i))[:18]
    assert sorted(set(range(30)) - set(gone)) == stay.tolist()
    assert q8.evict(acc, pos, 10, 12, recent, sink).tolist() == list(range(10))
