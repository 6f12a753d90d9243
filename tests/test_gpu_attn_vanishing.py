"""A NaN in V reaches the rows that see its slot, however little they weigh it."""
import math

import pytest
import torch

from _long import BF, F32, rand

pytestmark = pytest.mark.gpu

TYPES = pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])


def _inputs(dtype, P, n, d=128):
    q, K, V = rand((2, 8, 1, d), dtype, 1).abs() + 0.5, rand((2, 2, n, d), dtype, 2), rand((2, 2, n, d), dtype, 3)
    return q, rand((2, P, d), dtype, 4), rand((2, P, d), dtype, 5), K, V, torch.full((2, 2), n, dtype=torch.int32, device="cuda")


@TYPES
@pytest.mark.parametrize("where", ["prefix", "own"])
@pytest.mark.parametrize("P", [100, 300, 5000])  # one key tile; two; many shares
def test_of_a_share_that_vanishes(kvc, dtype, where, P):
    q, Kp, Vp, K, V, ln = _inputs(dtype, P, 200)
    clean = kvc.kv_attn_shared(q, Kp, Vp, K, V, ln)
    assert clean[0].isfinite().all() and clean[1].isfinite().all()
    (K if where == "prefix" else Kp).add_(60.0)  # the other part's logits are about 900 below
    if where == "prefix":
        Vp[0, 10, 3] = math.nan
    else:
        V[:, 0, 10, 3] = math.nan
    o, lse = kvc.kv_attn_shared(q, Kp, Vp, K, V, ln)
    assert o[:, :4, 0, 3].isnan().all() and lse.isfinite().all()
    assert o[:, 4:].isfinite().all() and o[:, :4, 0, :3].isfinite().all() and o[:, :4, 0, 4:].isfinite().all()


@TYPES
def test_of_slots_that_weigh_nothing(kvc, dtype):
    """Logits below every number: their weights are 0, and 0 times a NaN is a NaN."""
    q, Kp, Vp, K, V, ln = _inputs(dtype, 300, 200)
    low = torch.finfo(dtype).min * 0.9  # times q's 0.5 and more in two channels: past float32
    K[0, 1, 32:48, :40], V[0, 1, 40, 9] = low, math.nan
    for o, lse in (kvc.kv_attn_shared(q, Kp, Vp, K, V, ln), kvc.kv_attn_shared(q, None, None, K, V, ln),
                   kvc.kv_attn_blocks(q, K, V, ln, kvc.kv_block_digest(K, 16), 16, 99)[:2]):
        assert o[0, 4:, 0, 9].isnan().all() and lse.isfinite().all() and int(o.isnan().sum()) == 4
