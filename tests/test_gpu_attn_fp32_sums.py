"""float32 logits whose terms cancel: their sums round where the tensor cores would cut off.

Channel 0 adds 64 * 64 = 2^12 to every logit and the last channel takes it away again; the 15 channels that share a step of 16
with each are 0, so that the two products are exact.  In between the sum is near 2^12.  Steps of 16 channels are joined two by
two and these one after the other, d / 32 additions that are off by half a step of 2^12 each at most, 2^-12:  with the small
products' 2^-17 (terms of about 60 in all, each to 2^-23) and 2^-19 for the rest a logit (and with it lse) is off by
less than d / 32 2^-12 + 2^-16.  Cut off at each step it would be off by 2^-12 for each on average, all to the same side."""
import pytest
import torch

from _long import F32, rand

pytestmark = pytest.mark.gpu


def _inputs(d, n, seed, B=2, Hkv=2, G=4):
    q, K, V = rand((B, Hkv * G, 1, d), F32, seed), rand((B, Hkv, n, d), F32, seed + 1), rand((B, Hkv, n, d), F32, seed + 2)
    for x in (q, K):
        x[..., :16] = 0
        x[..., -16:] = 0
        x[..., 0], x[..., -1] = 64.0, 64.0
    K[..., -1] = -64.0
    return q, K, V, torch.full((B, Hkv), n, dtype=torch.int32, device="cuda")


def _check(q, K, V, o, lse, what):
    G, d = q.shape[1] // K.shape[1], q.shape[3]
    bound = d / 32 * 2.0 ** -12 + 2.0 ** -16
    x = q.double().squeeze(2).unflatten(1, (-1, G)) @ K.double().transpose(-1, -2)
    err = (lse.double().squeeze(2).unflatten(1, (-1, G)) - x.logsumexp(-1)).abs().max()
    assert float(err) <= bound + 2.0 ** -22 * float(x.abs().max()), f"{what}: lse off by {float(err):.2e}"
    p = (x - x.logsumexp(-1, keepdim=True)).exp()
    got = o.double().squeeze(2).unflatten(1, (-1, G))
    assert bool(((got - p @ V.double()).abs() <= (2 * bound + 2.0 ** -18) * (p @ V.double().abs())).all()), f"{what}: o"


@pytest.mark.parametrize("d", [64, 128])
def test_blocks(kvc, d):
    q, K, V, ln = _inputs(d, 900, 1)
    o, lse, _ = kvc.kv_attn_blocks(q, K, V, ln, kvc.kv_block_digest(K, 32), 32, 99, scale=1.0)
    _check(q, K, V, o, lse, "blocks")


@pytest.mark.parametrize("d", [64, 128])
def test_shared(kvc, d):
    q, K, V, ln = _inputs(d, 700, 11)
    o, lse = kvc.kv_attn_shared(q, None, None, K, V, ln, scale=1.0)
    _check(q, K, V, o, lse, "own slots")
    o, lse = kvc.kv_attn_shared(q, K[1], V[1], None, None, None, scale=1.0)
    _check(q, K[1].expand(2, -1, -1, -1), V[1].expand(2, -1, -1, -1), o, lse, "prefix")
