"""Own slots keep 16 bits of their weights in bf16, alone and behind a prefix: only the prefix's weights are rounded to bf16."""
import pytest
import torch

from _long import BF, HALF, attend, check_rows, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", [
    # B, Hq, Hkv, nq, cap, d
    (3, 10, 5, 2, 700, 128),
    (2, 16, 1, 3, 90, 64),
    (1, 4, 2, 1, 20000, 128),
    (40, 8, 4, 1, 333, 64),
], ids=str)
def test_own_slots_alone(kvc, case):
    B, Hq, Hkv, nq, cap, d = case
    q, K, V = rand((B, Hq, nq, d), BF, 1), rand((B, Hkv, cap, d), BF, 2), rand((B, Hkv, cap, d), BF, 3)
    g = torch.Generator().manual_seed(4)
    ln = torch.randint(nq, cap + 1, (B, Hkv), generator=g, dtype=torch.int32)
    o, lse = kvc.kv_attn_shared(q, None, None, K, V, ln.cuda())
    G = Hq // Hkv
    for b in range(B):
        for h in range(Hkv):
            for t in range(nq):
                n, hs = int(ln[b, h]) - nq + t + 1, slice(h * G, h * G + G)
                check_rows(o[b, hs, t], lse[b, hs, t], q[b, hs, t], K[b, h, :n], V[b, h, :n], d ** -0.5, 2.0 ** -16, f"{b} {h} {t}")


@pytest.mark.parametrize("up", [0.0, 0.5, 2.0])
def test_own_slots_behind_a_prefix(kvc, up):
    """The prefix's part of the weights counts with 2^-8, the own slots' with 2^-16; `up` lifts the own logits."""
    B, Hq, Hkv, P, cap, d = 4, 8, 2, 600, 250, 128
    q, Kp, Vp = rand((B, Hq, 1, d), BF, 11).abs(), rand((Hkv, P, d), BF, 12), rand((Hkv, P, d), BF, 13)
    K, V = (rand((B, Hkv, cap, d), BF, 14).float() + up).to(BF), rand((B, Hkv, cap, d), BF, 15)
    ln = torch.full((B, Hkv), cap, dtype=torch.int32, device="cuda")
    o, lse = kvc.kv_attn_shared(q, Kp, Vp, K, V, ln)
    for b in range(B):
        for h in range(Hkv):
            hs = slice(4 * h, 4 * h + 4)
            x = q[b, hs, 0].double()
            k, v = torch.cat((Kp[h], K[b, h])).double(), torch.cat((Vp[h], V[b, h])).double()
            want, wl, mass, A = attend(x, k, v, d ** -0.5)
            p = torch.exp(d ** -0.5 * (x @ k[:P].T) - wl[:, None])
            dl = 2.0 ** -18 * A
            bound = ((2 * dl + 2.0 ** -18 + 2.0 ** -16 + (P + cap) * 2.0 ** -27)[:, None] * mass + 2.0 ** -8 * (p @ v[:P].abs())
                     + HALF[BF] * want.abs() + 1e-37)
            err = (o[b, hs, 0].double() - want).abs()
            assert bool((err <= bound).all()), f"{b} {h}: {float((err / bound).max()):.2f} of its bound"
