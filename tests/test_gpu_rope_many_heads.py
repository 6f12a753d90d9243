"""Prompts whose tokens have more rows than one warp has sent for at once."""
import pytest
import torch

from _long import BF, F32, rand
from test_gpu_rope import EPS, _near, _want

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", [
    # B, T, Hq, Hkv, d, rot, interleaved, dtype
    (1, 5003, 64, 8, 128, 128, False, BF),
    (1, 3001, 64, 8, 128, 64, True, BF),
    (2, 2500, 32, 8, 128, 128, False, F32),
    (1, 4000, 33, 17, 128, 32, True, F32),
    (1, 6007, 96, 16, 64, 64, False, BF),
    (3, 1700, 71, 1, 128, 96, False, BF),
], ids=str)
def test_many_heads(kvc, case):
    B, T, Hq, Hkv, d, rot, inter, dtype = case
    q, k, v = rand((B, T, Hq + 2 * Hkv, d), dtype, 1).transpose(1, 2).split([Hq, Hkv, Hkv], 1)
    f, _ = kvc.kv_rope_freqs(rot)
    pos = (torch.arange(B * T, device="cuda") * 13 % 90001).int().view(B, T)
    wq, wk = (1 + 0.3 * rand((d,), F32, 2)).to(dtype), (1 + 0.3 * rand((d,), F32, 3)).to(dtype)
    slot = torch.arange(B * Hkv, dtype=torch.int32, device="cuda").view(B, Hkv) % 5
    seq = torch.tensor([T - 3 * b for b in range(B)], dtype=torch.int32, device="cuda")
    K, V = torch.full((B, Hkv, T + 4, d), 3.0, dtype=dtype, device="cuda"), torch.full((B, Hkv, T + 4, d), 4.0, dtype=dtype, device="cuda")
    qo = torch.full((B, Hq, T, d), 5.0, dtype=dtype, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvc.kv_qk_norm_rope(q, k, v, f, pos, q_weight=wq, k_weight=wk, eps=EPS, interleaved=inter, slot=slot, seq=seq, q_out=qo, k_out=K,
                        v_out=V, dev_status=st)
    assert int(st) == 0
    wantq, wantk = (_want(x, w, f, pos, inter, EPS, False, 1.0) for x, w in ((q, wq), (k, wk)))
    for b in range(B):
        n = int(seq[b])
        _near(qo[b, :, :n], (wantq[0][b, :, :n], wantq[1][b, :, :n]), f"q {b}")
        assert (qo[b, :, n:] == 5).all()
        for h in range(Hkv):
            s = int(slot[b, h])
            _near(K[b, h, s:s + n], (wantk[0][b, h, :n], wantk[1][b, h, :n]), f"k {b} {h}")
            assert torch.equal(V[b, h, s:s + n], v[b, h, :n])
            assert (K[b, h, :s] == 3).all() and (K[b, h, s + n:] == 3).all() and (V[b, h, s + n:] == 4).all()
