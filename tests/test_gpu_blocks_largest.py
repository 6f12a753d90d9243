"""As many blocks as block-sparse attention takes, with one CTA a unit: its largest shared memory."""
import pytest
import torch

from _long import BF, check_rows, choose, rand

pytestmark = pytest.mark.gpu


def test_as_many_blocks_as_there_may_be_and_one_cta_a_unit(kvc):
    """12288 blocks, eight queries a head and more units than the GPU holds CTAs: the largest shared memory."""
    d, block, nb, nq, H = 128, 16, 12288, 250, 2
    K, V = rand((1, H, nb * block, d), BF, 40), rand((1, H, nb * block, d), BF, 41)
    K[0, 1] *= 0.01
    q = rand((1, 8 * H, nq, d), BF, 42)
    ln = torch.tensor([[nb * block, nb * block - 9]], dtype=torch.int32)
    dig = kvc.kv_block_digest(K, block, ln.cuda())
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse, sel = kvc.kv_attn_blocks(q, K, V, ln.cuda(), dig, block, 40, sink=2, recent=2, dev_status=st)
    assert int(st) == 0
    for h in range(H):
        for t in (0, 1, 123, 248, 249):
            hs, seen = slice(8 * h, 8 * h + 8), int(ln[0, h]) - nq + t + 1
            want = choose(q[0, hs, t].double(), dig[0, h].double(), seen, block, 40, 2, 2)
            assert sel[0, h, t].tolist() == want, f"h {h} t {t}"
            at = torch.cat([torch.arange(j * block, min(seen, (j + 1) * block)) for j in want]).cuda()
            check_rows(o[0, hs, t], lse[0, hs, t], q[0, hs, t], K[0, h, at], V[0, h, at], d ** -0.5, 2.0 ** -16, f"h {h} t {t}")
