"""Prompt attention whose keys are shared out, in a workspace of exactly the size asked for."""
import pytest
import torch

from _q8 import same_bits

pytestmark = pytest.mark.gpu

BF = torch.bfloat16

SHAPES = [
    # B, Hq, Hkv, Tq, Tk, d
    (1, 32, 8, 1300, 9000, 64),      # the last, partial round of tiles
    (1, 32, 8, 2500, 5100, 128),
    (3, 32, 8, 400, 6000, 128),      # ... of a batch: the split tiles are its last row's
    (1, 9, 1, 5000, 11000, 64),      # tiles of 256 rows of one head, the last of them partly filled
    (1, 32, 8, 16, 9000, 128),       # few rows: all tiles
    (2, 3, 1, 77, 5000, 64),
]


@pytest.mark.parametrize("case", SHAPES, ids=str)
def test_stays_inside_its_workspace(kvc, case):
    """What stands behind the workspace is not touched, whatever stood in it does not matter, and rows of
    padded sequences come out as those of calls of their own."""
    B, Hq, Hkv, Tq, Tk, d = case
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    Q, K, V = (torch.randn(B, h, t, d, generator=g, device="cuda").to(BF) for h, t in ((Hq, Tq), (Hkv, Tk), (Hkv, Tk)))
    need = kvc.kv_workspace_size(kvc.KV_OP_ATTN_PROMPT, B, Hq, Hkv, Tk, d, Tq, 0)
    assert need > 0
    # at every alignment that the call takes
    for shift, fill in ((0, 0xFF), (16, 0x7F)):
        room = torch.full((need + shift + 4096,), fill, dtype=torch.uint8, device="cuda")
        o, lse = kvc.kv_attn_prompt(Q, K, V, workspace=room[shift:shift + need])
        torch.cuda.synchronize()
        assert (room[shift + need:] == fill).all() and (room[:shift] == fill).all()
        o2, lse2 = kvc.kv_attn_prompt(Q, K, V)
        assert same_bits(o, o2) and same_bits(lse, lse2)
    # lengths of its own in each batch row, none in the first
    lens = torch.tensor([0] + [Tq - 3] * (B - 1) if B > 1 else [Tq - 130 if Tq > 130 else 1], dtype=torch.int32, device="cuda")
    keys = (lens + (Tk - Tq)).to(torch.int32)
    out, l3 = torch.full_like(Q, 5.0), torch.full((B, Hq, Tq), 5.0, device="cuda")
    kvc.kv_attn_prompt(Q, K, V, seq_q=lens, seq_k=keys, out=out, lse_out=l3)
    torch.cuda.synchronize()
    for b in range(B):
        n, m = int(lens[b]), int(keys[b])
        assert (out[b, :, n:] == 5).all() and (l3[b, :, n:] == 5).all()
        if n == 0:
            continue
        hidden = ~torch.ones((n, m), dtype=torch.bool, device="cuda").tril(m - n)
        for h in (0, Hq - 1):
            x = (Q[b, h, :n].double() @ K[b, h // (Hq // Hkv), :m].double().T * d ** -0.5).masked_fill(hidden, float("-inf"))
            want = x.softmax(-1) @ V[b, h // (Hq // Hkv), :m].double()
            # weights and the result rounded to bf16, half a step of 2^-8 each, and fp32 sums
            mass = x.softmax(-1) @ V[b, h // (Hq // Hkv), :m].double().abs()
            err = (out[b, h, :n].double() - want).abs()
            assert (err <= (2.0 ** -8 + 2.0 ** -12) * mass + 2.0 ** -8 * want.abs() + 1e-30).all()
            wl = x.logsumexp(-1)
            assert ((l3[b, h, :n] - wl).abs() <= 2.0 ** -13 + 2.0 ** -22 * wl.abs()).all()
