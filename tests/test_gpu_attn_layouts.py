"""Prompt attention with every tensor in a layout of its own, and two calls at once."""
import pytest
import torch

from _q8 import same_bits

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _lay(kind, B, H, T, d, dtype):
    """[B][H][T][d] over other memory: rows of d + 8 elements stand on 16-byte boundaries only."""
    e = lambda *s: torch.full(s, 9.0, dtype=dtype, device="cuda")  # noqa: E731
    return {"dense": lambda: e(B, H, T, d), "token": lambda: e(B, T, H, d).transpose(1, 2),
            "heads first": lambda: e(H, B, T, d).transpose(0, 1),
            "slice": lambda: e(B, H, T + 3, d + 8)[:, :, 2:T + 2, 8:]}[kind]()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("shape", [(2, 4, 2, 200, 230, 64), (1, 3, 1, 300, 300, 128), (2, 8, 2, 9, 4000, 128)], ids=str)
def test_layouts_give_the_same_bits(kvc, dtype, shape):
    """Inputs and the output in any strides: the dense call's bits, and nothing written beside the rows."""
    B, Hq, Hkv, Tq, Tk, d = shape
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    q, k, v = (torch.randn(B, h, t, d, generator=g, device="cuda").to(dtype) for h, t in ((Hq, Tq), (Hkv, Tk), (Hkv, Tk)))
    want, lse = kvc.kv_attn_prompt(q, k, v)
    kinds = ["dense", "token", "heads first", "slice"]
    for i in range(4):
        a = [_lay(kinds[(i + j) % 4], B, h, t, d, dtype).copy_(x)
             for j, (x, h, t) in enumerate(((q, Hq, Tq), (k, Hkv, Tk), (v, Hkv, Tk)))]
        out = _lay(kinds[(i + 3) % 4], B, Hq, Tq, d, dtype)
        o, l2 = kvc.kv_attn_prompt(*a, out=out)
        torch.cuda.synchronize()
        assert o is out and same_bits(o, want) and same_bits(l2, lse)
        if kinds[(i + 3) % 4] == "slice":
            assert (out._base[..., :8] == 9).all() and (out._base[:, :, :2] == 9).all() and (out._base[:, :, -1] == 9).all()


def test_two_prompts_and_a_scoring_at_once(kvc):
    """Kernels that hold tensor memory side by side on three streams: the bits of calls one after the other."""
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    ins = []
    for Hq, Hkv, T, d in ((16, 4, 1500, 128), (8, 8, 2000, 64)):
        ins.append([torch.randn(1, h, T, d, generator=g, device="cuda").to(BF) for h in (Hq, Hkv, Hkv)])
    want = [kvc.kv_attn_prompt(*x) for x in ins]
    q, k = ins[0][0][:, :, -64:].contiguous(), ins[0][1]
    s = kvc.kv_score_obs(q, k)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got, scores = [[], []], []
    for _ in range(8):
        for i in range(2):
            got[i].append(kvc.kv_attn_prompt(*ins[i], stream=streams[i]))
        with torch.cuda.stream(streams[2]):
            scores.append(kvc.kv_score_obs(q, k))
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in got[i]:
            assert same_bits(o, want[i][0]) and same_bits(lse, want[i][1])
    assert all(same_bits(x, s) for x in scores)
