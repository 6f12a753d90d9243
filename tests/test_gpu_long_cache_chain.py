"""The operators around a long cache together, as a server calls them."""
import pytest
import torch

from _long import BF, F32, check_rows, choose, digests, rand

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _project(x, Hq, Hkv):
    """Queries, keys and values of a fused projection [B][n][Hq + 2 Hkv][d]."""
    return x.transpose(1, 2).split([Hq, Hkv, Hkv], 1)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_prompt_then_block_sparse_steps(kvc, dtype):
    """A prompt's heads into a cache, its attention and its digests, then decode steps in a captured graph."""
    B, Hq, Hkv, d, T, cap, block, n_sel, sink, recent = 2, 8, 2, 128, 700, 720, 32, 9, 1, 2
    f, scale = kvc.kv_rope_freqs(d, 500000.0, "bands", factor=4.0, low=1.0, high=4.0, context=256)
    wq, wk = (1 + 0.2 * rand((d,), F32, 1)).to(dtype), (1 + 0.2 * rand((d,), F32, 2)).to(dtype)
    K = torch.zeros(B, Hkv, cap, d, dtype=dtype, device="cuda")
    V, ln = torch.zeros_like(K), torch.zeros(B, Hkv, dtype=torch.int32, device="cuda")
    make = lambda x, pos, q_out=None: kvc.kv_qk_norm_rope(  # noqa: E731
        *_project(x, Hq, Hkv), f, pos, q_weight=wq, k_weight=wk, eps=EPS, rot_scale=scale, slot=ln, q_out=q_out, k_out=K, v_out=V)[0]
    x = rand((B, T, Hq + 2 * Hkv, d), dtype, 3)
    pos = torch.arange(T, dtype=torch.int32, device="cuda").expand(B, T).contiguous()
    q = make(x, pos)
    o, lse = kvc.kv_attn_prompt(q, K[:, :, :T], V[:, :, :T])
    ln += T
    for b, h, t in ((0, 0, 0), (0, 5, 350), (1, 7, T - 1)):
        check_rows(o[b, h, t:t + 1], lse[b, h, t:t + 1], q[b, h, t:t + 1], K[b, h // 4, :t + 1], V[b, h // 4, :t + 1], d ** -0.5,
                   2.0 ** -8 if dtype == BF else 2.0 ** -20, f"prompt {b} {h} {t}")
    dig = kvc.kv_block_digest(K, block, ln, out=torch.zeros(B, Hkv, -(-cap // block), 2, d, dtype=dtype, device="cuda"))
    x1, p1 = rand((B, 1, Hq + 2 * Hkv, d), dtype, 4), torch.full((B, 1), T, dtype=torch.int32, device="cuda")
    q1 = torch.zeros(B, Hq, 1, d, dtype=dtype, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        make(x1, p1, q1)
        ln += 1
        p1 += 1
        kvc.kv_block_digest(K, block, ln, n_new=1, out=dig)
        got = kvc.kv_attn_blocks(q1, K, V, ln, dig, block, n_sel, sink=sink, recent=recent)
        whole = kvc.kv_attn_blocks(q1, K, V, ln, dig, block, 99)
    for step in range(cap - T):
        x1.copy_(rand((B, 1, Hq + 2 * Hkv, d), dtype, 10 + step))
        g.replay()
        if step in (0, 3, 19):
            n = T + step + 1
            assert (ln == n).all()
            assert torch.equal(dig, digests(K, ln.tolist(), block, dig))
            for b in range(B):
                for h in range(Hkv):
                    hs = slice(4 * h, 4 * h + 4)
                    check_rows(whole[0][b, hs, 0], whole[1][b, hs, 0], q1[b, hs, 0], K[b, h, :n], V[b, h, :n], d ** -0.5,
                               2.0 ** -16 if dtype == BF else 2.0 ** -20, f"all blocks {b} {h}")
                    want = choose(q1[b, hs, 0].double(), dig[b, h].double(), n, block, n_sel, sink, recent)
                    assert got[2][b, h, 0].tolist() == want
                    at = torch.cat([torch.arange(j * block, min(n, (j + 1) * block)) for j in want]).cuda()
                    check_rows(got[0][b, hs, 0], got[1][b, hs, 0], q1[b, hs, 0], K[b, h, at], V[b, h, at], d ** -0.5,
                               2.0 ** -16 if dtype == BF else 2.0 ** -20, f"chosen blocks {b} {h}")


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_rows_behind_a_common_prefix(kvc, dtype):
    """One prefix prepared once, a chunk of each row's own prompt behind it, then steps."""
    B, Hq, Hkv, d, P, n, cap = 5, 8, 2, 64, 600, 7, 16
    f, _ = kvc.kv_rope_freqs(d)
    xp = rand((1, P, 2 * Hkv, d), dtype, 1).transpose(1, 2)
    _, Kp, Vp = kvc.kv_qk_norm_rope(None, xp[:, :Hkv], xp[:, Hkv:], f, eps=EPS)
    K = torch.full((B, Hkv, cap, d), float("nan"), dtype=dtype, device="cuda")
    V, ln = K.clone(), torch.zeros(B, Hkv, dtype=torch.int32, device="cuda")
    first = P
    for step, m in enumerate((n, 1, 2)):
        x = rand((B, m, Hq + 2 * Hkv, d), dtype, 2 + step)
        pos = (first + torch.arange(m, dtype=torch.int32, device="cuda")).expand(B, m).contiguous()
        q, _, _ = kvc.kv_qk_norm_rope(*_project(x, Hq, Hkv), f, pos, eps=EPS, slot=ln, k_out=K, v_out=V)
        ln += m
        first += m
        o, lse = kvc.kv_attn_shared(q, Kp[0], Vp[0], K, V, ln)
        own = first - P
        for b in range(B):
            for h in range(Hkv):
                for t in range(m):
                    s, hs = own - m + t + 1, slice(4 * h, 4 * h + 4)
                    check_rows(o[b, hs, t], lse[b, hs, t], q[b, hs, t], torch.cat((Kp[0, h], K[b, h, :s])),
                               torch.cat((Vp[0, h], V[b, h, :s])), d ** -0.5, 2.0 ** -8 if dtype == BF else 2.0 ** -20,
                               f"step {step} b {b} h {h} t {t}")


def test_compressed_prefix_shared(kvc):
    """The prefix may itself be what eviction kept of a prompt."""
    Hq, Hkv, d, T, k, B = 8, 2, 128, 900, 200, 3
    K, V, Q = rand((1, Hkv, T, d), BF, 1), rand((1, Hkv, T, d), BF, 2), rand((1, Hq, 16, d), BF, 3)
    kept = kvc.compress_prefill(Q, K, V, k, 16, 0.2)
    q = rand((B, Hq, 1, d), BF, 4)
    o, lse = kvc.kv_attn_shared(q, kept["K"][0], kept["V"][0], None, None, None)
    for b in range(B):
        for h in range(Hkv):
            hs = slice(4 * h, 4 * h + 4)
            check_rows(o[b, hs, 0], lse[b, hs, 0], q[b, hs, 0], kept["K"][0, h], kept["V"][0, h], d ** -0.5, 2.0 ** -8, f"{b} {h}")
