"""Argument checks of prompt attention and the 8-bit slot cache, without a GPU: refused calls
return before anything is launched."""
import ctypes

import pytest

P16 = 256  # an aligned address that is never used: the calls are refused before


@pytest.fixture(scope="module")
def api():
    from kv_cache_compression_obs_gb300.build import build
    build()
    from kv_cache_compression_obs_gb300 import api
    return api


def _cache(api, base=P16, **kw):
    f = dict(B=1, Hkv=2, cap=128, d=64, block=32, dtype=0, format=0)
    f.update({k: v for k, v in kw.items() if k in f})
    ptr = {n: base + 256 * i for i, n in enumerate(("K", "V", "Ks", "Vs", "Kt", "Vt", "pos", "acc", "len"))}
    ptr.update({k: v for k, v in kw.items() if k in ptr})
    return api._Q8Cache(*[ptr[n] for n in ("K", "V", "Ks", "Vs", "Kt", "Vt", "pos", "acc", "len")],
                        *[f[n] for n in ("B", "Hkv", "cap", "d", "block", "dtype", "format")])


BAD_CACHES = [(dict(cap=100), -1), (dict(cap=0), -1), (dict(block=48, cap=96), -2), (dict(block=16), -2), (dict(d=96), -2),
              (dict(dtype=3), -1), (dict(format=2), -1), (dict(B=-1), -1), (dict(Hkv=0), -1), (dict(K=0), -1),
              (dict(V=P16 + 8), -1), (dict(Ks=0), -1), (dict(Kt=P16 + 4), -1), (dict(pos=P16 + 2), -1), (dict(len=0), -1)]


@pytest.mark.parametrize("kw,want", BAD_CACHES, ids=str)
def test_bad_caches_are_refused_by_every_call(api, kw, want):
    lib, c, ok = api.library_handle(), _cache(api, **kw), _cache(api, 1 << 20)
    ref = ctypes.byref
    assert lib.kv_compact_q8(P16, P16, None, None, 64, 64, ref(c), None, None) == want
    assert lib.h2o_decode_step_q8(P16, P16, P16, ref(c), 2, 9, None, P16, 0.1, P16, P16, 1 << 40, None, None) == want
    assert lib.kv_evict_q8(ref(c), 20, 5, 0, P16, ref(ok), None, None) == want
    assert lib.kv_evict_q8(ref(ok), 20, 5, 0, P16, ref(c), None, None) == want


def test_compact_refusals(api):
    lib, c = api.library_handle(), ctypes.byref(_cache(api))
    call = lambda T, k, idx=P16, K=P16, out=c: lib.kv_compact_q8(K, P16, None, idx, T, k, out, None, None)  # noqa: E731
    assert call(10, 11) == -1                  # k > T
    assert call(10, 0) == -1
    assert call(0, 0) == -1
    assert call(200, 129) == -1                # k > cap
    assert call(100, 50, None) == -1           # every row, but k < T
    assert call(100, 50, K=P16 + 2) == -1      # alignment
    assert call(100, 50, K=None) == -1
    assert call(100, 50, out=None) == -1
    assert call(100, 50, out=ctypes.byref(_cache(api, B=0))) == 0


def test_decode_refusals(api):
    lib = api.library_handle()

    def call(Hq=4, new_pos=9, q=P16, ln=P16, scale=0.1, ws=P16, nbytes=1 << 40, row_pos=None, **kw):
        return lib.h2o_decode_step_q8(q, P16, P16, ctypes.byref(_cache(api, **kw)), Hq, new_pos, row_pos, ln, scale, P16,
                                      ws, nbytes, None, None)
    assert call(Hq=3) == -1
    assert call(Hq=0) == -1
    assert call(Hq=18) == -2                   # nine query heads a KV head
    assert call(new_pos=-1) == -1
    assert call(scale=float("nan")) == -1
    assert call(q=None) == -1
    assert call(q=P16 + 8) == -1
    assert call(ln=None) == -1
    assert call(ws=None, cap=1 << 17) == -5    # short caches need none
    assert call(nbytes=100, cap=1 << 17) == -5
    assert call(ws=P16 + 8, cap=1 << 17) == -5
    assert call(B=0) == 0
    assert lib.kv_workspace_size(8, 2, 8, 2, 1 << 17, 64, 0, 0) > 0
    assert lib.kv_workspace_size(8, 2, 8, 2, 128, 64, 0, 0) == 0
    assert lib.kv_workspace_size(8, 2, 7, 2, 128, 64, 0, 0) == 0


def test_evict_refusals(api):
    lib = api.library_handle()

    def call(keep=20, recent=5, sink=0, idx=P16, base=1 << 20, src={}, **kw):
        return lib.kv_evict_q8(ctypes.byref(_cache(api, **src)), keep, recent, sink, idx,
                               ctypes.byref(_cache(api, base, **kw)), None, None)
    assert call(keep=5) == -1                  # nothing left to choose
    assert call(keep=8, sink=3) == -1
    assert call(keep=2 ** 31 - 1, recent=2 ** 31 - 1, sink=2 ** 31 - 1) == -1
    assert call(recent=-1) == -1 and call(sink=-1) == -1
    assert call(keep=129) == -1                # more than the destination holds
    assert call(idx=None) == -1
    assert call(base=P16) == -1                # into itself
    assert call(V=P16 + 256) == -1             # one array in common
    assert call(acc=None) == -1 and call(src=dict(acc=None)) == -1
    for kw in (dict(B=2), dict(Hkv=3), dict(d=128), dict(block=64), dict(dtype=1), dict(format=1)):
        assert call(**kw) == -1, kw
    assert call(src=dict(B=0), B=0) == 0


def test_prompt_attention_refusals(api):
    lib = api.library_handle()

    def call(B=1, Hq=4, Hkv=2, Tq=10, Tk=10, d=64, st=None, sq=None, sk=None, n=0, scale=0.1, dt=0, q=P16, k=P16, o=P16,
             lse=P16):
        arr = None if st is None else (ctypes.c_int64 * 12)(*st)
        return lib.kv_attn_prompt(q, k, k, B, Hq, Hkv, Tq, Tk, d, arr, sq, sk, n, scale, dt, o, lse, None, 0, None, None)
    assert call(Hq=3) == -1 and call(Hkv=0) == -1 and call(Tq=-1) == -1 and call(dt=2) == -1
    assert call(d=96) == -2
    assert call(scale=float("nan")) == -1
    assert call(n=2) == -1                                        # packed without offsets
    assert call(n=2, sq=P16, sk=P16, B=2) == -1                   # packed in two rows
    assert call(n=-1) == -1
    assert call(q=None) == -1 and call(k=None) == -1 and call(o=None) == -1
    assert call(q=P16 + 4) == -1 and call(lse=P16 + 2) == -1 and call(sq=P16 + 1) == -1
    dense = [4 * 640, 640, 64, 2 * 640, 640, 64, 2 * 640, 640, 64, 4 * 640, 640, 64]
    for i, bad in ((1, 636), (4, 0), (5, -64), (11, 63), (8, 1 << 40)):
        st = list(dense)
        st[i] = bad
        assert call(st=st) == -1, (i, bad)
    assert call(B=0) == 0 and call(Tq=0) == 0                     # nothing to do
    assert lib.kv_workspace_size(7, 1, 7, 2, 128, 64, 128, 0) == 0


def test_binding_checks_shapes(api):
    import torch
    x = torch.zeros(1, 2, 8, 64)
    with pytest.raises(ValueError):
        api.kv_attn_prompt(x, x, x[:, :, :4])
    with pytest.raises(ValueError):
        api.kv_attn_prompt(x, x, x, packed=True)
    with pytest.raises(ValueError):
        api.kv_attn_prompt(x, x, x, seq_q=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        api.kv_attn_prompt(x, x, x)                               # not on a GPU
    with pytest.raises(ValueError):
        api.q8_cache(1, 2, 100, 64, 64, device="cpu")
    with pytest.raises(TypeError):
        api.q8_cache(1, 2, 128, 64, 64, codes=torch.uint8, device="cpu")
    c = api.q8_cache(1, 2, 128, 64, 64, device="cpu")
    with pytest.raises(ValueError):
        api.kv_compact_q8(x, x, None, None, c)                    # not on a GPU
    with pytest.raises(ValueError):
        api.kv_evict_q8(dict(c, acc=None), 10, 2, c)
    with pytest.raises(ValueError):
        api.h2o_decode_step_q8(x[:, :, 0], x[:, :, 0], x[:, :, 0], dict(c, pos=c["acc"]), 5)


@pytest.mark.parametrize("tq,W", [(10, 0), (10, 11), (9, 4)])
def test_binding_checks_the_observed_queries(api, tq, W):
    """More observed queries than the prompt has would be fewer, without a word."""
    import torch
    kv = torch.zeros(1, 2, 10, 64)
    with pytest.raises(ValueError):
        api.compress_prefill_q8(torch.zeros(1, 4, tq, 64), kv, kv, W=W, k=4, recent=2, r=None)
