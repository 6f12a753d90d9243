"""Argument checks of rotary positions, block digests, block-sparse and shared-prefix attention, without a GPU:
refused calls return before anything is launched."""
import ctypes
import math

import pytest

P16 = 256  # an aligned address that is never used: the calls are refused before


@pytest.fixture(scope="module")
def api():
    from kv_cache_compression_obs_gb300.build import build
    build()
    from kv_cache_compression_obs_gb300 import api
    return api


def _heads(api, strides=None, **kw):
    f = dict(q=P16, k=P16, v=P16, q_out=P16, k_out=P16, v_out=P16, q_weight=P16, k_weight=P16, inv_freq=P16, pos=P16, slot=P16,
             seq=P16, B=2, Hq=4, Hkv=2, T=3, cap=8, d=64, rot=64, eps=1e-6, rot_scale=1.0, flags=2, dtype=0)
    f.update(kw)
    st = (ctypes.c_int64 * 18)(*(strides or [4096, 256, 64] * 6))
    return api._QkvHeads(*[f[n] for n in ("q", "k", "v", "q_out", "k_out", "v_out", "q_weight", "k_weight", "inv_freq", "pos",
                                          "slot", "seq")], st,
                         *[f[n] for n in ("B", "Hq", "Hkv", "T", "cap", "d", "rot", "eps", "rot_scale", "flags", "dtype")])


NONE = dict(q=None, k=None, v=None, q_out=None, k_out=None, v_out=None)


@pytest.mark.parametrize("kw,want", [
    (dict(d=96), -2), (dict(rot=65), -1), (dict(rot=66), -1), (dict(rot=-2), -1), (dict(dtype=2), -1), (dict(B=-1), -1),
    (dict(T=-1), -1), (dict(Hq=0), -1), (dict(Hkv=0), -1), (dict(eps=-1.0), -1), (dict(eps=math.inf), -1), (dict(eps=math.nan), -1),
    (dict(rot_scale=math.nan), -1), (dict(flags=8), -1), (dict(q_out=None), -1), (dict(q=None), -1), (dict(k=P16 + 8), -1),
    (dict(v_out=P16 + 2), -1), (dict(inv_freq=None), -1), (dict(inv_freq=P16 + 4), -1), (dict(pos=P16 + 2), -1),
    (dict(slot=P16 + 1), -1), (dict(seq=P16 + 1), -1), (dict(q_weight=P16 + 8), -1), (dict(k_weight=P16 + 2), -1), (dict(strides=[4096, 256, 60] * 6), -1),
    (dict(strides=[4096, 256, 64] * 3 + [0, 256, 64] * 3), -1), (dict(strides=[-4096, 256, 64] * 6), -1),
    (dict(B=0), 0), (dict(T=0), 0), (NONE, 0), (dict(cap=-1), -1)], ids=str)
def test_heads_refusals(api, kw, want):
    kw = dict(kw)
    assert api.library_handle().kv_qk_norm_rope(ctypes.byref(_heads(api, **kw)), None, None) == want
    assert api.library_handle().kv_qk_norm_rope(None, None, None) == -1


def test_frequencies(api):
    """Against the formulas, and refusals."""
    rot, theta, ctx, f = 64, 500000.0, 8192.0, 8.0
    plain = [theta ** (-2 * i / rot) for i in range(rot // 2)]
    got, scale = api.kv_rope_freqs(rot, theta, device="cpu")
    near = lambda a, b: all(abs(x - y) <= 1e-13 * abs(y) for x, y in zip(a.tolist(), b))  # noqa: E731
    assert near(got, plain) and scale == 1.0 and len(got) == 32
    assert near(api.kv_rope_freqs(rot, theta, "linear", f, device="cpu")[0], [x / f for x in plain])
    base = api.kv_rope_freqs(rot, theta, "base", f, device="cpu")[0]
    assert near(base, [(theta * f ** (rot / (rot - 2))) ** (-2 * i / rot) for i in range(32)])
    assert abs(base[-1].item() * f / plain[-1] - 1) < 1e-12
    bands = []
    for x in plain:
        keep = min(1.0, max(0.0, (ctx * x / (2 * math.pi) - 1.0) / (4.0 - 1.0)))
        bands.append(x * keep + x / f * (1 - keep))
    assert near(api.kv_rope_freqs(rot, theta, "bands", f, 1.0, 4.0, ctx, device="cpu")[0], bands)
    at = lambda turns: rot * math.log(ctx / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
    first, last = max(0, math.floor(at(32.0))), min(rot - 1, math.ceil(at(1.0)))
    ramp = [min(1.0, max(0.0, (i - first) / (last - first))) for i in range(32)]
    got, scale = api.kv_rope_freqs(rot, theta, "yarn", f, 1.0, 32.0, ctx, device="cpu")
    assert near(got, [x * (1 - r) + x / f * r for x, r in zip(plain, ramp)])
    assert abs(scale - (0.1 * math.log(f) + 1)) < 1e-6
    assert api.kv_rope_freqs(0, device="cpu")[0].numel() == 0
    for bad in (dict(rot=63), dict(rot=-2), dict(rot=8, theta=-1.0), dict(rot=8, theta=math.inf),
                dict(rot=8, scaling="linear", factor=0.5), dict(rot=8, scaling="bands", low=2.0, high=2.0),
                dict(rot=8, scaling="yarn", context=0.0), dict(rot=8, theta=1.0, scaling="yarn")):
        with pytest.raises(api.KvcError):
            api.kv_rope_freqs(**bad, device="cpu")
    with pytest.raises(ValueError):
        api.kv_rope_freqs(8, scaling="other", device="cpu")


@pytest.mark.parametrize("kw,want", [
    (dict(d=32), -2), (dict(block=24), -2), (dict(block=256), -2), (dict(block=0), -2), (dict(dtype=3), -1), (dict(B=-1), -1),
    (dict(Hkv=0), -1), (dict(cap=0), -1), (dict(n_new=0), -1), (dict(K=None), -1), (dict(K=P16 + 8), -1), (dict(digest=None), -1),
    (dict(digest=P16 + 8), -1), (dict(ln=P16 + 2), -1), (dict(B=0), 0), (dict(B=1 << 30, Hkv=1 << 30, cap=1 << 30), -1)], ids=str)
def test_digest_refusals(api, kw, want):
    f = dict(K=P16, ln=P16, B=1, Hkv=2, cap=100, d=64, block=32, n_new=1, dtype=0, digest=P16)
    f.update(kw)
    assert api.library_handle().kv_block_digest(*f.values(), None, None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(Hq=5), -1), (dict(Hq=18), -2), (dict(d=96), -2), (dict(block=48), -2), (dict(cap=16 * 12289, block=16), -2), (dict(nq=-1), -1),
    (dict(cap=0), -1), (dict(n_sel=2), -1), (dict(sink=-1), -1), (dict(recent=0), -1), (dict(scale=0.0), -1), (dict(scale=-1.0), -1),
    (dict(scale=math.inf), -1), (dict(scale=math.nan), -1), (dict(dtype=2), -1), (dict(q=None), -1), (dict(V=P16 + 8), -1),
    (dict(digest=None), -1), (dict(ln=None), -1), (dict(o=P16 + 4), -1), (dict(lse=P16 + 2), -1), (dict(sel=P16 + 2), -1),
    (dict(strides=[512, 128, 60, 512, 128, 64]), -1), (dict(strides=[512, 128, 64, 0, 128, 64]), -1), (dict(B=0), 0), (dict(nq=0), 0)],
    ids=str)
def test_blocks_refusals(api, kw, want):
    f = dict(q=P16, K=P16, V=P16, ln=P16, digest=P16, B=2, Hq=4, Hkv=2, nq=2, cap=100, d=64, block=32, n_sel=3, sink=1, recent=2,
             strides=None, scale=0.1, dtype=0, o=P16, lse=P16, sel=P16)
    f.update(kw)
    if f["strides"]:
        f["strides"] = (ctypes.c_int64 * 6)(*f["strides"])
    assert api.library_handle().kv_attn_blocks(*f.values(), None, None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(Hq=5), -1), (dict(d=96), -2), (dict(nq=-1), -1), (dict(P=-1), -1), (dict(cap=-1), -1), (dict(scale=0.0), -1),
    (dict(scale=math.nan), -1), (dict(dtype=2), -1), (dict(q=None), -1), (dict(Kp=None), -1), (dict(Vp=P16 + 8), -1), (dict(K=None), -1),
    (dict(ln=None), -1), (dict(ln=P16 + 2), -1), (dict(o=None), -1), (dict(lse=P16 + 2), -1), (dict(ws=None), -5), (dict(nbytes=64), -5),
    (dict(ws=P16 + 8), -5), (dict(strides=[512, 128, 64, 640, 60, 640, 64, 512, 128, 64]), -1),
    (dict(strides=[512, 128, 64, 640, 64, 640, -64, 512, 128, 64]), -1), (dict(B=0), 0), (dict(nq=0), 0),
    (dict(B=1 << 20, nq=1 << 12), -1), (dict(B=1 << 16, cap=1 << 20), -2)], ids=str)
def test_shared_refusals(api, kw, want):
    f = dict(q=P16, Kp=P16, Vp=P16, K=P16, V=P16, ln=P16, B=2, Hq=4, Hkv=2, nq=2, P=10, cap=20, d=64, strides=None, scale=0.1, dtype=0,
             o=P16, lse=P16, ws=P16, nbytes=1 << 40)
    f.update(kw)
    if f["strides"]:
        f["strides"] = (ctypes.c_int64 * 10)(*f["strides"])
    assert api.library_handle().kv_attn_shared(*f.values(), None, None) == want


def test_shared_workspace(api):
    size = lambda B, Hq, Hkv, P, d, nq: api.kv_workspace_size(api.KV_OP_ATTN_SHARED, B, Hq, Hkv, max(1, P), d, nq, P)  # noqa: E731
    assert size(64, 32, 8, 32768, 128, 1) >= 64 * 32 * 128 * 4
    assert size(2, 4, 2, 0, 64, 1) > 0          # the own slots' shares
    assert size(2, 4, 3, 10, 64, 1) == 0 and size(2, 4, 2, 10, 96, 1) == 0 and size(1 << 30, 8, 2, 10, 64, 1) == 0


def test_binding_refusals(api):
    """What the binding itself refuses, on CPU tensors: nothing is passed on."""
    import torch
    q, k, v = (torch.zeros(2, h, 3, 64, dtype=torch.bfloat16) for h in (4, 2, 2))
    with pytest.raises(ValueError):
        api.kv_qk_norm_rope(None, None, None, None)
    for call in (lambda: api.kv_qk_norm_rope(q, k, v, None), lambda: api.kv_block_digest(k, 16),
                 lambda: api.kv_attn_blocks(q, k, v, torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2, 1, 2, 64), 16, 2),
                 lambda: api.kv_attn_shared(q, k[0], v[0], None, None, None)):
        with pytest.raises(ValueError):
            call()


def test_binding_plans(api):
    """The binding's checks of shapes, strides and types."""
    import torch
    sig = lambda *ts: tuple(None if t is None else (t.shape, t.stride(), t.dtype, 0) for t in ts)  # noqa: E731
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)  # noqa: E731
    i32 = torch.int32
    q, k = z(2, 4, 3, 64), z(2, 2, 3, 64)
    good = dict(q=q, k=k, v=k, q_out=q, k_out=k, v_out=k, f=z(32, dtype=torch.float64), pos=z(2, 3, dtype=i32), wq=z(64), wk=z(64),
                slot=z(2, 2, dtype=i32), seq=z(2, dtype=i32), st=None)
    assert api._rope_plan(sig(*good.values()))[1:] == (2, 4, 2, 3, 3, 64, 64, 0, 0)
    for name, t in dict(k=z(2, 2, 4, 64), v=z(2, 3, 3, 64), q_out=z(2, 4, 4, 64), k_out=z(2, 3, 3, 64), f=z(32), pos=z(2, 3),
                        wq=z(32), slot=z(2, 3, dtype=i32), seq=z(3, dtype=i32), v_out=z(2, 2, 5, 64)).items():
        with pytest.raises(ValueError):
            api._rope_plan(sig(*{**good, name: t}.values()))
    on_two = sig(*good.values())
    for dev in (1, -1):
        with pytest.raises(ValueError):
            api._rope_plan(on_two[:1] + (on_two[1][:3] + (dev,),) + on_two[2:])
    with pytest.raises(TypeError):
        api._rope_plan(sig(*[z(2, 2, 3, 64, dtype=torch.float16)] * 6, *[None] * 7))
    K, ln, dig = z(2, 2, 100, 64), z(2, 2, dtype=i32), z(2, 2, 7, 2, 64)
    good = dict(q=q, K=K, V=K, ln=ln, dig=dig, o=None, lse=None, sel=None, st=None)
    assert api._blocks_plan(sig(*good.values()), 16, 4)[:7] == (2, 4, 2, 3, 100, 64, 0)
    for name, t in dict(K=z(2, 2, 90, 64), V=z(2, 2, 100, 64).transpose(0, 1), ln=z(2, 2), dig=z(2, 2, 6, 2, 64), o=z(2, 4, 4, 64),
                        lse=z(2, 4, 3), sel=z(2, 2, 3, 5, dtype=i32)).items():
        with pytest.raises(ValueError):
            api._blocks_plan(sig(*{**good, name: t}.values()), 16, 4)
    with pytest.raises(ValueError):
        api._blocks_plan(sig(*good.values()), 0, 4)
    Kp = z(2, 50, 64)
    good = dict(q=q, kp=Kp, vp=Kp, K=K, V=K, ln=ln, o=None, lse=None, ws=None, st=None)
    assert api._shared_plan(sig(*good.values()))[:7] == (2, 4, 2, 3, 50, 100, 64)
    for name, t in dict(kp=z(3, 50, 64), vp=z(2, 51, 64), K=None, ln=None, V=z(2, 2, 99, 64), q=z(3, 4, 3, 64)).items():
        with pytest.raises(ValueError):
            api._shared_plan(sig(*{**good, name: t}.values()))
