"""The cases on which the operators around a long cache are measured.

Four operators, in the order in which a server calls them:

  rope     the heads of a projection made ready: RMS norm of each query and key head, rotary positions,
           queries laid out by head, keys and values written into the slots of a cache;
  digest   per block of cache slots and channel the least and the largest key;
  blocks   attention of one or a few new tokens per row over the blocks that their digests choose;
  shared   attention of a batch over one common prefix and each row's own slots.

The formulas:
  rope     y = x w / sqrt(mean x^2 + eps); the pair (a, b) = (y_i, y_{i + rot/2}) (or (y_2i, y_{2i+1})) turns by
           pos f_i: (a cos - b sin, b cos + a sin) times the rotation's scale; what is behind rot stays y;
  blocks   u_j = max over a group's queries g of sum_c q_gc (q_gc >= 0 ? top_jc : low_jc), which no logit of
           block j passes; the first `sink` and last `recent` blocks of those that a token sees and the best of
           the others by (u descending, j ascending) up to n_sel; softmax over the slots that it sees of these;
  shared   softmax over the prefix and the row's own slots.  The n new tokens of a row are its last n slots:
           token t sees the slots j <= t + len - n.
"""
import math

import numpy as np
import torch

own = False

BF16, F32 = "bf16", "f32"
TYPE = {BF16: torch.bfloat16, F32: torch.float32}
EPS = 1e-6
SINKS = 4


def listed():
    return [
        # one new token of one request, far behind a long context: latency
        dict(name="rope-token", op="rope", B=1, T=1, Hq=32, Hkv=8, d=128, rot=128, pairs="half", dtype=BF16, far=131071,
             factor=1.0, norm=True, cap=4096),
        # the new tokens of 64 requests, positions scaled for a longer context
        dict(name="rope-batch", op="rope", B=64, T=1, Hq=32, Hkv=8, d=128, rot=128, pairs="half", dtype=BF16, far=500000,
             factor=8.0, norm=True, cap=1024),
        # a float32 prompt of odd length, half of each head turned, neighbours as pairs
        dict(name="rope-part", op="rope", B=2, T=1237, Hq=4, Hkv=4, d=64, rot=32, pairs="next", dtype=F32, far=0, factor=1.0,
             norm=True, cap=1237),
        # the long prompt of the grouped-head prefill configuration, from the projection's layout to the cache's
        dict(name="rope-prompt", op="rope", B=1, T=32768, Hq=32, Hkv=8, d=128, rot=128, pairs="half", dtype=BF16, far=0,
             factor=1.0, norm=True, cap=32768),
        # after a decode step: the one block of each head that the new token is in
        dict(name="digest-step", op="digest", B=8, H=8, cap=32768, least=20000, most=32768, d=128, block=64, n_new=1, dtype=BF16),
        # after prefill: every block of eight 32K prompts, odd ends
        dict(name="digest-prompt", op="digest", B=8, H=8, cap=32768, least=31000, most=32768, d=128, block=64, n_new=32768,
             dtype=BF16),
        # one request of 8K tokens: latency
        dict(name="blocks-short", op="blocks", B=1, Hq=32, Hkv=8, nq=1, cap=8192, least=8000, most=8191, d=128, block=32, n_sel=32,
             sink=1, recent=2, dtype=BF16),
        # five drafted tokens a row, every head with its own keys, different lengths
        dict(name="blocks-draft", op="blocks", B=2, Hq=32, Hkv=32, nq=5, cap=16384, least=900, most=16001, d=128, block=64, n_sel=24,
             sink=1, recent=2, dtype=BF16),
        # eight requests of 128K tokens, a 32nd of the blocks
        dict(name="blocks-long", op="blocks", B=8, Hq=32, Hkv=8, nq=1, cap=131072, least=120000, most=131071, d=128, block=64,
             n_sel=64, sink=1, recent=4, dtype=BF16),
        # four requests behind a 4K system prompt, few tokens of their own: latency
        dict(name="shared-few", op="shared", B=4, Hq=32, Hkv=8, nq=1, P=4096, cap=512, least=40, most=500, d=128, dtype=BF16),
        # three drafted tokens a row, every head with its own keys, odd lengths
        dict(name="shared-draft", op="shared", B=24, Hq=32, Hkv=32, nq=3, P=8191, cap=1024, least=3, most=1001, d=128, dtype=BF16),
        # 64 requests behind a 32K prefix
        dict(name="shared-many", op="shared", B=64, Hq=32, Hkv=8, nq=1, P=32768, cap=2048, least=200, most=2047, d=128, dtype=BF16),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "digest", "blocks", "shared"])
    d = rng.choice([64, 128, 128])
    dtype = rng.choice([BF16, BF16, BF16, F32])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    G = rng.choice([1, 2, 3, 4, 8])
    e = 2 if dtype == BF16 else 4
    if op == "rope":
        rows = _log_int(rng, 1, max(1, int(4.0e8 / (e * d * Hkv * (G + 2)))))
        B = rng.choice([1, rng.randint(1, 96)])
        T = rng.choice([1, max(1, rows // B)])
        rot = rng.choice([d, d, d // 2, d // 4, 24])
        return dict(op=op, B=B, T=T, Hq=Hkv * G, Hkv=Hkv, d=d, rot=rot, pairs=rng.choice(["half", "next"]), dtype=dtype,
                    far=rng.choice([0, _log_int(rng, 100, 1000000)]), factor=rng.choice([1.0, 4.0, 8.0]),
                    norm=rng.random() < 0.8, cap=T + rng.randint(0, 300))
    block = rng.choice([16, 32, 64, 64, 128])
    if op == "shared":
        P = _log_int(rng, 30, 40000)
        B = _log_int(rng, 1, 80)
        nq = rng.choice([1, 1, 2, 3, 5])
        cap = _log_int(rng, 8, 4000)
        most = rng.randint(nq, cap)
        c = dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, nq=nq, P=P, cap=cap, least=rng.choice([most, rng.randint(0, most)]),
                 most=most, d=d, dtype=dtype)
        room = 3.0e9 if dtype == F32 else 3.6e10  # float32 calls are the small ones
        while work(c)["flops"] > room or 2.0 * e * c["B"] * Hkv * cap * d > 6.0e8:
            if c["B"] > 4:
                c["B"] = c["B"] * 2 // 3
            else:
                c["P"], c["cap"] = c["P"] * 2 // 3, max(c["most"], c["cap"] * 2 // 3)
                c["most"], c["least"] = max(nq, c["most"] * 2 // 3), c["least"] * 2 // 3
        return c
    cap = _log_int(rng, 2 * block, 131072)
    B = rng.randint(1, max(1, min(16, int((5.0e8 if op == "digest" else 3.0e9) / (e * cap * Hkv * d)))))
    most = rng.randint(cap // 2, cap)
    least = rng.choice([most, rng.randint(0, most)])
    if op == "digest":
        return dict(op=op, B=B, H=Hkv, cap=cap, least=least, most=most, d=d, block=block,
                    n_new=rng.choice([cap, 1, rng.randint(1, cap)]), dtype=dtype)
    nq = rng.choice([1, 1, 1, 2, 4, 7])
    sink, recent = rng.choice([0, 1, 2]), rng.choice([1, 1, 2, 4])
    n_sel = rng.randint(sink + recent, sink + recent + 60)
    c = dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, nq=nq, cap=cap, least=least, most=most, d=d, block=block, n_sel=n_sel, sink=sink,
             recent=recent, dtype=dtype)
    while c["B"] > 1 and work(c)["bytes"] > 1.8e8:
        c["B"] -= 1
    return c


# ---- inputs -----------------------------------------------------------------------------------


def _rand(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _lengths(c, seed, shape):
    """Lengths between least and most, the largest among them; made on the host, as a scheduler has them."""
    r = np.random.default_rng([seed, 7])
    ln = r.integers(c["least"], c["most"] + 1, size=shape)
    ln.reshape(-1)[0] = c["most"]
    return torch.from_numpy(ln.astype(np.int32)).cuda()


def _keys(g, t, H, n, d):
    """Keys as a prompt's segments leave them: a common offset with a few large channels, a centre for each segment
    of 256 tokens, noise; the first keys draw more attention than the others."""
    x = torch.randn(H, n, d, generator=g, device="cuda")
    x += torch.randn(H, (n + 255) // 256, d, generator=g, device="cuda").mul_(0.7).repeat_interleave(256, 1)[:, :n]
    offset = torch.randn(H, 1, d, generator=g, device="cuda")
    offset[:, :, :: max(1, d // 4)] *= 6
    x += offset
    x[:, :SINKS] *= 1.5
    return x.to(t)


def _frequencies(c):
    """theta^(-2i/rot); with a factor, the slow ones divided by it and those between blended, as models scaled for a
    longer context have them, and the scale that goes with it."""
    f = 500000.0 ** (-np.arange(0, c["rot"], 2, dtype=np.float64) / c["rot"])
    if c["factor"] != 1.0:
        turns = 8192.0 * f / (2 * math.pi)
        keep = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        f = f * keep + f / c["factor"] * (1 - keep)
    return f, (1.0 if c["factor"] == 1.0 else 0.1 * math.log(c["factor"]) + 1.0)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = {"case": c}
    B, d, t = c["B"], c["d"], TYPE[c["dtype"]]
    if c["op"] == "rope":
        T, Hq, Hkv = c["T"], c["Hq"], c["Hkv"]
        x = torch.empty(B, T, Hq + 2 * Hkv, d, dtype=t, device="cuda")  # as one projection of q, k and v leaves them
        for b in range(B):
            x[b] = _rand(g, T, Hq + 2 * Hkv, d) * 1.7
        q, k, v = x.transpose(1, 2).split([Hq, Hkv, Hkv], 1)
        st.update(q=q, k=k, v=v)
        st["wq"] = (1 + 0.2 * _rand(g, d)).to(t) if c["norm"] else None
        st["wk"] = (1 + 0.2 * _rand(g, d)).to(t) if c["norm"] else None
        f, st["rot_scale"] = _frequencies(c)
        st["inv_freq"] = torch.from_numpy(f).cuda()
        r = np.random.default_rng([seed, 3])
        first = r.integers(0, c["far"] + 1, size=(B, 1))
        first[0] = c["far"]
        st["pos"] = torch.from_numpy((first + np.arange(T)).astype(np.int32)).cuda()
        slot = r.integers(0, c["cap"] - T + 1, size=(B, Hkv))
        st["slot"] = torch.from_numpy(slot.astype(np.int32)).cuda()
        st["q_out"] = torch.zeros(B, Hq, T, d, dtype=t, device="cuda")
        st["K"] = torch.zeros(B, Hkv, c["cap"], d, dtype=t, device="cuda")
        st["V"] = torch.zeros(B, Hkv, c["cap"], d, dtype=t, device="cuda")
        return st
    H = c["H"] if c["op"] == "digest" else c["Hkv"]
    st["K"] = torch.empty(B, H, c["cap"], d, dtype=t, device="cuda")
    for b in range(B):
        st["K"][b] = _keys(g, t, H, c["cap"], d)
    st["len"] = _lengths(c, seed, (B, H))
    nb = (c["cap"] + c.get("block", 1) - 1) // c.get("block", 1)
    if c["op"] == "digest":
        st["digest"] = torch.zeros(B, H, nb, 2, d, dtype=t, device="cuda")
        return st
    st["V"] = torch.empty_like(st["K"])
    for b in range(B):
        st["V"][b] = _rand(g, H, c["cap"], d)
    # queries lean towards one of the segments, as those of a model that looks something up
    G = c["Hq"] // H
    q = _rand(g, B, H, G * c["nq"], d)
    if c["op"] == "blocks":
        st["digest"] = torch.zeros(B, H, nb, 2, d, dtype=t, device="cuda")
        st["digest"].copy_(_digest_of(st["K"], st["len"], c["block"], st["digest"]))
        at = torch.randint(0, c["cap"], (B, H, 1, 1), generator=g, device="cuda").expand(B, H, 1, d)
        q += 0.5 * st["K"].gather(2, at).float()
    else:
        st["Kp"] = _keys(g, t, H, c["P"], d)
        st["Vp"] = _rand(g, H, c["P"], d).to(t)
    st["q"] = q.to(t).view(B, c["Hq"], c["nq"], d)
    return st


# ---- the plain forms --------------------------------------------------------------------------


def _digest_of(K, ln, block, old):
    """Least and largest key of each block's filled slots; blocks without one as in `old`."""
    B, H, cap, d = K.shape
    nb = (cap + block - 1) // block
    out = old.clone()
    at = torch.arange(nb * block, device=K.device)
    for b in range(B):
        x = torch.zeros(H, nb * block, d, dtype=torch.float32, device=K.device)
        x[:, :cap] = K[b]
        hidden = (at >= ln[b][:, None])[..., None]
        low = x.masked_fill(hidden, math.inf).view(H, nb, block, d).amin(2)
        top = x.masked_fill(hidden, -math.inf).view(H, nb, block, d).amax(2)
        new = torch.stack((low, top), 2).to(K.dtype)
        some = torch.arange(nb, device=K.device) * block < ln[b][:, None]
        out[b] = torch.where(some[..., None, None], new, old[b])
    return out


def _rope_one(x, w, c, cos, sin, scale):
    x = x.float()
    if c["norm"]:
        x = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
        x = x * w.float()
    rot = c["rot"]
    y, rest = x[..., :rot], x[..., rot:]
    if c["pairs"] == "half":
        a, b = y[..., :rot // 2], y[..., rot // 2:]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((y * scale, rest), -1)


def _rope_plain(st):
    c = st["case"]
    T, B, d = c["T"], c["B"], c["d"]
    for b in range(B) if B * T > 4096 else [slice(0, B)]:
        b = b if isinstance(b, slice) else slice(b, b + 1)
        angle = st["pos"][b].double()[:, None, :, None] * st["inv_freq"]  # far positions need 64 bits
        cos, sin = angle.cos().float(), angle.sin().float()
        st["q_out"][b] = _rope_one(st["q"][b], st["wq"], c, cos, sin, st["rot_scale"]).to(st["q"].dtype)
        k = _rope_one(st["k"][b], st["wk"], c, cos, sin, st["rot_scale"]).to(st["q"].dtype)
        at = (st["slot"][b].long()[..., None] + torch.arange(T, device=k.device))[..., None].expand(-1, -1, T, d)
        st["K"][b].scatter_(2, at, k)
        st["V"][b].scatter_(2, at, st["v"][b])
    return {"q": st["q_out"], "K": st["K"], "V": st["V"]}


def _digest_plain(st):
    c, K, out = st["case"], st["K"], st["digest"]
    B, H, cap, d = K.shape
    block, ln = c["block"], st["len"]
    if c["n_new"] >= cap:
        out.copy_(_digest_of(K, ln, block, out))
        return out
    # the blocks from the one that the first of the newest slots is in
    nb = (c["n_new"] + block - 2) // block + 1
    first = ((ln - c["n_new"]).clamp_min(0) // block).long()
    which = first[..., None] + torch.arange(nb, device=K.device)
    slots = which[..., None] * block + torch.arange(block, device=K.device)
    x = K.gather(2, slots.view(B, H, -1, 1).clamp_max(cap - 1).expand(B, H, nb * block, d)).float().view(B, H, nb, block, d)
    hidden = (slots >= ln[..., None, None])[..., None]
    new = torch.stack((x.masked_fill(hidden, math.inf).amin(3), x.masked_fill(hidden, -math.inf).amax(3)), 3).to(out.dtype)
    some = (which * block < ln[..., None])[..., None, None]
    at = which.clamp_max(out.shape[2] - 1)[..., None, None].expand(B, H, nb, 2, d)
    # blocks past the end keep what they hold: of equal targets the first is written last
    for i in range(nb - 1, -1, -1):
        a = at[:, :, i:i + 1]
        out.scatter_(2, a, torch.where(some[:, :, i:i + 1], new[:, :, i:i + 1], out.gather(2, a)))
    return out


def _choose(u, seen_blocks, c):
    """u [..., nb] -> the chosen blocks [..., n_sel] ascending, -1 behind the last."""
    nb, n_sel = u.shape[-1], c["n_sel"]
    j = torch.arange(nb, device=u.device)
    have = j < seen_blocks[..., None]
    safe = (j < c["sink"]) | (j >= seen_blocks[..., None] - c["recent"])
    rank = torch.where(have, torch.where(safe, math.inf, u), -math.inf)
    order = rank.sort(dim=-1, descending=True, stable=True).indices[..., :n_sel]
    order = torch.where(order < seen_blocks[..., None], order, nb).sort(-1).values
    sel = torch.full(u.shape[:-1] + (n_sel,), -1, dtype=torch.int32, device=u.device)
    sel[..., :order.shape[-1]] = torch.where(order < nb, order, -1)
    return sel


def _blocks_plain(st):
    c = st["case"]
    B, Hkv, cap, d = st["K"].shape
    nq, block, G = c["nq"], c["block"], c["Hq"] // c["Hkv"]
    q = st["q"].view(B, Hkv, G, nq, d)
    t = torch.arange(nq, device=q.device)
    o = torch.empty(B, Hkv, G, nq, d, dtype=st["q"].dtype, device=q.device)
    lse = torch.empty(B, Hkv, G, nq, device=q.device)
    sels = []
    for b in range(B):
        # 64 bits: two bounds may be very near, and which is larger decides
        x = q[b].double().reshape(Hkv, G * nq, d)
        dig = st["digest"][b].double()
        u = x.clamp_min(0) @ dig[:, :, 1].transpose(1, 2) + x.clamp_max(0) @ dig[:, :, 0].transpose(1, 2)
        u = u.view(Hkv, G, nq, -1).amax(1)
        seen = (st["len"][b].long()[:, None] - nq + t + 1).clamp_min(0)
        sel = _choose(u, (seen + block - 1) // block, c)
        sels.append(sel)
        slots = (sel.long()[..., None] * block + torch.arange(block, device=q.device)).view(Hkv, nq, -1)
        ok = (sel >= 0).repeat_interleave(block, -1) & (slots < seen[..., None])
        at = slots.clamp(0, cap - 1).view(Hkv, -1, 1).expand(Hkv, nq * slots.shape[-1], d)
        k = st["K"][b].gather(1, at).float().view(Hkv, nq, -1, d)
        v = st["V"][b].gather(1, at).float().view(Hkv, nq, -1, d)
        v = v.masked_fill_(~ok[..., None], 0.0)
        s = (q[b].float() * d ** -0.5).transpose(1, 2) @ k.transpose(2, 3)  # [Hkv][nq][G][slots]
        s = s.masked_fill_(~ok[:, :, None], -math.inf)
        top = s.amax(-1, keepdim=True)
        p = (s - torch.where(top == -math.inf, 0.0, top)).exp()
        z = p.sum(-1, keepdim=True)
        y = torch.where(z > 0, p @ v / z, 0.0)
        o[b] = y.transpose(1, 2).to(o.dtype)
        lse[b] = (top + z.log()).squeeze(-1).transpose(1, 2)
    return {"o": o.view(st["q"].shape), "lse": lse.view(B, -1, nq), "sel": torch.stack(sels)}


def _shared_plain(st):
    c = st["case"]
    B, Hkv, cap, d = st["K"].shape
    nq, G, P = c["nq"], c["Hq"] // c["Hkv"], c["P"]
    q = st["q"].float().view(B, Hkv, G * nq, d) * d ** -0.5
    x = q.transpose(0, 1).reshape(Hkv, B * G * nq, d) @ st["Kp"].float().transpose(1, 2)
    top = x.amax(-1, keepdim=True)
    p = x.sub_(top).exp_()
    zp = p.sum(-1, keepdim=True)
    op = p @ st["Vp"].float()
    fold = lambda y: y.reshape(Hkv, B, G, nq, -1).transpose(0, 1)  # noqa: E731
    top, zp, op = fold(top), fold(zp), fold(op)
    y = (q @ st["K"].float().transpose(2, 3)).view(B, Hkv, G, nq, cap)
    seen = st["len"].long()[:, :, None] - nq + torch.arange(nq, device=q.device) + 1
    ok = torch.arange(cap, device=q.device) < seen[..., None]
    y = y.masked_fill_(~ok[:, :, None], -math.inf)
    big = torch.maximum(top, y.amax(-1, keepdim=True))
    w = (y - big).exp_()
    vf = st["V"].float().masked_fill_(~ok.any(2)[..., None], 0.0)
    f = (top - big).exp()
    z = zp * f + w.sum(-1, keepdim=True)
    o = (op * f + (w.view(B, Hkv, G * nq, cap) @ vf).view(B, Hkv, G, nq, d)) / z
    lse = big + z.log()
    return {"o": o.reshape(B, -1, nq, d).to(st["q"].dtype), "lse": lse.reshape(B, -1, nq)}


def run(state):
    st = state
    c = st["case"]
    op = c["op"]
    if not own:
        return {"rope": _rope_plain, "digest": _digest_plain, "blocks": _blocks_plain, "shared": _shared_plain}[op](st)
    from kv_cache_compression_obs_gb300 import api
    if op == "rope":
        q, K, V = api.kv_qk_norm_rope(st["q"], st["k"], st["v"], st["inv_freq"], st["pos"], q_weight=st["wq"], k_weight=st["wk"],
                                      eps=EPS if c["norm"] else None, interleaved=c["pairs"] == "next",
                                      rot_scale=st["rot_scale"], slot=st["slot"], q_out=st["q_out"], k_out=st["K"], v_out=st["V"])
        return {"q": q, "K": K, "V": V}
    if op == "digest":
        return api.kv_block_digest(st["K"], c["block"], st["len"], n_new=c["n_new"], out=st["digest"])
    if op == "blocks":
        o, lse, sel = api.kv_attn_blocks(st["q"], st["K"], st["V"], st["len"], st["digest"], c["block"], c["n_sel"],
                                         sink=c["sink"], recent=c["recent"])
        return {"o": o, "lse": lse, "sel": sel}
    o, lse = api.kv_attn_shared(st["q"], st["Kp"], st["Vp"], st["K"], st["V"], st["len"])
    return {"o": o, "lse": lse}


# ---- what a pass cannot do without --------------------------------------------------------------


def work(case):
    c = dict(case)
    e, d, B = (2 if c["dtype"] == BF16 else 4), c["d"], c["B"]
    if c["op"] == "rope":
        rows = B * c["T"]
        heads = c["Hq"] + 2 * c["Hkv"]
        return {"bytes": rows * (2.0 * e * d * heads + 4) + 4.0 * B * c["Hkv"] + 4.0 * c["rot"] + (2.0 * e * d if c["norm"] else 0),
                "flops": rows * (c["Hq"] + c["Hkv"]) * ((4.0 * d if c["norm"] else 0) + 4.0 * c["rot"])}
    mid = (c["least"] + c["most"]) / 2.0
    if c["op"] == "digest":
        n = min(mid, c["n_new"] + (c["block"] - 1) / 2.0 if c["n_new"] < c["cap"] else mid)
        units = B * c["H"]
        return {"bytes": units * (n * e * d + max(1.0, n / c["block"]) * 2 * e * d + 4), "flops": 2.0 * units * n * d}
    units, rows = B * c["Hkv"], B * c["Hq"] * c["nq"]
    ends = rows * (2.0 * e * d + 4) + 4.0 * units
    if c["op"] == "blocks":
        nb = mid / c["block"]
        read = min(mid, c["n_sel"] * c["block"])  # slots of one token; several tokens' choices may be the same
        return {"bytes": ends + units * (nb * 2 * e * d + read * 2 * e * d + 4.0 * c["nq"] * c["n_sel"]),
                "flops": rows * (4.0 * nb * d + 4.0 * read * d)}
    return {"bytes": ends + 2.0 * e * d * (c["Hkv"] * c["P"] + units * mid), "flops": 4.0 * rows * d * (c["P"] + mid)}


# ---- the definitions in 64 bits -------------------------------------------------------------------


def _exact_rope(st):
    c = st["case"]
    B, T, d, rot = c["B"], c["T"], c["d"], c["rot"]
    if B * T * (c["Hq"] + c["Hkv"]) * d > 4e8:
        return None
    m = rot // 2
    i = torch.arange(m, device="cuda")
    ia, ib = (i, i + m) if c["pairs"] == "half" else (2 * i, 2 * i + 1)
    out = {"K": torch.zeros(st["K"].shape, dtype=torch.float64, device="cuda")}
    out["V"] = out["K"].clone()
    out["q"] = torch.zeros(st["q_out"].shape, dtype=torch.float64, device="cuda")

    def one(x, w, b):
        y = x.to(torch.float64)
        if c["norm"]:
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / d + EPS) * w.to(torch.float64)
        turn = torch.exp(1j * torch.outer(st["pos"][b].double(), st["inv_freq"])) * st["rot_scale"]
        z = torch.complex(y[..., ia], y[..., ib]) * turn
        y = y.clone()
        y[..., ia], y[..., ib] = z.real, z.imag
        return y

    for b in range(B):
        for h in range(c["Hq"]):
            out["q"][b, h] = one(st["q"][b, h], st["wq"], b)
        for h in range(c["Hkv"]):
            s = int(st["slot"][b, h])
            out["K"][b, h, s:s + T] = one(st["k"][b, h], st["wk"], b)
            out["V"][b, h, s:s + T] = st["v"][b, h].double()
    return out


def _exact_digest(st):
    c = st["case"]
    B, H, cap, d = st["K"].shape
    block = c["block"]
    out = st["digest"].double()
    for u, n in enumerate(st["len"].view(-1).tolist()):
        x = st["K"].view(B * H, cap, d)[u]
        y = out.view(B * H, -1, 2, d)[u]
        first = 0 if c["n_new"] >= cap else max(0, n - c["n_new"]) // block
        full = n // block
        if full > first:
            z = x[first * block:full * block].double().view(full - first, block, d)
            y[first:full, 0], y[first:full, 1] = z.min(1).values, z.max(1).values
        if n % block and full >= first:
            z = x[full * block:n].double()
            y[full, 0], y[full, 1] = z.min(0).values, z.max(0).values
    return out


def _exact_blocks(st):
    c = st["case"]
    B, Hkv, cap, d = st["K"].shape
    nq, block, G, U = c["nq"], c["block"], c["Hq"] // c["Hkv"], B * Hkv
    q = st["q"].double().view(U, G, nq, d)
    K, V, dig = st["K"].view(U, cap, d), st["V"].view(U, cap, d), st["digest"].view(U, -1, 2, d)
    o = torch.zeros(U, G, nq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((U, G, nq), -math.inf, dtype=torch.float64, device="cuda")
    for u, n in enumerate(st["len"].view(-1).tolist()):
        low, top = dig[u, :, 0].double(), dig[u, :, 1].double()
        for t in range(nq):
            seen = n - nq + t + 1
            if seen <= 0:
                continue
            nb = -(-seen // block)
            bound = torch.full((nb,), -math.inf, dtype=torch.float64, device="cuda")
            for g in range(G):
                x = q[u, g, t]
                bound = torch.maximum(bound, torch.maximum(x * low[:nb], x * top[:nb]).sum(1))
            bound = bound.cpu().numpy()
            fixed = set(range(min(nb, c["sink"]))) | set(range(max(0, nb - c["recent"]), nb))
            others = np.array([j for j in range(nb) if j not in fixed], dtype=np.int64)
            best = others[np.lexsort((others, -bound[others]))][:max(0, c["n_sel"] - len(fixed))]
            chosen = sorted(fixed | set(best.tolist()))
            at = torch.cat([torch.arange(j * block, min(seen, (j + 1) * block)) for j in chosen]).cuda()
            x = q[u, :, t] @ K[u].index_select(0, at).double().T / math.sqrt(d)
            lse[u, :, t] = torch.logsumexp(x, -1)
            o[u, :, t] = torch.softmax(x, -1) @ V[u].index_select(0, at).double()
    return {"o": o.view(st["q"].shape), "lse": lse.view(B, -1, nq), "sel": None}


def _exact_shared(st):
    c = st["case"]
    B, Hkv, cap, d = st["K"].shape
    nq, G = c["nq"], c["Hq"] // c["Hkv"]
    q = st["q"].double().view(B, Hkv, G, nq, d)
    o = torch.zeros_like(q)
    lse = torch.zeros(q.shape[:-1], dtype=torch.float64, device="cuda")
    lens = st["len"].tolist()
    for h in range(Hkv):
        kp, vp = st["Kp"][h].double(), st["Vp"][h].double()
        for b in range(B):
            for t in range(nq):
                n = max(0, lens[b][h] - nq + t + 1)
                k, v = torch.cat((kp, st["K"][b, h, :n].double())), torch.cat((vp, st["V"][b, h, :n].double()))
                x = q[b, h, :, t] @ k.T / math.sqrt(d)
                lse[b, h, :, t] = torch.logsumexp(x, -1)
                o[b, h, :, t] = torch.softmax(x, -1) @ v
    return {"o": o.view(st["q"].shape), "lse": lse.view(B, -1, nq)}


def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _exact_rope, "digest": _exact_digest, "blocks": _exact_blocks, "shared": _exact_shared}[case["op"]](st)
