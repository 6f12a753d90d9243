"""The cases on which prompt attention and the 8-bit slot cache are measured.

Four operators, in the order in which a server calls them:

  prompt   causal attention of whole prompts (or of a chunk behind cached keys), grouped heads,
           sequences of different lengths packed along the token axis;
  compact  the kept rows of a prompt gathered into a slot cache of 8-bit codes with one float32
           scale per block of slots and head (the rows of the last, unfinished block stay as they are);
  decode   one decode step over such a cache: attention of one new token per row, its weights added
           to the slots' accumulators, the token appended (a block that becomes full is quantised);
  evict    the slots with the least accumulated attention dropped from such a cache, the others moved
           together into another cache.

The formulas, with c = codes of a block, a = its scale and top = 127 (int8) or 448 (e4m3):
  a = max(max|x| / top, 2^-126) over the block's rows and d, c = round(x (1 / a)) to nearest even,
  the value that a code stands for = c a (all in float32);
  o_i = sum_j p_ij v_j, p_ij = exp(scale q_i.k_j - lse_i) over the keys j that row i sees.
The 8-bit codes are returned as they are, beside their scales: they follow from float32 operations
that are all rounded to nearest, so two implementations give the same codes.
"""
import math

import numpy as np
import torch

own = False

BF16, F32 = "bf16", "f32"
S8, E4M3 = "s8", "e4m3"
CODE = {S8: torch.int8, E4M3: torch.float8_e4m3fn}
TOP = {S8: 127.0, E4M3: 448.0}
TYPE = {BF16: torch.bfloat16, F32: torch.float32}
SINKS = 4


def listed():
    return [
        # the smallest prompt that the package's configurations hold: four float32 heads, one sequence
        dict(name="prompt-tiny", op="prompt", Hq=4, Hkv=4, d=64, dtype=F32, lens="512", prefix="0", layout="head"),
        # one layer of a 32-head model over a 4K prompt
        dict(name="prompt-layer", op="prompt", Hq=32, Hkv=32, d=128, dtype=BF16, lens="4096", prefix="0", layout="head"),
        # a server's batch of requests: odd lengths, one token, none; Q, K and V as a projection lays them out
        dict(name="prompt-packed", op="prompt", Hq=32, Hkv=8, d=128, dtype=BF16,
             lens="4097,1,733,0,2048,129,5001,63,1900,257,31,1200", prefix="0", layout="token"),
        # a chunk of a long prompt behind the keys of the chunks before it
        dict(name="prompt-chunk", op="prompt", Hq=32, Hkv=8, d=128, dtype=BF16, lens="2000", prefix="30001", layout="head"),
        # the long prompt of the grouped-head prefill configuration, whole
        dict(name="prompt-long", op="prompt", Hq=32, Hkv=8, d=128, dtype=BF16, lens="32768", prefix="0", layout="head"),
        # the smallest compaction: the tiny configuration's 102 of 512 positions
        dict(name="compact-tiny", op="compact", B=1, H=4, T=512, k=102, d=64, block=32, dtype=F32, fmt=S8),
        # 32 layers of an 8-KV-head model, a tenth of a 32K prompt kept
        dict(name="compact-layers", op="compact", B=32, H=8, T=32768, k=3276, d=128, block=64, dtype=BF16, fmt=S8),
        # one sequence, one layer, a short cache: latency
        dict(name="decode-short", op="decode", B=1, Hq=32, Hkv=8, cap=2048, least=1638, most=1638, d=128, block=64,
             dtype=BF16, fmt=S8),
        # eight requests of different lengths, every head with its own keys
        dict(name="decode-ragged", op="decode", B=8, Hq=32, Hkv=32, cap=8192, least=700, most=8191, d=128, block=64,
             dtype=BF16, fmt=E4M3),
        # eight long contexts
        dict(name="decode-long", op="decode", B=8, Hq=32, Hkv=8, cap=131072, least=131000, most=131071, d=128, block=64,
             dtype=BF16, fmt=S8),
        # one layer of a 32-head model: a full cache down to a fifth of an 8K prompt
        dict(name="evict-layer", op="evict", B=1, H=32, cap=2048, least=2048, most=2048, keep=1638, recent=819, sink=0,
             d=128, block=64, dtype=BF16, fmt=E4M3),
        # eight requests' long caches, different lengths, down to half of the capacity
        dict(name="evict-long", op="evict", B=8, H=8, cap=65536, least=60000, most=65536, keep=32768, recent=64, sink=4,
             d=128, block=64, dtype=BF16, fmt=S8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "compact", "decode", "evict"])
    d = rng.choice([64, 128, 128])
    dtype = rng.choice([BF16, BF16, BF16, F32])
    fmt = rng.choice([S8, E4M3])
    block = rng.choice([32, 64, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    G = rng.choice([1, 2, 3, 4, 8])
    if op == "prompt":
        # at most a quarter of the long prompt's products; float32 prompts are the small ones
        room = 2.0e11 if dtype == F32 else 2.0e12
        total = _log_int(rng, 60, 24000 if dtype == BF16 else 4000)
        n = rng.randint(1, 9)
        cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        prefix = [rng.randint(0, 4000) if rng.random() < 0.3 else 0 for _ in lens]
        while 4.0 * d * Hkv * G * sum(a * (a / 2 + p) for a, p in zip(lens, prefix)) > room:
            lens = [a * 2 // 3 for a in lens]
        return dict(op=op, Hq=Hkv * G, Hkv=Hkv, d=d, dtype=dtype, lens=",".join(map(str, lens)),
                    prefix=",".join(map(str, prefix)), layout=rng.choice(["head", "token"]))
    if op == "compact":
        T = _log_int(rng, 100, 40000)
        B = max(1, min(32, int(2.0e9 / (4.0 * T * Hkv * d))))
        return dict(op=op, B=rng.randint(1, B), H=Hkv, T=T, k=rng.choice([T, rng.randint(1, T), max(1, T // 10)]), d=d,
                    block=block, dtype=dtype, fmt=fmt)
    cap = (_log_int(rng, 2 * block, 100000) + block - 1) // block * block
    B = rng.randint(1, max(1, min(16, int(4.0e9 / (2.0 * cap * Hkv * d)))))
    most = rng.randint(cap // 2, cap - 1)
    least = rng.choice([most, rng.randint(0, most)])
    if op == "decode":
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, cap=cap, least=least, most=most, d=d, block=block, dtype=dtype,
                    fmt=fmt)
    keep = rng.randint(max(2, cap // 8), cap - 1)
    return dict(op=op, B=B, H=Hkv, cap=cap, least=least, most=most, keep=keep, recent=rng.randint(0, keep // 2),
                sink=rng.choice([0, min(SINKS, keep // 4)]), d=d, block=block, dtype=dtype, fmt=fmt)


# ---- inputs -----------------------------------------------------------------------------------


def _rand(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _ints(text):
    return [int(x) for x in text.split(",")]


def _lengths(c, seed, shape):
    """Lengths between least and most, the largest among them; made on the host, as a scheduler has them."""
    r = np.random.default_rng([seed, 5])
    ln = r.integers(c["least"], c["most"] + 1, size=shape)
    ln.reshape(-1)[0] = c["most"]
    return torch.from_numpy(ln.astype(np.int32)).cuda()


def _codes(g, c, *shape):
    """Codes as a quantised cache holds them: about normal, the largest at the top of the range."""
    x = (_rand(g, *shape) * 0.28).clamp_(-1, 1)
    x[..., 0, :1] = 1.0
    return (x * TOP[c["fmt"]]).round_().to(CODE[c["fmt"]]) if c["fmt"] == S8 else (x * TOP[c["fmt"]]).to(CODE[c["fmt"]])


def _cache(g, c, H, cap, lens):
    """A filled 8-bit slot cache: codes and scales of the full blocks, the unfinished block's rows, positions
    that ascend along the slots (with gaps, as evictions leave them) and accumulated attention."""
    B, d, block, t = c["B"], c["d"], c["block"], TYPE[c["dtype"]]
    nb = cap // block
    st = {}
    for name in ("K", "V"):
        st[name] = torch.empty(B, H, cap, d, dtype=CODE[c["fmt"]], device="cuda")
        for b in range(B):
            st[name][b] = _codes(g, c, H, nb, block, d).view(H, cap, d)
        st[name + "s"] = (0.5 + torch.rand(B, H, nb, generator=g, device="cuda")) * (4.0 / TOP[c["fmt"]])
        st[name + "t"] = _rand(g, B, H, block, d).to(t)
    gaps = torch.randint(1, 4, (B, H, cap), generator=g, device="cuda", dtype=torch.int32)
    st["pos"] = torch.cumsum(gaps, -1, dtype=torch.int32) - gaps[..., :1]
    # a power law, a few ties among the small values, as accumulated attention has
    st["acc"] = torch.rand(B, H, cap, generator=g, device="cuda").clamp_min(1e-4).pow(-0.7).mul_(512).floor_().div_(512)
    st["len"] = lens
    return st


def _empty_cache(c, H, cap):
    B, d, block, t = c["B"], c["d"], c["block"], TYPE[c["dtype"]]
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    return {"K": z(B, H, cap, d, dtype=torch.uint8).view(CODE[c["fmt"]]), "Ks": z(B, H, cap // block),
            "V": z(B, H, cap, d, dtype=torch.uint8).view(CODE[c["fmt"]]), "Vs": z(B, H, cap // block),
            "Kt": z(B, H, block, d, dtype=t), "Vt": z(B, H, block, d, dtype=t), "pos": z(B, H, cap, dtype=torch.int32),
            "acc": z(B, H, cap), "len": z(B, H, dtype=torch.int32)}


def _up(n, m):
    return (n + m - 1) // m * m


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = {"case": c}
    if c["op"] == "prompt":
        lens, prefix = _ints(c["lens"]), _ints(c["prefix"])
        prefix = prefix * len(lens) if len(prefix) == 1 else prefix
        keys = [a + p for a, p in zip(lens, prefix)]
        t, tq, tk = TYPE[c["dtype"]], sum(lens), sum(keys)

        def heads(H, n):
            if c["layout"] == "token":  # [tokens][heads][d], seen as [1][heads][tokens][d]
                return _rand(g, n, H, c["d"]).to(t).transpose(0, 1).unsqueeze(0)
            return _rand(g, 1, H, n, c["d"]).to(t)

        st.update(q=heads(c["Hq"], tq), k=heads(c["Hkv"], tk), v=heads(c["Hkv"], tk), lens=lens, keys=keys)
        st["k"][:, :, :SINKS] *= 2  # the first keys draw more attention than the others
        st["seq_q"] = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
        st["seq_k"] = torch.tensor(np.cumsum([0] + keys), dtype=torch.int32, device="cuda")
        return st
    if c["op"] == "compact":
        B, H, T, k, d, t = c["B"], c["H"], c["T"], c["k"], c["d"], TYPE[c["dtype"]]
        st["K"] = torch.empty(B, H, T, d, dtype=t, device="cuda")
        st["V"] = torch.empty(B, H, T, d, dtype=t, device="cuda")
        for b in range(B):
            st["K"][b] = _rand(g, H, T, d)
            st["V"][b] = _rand(g, H, T, d)
        st["s"] = torch.rand(B, H, T, generator=g, device="cuda").pow(4)
        if k == T:
            st["idx"] = torch.arange(T, dtype=torch.int32, device="cuda").expand(B, H, T).contiguous()
        else:
            order = torch.rand(B, H, T, generator=g, device="cuda").argsort(-1)[..., :k]
            st["idx"] = order.sort(-1).values.to(torch.int32).contiguous()
        st["cache"] = _empty_cache(c, H, _up(k, c["block"]))
        return st
    if c["op"] == "decode":
        st["cache"] = _cache(g, c, c["Hkv"], c["cap"], _lengths(c, seed, (c["B"], c["Hkv"])))
        t = TYPE[c["dtype"]]
        st["q"] = _rand(g, c["B"], c["Hq"], c["d"]).to(t)
        st["k_new"] = _rand(g, c["B"], c["Hkv"], c["d"]).to(t)
        st["v_new"] = _rand(g, c["B"], c["Hkv"], c["d"]).to(t)
        st["new_pos"] = 4 * c["cap"]
        st["len_out"] = torch.zeros_like(st["cache"]["len"])  # apart from len: the step can be taken again
        return st
    st["cache"] = _cache(g, c, c["H"], c["cap"], _lengths(c, seed, (c["B"], c["H"])))
    st["into"] = _empty_cache(c, c["H"], _up(c["keep"], c["block"]))
    return st


# ---- the plain forms --------------------------------------------------------------------------


def _quantise(x, fmt):
    """x [..., rows, d] float32 -> codes and one scale for each [rows, d]."""
    big = x.abs().amax((-2, -1))
    scale = torch.maximum(big / torch.full_like(big, TOP[fmt]), torch.full_like(big, 2.0 ** -126))
    y = x * (torch.ones_like(scale) / scale)[..., None, None]
    return (y.round().clamp(-127, 127) if fmt == S8 else y).to(CODE[fmt]), scale


def _prompt_plain(st):
    c = st["case"]
    q, k, v = st["q"][0], st["k"][0], st["v"][0]
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    G = Hq // Hkv
    o = torch.empty(Hq, q.shape[1], d, dtype=q.dtype, device=q.device)
    lse = torch.empty(Hq, q.shape[1], device=q.device)
    q0 = k0 = 0
    for nq, nk in zip(st["lens"], st["keys"]):
        kf, vf = k[:, k0:k0 + nk].float(), v[:, k0:k0 + nk].float()
        step = max(1, int(1.5e9 // max(1, Hq * nk)))  # rows at a time: the scores are held whole
        for a in range(0, nq, step):
            b = min(nq, a + step)
            seen = nk - nq + b  # no row of the chunk sees a later key
            x = (q[:, q0 + a:q0 + b].float() * d ** -0.5).reshape(Hkv, G * (b - a), d) @ kf[:, :seen].transpose(1, 2)
            x = x.view(Hq, b - a, seen)
            row = torch.arange(nk - nq + a, nk - nq + b, device=q.device)
            x = x.masked_fill_(torch.arange(seen, device=q.device) > row[:, None], -math.inf)
            top = x.amax(-1, keepdim=True)
            p = x.sub_(top).exp_()
            z = p.sum(-1, keepdim=True)
            y = p.view(Hkv, G * (b - a), seen) @ vf[:, :seen]
            o[:, q0 + a:q0 + b] = (y.view(Hq, b - a, d) / z).to(o.dtype)
            lse[:, q0 + a:q0 + b] = (top + z.log()).squeeze(-1)
        q0, k0 = q0 + nq, k0 + nk
    return {"o": o.unsqueeze(0), "lse": lse.unsqueeze(0)}


def _store(into, name, x, n_new, block, fmt, codes=None, scale=None):
    """The rows x [B][H][m][d] (float32, m a whole number of blocks) as blocks and the unfinished block of `into`."""
    B, H, m, d = x.shape
    nb = m // block
    if codes is None:
        codes, scale = _quantise(x.view(B, H, nb, block, d), fmt)
    blocks = torch.arange(nb, device=x.device)
    full = blocks < (n_new // block)[..., None]
    out = into[name].view(B, H, -1, block, d)[:, :, :nb]
    old = out.view(torch.uint8)
    old.copy_(torch.where(full[..., None, None], codes.view(torch.uint8), old))
    into[name + "s"][:, :, :nb] = torch.where(full, scale, into[name + "s"][:, :, :nb])
    at = torch.arange(block, device=x.device)
    src = ((n_new // block) * block).long()[..., None] + at
    rows = x.gather(2, src.clamp_max(m - 1)[..., None].expand(B, H, block, d)).to(into[name + "t"].dtype)
    mine = at < (n_new % block)[..., None]
    into[name + "t"].copy_(torch.where(mine[..., None], rows, into[name + "t"]))


def _pad_rows(x, m):
    """x [B][H][k][...] with zero rows up to m."""
    y = torch.zeros(*x.shape[:2], m, *x.shape[3:], dtype=x.dtype, device=x.device)
    y[:, :, :x.shape[2]] = x
    return y


def _compact_plain(st):
    c, into = st["case"], st["cache"]
    k, d, block = c["k"], c["d"], c["block"]
    at = st["idx"].long()
    n_new = torch.full((c["B"], c["H"]), k, dtype=torch.int32, device=at.device)
    m = into["K"].shape[2]
    for name in ("K", "V"):
        x = st[name].gather(2, at[..., None].expand(*at.shape, d)).float()
        _store(into, name, _pad_rows(x, m), n_new, block, c["fmt"])
    into["pos"][..., :k] = st["idx"]
    into["acc"][..., :k] = st["s"].gather(2, at)
    into["len"].copy_(n_new)
    return into


def _values(cache, name):
    """Every slot's row in float32: code times scale, or the unfinished block's own row; [B][H][cap][d]."""
    code, scale, tail = cache[name], cache[name + "s"], cache[name + "t"]
    B, H, cap, d = code.shape
    block = tail.shape[2]
    x = (code.float().view(B, H, -1, block, d) * scale[..., None, None]).view(B, H, cap, d)
    ln = cache["len"].long()
    # the unfinished block: none where the cache is full
    last = (ln // block).clamp_max(cap // block - 1)
    rows = torch.where((ln < cap)[..., None, None], tail.float(),
                       x.view(B, H, -1, block * d).gather(2, last[..., None, None].expand(B, H, 1, block * d))
                       .view(B, H, block, d))
    x.view(B, H, -1, block * d).scatter_(2, last[..., None, None].expand(B, H, 1, block * d),
                                         rows.view(B, H, 1, block * d))
    return x


def _decode_plain(st):
    c, cache = st["case"], st["cache"]
    B, Hkv, cap, d = cache["K"].shape
    Hq, block = c["Hq"], c["block"]
    ln = cache["len"].long()
    slot = (ln % block)[..., None, None].expand(B, Hkv, 1, d)
    cache["Kt"].scatter_(2, slot, st["k_new"].unsqueeze(2))
    cache["Vt"].scatter_(2, slot, st["v_new"].unsqueeze(2))
    kf, vf = _values(cache, "K"), _values(cache, "V")
    x = (st["q"].float() * d ** -0.5).view(B, Hkv, Hq // Hkv, d) @ kf.transpose(2, 3)
    at = torch.arange(cap, device=x.device)
    seen = at <= ln[..., None]
    x = x.masked_fill_(~seen.unsqueeze(2), -math.inf)
    p = (x - x.amax(-1, keepdim=True)).exp_()
    p = p / p.sum(-1, keepdim=True)
    # the slots behind a unit's last row weigh nothing, whatever they hold
    vf = vf.masked_fill_(~seen.unsqueeze(-1), 0.0)
    o = (p @ vf).view(B, Hq, d)
    mass = p.sum(2)
    acc, pos = cache["acc"], cache["pos"]
    new = at == ln[..., None]
    acc.copy_(torch.where(new, mass, torch.where(seen, acc + mass, acc)))
    pos.copy_(torch.where(new, torch.full_like(pos, st["new_pos"]), pos))
    done = ((ln + 1) % block == 0)
    which = (ln // block)[..., None]
    for name in ("K", "V"):
        codes, scale = _quantise(cache[name + "t"].float(), c["fmt"])
        raw = cache[name].view(torch.uint8).view(B, Hkv, -1, block * d)
        at_b = which[..., None].expand(B, Hkv, 1, block * d)
        raw.scatter_(2, at_b, torch.where(done[..., None, None], codes.view(torch.uint8).view(B, Hkv, 1, block * d),
                                          raw.gather(2, at_b)))
        s = cache[name + "s"]
        s.scatter_(2, which, torch.where(done, scale, s.gather(2, which).squeeze(-1)).unsqueeze(-1))
    st["len_out"].copy_(ln + 1)
    return {"o": o, "len_out": st["len_out"], **{n: cache[n] for n in cache if n != "len"}}


def _evict_plain(st):
    c, cache, into = st["case"], st["cache"], st["into"]
    B, H, cap, d = cache["K"].shape
    keep, block = c["keep"], c["block"]
    ln = cache["len"]
    at = torch.arange(cap, device=ln.device)
    have = at < ln[..., None]
    safe = (at >= ln[..., None] - c["recent"]) | (cache["pos"] < c["sink"])
    rank = torch.where(have, torch.where(safe, math.inf, cache["acc"]), -math.inf)
    order = rank.flip(-1).sort(dim=-1, descending=True, stable=True).indices  # of equals the later slot stays
    kept = (cap - 1 - order)[..., :min(keep, cap)].sort(-1).values
    n_new = ln.clamp_max(keep)
    # where fewer than `keep` are held, the slots behind them sort last and are cut off
    kept = torch.where(kept < ln[..., None], kept, cap).sort(-1).values
    mine = torch.arange(kept.shape[-1], device=ln.device) < n_new[..., None]
    idx = torch.where(mine, kept, -1).to(torch.int32)
    src = torch.where(mine, kept, 0)
    m = into["K"].shape[2]
    src_m = torch.zeros(B, H, m, dtype=torch.int64, device=ln.device)
    src_m[..., :src.shape[-1]] = src
    lead = src_m.view(B, H, -1, block)
    # a block that moves as it is keeps its codes and scale
    whole = (lead[..., -1] - lead[..., 0] == block - 1) & (lead[..., 0] % block == 0) \
        & (lead[..., -1] < (ln // block * block)[..., None])
    for name in ("K", "V"):
        x = _values(cache, name).gather(2, src_m[..., None].expand(B, H, m, d))
        codes, scale = _quantise(x.view(B, H, -1, block, d), c["fmt"])
        old = cache[name].view(torch.uint8).gather(2, src_m[..., None].expand(B, H, m, d)).view(B, H, -1, block, d)
        codes = torch.where(whole[..., None, None], old, codes.view(torch.uint8))
        scale = torch.where(whole, cache[name + "s"].gather(2, lead[..., 0] // block), scale)
        _store(into, name, x, n_new, block, c["fmt"], codes, scale)
    k = kept.shape[-1]
    into["pos"][..., :k] = torch.where(mine, cache["pos"].gather(2, src), into["pos"][..., :k])
    into["acc"][..., :k] = torch.where(mine, cache["acc"].gather(2, src), into["acc"][..., :k])
    into["len"].copy_(n_new)
    return {"idx": idx, **into}


def run(state):
    st = state
    op = st["case"]["op"]
    if not own:
        return {"prompt": _prompt_plain, "compact": _compact_plain, "decode": _decode_plain, "evict": _evict_plain}[op](st)
    from kv_cache_compression_obs_gb300 import api
    c = st["case"]
    if op == "prompt":
        o, lse = api.kv_attn_prompt(st["q"], st["k"], st["v"], seq_q=st["seq_q"], seq_k=st["seq_k"], packed=True)
        return {"o": o, "lse": lse}
    if op == "compact":
        return api.kv_compact_q8(st["K"], st["V"], st["s"], st["idx"], st["cache"])
    if op == "decode":
        o = api.h2o_decode_step_q8(st["q"], st["k_new"], st["v_new"], st["cache"], st["new_pos"], len_out=st["len_out"])
        return {"o": o, "len_out": st["len_out"], **{n: st["cache"][n] for n in st["cache"] if n != "len"}}
    idx = api.kv_evict_q8(st["cache"], c["keep"], c["recent"], st["into"], sink=c["sink"])
    return {"idx": idx, **st["into"]}


# ---- what a pass cannot do without --------------------------------------------------------------


def _pairs(c):
    lens, prefix = _ints(c["lens"]), _ints(c["prefix"])
    prefix = prefix * len(lens) if len(prefix) == 1 else prefix
    return lens, prefix, sum(a * p + a * (a + 1) / 2 for a, p in zip(lens, prefix))


def work(case):
    c = dict(case)
    e, d = (2 if c["dtype"] == BF16 else 4), c["d"]
    if c["op"] == "prompt":
        lens, prefix, pairs = _pairs(c)
        tq, tk = sum(lens), sum(lens) + sum(prefix)
        return {"bytes": e * d * (2 * c["Hq"] * tq + 2 * c["Hkv"] * tk) + 4 * c["Hq"] * tq, "flops": 4.0 * d * c["Hq"] * pairs}
    if c["op"] == "compact":
        rows = c["B"] * c["H"] * c["k"]
        return {"bytes": rows * (2.0 * d * (e + 1) + 16 + 8.0 / c["block"]), "flops": 6.0 * rows * d}
    mid = (c["least"] + c["most"]) / 2.0
    if c["op"] == "decode":
        units, G = c["B"] * c["Hkv"], c["Hq"] // c["Hkv"]
        rest = (mid % c["block"]) if c["least"] == c["most"] else c["block"] / 2.0
        return {"bytes": units * (mid * (2.0 * d + 8 + 8.0 / c["block"]) + rest * 2.0 * d * e + 2 * d * e * 2 + G * d * (e + 4)),
                "flops": 4.0 * units * G * mid * d}
    units = c["B"] * c["H"]
    kept = min(c["keep"], mid)
    return {"bytes": units * (4.0 * mid + kept * (4.0 * d + 16 + 4 + 16.0 / c["block"])), "flops": 6.0 * units * kept * d}


# ---- the definitions in 64 bits -------------------------------------------------------------------


def _exact_prompt(st):
    c = st["case"]
    if 4.0 * c["d"] * c["Hq"] * _pairs(c)[2] > 1.2e13:
        return None
    G, d = c["Hq"] // c["Hkv"], c["d"]
    q, k, v = (st[n][0].double() for n in "qkv")
    o = torch.zeros(c["Hq"], q.shape[1], d, dtype=torch.float64, device="cuda")
    lse = torch.full(o.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    q0 = k0 = 0
    for nq, nk in zip(st["lens"], st["keys"]):
        for h in range(c["Hq"]):
            kk, vv = k[h // G, k0:k0 + nk], v[h // G, k0:k0 + nk]
            for a in range(0, nq, 4096):
                b = min(nq, a + 4096)
                n = nk - nq + b
                x = torch.einsum("id,jd->ij", q[h, q0 + a:q0 + b], kk[:n]) / math.sqrt(d)
                hidden = torch.ones(b - a, n, dtype=torch.bool, device="cuda").triu(nk - nq + a + 1)
                x[hidden] = -math.inf
                lse[h, q0 + a:q0 + b] = torch.logsumexp(x, -1)
                o[h, q0 + a:q0 + b] = torch.softmax(x, -1) @ vv[:n]
        q0, k0 = q0 + nq, k0 + nk
    return {"o": o[None], "lse": lse[None]}


def _nothing(names):
    return {n: None for n in names}


def _exact_scales(x, block, fmt, n_new, m):
    """x: list of units' rows in 64 bits -> their full blocks' scales, [units][m / block]."""
    out = torch.zeros(len(x), m // block, dtype=torch.float64, device="cuda")
    for u, r in enumerate(x):
        f = int(n_new[u]) // block
        if f:
            out[u, :f] = (r[:f * block].reshape(f, -1).abs().max(1).values / TOP[fmt]).clamp_min(2.0 ** -126)
    return out


def _exact_compact(st):
    c = st["case"]
    B, H, k, d, block = c["B"], c["H"], c["k"], c["d"], c["block"]
    m = st["cache"]["K"].shape[2]
    out = _nothing(["K", "V", "pos", "len"])
    idx = st["idx"].view(B * H, k).long()
    for name in ("K", "V"):
        rows = st[name].view(B * H, -1, d)
        sc = torch.zeros(B * H, m // block, dtype=torch.float64, device="cuda")
        tail = torch.zeros(B * H, block, d, dtype=torch.float64, device="cuda")
        for u in range(B * H):
            x = rows[u].index_select(0, idx[u]).double()
            sc[u] = _exact_scales([x], block, c["fmt"], [k], m)[0]
            tail[u, :k % block] = x[k - k % block:]
        out[name + "s"], out[name + "t"] = sc.view(B, H, -1), tail.view(B, H, block, d)
    acc = torch.zeros(B * H, m, dtype=torch.float64, device="cuda")
    acc[:, :k] = torch.stack([a[i] for a, i in zip(st["s"].view(B * H, -1).double(), idx)])
    out["acc"] = acc.view(B, H, m)
    return out


def _rows64(cache, name, u, n):
    """The first n rows that unit u of a cache holds, in 64 bits."""
    d = cache[name].shape[-1]
    tail = cache[name + "t"]
    block = tail.shape[2]
    f = n // block * block
    code = cache[name].view(-1, cache[name].shape[2], d)[u, :f].to(torch.float32).double()
    scale = cache[name + "s"].view(-1, cache[name + "s"].shape[2])[u, :f // block].double()
    return torch.cat([code * scale.repeat_interleave(block)[:, None], tail.view(-1, block, d)[u, :n - f].double()])


def _exact_decode(st):
    c, cache = st["case"], st["cache"]
    B, Hkv, cap, d = cache["K"].shape
    G, block = c["Hq"] // Hkv, c["block"]
    U = B * Hkv
    q = st["q"].double().view(U, G, d)
    kn, vn = st["k_new"].double().view(U, d), st["v_new"].double().view(U, d)
    lens = cache["len"].view(-1).tolist()
    o = torch.zeros(U, G, d, dtype=torch.float64, device="cuda")
    acc = cache["acc"].double().view(U, cap).clone()
    out = _nothing(["K", "V", "pos", "len_out"])
    sc = {n: cache[n].double().view(U, -1).clone() for n in ("Ks", "Vs")}
    tail = {n: cache[n].double().view(U, block, d).clone() for n in ("Kt", "Vt")}
    for u, n in enumerate(lens):
        k, v = torch.cat([_rows64(cache, "K", u, n), kn[u:u + 1]]), torch.cat([_rows64(cache, "V", u, n), vn[u:u + 1]])
        p = torch.softmax(q[u] @ k.T / math.sqrt(d), -1)
        o[u] = p @ v
        acc[u, :n] += p[:, :n].sum(0)
        acc[u, n] = p[:, n].sum()
        for name, x in (("K", kn), ("V", vn)):
            tail[name + "t"][u, n % block] = x[u]
            if (n + 1) % block == 0:
                sc[name + "s"][u, n // block] = max(float(tail[name + "t"][u].abs().max()) / TOP[c["fmt"]], 2.0 ** -126)
    out.update(o=o.view(B, -1, d), acc=acc.view(B, Hkv, cap))
    out.update({n: x.view(B, Hkv, -1) for n, x in sc.items()}, **{n: x.view(B, Hkv, block, d) for n, x in tail.items()})
    return out


def _exact_evict(st):
    c, cache = st["case"], st["cache"]
    B, H, cap, d = cache["K"].shape
    U, keep, block, m = B * H, c["keep"], c["block"], st["into"]["K"].shape[2]
    lens = cache["len"].view(-1).tolist()
    out = _nothing(["K", "V", "pos", "len", "idx"])
    z = lambda *s: torch.zeros(U, *s, dtype=torch.float64, device="cuda")  # noqa: E731
    acc, sc, tail = z(m), {"K": z(m // block), "V": z(m // block)}, {"K": z(block, d), "V": z(block, d)}
    for u, n in enumerate(lens):
        a = cache["acc"].view(U, cap)[u, :n].cpu().numpy().astype(np.float64)
        pos = cache["pos"].view(U, cap)[u, :n].cpu().numpy()
        slots = np.arange(n)
        free = slots[(slots < n - c["recent"]) & (pos >= c["sink"])]
        drop = max(0, n - keep)
        gone = free[np.lexsort((free, a[free]))[:drop]]  # the least (weight, slot) go
        left = np.setdiff1d(slots, gone)
        at = torch.from_numpy(left).cuda()
        nn = len(left)
        acc[u, :nn] = torch.from_numpy(a[left]).cuda()
        for name in ("K", "V"):
            x = _rows64(cache, name, u, n)[at]
            sc[name][u] = _exact_scales([x], block, c["fmt"], [nn], m)[0]
            for b in range(nn // block):
                lo = int(left[b * block])
                if lo % block == 0 and int(left[b * block + block - 1]) == lo + block - 1 < n // block * block:
                    sc[name][u, b] = cache[name + "s"].view(U, -1)[u, lo // block].double()
            tail[name][u, :nn % block] = x[nn - nn % block:]
    out["acc"] = acc.view(B, H, m)
    for name in ("K", "V"):
        out[name + "s"], out[name + "t"] = sc[name].view(B, H, -1), tail[name].view(B, H, block, d)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return {"prompt": _exact_prompt, "compact": _exact_compact, "decode": _exact_decode, "evict": _exact_evict}[case["op"]](st)
