"""Inputs and tolerances of the tests of prompt attention and the 8-bit slot cache.

A logit l = scale <q, k> computed in fp32 is off by at most about
dl = c A, A = scale sum_i |q_i k_i|: with products of exact operands c = (number of
roundings) 2^-23 (tensor cores may truncate, a step twice half a step), so
  CUDA cores       c = d 2^-24 <= 2^-17 for d <= 128 (one rounding a term),
  tensor cores     c = (d / 16 + 2) 2^-23 < 2^-19, with 2^-22 more where an operand is
                   split into hi + lo fp16 (22 bits): 2^-18 covers both.
A weight p = exp(l - lse) is then off by a factor 1 +- (2 dl + 2^-18): the error of l and
of lse, and 2^-18 for the exponentials (2^-22 each), the normaliser's sum and the products'
sums.  So |o - o_exact| <= (2 dl + 2^-18 [+ 2^-8 where weights are rounded to bf16])
sum_j p_j |v_j| + half a step of the output's type, 2^-8 |o| for bf16.
lse: dl + 2^-20 + 2^-22 |lse|.  acc: (2 dl + 2^-18) sum_g p_g + 2^-23 |acc|.
"""
import numpy as np
import torch

CODES = {"s8": torch.int8, "e4m3": torch.float8_e4m3fn}
C_CUDA, C_TC = 2.0 ** -17, 2.0 ** -18


def np64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def within(got, want, bound, what):
    err = np.abs(np.asarray(got, np.float64) - want)
    bad = ~(err <= bound)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(np.isnan(err), np.inf, err) / np.maximum(bound, 1e-300)), err.shape)
        raise AssertionError(f"{what}: {int(bad.sum())}/{bad.size} outside; worst at {i}: got {np.asarray(got)[i]!r} "
                             f"want {want[i]!r} err {err[i]:.3e} bound {np.broadcast_to(bound, err.shape)[i]:.3e}")


def filled_cache(api, B, H, cap, d, block, dtype, fmt, lens, seed, device="cuda", acc=True):
    """A cache whose units hold `lens` slots: every part random, the unused slots too."""
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    c = api.q8_cache(B, H, cap, d, block, dtype, CODES[fmt], device)
    for n in ("K", "V"):
        x = torch.randn(B, H, cap, d, generator=g) * 0.3
        x = (x.clamp(-1, 1) * (127 if fmt == "s8" else 448))
        c[n].copy_((x.round() if fmt == "s8" else x).to(CODES[fmt]))
        c[n + "s"].copy_(torch.rand(B, H, cap // block, generator=g) * 0.02 + 0.005)
        c[n + "t"].copy_(torch.randn(B, H, block, d, generator=g).to(dtype))
    c["pos"].copy_(torch.randint(1, 4, (B, H, cap), generator=g, dtype=torch.int32).cumsum(-1, dtype=torch.int32) - 1)
    c["acc"].copy_((torch.rand(B, H, cap, generator=g) * 64).floor() / 16)  # many ties
    c["len"].copy_(torch.as_tensor(lens, dtype=torch.int32).reshape(B, H))
    if not acc:
        c["acc"] = None
    return c


def clone(c):
    return {n: None if t is None else t.clone() for n, t in c.items()}


def unit_rows(oracle_q8, c, name, b, h, n):
    """Float64 rows that unit (b, h) of a cache stands for."""
    return oracle_q8.rows(np64(c[name][b, h]), c[name + "s"][b, h].cpu().numpy(), np64(c[name + "t"][b, h]), n,
                          c[name + "t"].shape[2])


def _bytes(t):
    return t.contiguous().reshape(-1).view(torch.uint8)


def same_bits(a, b):
    if a is None or b is None:
        return a is b
    return a.dtype == b.dtype and a.shape == b.shape and torch.equal(_bytes(a), _bytes(b))


def check_written(oracle_q8, before, after, name, u, x, n, fmt):
    """Unit u's K or V after `n` slots of float64 rows x were written: bit-exact codes, scales and
    unfinished rows, everything behind them as before."""
    b, h = u
    block = after[name + "t"].shape[2]
    f = n // block
    code, scale, tail = np64(after[name][b, h]), after[name + "s"][b, h].cpu().numpy(), after[name + "t"][b, h]
    for i in range(f):
        want, a = oracle_q8.quantise(x[i * block:(i + 1) * block].astype(np.float32), fmt)
        assert scale[i] == a, (u, name, i, scale[i], a)
        np.testing.assert_array_equal(code[i * block:(i + 1) * block], want, err_msg=f"{u} {name} block {i}")
    want_tail = before[name + "t"][b, h].clone()
    want_tail[:n - f * block] = torch.from_numpy(x[f * block:n].astype(np.float32)).to(want_tail.dtype).to(want_tail.device)
    assert same_bits(tail, want_tail), (u, name, "unfinished rows")
    assert same_bits(after[name][b, h, f * block:], before[name][b, h, f * block:])
    assert same_bits(after[name + "s"][b, h, f:], before[name + "s"][b, h, f:])
