"""Float64 references and tolerances of the tests of rotary positions, block digests, block-sparse
and shared-prefix attention.

Attention: with A = scale max_j sum_c |q_c k_jc| a logit is off by dl = c A, c = 2^-18 where the products of
bf16 operands are exact and their sums may be cut off (d / 16 steps of 2^-23), 2^-17 for fp32
operands in two tf32 parts (products to 2^-21, 3 d / 8 steps).  A weight is off by a factor
1 +- (2 dl + 2^-18) (the logit, the normaliser; exponentials 2^-22 and products' sums), and by w more
where weights are rounded: 2^-8 for the prefix's bf16 weights (half a step), 2^-16 where they enter as
two bf16 parts, 2^-20 as two tf32 parts.  A sum over n slots that may be cut off at every 16th
adds n / 16 steps of 2^-23.  So with mass = sum_j p_j |v_j|
    |o - o_exact| <= (2 dl + 2^-18 + w + n 2^-27) mass + half a step of the type |o|,
    |lse - lse_exact| <= dl + 2^-20 + 2^-22 |lse| + n 2^-28 (its sum of fp32 weights, shared out over lanes).

Rotary positions: an angle is off by less than 2^-23 rad (its fraction of a turn cut at 2^-32, rounded to 24
bits below half a turn; the frequency's own 2^-55 turns times the position, 2^-30 rad up to 2^20), so
cosine and sine by 2^-22 with their own two units in the last place.  The norm's factor is off by 2^-20
(a sum of at most 19 roundings, halved by the root; the root's 2^-22; two products), so a turned
element by (2^-20 + 2^-22 + 2^-23) (|a| + |b|) rot_scale <= 2^-19 (|a| + |b|) rot_scale.
"""
import math

import numpy as np
import torch

BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}  # half a step, relative


def rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def attend(q, k, v, scale):
    """q [r][d], k, v [n][d] in float64 -> o, lse, mass (sum p |v|), A."""
    if k.shape[0] == 0:
        z = torch.zeros_like(q)
        return z, torch.full((len(q),), -math.inf, dtype=q.dtype, device=q.device), z, torch.zeros(len(q), device=q.device).double()
    x = scale * (q @ k.T)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse[:, None])
    return p @ v, lse, p @ v.abs(), scale * (q.abs() @ k.abs().T).amax(-1)


def check_rows(o, lse, q, k, v, scale, w, what):
    """Rows o, lse (as computed) of queries q over keys k and values v (as given)."""
    bf = q.dtype == BF
    want, wl, mass, A = attend(q.double(), k.double(), v.double(), scale)
    n = k.shape[0]
    dl = (2.0 ** -18 if bf else 2.0 ** -17) * A
    bound = (2 * dl + 2.0 ** -18 + w + n * 2.0 ** -27)[:, None] * mass + HALF[q.dtype] * want.abs() + 1e-37
    err = (o.double() - want).abs()
    assert bool((err <= bound).all()), f"{what}: o off by {float((err / bound).max()):.2f} of its bound"
    if lse is not None:
        empty = wl == -math.inf
        assert torch.equal(lse == -math.inf, empty), what
        el = (lse.double() - wl).abs()[~empty]
        bl = (dl + 2.0 ** -20 + 2.0 ** -22 * wl.abs() + n * 2.0 ** -28)[~empty]
        assert bool((el <= bl).all()), f"{what}: lse off by {float((el / bl).max()):.2f} of its bound"


def digests(K, lens, block, old, n_new=None):
    """K [B][H][cap][d] (any float type), lens [B][H] list -> digest as kv_block_digest leaves it over `old`."""
    out = old.clone()
    B, H, cap, d = K.shape
    for b in range(B):
        for h in range(H):
            n = int(lens[b][h])
            first = 0 if n_new is None else max(0, n - n_new) // block
            for j in range(first, -(-n // block)):
                x = K[b, h, j * block:min(n, (j + 1) * block)]
                out[b, h, j, 0], out[b, h, j, 1] = x.amin(0), x.amax(0)
    return out


def choose(q, dig, seen, block, n_sel, sink, recent):
    """q [G][d], dig [nb][2][d] in float64 -> the chosen blocks, ascending."""
    nb = -(-seen // block)
    if nb <= n_sel:
        return list(range(nb))
    q, dig = q.cpu().numpy(), dig[:nb].cpu().numpy()
    with np.errstate(all="ignore"):
        u = (np.maximum(q, 0) @ dig[:, 1].T + np.minimum(q, 0) @ dig[:, 0].T)
    u = np.where(np.isnan(u), np.inf, u).max(0)
    fixed = list(range(sink)) + list(range(nb - recent, nb))
    mid = np.arange(sink, nb - recent)
    best = mid[np.lexsort((mid, -u[mid]))][:n_sel - len(fixed)]
    return sorted(fixed + best.tolist())
