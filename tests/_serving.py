"""Plain 64-bit implementations of the calls around the paged cache, and the
pools, tables and batches that their tests share."""
import math

import numpy as np
import torch

PAGE = 128


def tiles(L):
    return -(-L // PAGE)


# ------------------------------------------------------------------- rotary positions


def rotate(x, pos, inv_freq, factor, off, interleaved, inverse=False):
    """x [..., d] (64 bits) turned at the positions pos (broadcast against x's leading axes)."""
    x = x.double()
    rot = 2 * inv_freq.shape[0]
    t = pos.double()[..., None] * inv_freq.double()
    c, s = factor * torch.cos(t), factor * torch.sin(t) * (-1 if inverse else 1)
    y = x.clone()
    z = x[..., off:off + rot]
    a, b = (z[..., 0::2], z[..., 1::2]) if interleaved else (z[..., :rot // 2], z[..., rot // 2:])
    ra, rb = a * c - b * s, b * c + a * s
    if interleaved:
        y[..., off:off + rot] = torch.stack([ra, rb], -1).flatten(-2)
    else:
        y[..., off:off + rot] = torch.cat([ra, rb], -1)
    return y


def rotate_tolerance(x, inv_freq, factor, off, interleaved):
    """What fp32 arithmetic and one rounding to bf16 may be off by, per entry.

    The angle: its fraction of a turn is cut at 2^-32 and rounded to a float
    (2^-25 of half a turn: 9.4e-8 rad), sincospif is good to 2 ulp (1.2e-7),
    the factor, two products and a sum round at 2^-24 each: below 6e-7 of
    factor * (|a| + |b|).  Copied entries are exact."""
    rot = 2 * inv_freq.shape[0]
    z = x.double().abs()[..., off:off + rot]
    a, b = (z[..., 0::2], z[..., 1::2]) if interleaved else (z[..., :rot // 2], z[..., rot // 2:])
    w = 6e-7 * factor * (a + b)
    part = torch.stack([w, w], -1).flatten(-2) if interleaved else torch.cat([w, w], -1)
    tol = torch.zeros_like(x, dtype=torch.float64)
    tol[..., off:off + rot] = part
    return tol


def assert_rounded(got, want, tol, what=""):
    """got (bf16) is want (64 bits), off by tol and then rounded: half a step is 2^-8 of the value."""
    err = (got.double() - want).abs()
    allowed = tol + (want.abs() + tol) * 2.0 ** -8 + 1e-40
    bad = ~(err <= allowed)
    assert not bad.any(), f"{what}: {int(bad.sum())} entries off, worst {float((err - allowed).max()):.3e}"


# ------------------------------------------------------------------------- the cache


def random_tables(L, spare, rng, width=None):
    """Page table over shuffled pages for sequences of these lengths: (table, pages)."""
    need = sum(tiles(x) for x in L)
    order = [int(p) for p in rng.permutation(need + spare)]
    width = width or max(1, max(tiles(x) for x in L))
    # entries past a sequence's last page name a page of somebody else
    table = np.full((len(L), width), order[0] if order else 0, dtype=np.int32)
    at = 0
    for b, x in enumerate(L):
        table[b, :tiles(x)] = order[at:at + tiles(x)]
        at += tiles(x)
    return torch.from_numpy(table), need + spare


def fill_pool(k, L, table, pages):
    """Pool [pages][Hkv][128][d] of the sequences' rows k[b] [Hkv, L_b, d]; NaN everywhere else."""
    Hkv, _, d = k[0].shape
    pool = torch.full((pages, Hkv, PAGE, d), float("nan"), dtype=k[0].dtype)
    for b, x in enumerate(L):
        for j in range(tiles(x)):
            n = min(PAGE, x - j * PAGE)
            pool[table[b, j], :, :n] = k[b][:, j * PAGE:j * PAGE + n]
    return pool


def offsets(n):
    return torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32)


# -------------------------------------------------------------- attention of a chunk


def chunk_place(cu, b, block, G, T, B):
    """Place and half of block `block` of sequence b, and the number of places."""
    m = PAGE // G
    return cu[b] // (2 * m) + b + block // 2, block % 2, T // (2 * m) + B


def chunk_reference(q, k, v, L, scale, causal, a, splits, keep=None):
    """One sequence: q [n, Hq, d], k / v [Hkv, >= L, d] -> o [n, Hq, d], weights |P||V| / l, and the vote
    statistic c [Hkv, blocks, tiles] (nan: not seen by the block), all in 64 bits.

    keep: bool [Hkv, blocks, tiles] decisions to use in place of the vote's."""
    n, Hq, d = q.shape
    Hkv = k.shape[0]
    G = Hq // Hkv
    m = PAGE // G
    nT, blocks = tiles(L), -(-n // m) if n else 0
    per = -(-nT // splits) if nT else 1
    ln_lam = math.log(min(1.0, a / L)) if a > 0 and L > 0 else -math.inf
    o = torch.zeros(n, Hq, d, dtype=torch.float64)
    weight = torch.zeros(n, Hq, d, dtype=torch.float64)
    c = torch.full((Hkv, blocks, nT), math.nan, dtype=torch.float64)
    for h in range(Hkv):
        kk, vv = k[h, :L].double(), v[h, :L].double()
        for blk in range(blocks):
            i0, i1 = blk * m, min(n, blk * m + m)
            rows = q[i0:i1, h * G:(h + 1) * G].double().reshape(-1, d)
            sees = torch.arange(i0, i1).repeat_interleave(G) + (L - n) if causal else torch.full((len(rows),), L - 1)
            S = rows @ kk.T * scale
            S[torch.arange(L)[None, :] > sees[:, None]] = -math.inf
            seen = 0 if sees.max() < 0 else min(nT, int(sees.max()) // PAGE + 1)
            top = None
            for j in range(seen):
                if j % per == 0:
                    top = torch.full((len(rows),), -math.inf, dtype=torch.float64)
                t = S[:, j * PAGE:(j + 1) * PAGE].amax(1)
                stat = torch.where(t == -math.inf, -math.inf, torch.where(top == -math.inf, math.inf, t - top))
                c[h, blk, j] = stat.max()
                kept = bool(keep[h, blk, j]) if keep is not None else not bool(c[h, blk, j] < ln_lam)
                top = torch.maximum(top, t)
                if not kept:
                    S[:, j * PAGE:(j + 1) * PAGE] = -math.inf
            mx = S.amax(1, keepdim=True) if L else torch.full((len(rows), 1), -math.inf, dtype=torch.float64)
            P = torch.exp(S - torch.where(mx == -math.inf, 0.0, mx))
            l = P.sum(1, keepdim=True)
            inv = torch.where(l > 0, 1.0 / l, 0.0)
            o[i0:i1, h * G:(h + 1) * G] = (P @ vv * inv).view(i1 - i0, G, d)
            weight[i0:i1, h * G:(h + 1) * G] = (P @ vv.abs() * inv).view(i1 - i0, G, d)
    return o, weight, c


def assert_attention(got, o, weight, what=""):
    """Each weight is rounded to bf16 once (half a step, 2^-8 of it), so the sums of weighted values are off
    by 2^-8 sum p|v| / l at most; scores in fp32 and exp2 add below 2^-11 of the same sum, the output rounds
    once more to bf16."""
    tol = (2.0 ** -8 + 2.0 ** -11) * weight
    assert_rounded(got, o, tol + 1e-30, what)
