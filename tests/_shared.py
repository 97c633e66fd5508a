"""Plain 64-bit implementations of the calls over shared pages, of the record of
attention weights and of eviction, and the batches that their tests share."""
import math

import torch

from _serving import PAGE, tiles


def sequence(pool, row, L):
    """Rows [Hkv, L, d] of a sequence with these pages."""
    n = tiles(L)
    return pool[row[:n].long()].transpose(0, 1).flatten(1, 2)[:, :L]


def scores(q, k, scale):
    """[n, Hq, d] x [Hkv, L, d] -> scores [Hkv, n, G, L] and what fp32 arithmetic may be off by in them.

    A product of two bf16 is exact in fp32; the 2^-24 of a sum's rounding (twice that where the sum is
    truncated) is made at most d times, relative to the sum of the products' magnitudes."""
    n, Hq, d = q.shape
    Hkv = k.shape[0]
    r = q.double().view(n, Hkv, Hq // Hkv, d)
    S = torch.einsum("nhgd,hkd->hngk", r, k.double()) * scale
    size = torch.einsum("nhgd,hkd->hngk", r.abs(), k.double().abs()) * scale
    return S, size * (d * 2.0 ** -23)


def softmax(q, k, scale, sees):
    """Weights [Hkv, n, G, L] of rows whose last visible key is sees[i], and their relative tolerance."""
    S, off = scores(q, k, scale)
    L = k.shape[1]
    hidden = torch.arange(L, device=S.device) > sees[:, None, None]
    S = S.masked_fill(hidden, -math.inf)
    P = torch.softmax(S, -1)
    P = torch.where(hidden | (sees < 0)[:, None, None], torch.zeros_like(P), P)
    # Scores are off by `off` in the weight and in the sum; the sum of L terms rounds along a thread's 64
    # pairs, the tiles and the partial results (2^-24 each); exp2 is good to 2^-22, its argument and the
    # logarithm of the sum round at 2^-24 of numbers below |s| + log2 L (in units of log2, 1.45 of them).
    worst = off.masked_fill(hidden, 0.0).amax(-1, keepdim=True)
    top = S.masked_fill(hidden, 0.0).abs().amax(-1, keepdim=True)
    rel = 2.0 * worst + (64 + 8 + 2 * tiles(L)) * 2.0 ** -24 + 4 * 2.0 ** -22 + 4 * 1.45 * (top + math.log(L + 1.0)) * 2.0 ** -24
    return P, rel


def assert_close(got, want, tol, what=""):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} entries off, worst {float((err - tol).max()):.3e}"


def tree_batch(rng, B, groups, root, doc, own):
    """(lengths, tables as lists, pages): sequences that share root tokens, groups of them doc more, own[b] to themselves."""
    used = {}
    lens, table = [], []

    def page(name):
        return used.setdefault(name, len(used))

    for b in range(B):
        g = b % max(1, groups)
        L = root + doc + own[b]
        row = []
        for j in range(tiles(L)):
            if groups and j < root // PAGE:
                row.append(page(("root", j)))
            elif groups and j < (root + doc) // PAGE:
                row.append(page(("doc", g, j)))
            else:
                row.append(page(("own", b, j)))
        lens.append(L)
        table.append(row)
    order = [int(x) for x in rng.permutation(len(used) + 3)]
    table = [[order[p] for p in row] for row in table]
    width = max(1, max(len(r) for r in table))
    return lens, [r + [order[-1]] * (width - len(r)) for r in table], len(used) + 3


def choose(weight, keep, recent):
    """Kept keys of one head, ascending, by the definition: weight [L] in 64 bits."""
    L = weight.shape[0]
    if L <= keep:
        return torch.arange(L)
    newest = min(recent, keep)
    w = torch.where(torch.isnan(weight), torch.full_like(weight, -math.inf), weight).tolist()
    nan = torch.isnan(weight).tolist()
    old = sorted(range(L - newest), key=lambda k: (nan[k], -w[k], k))[:keep - newest]
    return torch.tensor(sorted(old) + list(range(L - newest, L)), dtype=torch.long)


def evict(pools, weights, refs, table, lens, keep, recent, rows=None):
    """The state after an eviction: (result, refs, table, lens); pools and weights (CPU) are changed in place."""
    rows = list(range(len(keep))) if rows is None else rows
    refs, table, lens = list(refs), [list(r) for r in table], list(lens)
    was = [list(r) for r in table]
    free = [p for p, n in enumerate(refs) if n == 0]
    cut = [(r, min(k, lens[r])) for r, k in zip(rows, keep)]
    need = sum(refs[was[r][j]] > 1 for r, k in cut if k < lens[r] for j in range(tiles(k)))
    if need > len(free):
        return need - len(free), refs, table, lens
    held = list(refs)
    old_pools, old_weights = [p.clone() for p in pools], [w.clone() for w in weights]
    per = len(pools) // len(weights)
    for r, k in cut:
        L = lens[r]
        if k < L:
            for j in range(tiles(L)):
                p = was[r][j]
                if j >= tiles(k) or held[p] > 1:
                    refs[p] -= 1
                    if j < tiles(k):
                        table[r][j] = free.pop(0)
                        refs[table[r][j]] = 1
        for j in range(tiles(k), len(table[r])):
            table[r][j] = -1
        if k < L:
            for i, w in enumerate(weights):
                for h in range(w.shape[1]):
                    src = choose(old_weights[i][r, h, :L].double(), k, recent)
                    w[r, h] = 0
                    w[r, h, :k] = old_weights[i][r, h, src]
                    for q in range(i * per, i * per + per):
                        for d, s in enumerate(src.tolist()):
                            pools[q][table[r][d // PAGE], h, d % PAGE] = old_pools[q][was[r][s // PAGE], h, s % PAGE]
        lens[r] = k
    return 0, refs, table, lens
