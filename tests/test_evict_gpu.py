"""Eviction by accumulated weight against a plain model: pools, weights, tables, lengths and counts, bit for bit."""
import math

import numpy as np
import pytest
import torch

from _serving import PAGE, tiles
from _shared import evict

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss():
    import block_sparse_attention_sm_gb300 as ss

    ss.build()
    return ss


def make(rng, lens, layers, Hkv, row, per=2, shared=0, spare=8, kind="skewed", dtype=torch.bfloat16):
    """State on the CPU; the first `shared` pages are held by all sequences that have them full."""
    width = max(1, max(tiles(L) for L in lens)) + 1
    pages = shared + sum(tiles(L) for L in lens) + spare
    order = [int(x) for x in rng.permutation(pages)]
    front, rest = order[:shared], iter(order[shared:])
    table, refs = [], [0] * pages
    for L in lens:
        mine = front[:L // PAGE]
        mine = mine + [next(rest) for _ in range(tiles(L) - len(mine))]
        for p in mine:
            refs[p] += 1
        table.append(mine + [-1] * (width - len(mine)))
    g = torch.Generator().manual_seed(int(rng.integers(1 << 30)))
    pools = [torch.randn(pages, Hkv, PAGE, row, generator=g).to(dtype) for _ in range(layers * per)]
    shape = (len(lens), Hkv, width * PAGE)
    weights = []
    for _ in range(layers):
        w = torch.rand(shape, generator=g) ** 8 * 50
        if kind == "ties":
            w = w.round()
        elif kind == "equal":
            w = torch.full(shape, 0.25)
        elif kind == "odd":  # signs, zeros of both signs, infinities, NaN, denormals
            w = torch.randn(shape, generator=g)
            pick = torch.rand(shape, generator=g)
            for lo, x in ((0.1, 0.0), (0.2, -0.0), (0.25, math.inf), (0.3, -math.inf), (0.4, math.nan), (0.45, 1e-42)):
                w = torch.where((pick < lo) & (pick >= lo - 0.05), torch.tensor(x), w)
        weights.append(w)
    return pools, weights, refs, table, lens


def same(a, b):
    """Bit for bit (NaN included)."""
    view = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.cpu().contiguous().view(view), b.contiguous().view(view))


def check(ss, state, keep, recent, rows=None, out=False, **kw):
    pools, weights, refs, table, lens = state
    ints = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    gp, gw = [p.cuda() for p in pools], [w.cuda() for w in weights]
    gr, gt, gl = ints(refs), ints(table), ints(lens)
    more, new_w = {}, gw
    if out:
        new_w = [torch.full_like(w, 7.0) for w in gw]
        more = dict(out_weights=new_w, out_refs=torch.full_like(gr, 9), out_table=torch.full_like(gt, 9), out_lens=torch.full_like(gl, 9))
    result = ss.pages_evict(gp, gw, gr, gt, gl, ints(keep), rows=None if rows is None else ints(rows), recent=recent, **more, **kw)
    was = [w.clone() for w in weights]
    want, refs2, table2, lens2 = evict(pools, weights, refs, table, lens, keep, recent, rows)
    assert int(result) == want
    if out and want == 0:
        gr, gt, gl = more["out_refs"], more["out_table"], more["out_lens"]
    assert gr.tolist() == refs2
    assert gt.tolist() == table2
    assert gl.tolist() == lens2
    for a, b in zip(gp, pools):
        assert same(a, b)
    listed = list(range(len(keep))) if rows is None else rows
    for g, old, w in zip(new_w, was, weights):
        if out:  # the inputs are as they were; unlisted rows of the output too
            full = torch.full_like(w, 7.0)
            if want == 0:
                for r, k in zip(listed, keep):
                    full[r] = 0
                    n = min(k, lens[r])
                    full[r, :, :n] = w[r, :, :n]
            w = full
        assert same(g, w)
    if out:
        for g, old in zip(gw, was):
            assert same(g, old)


CASES = [  # lengths, keep, recent, layers, Hkv, row, shared
    ([1], [1], 0, 1, 1, 64, 0),
    ([1, 5], [0, 3], 0, 1, 2, 64, 0),
    ([300, 129, 128, 0], [100, 129, 127, 5], 32, 1, 2, 64, 0),
    ([900, 640, 1000], [300, 200, 448], 32, 1, 2, 64, 0),
    ([513, 700], [512, 1], 0, 2, 1, 128, 0),
    ([2000], [1999], 64, 1, 1, 128, 0),
    ([400, 500, 600], [200, 130, 300], 10, 2, 2, 64, 2),
    ([400, 130, 600], [400, 128, 10], 300, 1, 2, 128, 3),
    ([1500, 1400], [900, 128], 2000, 1, 3, 72, 4),
]


@pytest.mark.parametrize("out", [False, True])
@pytest.mark.parametrize("kind", ["skewed", "ties", "equal", "odd"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_the_model(ss, case, kind, out):
    lens, keep, recent, layers, Hkv, row, shared = CASES[case]
    rng = np.random.default_rng(case)
    check(ss, make(rng, lens, layers, Hkv, row, shared=shared, kind=kind), keep, recent, out=out)
