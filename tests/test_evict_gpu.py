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


def test_listed_rows(ss):
    rng = np.random.default_rng(20)
    for out in (False, True):
        state = make(rng, [300, 500, 129, 700, 64], 2, 2, 64, shared=1)
        check(ss, state, [100, 650, 129], 16, rows=[3, 0, 2], out=out)
        check(ss, state, [], 16, rows=[], out=out)


@pytest.mark.parametrize("out", [False, True])
def test_refused_without_free_pages(ss, out):
    """Shared pages must be replaced and there are too few free ones: nothing changes."""
    rng = np.random.default_rng(21)
    state = make(rng, [700, 650, 900], 1, 2, 64, shared=4, spare=3)
    before = [x.clone() for x in state[0] + state[1]]
    pools, weights, refs, table, lens = state
    for p in [p for p, n in enumerate(refs) if n == 0][3:]:  # (somebody else's)
        refs[p] = 1
    ints = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    gp, gw, gr, gt, gl = [p.cuda() for p in pools], [w.cuda() for w in weights], ints(refs), ints(table), ints(lens)
    r = ss.pages_evict(gp, gw, gr, gt, gl, ints([200, 200, 200]), recent=10)
    assert int(r) == 3  # two pages a sequence, three free
    assert gr.tolist() == refs and gt.tolist() == table and gl.tolist() == lens
    assert all(same(a, b) for a, b in zip(gp + gw, before))
    check(ss, state, [128, 200, 700], 10, out=out)  # one, two and none


@pytest.mark.parametrize("what", ["row", "twice", "keep", "length", "long"])
def test_wrong_arguments_change_nothing(ss, what):
    rng = np.random.default_rng(22)
    pools, weights, refs, table, lens = make(rng, [300, 500, 129], 1, 2, 64)
    rows, keep = [0, 1, 2], [100, 100, 100]
    if what == "row":
        rows[1] = 3
    elif what == "twice":
        rows[1] = 2
    elif what == "keep":
        keep[2] = -1
    elif what == "length":
        lens[1] = -5
    else:
        lens[1] = len(table[0]) * PAGE + 1
    ints = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    gp, gw, gr, gt, gl = [p.cuda() for p in pools], [w.cuda() for w in weights], ints(refs), ints(table), ints(lens)
    r = ss.pages_evict(gp, gw, gr, gt, gl, ints(keep), rows=ints(rows))
    assert int(r) == -1
    assert gr.tolist() == refs and gt.tolist() == table and gl.tolist() == lens
    assert all(same(a, b) for a, b in zip(gp + gw, pools + weights))
    ss.stream_status()


def test_many_layers_and_pools(ss):
    """More layers than a launch takes; one pool a layer (latent rows), three, and wide rows."""
    rng = np.random.default_rng(23)
    check(ss, make(rng, [200, 300], 19, 1, 8, shared=1), [100, 257], 5)
    check(ss, make(rng, [200, 300], 25, 2, 8, per=3), [100, 257], 5, out=True)
    check(ss, make(rng, [300, 200], 2, 1, 576, per=1), [130, 7], 0)
    check(ss, make(rng, [260], 1, 1, 3080, per=1), [200], 1)
    check(ss, make(rng, [260, 140], 1, 2, 36, dtype=torch.float32), [200, 100], 1)


def test_latent_pools_without_a_head_axis(ss):
    rng = np.random.default_rng(24)
    pools, weights, refs, table, lens = make(rng, [300, 290], 1, 1, 64, per=1)
    ints = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    flat = pools[0][:, 0].contiguous().cuda()
    gr, gt, gl, gw = ints(refs), ints(table), ints(lens), weights[0].cuda()
    assert int(ss.pages_evict([flat], [gw], gr, gt, gl, ints([100, 20]), recent=3)) == 0
    evict(pools, weights, refs, table, lens, [100, 20], 3)
    assert same(flat, pools[0][:, 0])


@pytest.mark.parametrize("kind", ["skewed", "ties", "odd"])
def test_long_sequences(ss, kind):
    """More keys than a choosing block holds in registers."""
    rng = np.random.default_rng(25)
    pools, weights, refs, table, lens = make(rng, [40000, 17000], 1, 1, 8, kind=kind, per=1)
    ints = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    gp, gw, gr, gt, gl = [p.cuda() for p in pools], [w.cuda() for w in weights], ints(refs), ints(table), ints(lens)
    keep, recent = [5000, 16999], 100
    assert int(ss.pages_evict(gp, gw, gr, gt, gl, ints(keep), recent=recent)) == 0
    from _shared import choose
    for r, k in enumerate(keep):
        src = choose(weights[0][r, 0, :lens[r]].double(), k, recent)
        assert same(gw[0][r, 0, :k], weights[0][r, 0, src]) and (gw[0][r, 0, k:] == 0).all()
        t = torch.tensor(table[r])
        old = pools[0][t[src // PAGE], 0, src % PAGE]
        assert same(gp[0][gt[r, :tiles(k)].long()].cpu()[:, 0].flatten(0, 1)[:k].contiguous(), old.contiguous())


def test_streams_and_graphs(ss):
    rng = np.random.default_rng(26)
    ints = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    states = [make(rng, [700, 400 + i], 2, 2, 64, shared=1) for i in range(2)]
    cuda = [([p.cuda() for p in s[0]], [w.cuda() for w in s[1]], ints(s[2]), ints(s[3]), ints(s[4])) for s in states]
    out = [dict(out_weights=[torch.zeros_like(w) for w in c[1]], out_refs=torch.zeros_like(c[2]), out_table=torch.zeros_like(c[3]),
                out_lens=torch.zeros_like(c[4])) for c in cuda]
    keep = ints([300, 200])
    saved = [[p.clone() for p in c[0]] for c in cuda]
    graphs = []
    for c, o in zip(cuda, out):
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            ss.pages_evict(*c, keep, recent=8, **o)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ss.pages_evict(*c, keep, recent=8, **o)
        graphs.append(g)
    for turn in range(2):
        for c, s in zip(cuda, saved):
            for p, x in zip(c[0], s):
                p.copy_(x)
        keep.copy_(torch.tensor([300 - 50 * turn, 200 + 9 * turn]))
        torch.cuda.synchronize()
        for g in graphs:
            with torch.cuda.stream(torch.cuda.Stream()):
                g.replay()
        torch.cuda.synchronize()
        for s, c, o in zip(states, cuda, out):
            pools, weights = [p.clone() for p in s[0]], [w.clone() for w in s[1]]
            want, refs, table, lens = evict(pools, weights, s[2], s[3], s[4], keep.tolist(), 8)
            assert want == 0 and o["out_refs"].tolist() == refs and o["out_table"].tolist() == table
            assert all(same(a, b) for a, b in zip(c[0], pools)) and all(same(a, b) for a, b in zip(o["out_weights"], weights))


@pytest.mark.parametrize("layers", [1, 16, 17, 40])
@pytest.mark.parametrize("out", [False, True])
def test_nothing_listed(ss, layers, out):
    """No sequence listed, layers of one launch and of several: the state is passed on as it is."""
    rng = np.random.default_rng(25)
    for rows in (None, []):
        check(ss, make(rng, [200, 300], layers, 1, 8, shared=1), [], 3, rows=rows, out=out)
