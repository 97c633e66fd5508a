"""Decode over shared pages and the record of attention weights against 64-bit arithmetic."""
import math

import numpy as np
import pytest
import torch

from _serving import PAGE, assert_attention, tiles
from _shared import assert_close, sequence, softmax, tree_batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss():
    import block_sparse_attention_sm_gb300 as ss

    ss.build()
    return ss


def make(rng, lens, table, pages, Hq, Hkv, d, peak=6.0):
    """Queries and pools on the GPU; what the pools hold behind the sequences' ends is NaN."""
    g = torch.Generator().manual_seed(int(rng.integers(1 << 30)))
    u = torch.nn.functional.normalize(torch.randn(Hkv, 1, d, generator=g), dim=-1)
    kp = torch.randn(pages, Hkv, PAGE, d, generator=g)
    kp += peak * u * (torch.rand(pages, Hkv, PAGE, 1, generator=g) < 0.02)
    vp = torch.randn(pages, Hkv, PAGE, d, generator=g)
    q = torch.randn(len(lens), Hkv, Hq // Hkv, d, generator=g) + peak * u
    seen = torch.zeros(pages, PAGE, dtype=torch.bool)
    for L, row in zip(lens, table):
        for j in range(tiles(L)):
            seen[row[j], :min(PAGE, L - j * PAGE)] = True
    for p in (kp, vp):
        p.transpose(1, 2)[~seen] = math.nan
    bf = lambda x: x.to(torch.bfloat16).cuda().contiguous()  # noqa: E731
    ints = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    return bf(q).view(len(lens), Hq, d), bf(kp), bf(vp), ints(table), ints(lens)


def check(ss, q, kp, vp, table, lens, plan, weights=True, **kw):
    B, Hq, d = q.shape
    Hkv, scale = kp.shape[1], 1.3 / math.sqrt(d)
    W = table.shape[1] * PAGE
    w = w0 = None
    if weights:
        w = torch.rand(B, Hkv, W, device="cuda")
        w0 = w.clone()
    o = ss.decode_shared(q, kp, vp, table, lens, plan, scale=scale, weights=w, **kw)
    assert ss.stream_status() is None
    for b, L in enumerate(lens.tolist()):
        if L == 0:
            assert (o[b] == 0).all()
            assert w is None or torch.equal(w[b], w0[b])
            continue
        k, v = sequence(kp, table[b], L), sequence(vp, table[b], L).double()
        P, rel = softmax(q[b:b + 1], k, scale, torch.tensor([L - 1], device="cuda"))
        want = torch.einsum("hngk,hkd->nhgd", P, v).reshape(Hq, d)
        weight = torch.einsum("hngk,hkd->nhgd", P, v.abs()).reshape(Hq, d)
        assert_attention(o[b], want, weight, f"sequence {b} of {L} keys")
        if w is not None:
            gain = P.sum((1, 2))
            tol = (P * rel).sum((1, 2)) + (w0[b, :, :L].double() + gain) * 2.0 ** -23 + 1e-37
            assert_close(w[b, :, :L], w0[b, :, :L].double() + gain, tol, f"weights of sequence {b}")
            assert torch.equal(w[b, :, L:], w0[b, :, L:])
    return o, w


SIZES = [  # B, groups, root, doc, own lengths up to, Hq, Hkv, d
    (1, 0, 0, 0, 1, 4, 1, 128),
    (1, 0, 0, 0, 3000, 8, 2, 128),
    (3, 0, 0, 0, 128, 8, 8, 64),
    (5, 1, 300, 0, 200, 8, 2, 128),
    (7, 1, 256, 0, 1, 12, 4, 64),
    (9, 3, 140, 700, 260, 10, 2, 128),
    (33, 1, 1100, 0, 130, 8, 2, 128),
    (40, 4, 513, 400, 300, 28, 4, 128),
    (70, 2, 384, 0, 90, 16, 2, 64),
    (65, 1, 128, 128, 5, 16, 1, 128),
    (130, 5, 260, 256, 40, 6, 2, 64),
    (3, 1, 129, 0, 10, 128, 1, 128),
    (4, 2, 640, 0, 20, 100, 1, 64),
]


@pytest.mark.parametrize("planned", [True, False])
@pytest.mark.parametrize("B,groups,root,doc,own,Hq,Hkv,d", SIZES)
def test_against_64_bits(ss, B, groups, root, doc, own, Hq, Hkv, d, planned):
    rng = np.random.default_rng(B * 1000 + own)
    owns = rng.integers(1, own + 1, B)
    lens, table, pages = tree_batch(rng, B, groups, root, doc, [int(x) for x in owns])
    q, kp, vp, table, lens = make(rng, lens, table, pages, Hq, Hkv, d)
    plan = ss.prefix_plan(table, lens) if planned else None
    check(ss, q, kp, vp, table, lens, plan)
    check(ss, q, kp, vp, table, lens, plan, weights=False)


@pytest.mark.parametrize("B", [2, 8, 9, 16])
def test_plans_of_small_batches(ss, B):
    """The sequences' places and the nodes above them, by one launch or two, and what they share with them."""
    rng = np.random.default_rng(B)
    lens, table, pages = tree_batch(rng, B, 2, 400, 300, [int(x) for x in rng.integers(1, 300, B)])
    q, kp, vp, table, lens = make(rng, lens, table, pages, 8, 2, 64)
    plans = [ss.prefix_plan(table, lens) for _ in range(3)]
    assert sorted(plans[0][8:8 + B].tolist()) == list(range(B))
    assert all(torch.equal(p, plans[0]) for p in plans)
    check(ss, q, kp, vp, table, lens, plans[0])
    order = torch.from_numpy(rng.permutation(B)).cuda()
    o, _ = check(ss, q, kp, vp, table, lens, plans[0], weights=False)
    swapped = table[order].contiguous()
    p, _ = check(ss, q[order].contiguous(), kp, vp, swapped, lens[order].contiguous(), ss.prefix_plan(swapped, lens[order].contiguous()),
                 weights=False)
    assert p.shape == o.shape


def batch(rng, B=12, groups=3, root=300, doc=200, own=300, Hq=8, Hkv=2, d=128):
    lens, table, pages = tree_batch(rng, B, groups, root, doc, [int(x) for x in rng.integers(1, own + 1, B)])
    return make(rng, lens, table, pages, Hq, Hkv, d)


def test_empty_sequences_and_unused_rows(ss):
    rng = np.random.default_rng(1)
    q, kp, vp, table, lens = batch(rng)
    for gone in ([0, 5], [11], list(range(12))):
        some = lens.clone()
        some[gone] = 0
        for plan in (None, ss.prefix_plan(table, some), ss.prefix_plan(table, lens)):  # (the last: sequences that have ended since)
            check(ss, q, kp, vp, table, some, plan)


def test_plan_holds_while_sequences_grow(ss):
    """Lengths grow under one plan, within their last pages and into new ones."""
    rng = np.random.default_rng(2)
    owns = [int(x) for x in rng.integers(1, 200, 9)]
    lens, table, pages = tree_batch(rng, 9, 2, 400, 260, [x + 400 for x in owns])
    q, kp, vp, table, full = make(rng, lens, table, pages, 8, 2, 64)
    short = full - torch.tensor([400 - int(x) for x in rng.integers(0, 3, 9)], dtype=torch.int32).cuda()
    plan = ss.prefix_plan(table, short)
    kept = plan.clone()
    for add in (0, 1, 90, 128, 397):
        check(ss, q, kp, vp, table, torch.minimum(short + add, full), plan)
    assert torch.equal(plan, kept)


def test_plan_of_other_sizes_is_not_used(ss):
    rng = np.random.default_rng(3)
    q, kp, vp, table, lens = batch(rng)
    want, _ = check(ss, q, kp, vp, table, lens, None)
    other = ss.prefix_plan(torch.cat([table, table[:, :1]], 1), lens)  # (of a wider table)
    assert torch.equal(ss.decode_shared(q, kp, vp, table, lens, other, scale=1.3 * 128 ** -0.5), want)
    with pytest.raises(ValueError, match="plan"):
        ss.decode_shared(q, kp, vp, table, lens, plan=torch.zeros(5, dtype=torch.int32, device="cuda"), scale=1.0)


def test_plan_that_holds_nothing_of_use(ss):
    """Whatever a plan's numbers are, nothing outside the given arrays is touched (guard bands around the outputs)."""
    rng = np.random.default_rng(4)
    q, kp, vp, table, lens = batch(rng, d=64)
    B, Hq, d = q.shape
    good = ss.prefix_plan(table, lens)
    band, n = 256, q.numel()
    for seed in range(6):
        g = torch.Generator(device="cuda").manual_seed(seed)
        plan = good.clone()
        plan[8:] = torch.randint(-3, 40 if seed < 3 else 1 << 30, plan[8:].shape, generator=g, device="cuda", dtype=torch.int32)
        room = torch.full((n + 2 * band,), 9.0, dtype=torch.bfloat16, device="cuda")
        W = table.shape[1] * PAGE * 2 * B
        cells = torch.full((W + 2 * band,), 9.0, device="cuda")
        ss.decode_shared(q, kp, vp, table, lens, plan, scale=0.1, out=room[band:band + n].view(q.shape),
                         weights=cells[band:band + W].view(B, 2, -1))
        assert ss.stream_status() is None
        assert (room[:band] == 9).all() and (room[-band:] == 9).all() and (cells[:band] == 9).all() and (cells[-band:] == 9).all()
    check(ss, q, kp, vp, table, lens, good)


def test_deep_chains(ss):
    """Sequences forked from one another a page at a time: more levels than a plan keeps."""
    rng = np.random.default_rng(5)
    lens, table = [], []
    for b in range(20):
        row = table[-1][:b] if b else []
        table.append(row + [100 + b, 200 + b][:2])
        lens.append(len(table[-1]) * PAGE - int(rng.integers(0, 100)))
    width = max(len(r) for r in table)
    q, kp, vp, table, lens = make(rng, lens, [r + [0] * (width - len(r)) for r in table], 300, 12, 4, 128)
    check(ss, q, kp, vp, table, lens, ss.prefix_plan(table, lens))


def test_identical_sequences(ss):
    rng = np.random.default_rng(6)
    q, kp, vp, table, lens = make(rng, [640] * 40 + [700] * 3, [[3, 1, 4, 0, 5, 6]] * 43, 9, 8, 2, 128)
    check(ss, q, kp, vp, table, lens, ss.prefix_plan(table, lens))
    check(ss, q, kp, vp, table, lens, None)


def test_one_sequence_cannot_reach_another(ss):
    """Infinities and NaN in one sequence's own keys, values or query change nothing for the others, bit for bit."""
    rng = np.random.default_rng(7)
    for Hq, Hkv, d in ((8, 2, 128), (7, 1, 64)):
        q, kp, vp, table, lens = batch(rng, Hq=Hq, Hkv=Hkv, d=d)
        plan = ss.prefix_plan(table, lens)
        for p in (plan, None):
            clean = ss.decode_shared(q, kp, vp, table, lens, p, scale=0.1)
            for bad in (math.nan, math.inf):
                for b in (0, 4):
                    q2, k2, v2 = q.clone(), kp.clone(), vp.clone()
                    page = int(table[b, (int(lens[b]) - 1) // PAGE])
                    v2[page, :, 0] = bad
                    k2[page, :, 0, 0] = bad
                    q2[b, 1] = math.nan
                    w = torch.zeros(12, Hkv, table.shape[1] * PAGE, device="cuda")
                    got = ss.decode_shared(q2, k2, v2, table, lens, p, scale=0.1, weights=w)
                    others = [i for i in range(12) if i != b]
                    assert torch.equal(got[others], clean[others])
                    assert torch.isfinite(w[others]).all() and torch.isnan(got[b, 1]).all()


def test_scores_of_any_size(ss):
    """Rows whose maximum grows by hundreds from tile to tile, falls, or stays equal."""
    rng = np.random.default_rng(8)
    q, kp, vp, table, lens = batch(rng, B=6, groups=1, root=1100, doc=0, own=600)
    scale = 1.3 * 128 ** -0.5
    u = torch.zeros(128, device="cuda")
    u[0] = 1.0
    steps = torch.arange(table.shape[1], device="cuda")
    for slope in (40.0, -40.0, 400.0, 0.0):
        k2 = kp.clone()
        for j in steps.tolist():
            k2[table[:, j].long()] = (torch.nan_to_num(kp[table[:, j].long()]).float() * 0.01 + slope * j * u).to(torch.bfloat16)
        q2 = (torch.randn(q.shape, device="cuda") * 0.1 + 8.0 * u).to(torch.bfloat16)
        v2 = torch.nan_to_num(vp)
        for plan in (ss.prefix_plan(table, lens), None):
            o = ss.decode_shared(q2, k2, v2, table, lens, plan, scale=scale)
            for b, L in enumerate(lens.tolist()):
                k, v = sequence(k2, table[b], L), sequence(v2, table[b], L).double()
                P, rel = softmax(q2[b:b + 1], k, scale, torch.tensor([L - 1], device="cuda"))
                want = torch.einsum("hngk,hkd->nhgd", P, v).reshape(8, 128)
                # (scores of thousands: what fp32 keeps of them is part of the weights' tolerance)
                size = torch.einsum("hngk,hkd->nhgd", P * (1.0 + 2.0 ** 8 * rel), v.abs()).reshape(8, 128)
                assert_attention(o[b], want, size, f"slope {slope}, sequence {b}")


def test_strides_outputs_and_workspaces(ss):
    rng = np.random.default_rng(9)
    q, kp, vp, table, lens = batch(rng)
    plan = ss.prefix_plan(table, lens)
    want = ss.decode_shared(q, kp, vp, table, lens, plan, scale=0.1)
    wide = torch.full((12, 12, 128), math.nan, dtype=torch.bfloat16, device="cuda")
    wide[:, :8] = q
    out = torch.empty_like(q)
    ws = ss.decode_shared_workspace(64, 8, 2, 4 * table.shape[1], 128, "cuda", weights=True)  # one for larger steps
    ws.fill_(255)
    assert ss.decode_shared(wide[:, :8], kp, vp, table, lens, plan, scale=0.1, out=out, workspace=ws) is out
    assert torch.equal(out, want)
    odd = torch.empty(ws.numel() + 16, dtype=torch.uint8, device="cuda")[16:]  # 16-byte aligned only
    assert torch.equal(ss.decode_shared(q, kp, vp, table, lens, plan, scale=0.1, workspace=odd), want)
    with pytest.raises(ss.SSError, match="workspace"):
        ss.decode_shared(q, kp, vp, table, lens, plan, scale=0.1, workspace=ws[:1024])


def test_the_same_from_run_to_run_streams_and_graphs(ss):
    """Two streams at once, a graph replayed on new lengths and data, two graphs; results bit for bit."""
    rng = np.random.default_rng(10)
    batches = [batch(rng, B=9 + i, own=400) for i in range(2)]
    scale = 0.11

    def step(x, stream=None):
        q, kp, vp, table, lens = x
        plan = ss.prefix_plan(table, lens, stream=stream)
        w = torch.zeros(q.shape[0], 2, table.shape[1] * PAGE, device="cuda")
        if stream is not None:
            torch.cuda.synchronize()
        o = ss.decode_shared(q, kp, vp, table, lens, plan, scale=scale, weights=w, stream=stream)
        return o, w

    want = [step(x) for x in batches]
    for _ in range(3):
        assert all(torch.equal(a, b) for x, y in zip(batches, want) for a, b in zip(step(x), y))
    streams = [torch.cuda.Stream() for _ in range(2)]
    weights = [torch.zeros_like(y[1]) for y in want]
    plans = [ss.prefix_plan(x[3], x[4]) for x in batches]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, (q, kp, vp, table, lens) in enumerate(batches):
            stream = streams[i] if i == 0 else streams[i].cuda_stream
            got[i].append(ss.decode_shared(q, kp, vp, table, lens, plans[i], scale=scale, stream=stream))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i][0]) for i in range(2) for o in got[i])
    del weights
    graphs, outs = [], []
    for x in batches:
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            step(x)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(x))
        graphs.append(g)
    for turn in range(3):
        for x in batches:  # other queries, shorter sequences
            x[0].copy_(torch.randn(x[0].shape, device="cuda"))
            x[4].copy_(torch.clamp(x[4] - turn * 7, min=0))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        for x, (o, w) in zip(batches, outs):
            a, b = step(x)
            assert torch.equal(o, a) and torch.equal(w, b)
    assert ss.stream_status() is None


def test_weights_add_up_over_steps(ss):
    rng = np.random.default_rng(11)
    q, kp, vp, table, lens = batch(rng, B=5, groups=1, own=500)
    total = torch.zeros(5, 2, table.shape[1] * PAGE, device="cuda")
    each = []
    for _ in range(4):
        q = torch.randn(q.shape, device="cuda").to(torch.bfloat16)
        one = torch.zeros_like(total)
        ss.decode_shared(q, kp, vp, table, lens, ss.prefix_plan(table, lens), scale=0.1, weights=total)
        ss.decode_shared(q, kp, vp, table, lens, None, scale=0.1, weights=one)
        # (each head's weights add up to 1: 4 heads of a group; every key's rounding is below 2^-22 of it)
        assert ((one.double().sum(-1) - 4.0).abs() < 1e-4).all()
        each.append(one)
    want = sum(x.double() for x in each)
    assert ((total.double() - want).abs() <= 1e-5 * want + 1e-12).all()


@pytest.mark.parametrize("B,L,Hq,Hkv,d,shared", [(1, 100000, 8, 1, 128, 0), (700, 260, 4, 1, 64, 256), (2, 40000, 16, 2, 64, 38400),
                                                 (1500, 130, 1, 1, 64, 0)])
def test_large_sizes(ss, B, L, Hq, Hkv, d, shared):
    rng = np.random.default_rng(B)
    n = tiles(L)
    first = shared // PAGE
    pages = first + B * (n - first)
    order = rng.permutation(pages)
    table = np.concatenate([np.tile(order[:first], (B, 1)), order[first:].reshape(B, n - first)], 1)
    g = torch.Generator(device="cuda").manual_seed(B)
    mk = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, kp, vp = mk(B, Hq, d), mk(pages, Hkv, PAGE, d), mk(pages, Hkv, PAGE, d)
    table, lens = torch.from_numpy(table).int().cuda(), torch.full((B,), L, dtype=torch.int32, device="cuda")
    w = torch.zeros(B, Hkv, n * PAGE, device="cuda")
    o = ss.decode_shared(q, kp, vp, table, lens, ss.prefix_plan(table, lens), scale=d ** -0.5, weights=w)
    for b in sorted({0, B // 2, B - 1}):
        k, v = sequence(kp, table[b], L), sequence(vp, table[b], L).double()
        P, rel = softmax(q[b:b + 1], k, d ** -0.5, torch.tensor([L - 1], device="cuda"))
        assert_attention(o[b], torch.einsum("hngk,hkd->nhgd", P, v).reshape(Hq, d),
                         torch.einsum("hngk,hkd->nhgd", P, v.abs()).reshape(Hq, d))
        assert_close(w[b, :, :L], P.sum((1, 2)), (P * rel).sum((1, 2)) + 1e-37)
    assert torch.isfinite(o.float()).all()


def test_pages_beyond_32_bits(ss):
    """Pages whose first element lies beyond 2^31 elements of the pool."""
    Hkv, d, pages = 8, 128, 17000
    kp = torch.empty((pages, Hkv, PAGE, d), dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    table = torch.tensor([[pages - 1, 3, pages - 2], [5, pages - 3, 0]], dtype=torch.int32, device="cuda")
    for p in (kp, vp):
        p[table.long().unique()] = torch.randn(6, Hkv, PAGE, d, device="cuda").to(torch.bfloat16)
    q = torch.randn(2, 16, d, device="cuda").to(torch.bfloat16)
    lens = torch.tensor([300, 384], dtype=torch.int32, device="cuda")
    check(ss, q, kp, vp, table, lens, ss.prefix_plan(table, lens))


def test_entries_that_name_no_page_read_zeros(ss):
    rng = np.random.default_rng(12)
    q, kp, vp, table, lens = batch(rng, B=3, groups=0, root=0, doc=0, own=500)
    lens.fill_(300)
    pages = kp.shape[0]
    wide = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    wide[:, :3] = torch.tensor([[0, 1, 2], [3, -7, 4], [5, pages, 6]])
    kp, vp = (torch.cat([torch.nan_to_num(x), torch.zeros_like(x[:1])]) for x in (kp, vp))  # page `pages`: zeros
    named = torch.where((wide < 0) | (wide >= pages), pages, wide)
    got = ss.decode_shared(q, kp[:pages], vp[:pages], wide, lens, ss.prefix_plan(wide, lens), scale=0.1)
    want = ss.decode_shared(q, kp, vp, named, lens, None, scale=0.1)
    assert torch.equal(got, want)
