"""The plan of shared pages against a model of it on the host, and decode steps of batches in any order."""
import numpy as np
import pytest
import torch

from _serving import PAGE, assert_attention, tiles
from _shared import sequence, softmax, tree_batch
from test_decode_shared_gpu import check, make

pytestmark = pytest.mark.gpu

HEAD, NODE, LEVELS = 8, 4, 7  # words in front, of a node; shared nodes above a sequence at most


@pytest.fixture(scope="module")
def ss():
    import block_sparse_attention_sm_gb300 as ss

    ss.build()
    return ss


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def tree(table, lens):
    """({(members, first tile, end tile)}, own tiles' start, nodes above from the root down) of each sequence, by the definition."""
    width = len(table[0])
    full = [min(max(L, 0) // PAGE, width) for L in lens]
    nodes, own, above = set(), [0] * len(lens), [[] for _ in lens]
    stack = [(list(range(len(lens))), 0, 0)]
    while stack:
        members, t, level = stack.pop()
        groups = {}
        for b in members:
            if full[b] > t and table[b][t] >= 0:
                groups.setdefault(table[b][t], []).append(b)
        for some in groups.values():
            if len(some) < 2:
                continue
            t1, one = t + 1, table[some[0]]
            while all(full[b] > t1 for b in some) and one[t1] >= 0 and all(table[b][t1] == one[t1] for b in some):
                t1 += 1
            if level < LEVELS:
                node = (tuple(some), t, t1)
                nodes.add(node)
                for b in some:
                    own[b] = t1
                    above[b].append(node)
            stack.append((some, t1, level + 1))
    return nodes, own, above


def check_plan(ss, table, lens):
    B = len(lens)
    plan = ss.prefix_plan(ints(table), ints(lens)).tolist()
    order = plan[HEAD:HEAD + B]
    assert sorted(order) == list(range(B))
    words = plan[HEAD + B:HEAD + B + 2 * B * NODE]
    at = [words[NODE * i:NODE * i + NODE] for i in range(2 * B)]
    up = plan[HEAD + B + 2 * B * NODE:]
    nodes, own, above = tree(table, lens)
    named = [None if n[1] == 0 else (tuple(sorted(order[n[0]:n[0] + n[1]])), n[2], n[3]) for n in at[B:]]
    got = [n for n in named if n is not None]
    assert len(got) == len(set(got)) and set(got) == nodes
    for i, b in enumerate(order):
        assert at[i][:3] == [i, 1, own[b]], f"sequence {b}"
        chain = up[LEVELS * i:LEVELS * i + LEVELS]
        want = above[b][::-1]
        assert [named[x - B] for x in chain[:len(want)]] == want and chain[len(want):] == [-1] * (LEVELS - len(want)), f"sequence {b}"


def forest(rng, B, width, negative=0.0, short=0.2):
    """Tables and lengths: rows that begin as an earlier one does, for any number of pages, and go on with pages of their own."""
    table, lens, fresh = [], [], 0
    for b in range(B):
        row = []
        if b and rng.random() < 0.8:
            other = table[int(rng.integers(max(0, b - 40), b))]
            row = list(other[:int(rng.integers(0, width + 1))])
        while len(row) < width:
            row.append(fresh)
            fresh += 1
        if rng.random() < negative:
            row[int(rng.integers(width))] = -int(rng.integers(1, 4))
        table.append(row)
        lens.append(int(rng.integers(0, PAGE)) if rng.random() < short else int(rng.integers(0, width * PAGE + 1)))
    names = rng.permutation(fresh + 1)
    return [[int(names[p]) if p >= 0 else p for p in row] for row in table], lens


@pytest.mark.parametrize("B", [1, 2, 3, 4, 5, 6, 7, 8, 9, 16, 40, 130, 1100])
def test_tree_against_the_model(ss, B):
    rng = np.random.default_rng(B)
    for width, negative, short in ((1, 0.0, 0.0), (4, 0.0, 0.2), (9, 0.3, 0.1), (37, 0.1, 0.0)):
        check_plan(ss, *forest(rng, B, width, negative, short))
        # all as full as they can be
        table, lens = forest(rng, B, width, negative)
        check_plan(ss, table, [width * PAGE] * B)


@pytest.mark.parametrize("B", [6200, 8192])
def test_tree_of_large_batches(ss, B):
    """More places than 48 KB of shared memory hold, up to the most that a plan takes."""
    rng = np.random.default_rng(B)
    check_plan(ss, *forest(rng, B, 6))
    check_plan(ss, [[b % 3, 10 + b % 7, 20 + b] for b in range(B)], [3 * PAGE - b % 2 * PAGE for b in range(B)])


def test_equal_rows_chains_and_single_pages(ss):
    check_plan(ss, [[5, 6, 7]] * 70, [3 * PAGE] * 40 + [2 * PAGE + 5] * 20 + [PAGE] * 5 + [PAGE - 1] * 5)
    check_plan(ss, [[5, 6, 7]] * 3, [0, 10 ** 9, 2 * PAGE])  # (longer than its table: as long as that)
    # every row shares one page more with its successors: more levels than are kept, with rows that stop at each
    deep = [list(range(b)) + [100 + b + 40 * j for j in range(30 - b)] for b in range(30)]
    check_plan(ss, deep, [30 * PAGE] * 30)
    check_plan(ss, deep[::-1] + deep, [30 * PAGE - 50 * b for b in range(30)] + [30 * PAGE] * 30)
    # long runs that differ at the last page, in words of every position of a comparing warp's
    rows = [[*range(1000)] for _ in range(24)]
    for b, at in enumerate([0, 1, 31, 32, 33, 511, 512, 513, 543, 544, 998, 999] * 2):
        rows[b][at] = 5000 + b % 12 if b < 12 else 6000 + b % 12
    check_plan(ss, rows, [1000 * PAGE] * 24)
    check_plan(ss, rows, [1000 * PAGE - b * 4111 for b in range(24)])


@pytest.mark.parametrize("B,Hq,Hkv,d", [(2, 8, 2, 64), (9, 8, 2, 128), (40, 28, 4, 128), (70, 4, 1, 64)])
def test_batches_in_any_order(ss, B, Hq, Hkv, d):
    """The same sequences in another order: each has the output and the weights that it had."""
    rng = np.random.default_rng(B + d)
    lens, table, pages = tree_batch(rng, B, 2, 400, 300, [int(x) for x in rng.integers(1, 300, B)])
    q, kp, vp, table, lens = make(rng, lens, table, pages, Hq, Hkv, d)
    scale, W = 1.3 * d ** -0.5, table.shape[1] * PAGE
    order = torch.from_numpy(rng.permutation(B)).cuda()

    def step(some):
        w = torch.zeros(B, Hkv, W, device="cuda")
        rows, n = table[some].contiguous(), lens[some].contiguous()
        return ss.decode_shared(q[some].contiguous(), kp, vp, rows, n, ss.prefix_plan(rows, n), scale=scale, weights=w), w

    (o, w), (p, x) = step(torch.arange(B, device="cuda")), step(order)
    assert ss.stream_status() is None
    for i, b in enumerate(order.tolist()):
        L = int(lens[b])
        k, v = sequence(kp, table[b], L), sequence(vp, table[b], L).double()
        P, rel = softmax(q[b:b + 1], k, scale, torch.tensor([L - 1], device="cuda"))
        size = torch.einsum("hngk,hkd->nhgd", P, v.abs()).reshape(Hq, d)
        # Each is off from the exact result by t + 2^-8 (|o| + t), t = (2^-8 + 2^-11) size, so from the other by twice
        # that: in size and |o| below what is allowed for these (the 1% is 2^-8 of t, for |o| differs from the exact one).
        assert_attention(p[i], o[b].double(), 2.02 * size + o[b].double().abs(), f"sequence {b}")
        tol = 2.0 * (P * rel).sum((1, 2)) + 1e-37
        assert ((w[b, :, :L].double() - x[i, :, :L].double()).abs() <= tol).all(), f"weights of sequence {b}"
        assert not x[i, :, L:].any() and not w[b, :, L:].any()


def test_sequences_that_become_shorter_need_a_new_plan(ss):
    """Rolled back inside a run that they shared, with a plan made anew; behind the run the old one goes on holding."""
    rng = np.random.default_rng(3)
    lens, table, pages = tree_batch(rng, 10, 2, 640, 260, [int(x) for x in rng.integers(150, 400, 10)])
    q, kp, vp, table, lens = make(rng, lens, table, pages, 8, 2, 128)
    plan = ss.prefix_plan(table, lens)
    own = lens - 900 // PAGE * PAGE  # keys behind the shared tiles
    check(ss, q, kp, vp, table, lens - torch.minimum(own, ints([0, 1, 5, 120, 129, 1000, 0, 3, 77, 150])), plan)
    short = lens.clone()
    short[[1, 4, 7]] = ints([700, 128, 39])
    check(ss, q, kp, vp, table, short, ss.prefix_plan(table, short))
