"""Page bookkeeping against a plain Python model: reserve, free, fork, copy, compact (GPU)."""
import numpy as np
import pytest
import torch

from _serving import PAGE, tiles

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import block_sparse_attention_sm_gb300 as ss

    ss.build()
    assert torch.cuda.is_available()


class Model:
    """The state as Python lists, with the same rules."""

    def __init__(self, pages, rows, width, pools, words, seed=0):
        self.refs, self.table, self.lens = [0] * pages, [[-1] * width for _ in range(rows)], [0] * rows
        self.width = width
        rng = np.random.default_rng(seed)
        self.pools = [rng.integers(-(1 << 31), 1 << 31, (pages, words), dtype=np.int64).astype(np.int32)
                      for _ in range(pools)]

    def free_pages(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def reserve(self, rows, add):
        need = sum(tiles(self.lens[r] + a) - tiles(self.lens[r]) for r, a in zip(rows, add))
        free = self.free_pages()
        if len(free) < need:
            return need - len(free)
        for r, a in zip(rows, add):
            for j in range(tiles(self.lens[r]), tiles(self.lens[r] + a)):
                p = free.pop(0)
                self.table[r][j], self.refs[p] = p, 1
            self.lens[r] += a
        return 0

    def free(self, rows):
        for r in rows:
            if 0 <= r < len(self.lens):
                for j in range(tiles(self.lens[r])):
                    self.refs[self.table[r][j]] -= 1
                    self.table[r][j] = -1
                self.lens[r] = 0

    def fork(self, src, dst):
        need = sum(self.lens[s] % PAGE != 0 for s in src)
        free = self.free_pages()
        if len(free) < need:
            return need - len(free)
        for s, d in zip(src, dst):
            L, row = self.lens[s], [-1] * self.width
            for j in range(L // PAGE):
                row[j] = self.table[s][j]
                self.refs[row[j]] += 1
            if L % PAGE:
                row[L // PAGE] = p = free.pop(0)
                self.refs[p] = 1
                for pool in self.pools:
                    pool[p] = pool[self.table[s][L // PAGE]]
            self.table[d], self.lens[d] = row, L
        return 0

    def compact(self):
        live = sum(r > 0 for r in self.refs)
        holes = [p for p in range(live) if self.refs[p] == 0]
        movers = [p for p in range(len(self.refs) - 1, live - 1, -1) if self.refs[p] > 0]
        to = dict(zip(movers, holes))
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
            for pool in self.pools:
                pool[b] = pool[a]
        for r, L in enumerate(self.lens):
            self.table[r] = [to.get(p, p) if j < tiles(L) else -1 for j, p in enumerate(self.table[r])]
        return live


class Device:
    def __init__(self, m):
        self.refs = torch.tensor(m.refs, dtype=torch.int32, device="cuda")
        self.table = torch.tensor(m.table, dtype=torch.int32, device="cuda")
        self.lens = torch.tensor(m.lens, dtype=torch.int32, device="cuda")
        self.pools = [torch.from_numpy(p.copy()).cuda() for p in m.pools]

    def state(self):
        return self.refs, self.table, self.lens

    def same(self, m):
        assert self.refs.tolist() == m.refs
        assert self.lens.tolist() == m.lens
        got = self.table.tolist()
        for r, L in enumerate(m.lens):
            assert got[r][:tiles(L)] == m.table[r][:tiles(L)], r
        used = [p for p, r in enumerate(m.refs) if r > 0]
        for a, b in zip(self.pools, m.pools):
            assert np.array_equal(a.cpu().numpy()[used], b[used])


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("pages,rows,width,pools,words", [
    (7, 3, 4, 1, 4),
    (40, 9, 6, 2, 32),
    (1000, 70, 20, 3, 8200),      # pages of more than one 32 KB chunk, not a whole number of them
    (20000, 200, 60, 1, 4),       # more pages than one round of the search
    (33, 6, 5, 70, 12),           # more pools than one launch takes
])
def test_random_histories(pages, rows, width, pools, words):
    """Reserves, forks, frees and compactions in a random order; every state equals the model's."""
    import block_sparse_attention_sm_gb300 as ss

    rng = np.random.default_rng(pages)
    m = Model(pages, rows, width, pools, words)
    dev = Device(m)
    refused = 0
    for step in range(30):
        used = [r for r in range(rows) if m.lens[r] > 0]
        idle = [r for r in range(rows) if m.lens[r] == 0]
        op = rng.choice(["reserve", "reserve", "fork", "free", "compact"])
        if op == "reserve":
            some = [int(r) for r in rng.permutation(rows)[:rng.integers(1, rows + 1)]]
            most = max(1, 2 * pages * PAGE // (rows + 1))
            add = [int(min(rng.integers(0, most), width * PAGE - m.lens[r])) for r in some]
            want = m.reserve(some, add)
            assert ss.pages_reserve(*dev.state(), ints(add), rows=ints(some)).item() == want
            refused += want > 0
        elif op == "fork" and used and idle:
            n = int(rng.integers(1, len(idle) + 1))
            dst = [int(r) for r in rng.permutation(idle)[:n]]
            src = [int(rng.choice(used)) for _ in dst]
            want = m.fork(src, dst)
            assert ss.pages_fork(dev.pools, *dev.state(), ints(src), ints(dst)).item() == want
            refused += want > 0
        elif op == "free" and used:
            some = [int(r) for r in rng.permutation(used)[:rng.integers(1, len(used) + 1)]]
            m.free(some)
            ss.pages_free(*dev.state(), ints(some + some[:1] + [rows, -1]))  # one of them twice, two that are none
        elif op == "compact":
            live = m.compact()
            assert ss.pages_compact(dev.pools, *dev.state()).item() == live
            assert dev.refs[live:].sum().item() == 0
        dev.same(m)


def test_reserve_all_rows_and_what_it_refuses():
    import block_sparse_attention_sm_gb300 as ss

    m = Model(10, 4, 5, 1, 4)
    dev = Device(m)
    assert m.reserve(range(3), [1, 0, 300]) == 0
    assert ss.pages_reserve(*dev.state(), ints([1, 0, 300])).item() == 0
    dev.same(m)
    for rows, add in (([0, 0], [1, 1]), ([4], [1]), ([-1], [1]), ([1], [-1]), ([1], [5 * PAGE + 1]), ([2], [2 ** 31 - 1])):
        assert ss.pages_reserve(*dev.state(), ints(add), rows=ints(rows)).item() == -1
        dev.same(m)
    assert ss.pages_reserve(*dev.state(), ints([4 * PAGE, 3 * PAGE]), rows=ints([1, 3])).item() == 1  # 7 pages of 6
    dev.same(m)
    assert ss.pages_reserve(*dev.state(), ints([])).item() == 0
    dev.same(m)


def test_fork_and_copy_refuse():
    import block_sparse_attention_sm_gb300 as ss

    m = Model(6, 5, 4, 2, 8)
    m.reserve([0, 1], [200, 128])
    dev = Device(m)
    for src, dst in (([0, 0], [2, 2]), ([0], [0]), ([0, 2], [2, 3]), ([0], [1]), ([5], [2]), ([0], [-1]), ([0], [5])):
        assert ss.pages_fork(dev.pools, *dev.state(), ints(src), ints(dst)).item() == -1, (src, dst)
        dev.same(m)
    before = [p.clone() for p in dev.pools]
    for src, dst in (([0, 1], [3, 3]), ([0, 1], [1, 2]), ([0], [0]), ([6], [1]), ([0], [-1])):
        assert ss.pages_copy(dev.pools, ints(src), ints(dst)).item() == -1, (src, dst)
        assert all(torch.equal(a, b) for a, b in zip(before, dev.pools))
    assert ss.pages_copy(dev.pools, ints([0, 0, 1]), ints([5, 4, 3])).item() == 0
    for a, b in zip(before, dev.pools):
        b = b.clone()
        assert torch.equal(b[[5, 4, 3]], a[[0, 0, 1]]) and torch.equal(b[:3], a[:3])
    # 4 free pages, 5 wanted (and an unused row forks to an unused row)
    m2 = Model(7, 8, 4, 1, 4)
    m2.reserve([0, 7], [130, 50])
    dev = Device(m2)
    assert ss.pages_fork(dev.pools, *dev.state(), ints([0, 0, 7, 7, 0]), ints([1, 2, 3, 4, 5])).item() == 1
    dev.same(m2)
    assert m2.fork([5], [6]) == 0
    assert ss.pages_fork(dev.pools, *dev.state(), ints([5]), ints([6])).item() == 0
    dev.same(m2)


def test_compact_out_of_place_and_many_rows():
    """The old counts and table stay as they are; thousands of forks of one sequence."""
    import block_sparse_attention_sm_gb300 as ss

    m = Model(6000, 2500, 3, 1, 4)
    m.reserve([0, 1], [300, 100])
    dev = Device(m)
    src, dst = [0] * 2400, list(range(2, 2402))
    assert m.fork(src, dst) == 0
    assert ss.pages_fork(dev.pools, *dev.state(), ints(src), ints(dst)).item() == 0
    dev.same(m)
    gone = list(range(0, 2402, 3))
    m.free(gone)
    ss.pages_free(*dev.state(), ints(gone))
    dev.same(m)
    old = dev.refs.clone(), dev.table.clone()
    new_refs, new_table = torch.full_like(dev.refs, -7), torch.full_like(dev.table, -7)
    live = ss.pages_compact(dev.pools, *dev.state(), out_refs=new_refs, out_table=new_table)
    assert torch.equal(dev.refs, old[0]) and torch.equal(dev.table, old[1])
    assert live.item() == m.compact()
    dev.refs, dev.table = new_refs, new_table
    dev.same(m)
    assert new_table.tolist() == m.table


@pytest.mark.slow
def test_lists_of_more_blocks_than_a_launch_has():
    """2^25 entries x 64 pools of 16-byte pages (34 GB): more than 2^31 blocks, so several launches; no result of 0
    stands for work that was not done."""
    import block_sparse_attention_sm_gb300 as ss

    n, pools = (1 << 25) + 3, 64
    pages = n + 1
    pool = torch.zeros(pools, pages, 4, dtype=torch.int32, device="cuda")
    pool[:, 0] = torch.arange(1, 4 * pools + 1, dtype=torch.int32, device="cuda").view(pools, 4)
    each = list(pool)
    i = torch.arange(n, dtype=torch.int32, device="cuda")
    assert ss.pages_copy(each, torch.zeros_like(i), i + 1).item() == 0
    torch.cuda.synchronize()
    same = lambda: all(bool((p[1:] == p[:1]).all()) for p in each)  # noqa: E731
    assert same()
    # a fork of row 0 (5 keys in page 0) into n rows: each takes a page, in order
    pool[:, 1:] = 0
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[0] = 1
    table = torch.zeros(n + 1, 1, dtype=torch.int32, device="cuda")
    table[1:] = -1
    lens = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    lens[0] = 5
    assert ss.pages_fork(each, refs, table, lens, torch.zeros_like(i), i + 1).item() == 0
    torch.cuda.synchronize()
    assert same()
    assert bool((refs == 1).all()) and bool((lens == 5).all())
    assert torch.equal(table[:, 0], torch.arange(n + 1, dtype=torch.int32, device="cuda"))
