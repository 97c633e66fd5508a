"""Prompts, their windows' weights, eviction, forks and shared decode steps together, as a serving loop uses them (GPU)."""
import pytest
import torch

from _serving import PAGE, assert_attention, offsets, tiles
from _shared import assert_close, choose, softmax

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
HQ, HKV, D, ROWS, WIDTH, PAGES = 8, 2, 64, 6, 8, 40
SCALE = D ** -0.5


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Loop:
    """One layer's cache with the record of weights, and beside it each sequence's keys and values a head."""

    def __init__(self):
        import block_sparse_attention_sm_gb300 as ss

        ss.build()
        self.ss = ss
        self.kp = torch.full((PAGES, HKV, PAGE, D), float("nan"), dtype=BF, device="cuda")
        self.vp = torch.full_like(self.kp, float("nan"))
        self.refs, self.table, self.lens = ints([0] * PAGES), ints([[-1] * WIDTH] * ROWS), ints([0] * ROWS)
        self.weights = torch.zeros(ROWS, HKV, WIDTH * PAGE, device="cuda")
        self.freq, _ = ss.rope_frequencies(D)
        self.seen = [0] * ROWS  # tokens of each sequence so far: the next one's position
        self.rows = [None] * ROWS
        self.g = torch.Generator(device="cuda").manual_seed(1)

    def state(self):
        return self.refs, self.table, self.lens

    def read(self, pool, b):
        L = int(self.lens[b])
        return pool[self.table[b, :tiles(L)].long()].transpose(0, 1).flatten(1, 2)[:, :L]

    def append(self, n):
        """n[b] new tokens of row b: their rotated queries [T, HQ, D]."""
        T = sum(n)
        proj = torch.randn(T, HQ + 2 * HKV, D, generator=self.g, device="cuda").to(BF)
        pos = ints([self.seen[b] + i for b in range(ROWS) for i in range(n[b])])
        short = self.ss.pages_reserve(*self.state(), ints(n))
        q, k, v = proj.split([HQ, HKV, HKV], 1)
        q = self.ss.rope_append_paged(q, k, v, self.kp, self.vp, self.table, offsets(n).cuda(), self.lens, self.freq, positions=pos,
                                      refused=short)
        assert short.item() == 0
        at = 0
        for b, x in enumerate(n):
            if x:
                new = self.read(self.kp, b), self.read(self.vp, b)
                if self.rows[b] is not None:  # what was there is as it was
                    assert all(torch.equal(a[:, :-x], o) for a, o in zip(new, self.rows[b]))
                assert torch.equal(new[1][:, -x:], v[at:at + x].transpose(0, 1))
                self.rows[b] = new
                self.seen[b] += x
                at += x
        return q

    def evict(self, rows, keep, recent):
        before, old = self.weights.clone(), list(self.rows)
        result = self.ss.pages_evict([self.kp, self.vp], [self.weights], *self.state(), ints(keep), rows=ints(rows), recent=recent)
        assert result.item() == 0
        for b, k in zip(rows, keep):
            L = old[b][0].shape[1]
            src = [choose(before[b, h, :L].double().cpu(), k, recent).cuda() for h in range(HKV)]
            self.rows[b] = tuple(torch.stack([x[h, src[h]] for h in range(HKV)]) for x in old[b])
            assert all(torch.equal(self.weights[b, h, :min(k, L)], before[b, h, src[h]]) for h in range(HKV))
            assert (self.weights[b, :, k:] == 0).all()
        self.same()

    def same(self):
        """Every sequence's keys and values are what the model says, and the counts add up."""
        held = [0] * PAGES
        for b in range(ROWS):
            if self.rows[b] is None:
                assert int(self.lens[b]) == 0
                continue
            assert torch.equal(self.read(self.kp, b), self.rows[b][0]) and torch.equal(self.read(self.vp, b), self.rows[b][1])
            for p in self.table[b, :tiles(int(self.lens[b]))].tolist():
                held[p] += 1
        assert self.refs.tolist() == held

    def decode(self, live, plan):
        """One token of each live row; checks the outputs and what the step adds to the record."""
        q = self.append([1 if b in live else 0 for b in range(ROWS)])
        rows = torch.zeros(ROWS, HQ, D, dtype=BF, device="cuda")
        rows[live] = q
        before = self.weights.clone()
        o = self.ss.decode_shared(rows, self.kp, self.vp, self.table, self.lens, plan, scale=SCALE, weights=self.weights)
        self.ss.stream_status()
        for b in range(ROWS):
            if self.rows[b] is None:
                assert (o[b] == 0).all() and torch.equal(self.weights[b], before[b])
                continue
            k, v = self.rows[b]
            L = k.shape[1]
            P, rel = softmax(rows[b:b + 1], k, SCALE, torch.tensor([L - 1], device="cuda"))
            assert_attention(o[b], torch.einsum("hngk,hkd->nhgd", P, v.double()).reshape(HQ, D),
                             torch.einsum("hngk,hkd->nhgd", P, v.double().abs()).reshape(HQ, D), f"row {b}")
            want = before[b, :, :L].double() + P.sum((1, 2))
            assert_close(self.weights[b, :, :L], want, (P * rel).sum((1, 2)) + want * 2.0 ** -23 + 1e-37, f"weights of row {b}")


def test_prompts_forks_and_evictions():
    loop = Loop()
    ss = loop.ss
    n = [600, 0, 0, 390, 0, 0]
    q = loop.append(n)
    # the prompts' last 16 tokens choose which keys are kept
    window = torch.cat([q[600 - 16:600], q[990 - 16:990]])
    cu = ints([0, 16, 16, 16, 32, 32, 32])
    ss.key_weights(window, loop.kp, loop.table, cu, loop.lens, loop.weights, scale=SCALE)
    for b, rows in ((0, window[:16]), (3, window[16:])):
        k = loop.rows[b][0]
        L = k.shape[1]
        P, rel = softmax(rows, k, SCALE, torch.arange(L - 16, L, device="cuda"))
        assert_close(loop.weights[b, :, :L], P.sum((1, 2)), (P * rel).sum((1, 2)) + 1e-5 * P.sum((1, 2)) + 1e-37)
    loop.evict([0, 3], [400, 200], 32)
    # the first prompt is answered three ways
    assert ss.pages_fork([loop.kp, loop.vp], *loop.state(), ints([0, 0]), ints([1, 2])).item() == 0
    for b in (1, 2):
        loop.rows[b], loop.seen[b] = loop.rows[0], loop.seen[0]
        loop.weights[b] = loop.weights[0]
    loop.same()
    plan = ss.prefix_plan(loop.table, loop.lens)
    for _ in range(4):
        loop.decode([0, 1, 2, 3], plan)
    # one of them is cut again: the pages that the others hold too are left alone
    loop.evict([1], [300], 64)
    plan = ss.prefix_plan(loop.table, loop.lens)
    for _ in range(3):
        loop.decode([0, 1, 2, 3], plan)
    # a sequence ends, another is cut to a page, a new prompt comes
    ss.pages_free(*loop.state(), ints([2]))
    loop.rows[2], loop.seen[2] = None, 0
    loop.weights[2] = 0
    loop.evict([3, 0], [128, 10], 4)
    loop.append([0, 0, 0, 0, 0, 140])
    plan = ss.prefix_plan(loop.table, loop.lens)
    loop.decode([0, 1, 3, 5], plan)
    live = ss.pages_compact([loop.kp, loop.vp], *loop.state()).item()
    loop.kp[live:] = float("nan")
    loop.same()
    loop.decode([0, 5], ss.prefix_plan(loop.table, loop.lens))
    loop.evict([0, 1, 3, 5], [0, 0, 0, 0], 0)
    assert int(loop.refs.sum()) == 0 and int(loop.lens.sum()) == 0


def test_a_captured_step():
    """Plan, decode with weights and an eviction captured into one graph and replayed while the sequences grow."""
    loop = Loop()
    ss = loop.ss
    loop.append([700, 0, 0, 0, 0, 0])
    assert ss.pages_fork([loop.kp, loop.vp], *loop.state(), ints([0, 0, 0]), ints([1, 2, 4])).item() == 0
    q = torch.randn(ROWS, HQ, D, generator=loop.g, device="cuda").to(BF)
    keep, rows, add = ints([500, 460]), ints([1, 4]), ints([3, 3, 3, 0, 3, 0])

    def step():
        a = ss.pages_reserve(*loop.state(), add)
        plan = ss.prefix_plan(loop.table, loop.lens)
        o = ss.decode_shared(q, loop.kp, loop.vp, loop.table, loop.lens, plan, scale=SCALE, weights=loop.weights)
        return a, o, ss.pages_evict([loop.kp, loop.vp], [loop.weights], *loop.state(), keep, rows=rows, recent=20)

    state = [loop.kp, loop.vp, loop.weights, *loop.state()]
    loop.kp.nan_to_num_()
    loop.vp.nan_to_num_()
    start = [x.clone() for x in state]

    def back():
        for x, s in zip(state, start):
            x.copy_(s)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            want = [x.clone() for x in step()]
    torch.cuda.synchronize()
    after = [x.clone() for x in state]
    back()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    back()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert want[0].item() == want[2].item() == 0
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert all(torch.equal(a, b) for a, b in zip(after, state))
    assert loop.lens.tolist() == [709, 500, 709, 0, 460, 0]
    ss.stream_status()
