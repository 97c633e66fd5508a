"""The calls around the paged cache together, as a serving loop uses them (GPU)."""
import numpy as np
import pytest
import torch

from _serving import PAGE, assert_attention, chunk_reference, offsets, rotate, tiles

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
HQ, HKV, D = 8, 2, 64


@pytest.fixture(scope="module", autouse=True)
def _built():
    import block_sparse_attention_sm_gb300 as ss

    ss.build()
    assert torch.cuda.is_available()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Loop:
    """One layer's cache, and beside it each sequence's keys and values as rows on the host."""

    def __init__(self, pages=64, rows=6, width=8):
        import block_sparse_attention_sm_gb300 as ss

        self.ss = ss
        self.kp = torch.full((pages, HKV, PAGE, D), float("nan"), dtype=BF, device="cuda")
        self.vp = torch.full_like(self.kp, float("nan"))
        self.refs, self.table, self.lens = ints([0] * pages), ints([[-1] * width] * rows), ints([0] * rows)
        self.freq, _ = ss.rope_frequencies(D, 10000.0)
        self.rows = [(torch.zeros(HKV, 0, D, dtype=BF), torch.zeros(HKV, 0, D, dtype=BF)) for _ in range(rows)]
        self.seed = 0

    def state(self):
        return self.refs, self.table, self.lens

    def step(self, n):
        """n[b] new tokens for row b: reserve, rotate and write, attend; checks the outputs."""
        ss = self.ss
        self.seed += 1
        g = torch.Generator().manual_seed(self.seed)
        T = sum(n)
        proj = torch.randn(T, HQ + 2 * HKV, D, generator=g).to(BF)
        result = ss.pages_reserve(*self.state(), ints(n))
        cu = offsets(n).cuda()
        q, k, v = proj.cuda().split([HQ, HKV, HKV], 1)
        q = ss.rope_append_paged(q, k, v, self.kp, self.vp, self.table, cu, self.lens, self.freq)
        o = ss.chunk_paged(q, self.kp, self.vp, self.table, cu, self.lens, scale=D ** -0.5, num_kv_splits=2).cpu()
        assert result.item() == 0
        ss.stream_status()
        q, at = q.cpu(), 0
        for b, x in enumerate(n):
            hk, hv = self.rows[b]
            pos = torch.arange(hk.shape[1], hk.shape[1] + x)
            # the keys as the cache has them: rounded to bf16 after the rotation (by the device)
            turned = rotate(proj[at:at + x, HQ:HQ + HKV], pos[:, None], self.freq.cpu(), 1.0, 0, False)
            dev = self.read(self.kp, b)[:, hk.shape[1]:hk.shape[1] + x]
            assert (dev.double() - turned.transpose(0, 1)).abs().max() <= 2.0 ** -8 * turned.abs().max() if x else True
            hk, hv = torch.cat([hk, dev], 1), torch.cat([hv, proj[at:at + x, HQ + HKV:].transpose(0, 1)], 1)
            assert torch.equal(self.read(self.kp, b), hk) and torch.equal(self.read(self.vp, b), hv)
            self.rows[b] = (hk, hv)
            if x:
                ref, weight, _ = chunk_reference(q[at:at + x], hk, hv, hk.shape[1], D ** -0.5, True, 0.0, 2)
                assert_attention(o[at:at + x], ref, weight, f"row {b}")
            at += x

    def read(self, pool, b):
        L = int(self.lens[b])
        pages = self.table[b, :tiles(L)].long()
        return pool[pages].permute(1, 0, 2, 3).reshape(HKV, -1, D)[:, :L].cpu()

    def fork(self, src, dst):
        result = self.ss.pages_fork([self.kp, self.vp], *self.state(), ints(src), ints(dst))
        assert result.item() == 0
        for s, d in zip(src, dst):
            self.rows[d] = self.rows[s]

    def free(self, rows):
        self.ss.pages_free(*self.state(), ints(rows))
        for r in rows:
            self.rows[r] = (self.rows[r][0][:, :0], self.rows[r][1][:, :0])

    def compact(self):
        live = self.ss.pages_compact([self.kp, self.vp], *self.state()).item()
        assert live == int((self.refs > 0).sum()) and not (self.refs[live:] > 0).any()
        # what lies behind the live pages may go: nothing may read it
        self.kp[live:] = float("nan")
        self.vp[live:] = float("nan")


def test_serving_loop():
    loop = Loop()
    loop.step([300, 0, 5, 128, 0, 0])     # prompts
    loop.step([1, 0, 1, 1, 0, 0])         # one token each
    loop.fork([0, 0, 3], [1, 4, 5])       # sampled further in several ways
    loop.step([1, 1, 1, 1, 1, 1])
    loop.step([4, 1, 60, 1, 130, 2])      # drafts, pieces of prompts and single tokens in one step
    loop.free([0, 3])
    loop.compact()
    loop.step([200, 1, 1, 70, 1, 3])      # new sequences in the freed rows
    loop.free([1, 2, 4, 5])
    loop.compact()
    loop.step([1, 0, 0, 2, 0, 0])
    loop.free([0, 3])
    assert int(loop.refs.sum()) == 0 and int(loop.lens.sum()) == 0


def test_decode_reads_the_appended_cache():
    """ss_attn_decode_paged over pages that the append call wrote gives the chunk call's rows."""
    from block_sparse_attention_sm_gb300 import capi

    loop = Loop(rows=3)
    loop.step([140, 3, 600])
    ss = loop.ss
    q = torch.randn(3, HQ, D, device="cuda").to(BF)
    od = torch.empty_like(q)
    assert capi.ss_attn_decode_paged(q, loop.kp, loop.vp, loop.table, loop.lens, od, 3, HQ, HKV, loop.kp.shape[0],
                                     loop.table.shape[1], D, D ** -0.5, 0.0, 1) == capi.SS_OK
    oc = ss.chunk_paged(q, loop.kp, loop.vp, loop.table, ints([0, 1, 2, 3]), loop.lens, scale=D ** -0.5)
    for b in range(3):
        k, v = loop.rows[b]
        ref, weight, _ = chunk_reference(q[b:b + 1].cpu(), k, v, k.shape[1], D ** -0.5, True, 0.0, 1)
        assert_attention(od[b:b + 1].cpu(), ref, weight)
        assert_attention(oc[b:b + 1].cpu(), ref, weight)


def _batch(seed):
    n, L = [3, 40, 1], [200, 40, 513]
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, pages = sum(n), 16
    mk = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF)  # noqa: E731
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.stack([order[:5], order[5:10], order[10:15]]).contiguous()
    return dict(qkv=mk(T, HQ + 2 * HKV, D), kp=mk(pages, HKV, PAGE, D), vp=mk(pages, HKV, PAGE, D), table=table,
                cu=offsets(n).cuda(), lens=ints(L))


def _pass(ss, s, freq, stream=None, splits=3):
    q, k, v = s["qkv"].split([HQ, HKV, HKV], 1)
    q = ss.rope_append_paged(q, k, v, s["kp"], s["vp"], s["table"], s["cu"], s["lens"], freq, stream=stream)
    return ss.chunk_paged(q, s["kp"], s["vp"], s["table"], s["cu"], s["lens"], scale=D ** -0.5, lambda_a=2.0,
                          num_kv_splits=splits, stream=stream)


def test_other_streams_and_two_at_once():
    """Calls given a stream run on it, two at once do not share anything."""
    import block_sparse_attention_sm_gb300 as ss

    freq, _ = ss.rope_frequencies(D)
    want = [_pass(ss, _batch(i), freq) for i in range(2)]
    batches, streams, got = [_batch(i) for i in range(2)], [torch.cuda.Stream() for _ in range(2)], [[], []]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            stream = streams[i] if i == 0 else streams[i].cuda_stream
            got[i].append(_pass(ss, batches[i], freq, stream=stream))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])
    ss.stream_status()


def test_captured_and_replayed():
    """A step captured into a graph with its page bookkeeping, replayed on new data; two graphs at once."""
    import block_sparse_attention_sm_gb300 as ss

    freq, _ = ss.rope_frequencies(D)
    graphs, batches, outs = [], [], []
    for i in range(2):
        s = _batch(10 + i)
        refs, rows, lens = ints([0] * 32), ints([[-1] * 4] * 3), ints([0, 0, 0])
        pool = [torch.randn(32, 64, device="cuda")]
        add, src, dst = ints([200]), ints([0]), ints([2])

        def step(s=s, refs=refs, rows=rows, lens=lens, pool=pool, add=add, src=src, dst=dst):
            o = _pass(ss, s, freq)
            a = ss.pages_reserve(refs, rows, lens, add, rows=src)
            b = ss.pages_fork(pool, refs, rows, lens, src, dst)
            live = ss.pages_compact(pool, refs, rows, lens)
            ss.pages_free(refs, rows, lens, dst)
            ss.pages_free(refs, rows, lens, src)
            return o, a, b, live

        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
        batches.append((s, refs, lens))
    for seed in (20, 30):
        new = [_batch(seed + i) for i in range(2)]
        want = [_pass(ss, {k: x.clone() for k, x in b.items()}, freq) for b in new]
        for (s, _, _), b in zip(batches, new):
            for k in s:
                s[k].copy_(b[k])
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        for (o, a, b, live), w, (_, refs, lens) in zip(outs, want, batches):
            assert torch.equal(o, w)
            assert (a.item(), b.item(), live.item()) == (0, 0, 3)
            assert int(refs.sum()) == 0 and int(lens.sum()) == 0
    ss.stream_status()


def test_refused_step_leaves_the_cache_alone():
    """A captured step whose reserve is refused writes nothing, though its places would lie in shared pages; it is
    replayed until the pages are there."""
    import block_sparse_attention_sm_gb300 as ss

    freq, _ = ss.rope_frequencies(D)
    kp = torch.randn(4, HKV, PAGE, D, device="cuda").to(BF)
    vp = torch.randn_like(kp)
    refs, table, lens = ints([0] * 4), ints([[-1] * 4] * 3), ints([0] * 3)
    assert ss.pages_reserve(refs, table, lens, ints([256, 0, 200])).item() == 0
    assert ss.pages_fork([kp, vp], refs, table, lens, ints([0]), ints([1])).item() == 0  # two full pages are shared
    assert refs.tolist() == [2, 2, 1, 1]
    add, cu = ints([2, 1, 0]), ints([0, 2, 3, 3])
    proj = torch.randn(3, HQ + 2 * HKV, D, device="cuda").to(BF)
    q, k, v = proj.split([HQ, HKV, HKV], 1)
    out = torch.full((3, HQ, D), 9.0, dtype=BF, device="cuda")

    def step():
        refused = ss.pages_reserve(refs, table, lens, add)
        ss.rope_append_paged(q, k, v, kp, vp, table, cu, lens, freq, out=out, refused=refused)
        return refused, ss.chunk_paged(out, kp, vp, table, cu, lens, scale=D ** -0.5)

    before = [x.clone() for x in (kp, vp, refs, table, lens, out)]
    same = lambda: all(torch.equal(a, b) for a, b in zip(before, (kp, vp, refs, table, lens, out)))  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        refused, _ = step()
    torch.cuda.synchronize()
    assert refused.item() == 2 and same()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        refused, o = step()
    g.replay()
    assert refused.item() == 2 and same()
    add[1] = -1  # a wrong argument is a refusal too
    g.replay()
    assert refused.item() == -1 and same()
    add[1] = 1
    ss.pages_free(refs, table, lens, ints([2]))
    g.replay()
    assert refused.item() == 0 and lens.tolist() == [258, 257, 0] and refs.tolist() == [2, 2, 1, 1]
    assert torch.equal(kp[:2], before[0][:2]) and torch.equal(vp[:2], before[1][:2])
    turned = rotate(proj.cpu()[:, :HQ + HKV], torch.tensor([256, 257, 256])[:, None], freq.cpu(), 1.0, 0, False)
    assert (out.cpu().double() - turned[:, :HQ]).abs().max() <= 2.0 ** -8 * turned.abs().max()
    for t, (b, i) in enumerate(((0, 256), (0, 257), (1, 256))):
        page = int(table[b, 2])
        assert (kp[page, :, i - 256].cpu().double() - turned[t, HQ:]).abs().max() <= 2.0 ** -8 * turned.abs().max()
        assert torch.equal(vp[page, :, i - 256], v[t])
    for b, (t0, t1, L) in enumerate(((0, 2, 258), (2, 3, 257))):
        rows = [x[table[b, :3].long()].transpose(0, 1).reshape(HKV, -1, D)[:, :L].cpu() for x in (kp, vp)]
        ref, weight, _ = chunk_reference(out[t0:t1].cpu(), *rows, L, D ** -0.5, True, 0.0, 1)
        assert_attention(o[t0:t1].cpu(), ref, weight, f"row {b}")
    ss.stream_status()
