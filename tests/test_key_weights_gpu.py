"""The attention weight that cached keys receive from new tokens against 64-bit arithmetic."""
import math

import numpy as np
import pytest
import torch

from _serving import PAGE, offsets, random_tables, tiles
from _shared import assert_close, sequence, softmax

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss():
    import block_sparse_attention_sm_gb300 as ss

    ss.build()
    return ss


def make(rng, n, L, Hq, Hkv, d, pad=0, extra=0, peak=6.0):
    g = torch.Generator().manual_seed(int(rng.integers(1 << 30)))
    table, pages = random_tables(L, 3, rng)
    u = torch.nn.functional.normalize(torch.randn(Hkv, 1, d, generator=g), dim=-1)
    kp = torch.randn(pages, Hkv, PAGE, d, generator=g)
    kp += peak * u * (torch.rand(pages, Hkv, PAGE, 1, generator=g) < 0.02)
    seen = torch.zeros(pages, PAGE, dtype=torch.bool)
    for b, x in enumerate(L):
        for j in range(tiles(x)):
            seen[table[b, j], :min(PAGE, x - j * PAGE)] = True
    kp.transpose(1, 2)[~seen] = math.nan
    T = sum(n) + pad
    q = (torch.randn(T, Hkv, Hq // Hkv, d, generator=g) + peak * u).view(T, Hq, d)
    q[sum(n):] = math.nan  # rows behind the last sequence
    wide = torch.full((T, Hq + extra, d), math.nan)
    wide[:, :Hq] = q
    wide = wide.to(torch.bfloat16).cuda()
    ints = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    return wide[:, :Hq], kp.to(torch.bfloat16).cuda(), table.cuda(), offsets(n).cuda(), ints(L)


def check(ss, q, kp, table, cu, lens, causal=True, **kw):
    T, Hq, d = q.shape
    Hkv, scale, B = kp.shape[1], 1.3 / math.sqrt(d), table.shape[0]
    w = torch.rand(B, Hkv, table.shape[1] * PAGE, device="cuda")
    w0 = w.clone()
    assert ss.key_weights(q, kp, table, cu, lens, w, scale=scale, causal=causal, **kw) is w
    assert ss.stream_status() is None
    cu = cu.tolist()
    for b, L in enumerate(lens.tolist()):
        n = cu[b + 1] - cu[b]
        want, tol = w0[b].double(), torch.zeros_like(w0[b], dtype=torch.float64)
        if n > 0 and L > 0:
            k = sequence(kp, table[b], L)
            for i in range(0, n, 512):
                m = min(512, n - i)
                sees = torch.arange(L - n + i, L - n + i + m, device="cuda") if causal else torch.full((m,), L - 1, device="cuda")
                P, rel = softmax(q[cu[b] + i:cu[b] + i + m], k, scale, sees)
                want[:, :L] += P.sum((1, 2))
                tol[:, :L] += (P * rel).sum((1, 2))
            # the sum over rows: 64 pairs of a block's along a thread, then the blocks and parts
            tol[:, :L] += (want[:, :L]) * (64 + 4 + n * (Hq // Hkv) / 64) * 2.0 ** -24 + 1e-37
        assert_close(w[b], want, tol, f"sequence {b}: {n} tokens on {L} keys")
        assert torch.equal(w[b, :, L:], w0[b, :, L:])
    return w


SIZES = [  # new tokens, keys, Hq, Hkv, d
    ([1], [1], 4, 1, 128),
    ([1, 1, 1], [1, 128, 129], 8, 2, 64),
    ([3], [2000], 8, 2, 128),
    ([17, 5, 0, 9], [300, 700, 50, 9], 8, 8, 64),
    ([32, 32, 32], [1000, 4000, 333], 8, 2, 128),
    ([300], [300], 8, 2, 128),
    ([700, 1, 129], [900, 513, 129], 12, 4, 64),
    ([200, 10], [150, 4], 6, 2, 128),  # more tokens than keys: rows without keys
    ([33, 100], [0, 640], 10, 2, 128),
    ([2, 3], [600, 700], 128, 1, 128),
    ([50], [4097], 100, 1, 64),
    ([1500], [1500], 3, 1, 128),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n,L,Hq,Hkv,d", SIZES)
def test_against_64_bits(ss, n, L, Hq, Hkv, d, causal):
    rng = np.random.default_rng(sum(n) + sum(L))
    check(ss, *make(rng, n, L, Hq, Hkv, d, pad=3, extra=2), causal=causal)


def test_the_same_from_run_to_run_streams_and_graphs(ss):
    rng = np.random.default_rng(1)
    batches = [make(rng, [40, 200 + i, 1], [3000, 700, 129], 8, 2, 128) for i in range(2)]

    def run(x, stream=None, w=None):
        q, kp, table, cu, lens = x
        w = torch.zeros(3, 2, table.shape[1] * PAGE, device="cuda") if w is None else w
        return ss.key_weights(q, kp, table, cu, lens, w, scale=0.1, stream=stream)

    want = [run(x) for x in batches]
    assert all(torch.equal(run(x), y) for x, y in zip(batches, want))
    streams = [torch.cuda.Stream() for _ in range(2)]
    room = [[torch.zeros_like(y) for _ in range(8)] for y in want]
    torch.cuda.synchronize()
    for k in range(8):
        for i in range(2):
            run(batches[i], streams[i] if k % 2 else streams[i].cuda_stream, room[i][k])
    torch.cuda.synchronize()
    assert all(torch.equal(w, want[i]) for i in range(2) for w in room[i])
    graphs, outs = [], []
    for x in batches:
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            run(x)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(x))
        graphs.append(g)
    for turn in range(2):
        for x in batches:
            x[0].copy_(torch.randn(x[0].shape, device="cuda"))
            x[4][0] -= 100 * turn
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        for x, w in zip(batches, outs):
            assert torch.equal(w, run(x))
    assert ss.stream_status() is None


def test_single_tokens_as_in_the_decode(ss):
    """One token a sequence: the weights that the decode records."""
    rng = np.random.default_rng(2)
    q, kp, table, cu, lens = make(rng, [1] * 7, [1, 128, 300, 999, 5, 640, 2000], 8, 2, 128)
    W = table.shape[1] * PAGE
    a, b = torch.zeros(7, 2, W, device="cuda"), torch.zeros(7, 2, W, device="cuda")
    ss.key_weights(q, kp, table, cu, lens, a, scale=0.1)
    ss.decode_shared(q, kp, torch.nan_to_num(kp), table, lens, None, scale=0.1, weights=b)
    # both are off by the same tolerances as against 64 bits: below 2^-15 here (scores of at most 12)
    assert ((a - b).abs() <= 2.0 ** -14 * b + 1e-12).all()


def test_more_tokens_than_a_share_and_many_sequences(ss):
    rng = np.random.default_rng(3)
    n = [int(x) for x in rng.integers(0, 6, 300)]
    L = [int(x) + y for x, y in zip(rng.integers(0, 400, 300), n)]
    check(ss, *make(rng, n, L, 4, 2, 64, pad=5))
    check(ss, *make(rng, [64], [60000], 4, 1, 128))


@pytest.mark.parametrize("causal", [True, False])
def test_more_sequences_than_threads(ss, causal):
    rng = np.random.default_rng(5)
    n = [int(x) for x in rng.integers(0, 4, 1500)]
    n[700] = 90
    L = [int(x) * (int(y) > 0) + k for x, y, k in zip(rng.integers(0, 150, 1500), rng.integers(0, 5, 1500), n)]
    check(ss, *make(rng, n, L, 6, 3, 64, pad=2), causal=causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n,L,Hq,Hkv,d", [
    ([7], [50000], 2, 1, 128),  # one block of rows, cut: alternate tiles of keys
    ([900, 3], [100, 7], 4, 2, 64),  # one tile of keys, cut: alternate blocks of rows
    ([1000], [128], 128, 1, 128),  # a token a block
    ([2100, 40], [2100, 2400], 5, 5, 64),
    ([600], [9000], 35, 7, 128),
])
def test_items_that_are_cut(ss, n, L, Hq, Hkv, d, causal):
    rng = np.random.default_rng(sum(n) + sum(L) + Hq)
    check(ss, *make(rng, n, L, Hq, Hkv, d, pad=1), causal=causal)


def test_one_sequence_cannot_reach_another(ss):
    """Infinities and NaN in one sequence's keys or queries change nothing for the others, bit for bit."""
    rng = np.random.default_rng(4)
    q, kp, table, cu, lens = make(rng, [30, 9, 70], [500, 300, 70], 6, 2, 64)
    run = lambda q, kp: ss.key_weights(q, kp, table, cu, lens, torch.zeros(3, 2, table.shape[1] * PAGE, device="cuda"), scale=0.1)  # noqa: E731
    clean = run(q, kp)
    for b in range(3):
        for bad in (math.nan, math.inf):
            q2, k2 = q.clone(), kp.clone()
            q2[int(cu[b]) + 3, 1] = bad
            k2[int(table[b, 0]), :, 5] = bad
            got = run(q2, k2)
            others = [i for i in range(3) if i != b]
            assert torch.equal(got[others], clean[others])


def test_workspace_of_larger_sizes(ss):
    from block_sparse_attention_sm_gb300 import capi

    rng = np.random.default_rng(5)
    x = make(rng, [20, 3], [400, 100], 8, 2, 128)
    ws = torch.full((capi.ss_attn_key_weights_workspace_size(500, 64, 8, 2),), 255, dtype=torch.uint8, device="cuda")
    check(ss, *x, workspace=ws)
    with pytest.raises(ss.SSError, match="workspace"):
        check(ss, *x, workspace=ws[:4096])


def test_pages_beyond_32_bits(ss):
    Hkv, d, pages = 8, 128, 17000
    kp = torch.empty((pages, Hkv, PAGE, d), dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[pages - 1, 3, pages - 2], [5, pages - 3, 0]], dtype=torch.int32, device="cuda")
    kp[table.long().unique()] = torch.randn(6, Hkv, PAGE, d, device="cuda").to(torch.bfloat16)
    q = torch.randn(50, 16, d, device="cuda").to(torch.bfloat16)
    check(ss, q, kp, table, offsets([10, 40]).cuda(), torch.tensor([300, 384], dtype=torch.int32, device="cuda"))
