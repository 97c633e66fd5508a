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
