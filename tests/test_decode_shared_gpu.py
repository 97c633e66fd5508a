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
