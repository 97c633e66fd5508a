"""The calls over shared pages and the record of attention weights at the ends of their ranges."""
import numpy as np
import pytest
import torch

from _serving import PAGE, offsets
from _shared import assert_close, sequence, softmax, tree_batch
from test_decode_shared_gpu import check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss():
    import block_sparse_attention_sm_gb300 as ss

    ss.build()
    return ss


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_key_weights_of_items_that_take_seconds(ss):
    """A CTA's first item has three million steps, and short ones stand behind it: no wait is given up.

    All pages of the long sequence are the same one, so that its 384 million keys take little memory.
    304 tokens of 128 heads on one KV head are 152 pairs of blocks, about one a CTA; the last CTA has
    the two other sequences' as well."""
    many, d, G = 3_000_000, 128, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    mk = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    kp, n = mk(3, 1, PAGE, d), [304, 2, 3]
    q = mk(sum(n), G, d)
    table = torch.zeros(3, many, dtype=torch.int32, device="cuda")
    table[1, :1], table[2, :2] = 1, ints([2, 1])
    lens = ints([many * PAGE, 100, 200])
    w = torch.zeros(3, 1, many * PAGE, device="cuda")
    ss.key_weights(q, kp, table, offsets(n).cuda(), lens, w, scale=0.05, causal=False)
    assert ss.stream_status() is None
    for b, (at, L) in enumerate(((0, 0), (304, 100), (306, 200))):
        if b == 0:
            continue
        k = sequence(kp, table[b], L)
        P, rel = softmax(q[at:at + n[b]], k, 0.05, torch.full((n[b],), L - 1, device="cuda"))
        want = P.sum((1, 2))
        # (n * G rows, 64 pairs of a block's along a thread: see the tests of the record itself)
        assert_close(w[b, :, :L], want, (P * rel).sum((1, 2)) + want * (64 + 4 + n[b] * G / 64) * 2.0 ** -24 + 1e-37, f"sequence {b}")
        assert not w[b, :, L:].any()
    # The long sequence: 128 keys, each `many` times, all of a kind alike.  A row's sum adds `many` terms to one
    # number, each rounding at 2^-24 of it (and once more where the halves and streams are joined): in all below
    # many * 2^-24 = 0.18 of it either way.
    P, _ = softmax(q[:304], sequence(kp, table[0], PAGE), 0.05, torch.full((304,), PAGE - 1, device="cuda"))
    got, want = w[0].view(1, many, PAGE), P.sum((1, 2)) / many
    for at in (0, 1, many // 2, many - 1):
        ratio = got[:, at].double() / want
        assert ((ratio > 1 / 1.19) & (ratio < 1 / (1 - 0.19))).all(), ratio


def test_rows_whose_scores_are_all_minus_infinity(ss):
    """Scores of -2^200, below what fp32 holds, in all of a row: it gives zeros and adds nothing to the record, here and there."""
    d, L = 64, [300, 129, 128]
    g = torch.Generator(device="cuda").manual_seed(2)
    kp, vp = (torch.randn(7, 2, PAGE, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    kp[..., 0] = 2.0 ** 100
    q = torch.randn(3, 4, d, generator=g, device="cuda").to(torch.bfloat16)
    q[..., 0] = 0
    table, lens = ints([[0, 1, 2], [3, 4, -1], [5, -1, -1]]), ints(L)
    clean = torch.rand(3, 2, 3 * PAGE, generator=g, device="cuda")
    q[0, 1, 0] = q[1, 2:, 0] = q[2, :, 0] = -2.0 ** 100  # one of a group's heads, a whole group, all of a sequence
    gone = torch.zeros(3, 4, dtype=torch.bool, device="cuda")
    gone[0, 1] = gone[1, 2:] = gone[2] = True
    a, b = clean.clone(), clean.clone()
    o = ss.decode_shared(q, kp, vp, table, lens, ss.prefix_plan(table, lens), scale=0.1, weights=a)
    ss.key_weights(q, kp, table, offsets([1, 1, 1]).cuda(), lens, b, scale=0.1)
    assert ss.stream_status() is None
    assert (o[gone] == 0).all() and torch.isfinite(o.float()).all() and (o[~gone].abs().amax(-1) > 0).all()
    for i, n in enumerate(L):
        P, rel = softmax(torch.where(gone[i, :, None], torch.zeros_like(q[i]), q[i])[None], sequence(kp, table[i], n), 0.1,
                         torch.tensor([n - 1], device="cuda"))
        P = P * ~gone[i].view(2, 1, 2, 1)
        want = clean[i, :, :n].double() + P.sum((1, 2))
        for w in (a, b):
            assert_close(w[i, :, :n], want, (P * rel).sum((1, 2)) + want * 2.0 ** -22 + 1e-37, f"sequence {i}")
            assert torch.equal(w[i, :, n:], clean[i, :, n:])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv", [(57, 16, 4), (58, 16, 4), (76, 16, 4), (77, 16, 4)])
def test_joins_of_either_width(ss, B, Hq, Hkv, d):
    """Rows on both sides of the numbers up to which the join of partial results has 256 threads a row."""
    rng = np.random.default_rng(B + d)
    lens, table, pages = tree_batch(rng, B, 3, 520, 300, [int(x) for x in rng.integers(1, 300, B)])
    q, kp, vp, table, lens = make(rng, lens, table, pages, Hq, Hkv, d)
    check(ss, q, kp, vp, table, lens, ss.prefix_plan(table, lens))
