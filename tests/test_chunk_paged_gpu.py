"""Attention of packed new tokens over the paged cache against 64-bit arithmetic (GPU).

Pages behind a sequence's end hold NaN, unused table entries name other
sequences' pages, and every output has guard bands."""
import math

import numpy as np
import pytest
import torch

from _serving import (PAGE, assert_attention, chunk_place, chunk_reference, fill_pool, offsets, random_tables, tiles)

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    import block_sparse_attention_sm_gb300 as ss

    ss.build()
    assert torch.cuda.is_available()


def make(Hq, Hkv, d, n, L, seed, hot=0.2):
    """Queries and keys whose softmax weight lies on the keys of a few tiles."""
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    u = torch.nn.functional.normalize(torch.randn(Hkv, d, generator=g), dim=-1)
    G = Hq // Hkv
    q = torch.randn(sum(n), Hkv, G, d, generator=g) + 12 * u[:, None]
    k, v = [], []
    for x in L:
        kk = torch.randn(Hkv, x, d, generator=g)
        for j in range(tiles(x)):
            for h in range(Hkv):
                if j == 0 or rng.random() < hot:
                    kk[h, j * PAGE:(j + 1) * PAGE] += 12 * u[h]
        k.append(kk.to(BF))
        v.append(torch.randn(Hkv, x, d, generator=g).to(BF))
    return q.to(BF).view(sum(n), Hq, d), k, v


def check(Hq, Hkv, d, n, L, *, causal=True, a=0.0, splits=1, seed=0, pad=0, stride_pad=0, debug=True):
    import block_sparse_attention_sm_gb300 as ss
    from _parity import guarded
    from block_sparse_attention_sm_gb300 import capi

    rng = np.random.default_rng(seed)
    q, k, v = make(Hq, Hkv, d, n, L, seed)
    T, B, G = sum(n) + pad, len(n), Hq // Hkv
    table, pages = random_tables(L, 2, rng)
    width = table.shape[1]
    kp, vp = fill_pool(k, L, table, pages).cuda(), fill_pool(v, L, table, pages).cuda()
    cu = offsets(n)
    room = torch.full((T, Hq * d + stride_pad), float("nan"), dtype=BF)
    room[:sum(n), :Hq * d] = q.view(sum(n), -1)
    qd = room.cuda()[:, :Hq * d].unflatten(1, (Hq, d))
    scale = d ** -0.5
    units = capi.ss_attn_chunk_paged_units(T, B, Hq, Hkv)
    o = guarded((T, Hq, d), BF, "cuda", 7.0)
    extra, bands = {}, [o]
    if debug:
        bands += [guarded((units,), torch.int32, "cuda", -1), guarded((units, width), torch.uint8, "cuda", 9),
                  guarded((units, width), torch.float32, "cuda", 12345.0)]
        extra = dict(zip(("counts", "skip_mask", "vote_margin"), (x.t for x in bands[1:])))
    ss.chunk_paged(qd, kp, vp, table.cuda(), cu.cuda(), torch.tensor(L, dtype=torch.int32, device="cuda"),
                   scale=scale, causal=causal, lambda_a=a, num_kv_splits=splits, out=o.t, **extra)
    assert capi.ss_stream_status() == capi.SS_OK
    for x in bands:
        x.check("chunk")
    got = o.t.cpu()
    assert (got[sum(n):] == 7.0).all(), "rows behind the last sequence"
    if debug:
        mask, counts, margin = (extra[x].cpu() for x in ("skip_mask", "counts", "vote_margin"))
        seen_units = torch.zeros(units, dtype=torch.bool)
    cul = cu.tolist()
    skipped = evaluated = 0
    for b in range(B):
        if n[b] == 0:
            continue
        m = PAGE // G
        blocks = -(-n[b] // m)
        keep = None
        if debug:
            _, _, c = chunk_reference(q[cul[b]:cul[b + 1]], k[b], v[b], L[b], scale, causal, a, splits)
            ln_lam = math.log(min(1.0, a / L[b])) if a > 0 and L[b] > 0 else -math.inf
            nT = tiles(L[b])
            keep = torch.ones(Hkv, blocks, nT, dtype=torch.bool)
            for h in range(Hkv):
                for blk in range(blocks):
                    place, half, places = chunk_place(cul, b, blk, G, T, B)
                    unit = (h * places + place) * 2 + half
                    seen_units[unit] = True
                    for j in range(width):
                        if j >= nT or math.isnan(float(c[h, blk, j])):
                            assert mask[unit, j] == 2 and math.isnan(float(margin[unit, j]))
                            continue
                        stat, gpu = float(c[h, blk, j]), float(margin[unit, j])
                        evaluated += 1
                        skip = int(mask[unit, j]) == 1
                        assert int(mask[unit, j]) in (0, 1)
                        if math.isfinite(stat):
                            assert abs(gpu - stat) <= 1e-3 + 1e-5 * abs(stat)  # fp32 scores of |s| < 64
                        else:
                            assert gpu == stat
                        if abs(stat - ln_lam) > 1e-2:  # (elsewhere fp32 may decide otherwise)
                            assert skip == (stat < ln_lam)
                        keep[h, blk, j] = not skip
                        skipped += skip
                    assert int(counts[unit]) == int((mask[unit] == 1).sum())
        o_ref, weight, _ = chunk_reference(q[cul[b]:cul[b + 1]], k[b], v[b], L[b], scale, causal, a, splits, keep)
        assert_attention(got[cul[b]:cul[b + 1]], o_ref, weight, f"sequence {b}")
    if debug:
        assert (counts[~seen_units] == 0).all() and (mask[~seen_units] == 2).all()
    return skipped, evaluated


CASES = [
    # Hq, Hkv, d, new tokens, lengths
    (1, 1, 128, [1], [1]),
    (2, 1, 64, [1, 3], [130, 3]),
    (4, 1, 128, [5, 0, 1, 33], [300, 77, 0, 161]),          # a sequence without keys, one without tokens
    (8, 2, 128, [64, 65, 1], [64, 700, 128]),               # a full pair of blocks; one token more; a full page
    (3, 1, 64, [90, 2, 43], [90, 129, 1000]),               # groups that do not divide 128
    (7, 1, 128, [40, 18], [500, 18]),
    (16, 1, 128, [8, 17], [1030, 40]),
    (5, 5, 64, [257, 128], [257, 513]),                     # one head a group: 128 tokens a block
    (100, 1, 128, [3, 1], [200, 385]),                      # one token a block
    (128, 1, 64, [2], [129]),
]


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", CASES)
def test_chunk_dense(case, causal, splits):
    check(*case, causal=causal, splits=splits, seed=1, pad=5, debug=False)


@pytest.mark.parametrize("a", [0.0, 1.0, 16.0, 1e9])
@pytest.mark.parametrize("case,splits", [
    ((4, 1, 128, [130, 1, 40], [1500, 640, 2000]), 1),
    ((6, 2, 64, [50, 3], [900, 1281]), 2),
    ((8, 8, 128, [200], [1100]), 1),
    ((12, 1, 128, [1, 1, 30], [2100, 1, 700]), 5),
    ((3, 1, 128, [45], [1300]), 20),                        # more ranges than tiles
])
def test_chunk_votes(case, splits, a):
    skipped, evaluated = check(*case, a=a, splits=splits, seed=3)
    assert evaluated > 0
    if a == 0.0:
        assert skipped == 0
    if a == 16.0 and splits <= 2:
        assert skipped > 0


def test_chunk_strided_queries_and_padding():
    check(8, 2, 128, [70, 9], [300, 1000], seed=5, pad=200, stride_pad=64, a=8.0)


def test_chunk_shorter_than_its_new_tokens():
    """Rows whose place lies before the first key see nothing and give zeros."""
    check(4, 2, 128, [40, 300], [10, 130], seed=6)


def test_chunk_matches_decode_and_prefill():
    """One token a sequence is the paged decode; a whole prompt is the contiguous prefill (dense)."""
    import block_sparse_attention_sm_gb300 as ss
    from block_sparse_attention_sm_gb300 import capi

    Hq, Hkv, d, L = 8, 2, 128, [513, 128, 1000]
    q, k, v = make(Hq, Hkv, d, [1, 1, 1], L, 9)
    table, pages = random_tables(L, 1, np.random.default_rng(0))
    kp, vp = fill_pool(k, L, table, pages).cuda(), fill_pool(v, L, table, pages).cuda()
    lens, cu = torch.tensor(L, dtype=torch.int32, device="cuda"), offsets([1, 1, 1]).cuda()
    o = ss.chunk_paged(q.cuda(), kp, vp, table.cuda(), cu, lens, scale=d ** -0.5)
    od = torch.empty(3, Hq, d, dtype=BF, device="cuda")
    assert capi.ss_attn_decode_paged(q.cuda(), kp, vp, table.cuda(), lens, od, 3, Hq, Hkv, pages, table.shape[1], d,
                                     d ** -0.5, 0.0, 1) == capi.SS_OK
    # both round their weights and outputs to bf16: each within 2^-8 of weights and value of the other's
    assert (o.float() - od.float()).abs().max() <= 4 * 2.0 ** -8 * max(float(x.float().abs().max()) for x in v)
    n = 700
    q, k, v = make(Hq, Hkv, d, [n], [n], 10)
    table, pages = random_tables([n], 0, np.random.default_rng(1))
    o = ss.chunk_paged(q.cuda(), fill_pool(k, [n], table, pages).cuda(), fill_pool(v, [n], table, pages).cuda(),
                       table.cuda(), offsets([n]).cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"),
                       scale=d ** -0.5)
    op = ss.prefill(q.transpose(0, 1)[None].contiguous().cuda(), k[0][None].cuda(), v[0][None].cuda(), scale=d ** -0.5,
                    causal=True)
    assert (o.float() - op[0].transpose(0, 1).float()).abs().max() <= 4 * 2.0 ** -8 * float(v[0].float().abs().max())


def test_chunk_many_sequences():
    """More sequences than one step of the search looks at, most of them without tokens."""
    rng = np.random.default_rng(2)
    n = [int(x) for x in rng.integers(0, 3, 1100)]
    n[7] = 70
    L = [max(x, int(y)) for x, y in zip(n, rng.integers(0, 200, 1100))]
    check(4, 1, 64, n, L, seed=11, debug=False)


def test_chunk_bad_device_arrays_stay_in_bounds():
    """Pages outside the pool read zeros, offsets and lengths out of range are cut: no fault, guards intact."""
    import block_sparse_attention_sm_gb300 as ss
    from _parity import guarded
    from block_sparse_attention_sm_gb300 import capi

    Hq, Hkv, d, pages = 4, 1, 128, 3
    kp = torch.ones(pages, Hkv, PAGE, d, dtype=BF, device="cuda")
    q = torch.ones(10, Hq, d, dtype=BF, device="cuda")
    o = guarded((10, Hq, d), BF, "cuda", 7.0)
    table = torch.tensor([[0, 1 << 30], [-5, 2]], dtype=torch.int32, device="cuda")
    for cu, L in (([0, 4, 10], [256, 200]), ([0, 4, 1 << 30], [1 << 30, 5]), ([0, 9, 3], [100, 100]),
                  ([-3, 2, 5], [10, -7])):
        o.t.fill_(7.0)
        ss.chunk_paged(q, kp, kp, table, torch.tensor(cu, dtype=torch.int32, device="cuda"),
                       torch.tensor(L, dtype=torch.int32, device="cuda"), scale=0.1, out=o.t)
        assert capi.ss_stream_status() == capi.SS_OK
        o.check("o")
    # sequence 0 of the first batch: half its keys are of no page, so half the weight meets zeros
    o.t.fill_(7.0)
    ss.chunk_paged(q, kp, kp, table, offsets([1, 0]).cuda(), torch.tensor([256, 0], dtype=torch.int32, device="cuda"),
                   scale=0.1, out=o.t)
    want = 1.0 / (1.0 + math.exp(-0.1 * d))
    assert (o.t[0].float() - want).abs().max() <= 2.0 ** -8


def test_chunk_repeats_bit_for_bit():
    """Units are handed to clusters in any order; the results do not depend on it."""
    import block_sparse_attention_sm_gb300 as ss

    n, L = [33, 1, 200, 7, 1, 90], [900, 2000, 1300, 64, 129, 700]
    q, k, v = make(8, 4, 128, n, L, 21)
    table, pages = random_tables(L, 1, np.random.default_rng(3))
    args = (q.cuda(), fill_pool(k, L, table, pages).cuda(), fill_pool(v, L, table, pages).cuda(), table.cuda(),
            offsets(n).cuda(), torch.tensor(L, dtype=torch.int32, device="cuda"))
    for kw in (dict(num_kv_splits=1), dict(num_kv_splits=4, lambda_a=4.0)):
        first = ss.chunk_paged(*args, scale=128 ** -0.5, **kw)
        for _ in range(20):
            assert torch.equal(ss.chunk_paged(*args, scale=128 ** -0.5, **kw), first)
    one = args[0]
    # a row alone gives what it gives among others (decode: the last token of each sequence)
    last = torch.tensor([sum(n[:i + 1]) - 1 for i in range(len(n))], device="cuda")
    alone = ss.chunk_paged(one[last].contiguous(), *args[1:4], offsets([1] * len(n)).cuda(), args[5], scale=128 ** -0.5)
    among = ss.chunk_paged(*args, scale=128 ** -0.5)[last]
    assert (alone.float() - among.float()).abs().max() <= 4 * 2.0 ** -8 * max(float(x.float().abs().max()) for x in v)


def test_chunk_nan_query_stays_in_its_row():
    import block_sparse_attention_sm_gb300 as ss

    n, L = [20], [300]
    q, k, v = make(4, 2, 128, n, L, 22)
    table, pages = random_tables(L, 1, np.random.default_rng(3))
    rest = (fill_pool(k, L, table, pages).cuda(), fill_pool(v, L, table, pages).cuda(), table.cuda(), offsets(n).cuda(),
            torch.tensor(L, dtype=torch.int32, device="cuda"))
    for kw in (dict(), dict(lambda_a=4.0)):
        clean = ss.chunk_paged(q.cuda(), *rest, scale=128 ** -0.5, **kw)
        bad = q.clone()
        bad[7, 1] = float("nan")
        got = ss.chunk_paged(bad.cuda(), *rest, scale=128 ** -0.5, **kw)
        assert got[7, 1].isnan().all()
        got[7, 1] = clean[7, 1]
        assert torch.equal(got, clean)


@pytest.mark.slow
def test_chunk_and_append_beyond_32_bit_offsets():
    """Pages more than 2^32 elements into the pool, written by the append call and read by the attention."""
    import block_sparse_attention_sm_gb300 as ss

    Hq, Hkv, d = 8, 8, 128
    pages = (1 << 32) // (Hkv * PAGE * d) + 40  # 8.6 GB each for keys and values
    kp = torch.full((pages, Hkv, PAGE, d), float("nan"), dtype=BF, device="cuda")
    vp = torch.full_like(kp, float("nan"))
    L = [500, 129]
    q, k, v = make(Hq, Hkv, d, L, L, 23)
    far = [[pages - 1 - 3 * i for i in range(4)], [pages - 20 - i for i in range(4)]]
    table = torch.tensor(far, dtype=torch.int32, device="cuda")
    lens, cu = torch.tensor(L, dtype=torch.int32, device="cuda"), offsets(L).cuda()
    rows = [torch.cat([x.transpose(0, 1) for x in y]).contiguous().cuda() for y in (k, v)]
    ss.rope_append_paged(None, *rows, kp, vp, table, cu, lens)
    o = ss.chunk_paged(q.cuda(), kp, vp, table, cu, lens, scale=d ** -0.5).cpu()
    at = 0
    for b, x in enumerate(L):
        ref, weight, _ = chunk_reference(q[at:at + x], k[b], v[b], x, d ** -0.5, True, 0.0, 1)
        assert_attention(o[at:at + x], ref, weight, f"sequence {b}")
        at += x
    # a fork copies such a page too
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[table.flatten().long()] = 1
    refs[: pages - 30] = 1
    rowsT = torch.cat([table, torch.full((1, 4), -1, dtype=torch.int32, device="cuda")]).contiguous()
    lens3 = torch.tensor(L + [0], dtype=torch.int32, device="cuda")
    one = torch.tensor([0], dtype=torch.int32, device="cuda")
    assert ss.pages_fork([kp, vp], refs, rowsT, lens3, one, one + 2).item() == 0
    new, old = int(rowsT[2, 3]), far[0][3]
    assert new >= pages - 30 and new != old
    assert torch.equal(kp[new, :, :116], kp[old, :, :116]) and torch.equal(vp[new, :, :116], vp[old, :, :116])


def test_chunk_counts_without_the_vote():
    import block_sparse_attention_sm_gb300 as ss
    from block_sparse_attention_sm_gb300 import capi

    n, L = [3, 50], [300, 200]
    q, k, v = make(4, 2, 64, n, L, 24)
    table, pages = random_tables(L, 1, np.random.default_rng(3))
    counts = torch.full((capi.ss_attn_chunk_paged_units(53, 2, 4, 2),), -1, dtype=torch.int32, device="cuda")
    ss.chunk_paged(q.cuda(), fill_pool(k, L, table, pages).cuda(), fill_pool(v, L, table, pages).cuda(), table.cuda(),
                   offsets(n).cuda(), torch.tensor(L, dtype=torch.int32, device="cuda"), scale=0.125, counts=counts)
    assert (counts == 0).all()


@pytest.mark.parametrize("a", [0.0, 4.0])
def test_chunk_in_parts(a):
    """Few new tokens over a long cache: the tiles are dealt to parts and merged."""
    from block_sparse_attention_sm_gb300 import capi

    n, L = [1, 4], [128 * 40 + 7, 128 * 33]
    assert capi.ss_attn_chunk_paged_workspace_size(5, 2, 4, 1, 41, 128, 7) == 5 * 5 * 4 * 130 * 4  # 41 pages: 5 parts
    check(4, 1, 128, n, L, a=a, splits=7, seed=31)
    check(4, 1, 128, n, L, a=a, splits=7, seed=32, debug=False)
    check(2, 2, 64, n, L, a=a, splits=3, seed=33, causal=False)


@pytest.mark.parametrize("a", [0.0, 4.0])
def test_chunk_of_more_ranges_than_tiles(a):
    """Any count is allowed; beyond one range a tile nothing changes."""
    check(8, 2, 64, [3], [128 * 20 + 5], a=a, splits=2 ** 31 - 1, seed=31)


def test_chunk_and_append_of_no_tokens():
    import block_sparse_attention_sm_gb300 as ss
    from _parity import guarded
    from block_sparse_attention_sm_gb300 import capi

    L, Hq, Hkv, d = [100, 300], 4, 2, 64
    pool = torch.ones(4, Hkv, PAGE, d, dtype=BF, device="cuda")
    table = torch.tensor([[0, 1, 2], [1, 2, 3]], dtype=torch.int32, device="cuda")
    cu, lens = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.tensor(L, dtype=torch.int32, device="cuda")
    row = lambda h: torch.empty(0, h, d, dtype=BF, device="cuda")  # noqa: E731
    freq, _ = ss.rope_frequencies(d)
    assert ss.rope_append_paged(row(Hq), row(Hkv), row(Hkv), pool, pool.clone(), table, cu, lens, freq).shape == (0, Hq, d)
    units = capi.ss_attn_chunk_paged_units(0, 2, Hq, Hkv)
    bands = [guarded((units,), torch.int32, "cuda", -1), guarded((units, 3), torch.uint8, "cuda", 9),
             guarded((units, 3), torch.float32, "cuda", 5.0)]
    for a in (0.0, 2.0):
        o = ss.chunk_paged(row(Hq), pool, pool, table, cu, lens, scale=0.1, lambda_a=a, num_kv_splits=2, counts=bands[0].t,
                           skip_mask=bands[1].t, vote_margin=bands[2].t)
        assert o.shape == (0, Hq, d)
        assert (bands[0].t == 0).all() and (bands[1].t == 2).all() and bands[2].t.isnan().all()
    for x in bands:
        x.check("chunk of no tokens")
    assert (pool == 1).all() and capi.ss_stream_status() == capi.SS_OK


@pytest.mark.parametrize("a", [0.0, 4.0])
@pytest.mark.parametrize("Hq,Hkv,d,n,L,splits,spoilt", [
    (4, 1, 128, [1, 1], [128 * 9 + 5, 700], 1, [0]),           # a decoded token: its heads are its block's only rows
    (4, 1, 128, [2, 1], [128 * 8, 700], 1, [0, 1]),            # an even number of tiles
    (2, 2, 64, [1, 3], [128 * 6 + 1, 700], 3, [0]),            # one head a group, ranges of the vote
    (1, 1, 128, [130], [1500], 1, list(range(128))),           # the first block of a pair
    (1, 1, 128, [130], [1400], 2, [128, 129]),                 # the second
    (4, 1, 128, [1, 4], [128 * 40 + 7, 128 * 33], 7, [0]),     # dealt to parts
    (4, 1, 128, [1, 4], [128 * 40 + 7, 128 * 33], 7, [1, 2, 3, 4]),
])
def test_chunk_nan_queries_that_fill_a_block(Hq, Hkv, d, n, L, splits, spoilt, a):
    """NaN rows alone in their block give NaN, not the zeros of a row without keys, and leave the others alone."""
    import block_sparse_attention_sm_gb300 as ss
    from block_sparse_attention_sm_gb300 import capi

    q, k, v = make(Hq, Hkv, d, n, L, 41)
    table, pages = random_tables(L, 1, np.random.default_rng(3))
    T, B, width = sum(n), len(n), table.shape[1]
    args = (fill_pool(k, L, table, pages).cuda(), fill_pool(v, L, table, pages).cuda(), table.cuda(), offsets(n).cuda(),
            torch.tensor(L, dtype=torch.int32, device="cuda"))
    kw = dict(scale=d ** -0.5, lambda_a=a, num_kv_splits=splits)
    clean = ss.chunk_paged(q.cuda(), *args, **kw)
    bad = q.clone()
    bad[spoilt] = float("nan")
    got = ss.chunk_paged(bad.cuda(), *args, **kw)
    assert got[spoilt].isnan().all()
    rest = [t for t in range(T) if t not in spoilt]
    assert torch.equal(got[rest], clean[rest])
    # the first tile of a range is kept, whatever the rows hold
    units = capi.ss_attn_chunk_paged_units(T, B, Hq, Hkv)
    mask = torch.full((units, width), 9, dtype=torch.uint8, device="cuda")
    margin = torch.zeros(units, width, device="cuda")
    ss.chunk_paged(bad.cuda(), *args, **kw, skip_mask=mask, vote_margin=margin)
    cu = offsets(n).tolist()
    b = next(b for b in range(B) if cu[b] <= spoilt[0] < cu[b + 1])
    place, half, places = chunk_place(cu, b, (spoilt[0] - cu[b]) // (PAGE // (Hq // Hkv)), Hq // Hkv, T, B)
    per = -(-tiles(L[b]) // splits)
    for h in range(Hkv):
        unit = (h * places + place) * 2 + half
        for j in range(0, tiles(L[b]), per):
            assert int(mask[unit, j]) == 0 and float(margin[unit, j]) == math.inf
    assert capi.ss_stream_status() == capi.SS_OK


def test_chunk_workspace_made_once():
    """A workspace of the largest step serves the smaller ones, which need more of it."""
    import block_sparse_attention_sm_gb300 as ss
    from block_sparse_attention_sm_gb300 import capi

    Hq, Hkv, d, width, splits = 4, 2, 128, 64, 6
    ws, nbytes = ss.chunk_paged_workspace(5000, 3, Hq, Hkv, width, d, splits, "cuda")
    assert capi.ss_attn_chunk_paged_workspace_size(5000, 3, Hq, Hkv, width, d, splits) == 0 < nbytes
    for n, L in (([1900, 60, 40], [2000, 100, 64 * PAGE]), ([1], [64 * PAGE]), ([63], [60 * PAGE + 1]), ([3, 1], [40 * PAGE, 8000])):
        q, k, v = make(Hq, Hkv, d, n, L, 51)
        table, pages = random_tables(L, 1, np.random.default_rng(5), width=width)
        args = (q.cuda(), fill_pool(k, L, table, pages).cuda(), fill_pool(v, L, table, pages).cuda(), table.cuda(),
                offsets(n).cuda(), torch.tensor(L, dtype=torch.int32, device="cuda"))
        for a in (0.0, 4.0):
            kw = dict(scale=d ** -0.5, lambda_a=a, num_kv_splits=splits)
            assert torch.equal(ss.chunk_paged(*args, **kw, workspace=ws), ss.chunk_paged(*args, **kw))
    assert capi.ss_stream_status() == capi.SS_OK


@pytest.mark.parametrize("a,splits", [(0.0, 1), (16.0, 1), (16.0, 3), (1e4, 1)])
@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (3, 1, 64)])
def test_chunk_votes_over_long_caches(Hq, Hkv, d, a, splits):
    """256 tiles a unit: the rings and the softmax's state go round many times, with most tiles skipped and with none."""
    skipped, evaluated = check(Hq, Hkv, d, [70, 1, 129], [128 * 256 + 5, 128 * 201, 128 * 255], a=a, splits=splits, seed=61)
    assert evaluated > 1000 and (skipped > evaluated // 2 if a == 16.0 else skipped == 0 if a == 0.0 else True)
