"""What the calls around the paged cache refuse before any launch, and their host-side arithmetic (CPU)."""
import math

import pytest
import torch

import block_sparse_attention_sm_gb300 as ss
from block_sparse_attention_sm_gb300 import capi as _capi

BF, I32 = torch.bfloat16, torch.int32
FAKE = 1 << 20  # a 16-byte-aligned non-null address; never dereferenced here


@pytest.fixture(scope="module")
def capi():
    ss.build()
    _capi.load()
    return _capi


# ------------------------------------------------------------------------- frequencies


def test_frequencies(capi):
    rot, base, orig, factor = 64, 10000.0, 4096, 8.0
    plain = [base ** (-2.0 * i / rot) for i in range(rot // 2)]

    def get(**kw):
        w, f = ss.rope_frequencies(rot, base, original_length=orig, device="cpu", **kw)
        assert w.dtype == torch.float64 and w.shape == (rot // 2,)
        return w.tolist(), f

    close = lambda a, b: all(math.isclose(x, y, rel_tol=1e-13) for x, y in zip(a, b))  # noqa: E731
    w, f = get()
    assert close(w, plain) and f == 1.0
    w, f = get(scaling="linear", factor=factor)
    assert close(w, [x / factor for x in plain]) and f == 1.0
    w, f = get(scaling="base", factor=factor)
    assert math.isclose(w[-1], plain[-1] / factor, rel_tol=1e-12) and w[0] == 1.0  # the last pair stretches by factor
    w, f = get(scaling="yarn", factor=factor)
    assert math.isclose(f, 0.1 * math.log(factor) + 1, rel_tol=1e-6)
    turns = [orig * x / (2 * math.pi) for x in plain]
    for x, y, t in zip(w, plain, turns):
        assert y / factor * (1 - 1e-12) <= x <= y * (1 + 1e-12)
        if t > 32 * base ** (2.0 / rot):
            assert math.isclose(x, y, rel_tol=1e-13)
        if t < 1 / base ** (2.0 / rot):
            assert math.isclose(x, y / factor, rel_tol=1e-13)
    w, f = get(scaling="wavelength", factor=factor)
    for x, y, t in zip(w, plain, turns):
        s = min(1.0, max(0.0, (t - 1) / 3))
        assert math.isclose(x, y * s + y / factor * (1 - s), rel_tol=1e-13) and f == 1.0


@pytest.mark.parametrize("kw", [
    dict(rot_dim=0), dict(rot_dim=7), dict(base=1.0), dict(base=float("nan")), dict(scaling=_capi.SS_ROPE_LINEAR, factor=0.5),
    dict(scaling=_capi.SS_ROPE_LINEAR, factor=float("inf")), dict(scaling=_capi.SS_ROPE_BASE, factor=2.0, rot_dim=2),
    dict(scaling=_capi.SS_ROPE_YARN, factor=2.0, original_length=0, lo=1.0, hi=32.0),
    dict(scaling=_capi.SS_ROPE_YARN, factor=2.0, original_length=10, lo=4.0, hi=4.0),
    dict(scaling=_capi.SS_ROPE_WAVELENGTH, factor=2.0, original_length=10, lo=0.0, hi=4.0),
    dict(scaling=9, factor=2.0),
])
def test_frequencies_refuse(capi, kw):
    args = dict(rot_dim=64, base=10000.0)
    args.update(kw)
    assert capi.ss_rope_frequencies(**args)[0] == capi.SS_ERR_INVALID_ARG


# ------------------------------------------------------------------------- C entry points


@pytest.mark.parametrize("kw,expect", [
    (dict(x=None), "INVALID_ARG"), (dict(positions=None), "INVALID_ARG"), (dict(inv_freq=None), "INVALID_ARG"),
    (dict(x=FAKE + 1), "INVALID_ARG"), (dict(inv_freq=FAKE + 4), "INVALID_ARG"),
    (dict(rot_dim=0), "INVALID_ARG"), (dict(rot_dim=63), "INVALID_ARG"), (dict(rot_dim=130), "INVALID_ARG"),
    (dict(rot_offset=1), "INVALID_ARG"), (dict(rot_offset=-2), "INVALID_ARG"), (dict(B=-1), "INVALID_ARG"),
    (dict(attn_factor=float("nan")), "INVALID_ARG"), (dict(out_strides=(512, 64, 128)), "INVALID_ARG"),
    (dict(out_strides=(0, 512, 128)), "INVALID_ARG"), (dict(x_strides=(-512, 512, 128)), "INVALID_ARG"),
    (dict(out=FAKE, x_strides=(4096, 1024, 256)), "INVALID_ARG"),   # in place with other strides
    (dict(d=1 << 17), "UNSUPPORTED"), (dict(position_stride=-4), "INVALID_ARG"),
    (dict(L=0, x=None), "OK"),
])
def test_rope_rejects(capi, kw, expect):
    args = dict(x=FAKE, out=2 * FAKE, B=2, H=2, L=4, d=128, positions=FAKE, inv_freq=FAKE, rot_dim=128, stream=0)
    args.update(kw)
    assert capi.ss_rope(**args) == getattr(capi, "SS_OK" if expect == "OK" else "SS_ERR_" + expect)


@pytest.mark.parametrize("kw,expect", [
    (dict(k=None), "INVALID_ARG"), (dict(q_out=None), "INVALID_ARG"), (dict(v_pages=None), "INVALID_ARG"),
    (dict(k_pages=FAKE + 2), "INVALID_ARG"), (dict(cu_seqlens=None), "INVALID_ARG"), (dict(seq_lens=None), "INVALID_ARG"),
    (dict(page_table=FAKE + 2), "INVALID_ARG"), (dict(T=-1), "INVALID_ARG"), (dict(B=0), "INVALID_ARG"),
    (dict(num_pages=0), "INVALID_ARG"), (dict(max_pages=1 << 25), "INVALID_ARG"), (dict(rot_dim=200), "INVALID_ARG"),
    (dict(inv_freq=None), "INVALID_ARG"), (dict(q_out_strides=(1024, 0)), "INVALID_ARG"),
    (dict(q_out=FAKE, q_strides=(4096, 128)), "INVALID_ARG"), (dict(d=1 << 17), "UNSUPPORTED"), (dict(T=0), "OK"),
])
def test_append_rejects(capi, kw, expect):
    args = dict(q=FAKE, q_out=2 * FAKE, k=FAKE, v=FAKE, T=5, B=2, Hq=8, Hkv=2, d=128, cu_seqlens=FAKE, seq_lens=FAKE,
                inv_freq=FAKE, rot_dim=128, k_pages=FAKE, v_pages=FAKE, page_table=FAKE, num_pages=4, max_pages=4, stream=0)
    args.update(kw)
    assert capi.ss_rope_append_paged(**args) == getattr(capi, "SS_OK" if expect == "OK" else "SS_ERR_" + expect)


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), "INVALID_ARG"), (dict(q=FAKE + 8), "INVALID_ARG"), (dict(page_table=None), "INVALID_ARG"),
    (dict(cu_seqlens=None), "INVALID_ARG"), (dict(seq_lens=None), "INVALID_ARG"), (dict(o=None), "INVALID_ARG"),
    (dict(T=-1), "INVALID_ARG"), (dict(B=0), "INVALID_ARG"), (dict(Hq=9), "INVALID_ARG"), (dict(num_pages=0), "INVALID_ARG"),
    (dict(max_pages=1 << 25), "INVALID_ARG"), (dict(scale=0.0), "INVALID_ARG"), (dict(scale=float("inf")), "INVALID_ARG"),
    (dict(lambda_a=-1.0), "INVALID_ARG"), (dict(lambda_a=float("nan")), "INVALID_ARG"), (dict(num_kv_splits=0), "INVALID_ARG"),
    (dict(q_token_stride=1020), "INVALID_ARG"), (dict(q_token_stride=512), "INVALID_ARG"), (dict(d=96), "UNSUPPORTED"),
    (dict(Hq=258), "UNSUPPORTED"), (dict(num_kv_splits=2), "WORKSPACE"),
    (dict(num_kv_splits=2, workspace=FAKE, workspace_bytes=2 * 5 * 8 * 130 * 4 - 1), "WORKSPACE"), (dict(T=0), "OK"),
    (dict(Hkv=70000, Hq=70000), "INVALID_ARG"),
])
def test_chunk_rejects(capi, kw, expect):
    args = dict(q=FAKE, k_pages=FAKE, v_pages=FAKE, page_table=FAKE, cu_seqlens=FAKE, seq_lens=FAKE, o=FAKE, T=5, B=2, Hq=8,
                Hkv=2, num_pages=4, max_pages=64, d=128, scale=0.1, causal=True, lambda_a=0.0, num_kv_splits=1, stream=0)
    args.update(kw)
    assert capi.ss_attn_chunk_paged(**args) == getattr(capi, "SS_OK" if expect == "OK" else "SS_ERR_" + expect)


def test_chunk_refuses_test_only_debug_fields(capi):
    import ctypes

    for field in ("count_only", "fault_inject", "vote_chunk_tiles", "prefill_kernel"):
        dbg = capi.ss_debug_opts()
        setattr(dbg, field, 1)
        st = capi.load().ss_attn_chunk_paged(FAKE, 0, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 5, 2, 8, 2, 4, 4, 128, 0.1, 1, 0.0, 1,
                                             None, None, 0, ctypes.byref(dbg), None)
        assert st == capi.SS_ERR_UNSUPPORTED


def test_sizes(capi):
    ws = capi.ss_attn_chunk_paged_workspace_size
    assert ws(10, 2, 8, 2, 64, 128, 1) == 0
    assert ws(10, 2, 8, 2, 64, 128, 3) == 3 * 10 * 8 * 130 * 4
    assert ws(10, 2, 8, 2, 64, 128, 1000) == 8 * 10 * 8 * 130 * 4   # 64 pages: 8 parts of 8
    assert ws(10, 2, 8, 2, 9999, 128, 1000) == 19 * 10 * 8 * 130 * 4  # 76 clusters, 4 pairs
    assert ws(10, 2, 8, 2, 15, 128, 1000) == 0                       # fewer than 8 pages a part
    assert ws(8192, 4, 32, 8, 256, 128, 8) == 0                      # enough rows without parts
    assert capi.ss_attn_chunk_paged_units(1000, 7, 8, 2) == 2 * (1000 // 64 + 7) * 2
    assert capi.ss_attn_chunk_paged_units(1000, 7, 6, 2) == 2 * (1000 // 84 + 7) * 2
    assert capi.ss_attn_chunk_paged_units(10, 1, 258, 2) == 0
    assert capi.ss_pages_workspace_size(100, 7, 5) >= 4 * (3 * 100 + 2 * 5)


@pytest.mark.parametrize("m", [1, 8, 18, 42, 128])
def test_places_of_row_blocks_never_meet(m):
    """floor(cu[b] / 2m) + b leaves room for every sequence's pairs of blocks."""
    import random

    r = random.Random(m)
    for _ in range(300):
        n = [r.choice([0, 1, m, 2 * m, 2 * m + 1, r.randint(0, 9 * m)]) for _ in range(r.randint(1, 12))]
        cu = [sum(n[:i]) for i in range(len(n) + 1)]
        places = cu[-1] // (2 * m) + len(n)
        start = [cu[b] // (2 * m) + b for b in range(len(n))]
        for b, x in enumerate(n):
            end = start[b] + -(-x // (2 * m))
            assert end <= (start[b + 1] if b + 1 < len(n) else places)


@pytest.mark.parametrize("kw,expect", [
    (dict(page_refs=None), "INVALID_ARG"), (dict(page_refs=FAKE + 4), "INVALID_ARG"), (dict(page_table=None), "INVALID_ARG"),
    (dict(seq_lens=None), "INVALID_ARG"), (dict(num_pages=0), "INVALID_ARG"), (dict(num_rows=0), "INVALID_ARG"),
    (dict(max_pages=1 << 25), "INVALID_ARG"), (dict(n=-1), "INVALID_ARG"),
])
def test_pages_reject_state(capi, kw, expect):
    state = dict(page_refs=FAKE, num_pages=10, page_table=FAKE, num_rows=4, max_pages=4, seq_lens=FAKE, n=2)
    state.update(kw)
    ws = dict(workspace=FAKE, workspace_bytes=1 << 20, stream=0)
    want = getattr(capi, "SS_ERR_" + expect)
    assert capi.ss_pages_reserve(rows=None, add=FAKE, **state, **ws) == want
    assert capi.ss_pages_free(rows=FAKE, **state, stream=0) == want
    assert capi.ss_pages_fork([FAKE], 256, src_rows=FAKE, dst_rows=FAKE, **state, **ws) == want
    if "n" not in kw:
        state.pop("n")
        assert capi.ss_pages_compact([FAKE], 256, **state, **ws) == want


def test_pages_reject_pools_lists_and_workspaces(capi):
    state = dict(page_refs=FAKE, num_pages=10, page_table=FAKE, num_rows=4, max_pages=4, seq_lens=FAKE)
    ws = dict(workspace=FAKE, workspace_bytes=1 << 20, stream=0)
    bad, small = capi.SS_ERR_INVALID_ARG, capi.SS_ERR_WORKSPACE
    for pools, page_bytes in (([None], 256), ([FAKE + 8], 256), ([FAKE], 24), ([FAKE], 0)):
        assert capi.ss_pages_fork(pools, page_bytes, src_rows=FAKE, dst_rows=FAKE, n=2, **state, **ws) == bad
        assert capi.ss_pages_compact(pools, page_bytes, **state, **ws) == bad
        assert capi.ss_pages_copy(pools, page_bytes, 10, FAKE, FAKE, 2, **ws) == bad
    assert capi.ss_pages_copy([], 256, 10, FAKE, FAKE, 2, **ws) == bad
    assert capi.ss_pages_copy([FAKE], 256, 10, None, FAKE, 2, **ws) == bad
    assert capi.ss_pages_fork([FAKE], 256, src_rows=None, dst_rows=FAKE, n=2, **state, **ws) == bad
    assert capi.ss_pages_reserve(rows=None, add=FAKE, n=5, **state, **ws) == bad  # more entries than rows
    ws["workspace_bytes"] = 16
    assert capi.ss_pages_reserve(rows=None, add=FAKE, n=2, **state, **ws) == small
    assert capi.ss_pages_compact([FAKE], 256, **state, **ws) == small
    assert capi.ss_pages_copy([FAKE], 256, 10, FAKE, FAKE, 2, **ws) == small


# ----------------------------------------------------------------------------- helpers


def _z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


FREQ = torch.ones(32, dtype=torch.float64)


def test_rope_helper_refuses():
    x, pos = _z(2, 3, 5, 64), _z(5, dtype=I32)
    for kw, match in ((dict(x=x.float()), "element type"), (dict(x=_z(5, 64)), "expects x"),
                      (dict(x=x.transpose(2, 3)), "last axis"), (dict(positions=_z(4, dtype=I32)), "expected shape"),
                      (dict(positions=pos.long()), "element type"), (dict(inv_freq=FREQ.float()), "element type"),
                      (dict(inv_freq=torch.ones(33, dtype=torch.float64)), "entries"), (dict(rot_offset=2), "entries"),
                      (dict(out=_z(2, 3, 5, 32)), "expected shape"), (dict(out=_z(1, 3, 5, 64).expand(2, 3, 5, 64)), "overlap"),
                      (dict(), "CUDA tensor")):
        args = dict(x=x, positions=pos, inv_freq=FREQ)
        args.update(kw)
        with pytest.raises((ValueError, TypeError), match=match):
            ss.rope(**args)
    whole = _z(1, 3, 6, 64)
    with pytest.raises(ValueError, match="overlaps its input"):
        ss.rope(whole[:, :, 1:], pos, FREQ, out=whole[:, :, :5])


def test_append_helper_refuses():
    args = dict(q=_z(5, 4, 64), k=_z(5, 2, 64), v=_z(5, 2, 64), k_pages=_z(3, 2, 128, 64), v_pages=_z(3, 2, 128, 64),
                page_table=_z(2, 4, dtype=I32), cu_seqlens=_z(3, dtype=I32), seq_lens=_z(2, dtype=I32), inv_freq=FREQ)
    for kw, match in ((dict(q=_z(4, 4, 64)), "expects q"), (dict(v=None), "given together"), (dict(v=_z(5, 1, 64)), "v: expected"),
                      (dict(k_pages=_z(3, 2, 64, 64)), "k_pages"), (dict(v_pages=_z(2, 2, 128, 64)), "v_pages"),
                      (dict(page_table=_z(2, 4)), "page_table"), (dict(cu_seqlens=_z(2, dtype=I32)), "cu_seqlens"),
                      (dict(seq_lens=_z(3, dtype=I32)), "seq_lens"), (dict(positions=_z(4, dtype=I32)), "positions"),
                      (dict(out=_z(5, 4, 32)), "out"), (dict(q=None, out=_z(5, 4, 64)), "without q"),
                      (dict(rot_offset=64), "entries"), (dict(), "CUDA tensor")):
        with pytest.raises((ValueError, TypeError), match=match):
            ss.rope_append_paged(**{**args, **kw})


def test_chunk_helper_refuses():
    args = dict(q=_z(5, 4, 64), k_pages=_z(3, 2, 128, 64), v_pages=_z(3, 2, 128, 64), page_table=_z(2, 4, dtype=I32),
                cu_seqlens=_z(3, dtype=I32), seq_lens=_z(2, dtype=I32), scale=0.1)
    units = 2 * (5 // 128 + 2) * 2
    ss.build()
    for kw, match in ((dict(q=_z(5, 64, 4).transpose(1, 2)), "last axis"), (dict(q=_z(5, 8, 64)[:, ::2]), "heads of a token"),
                      (dict(k_pages=_z(3, 2, 128, 128)), "k_pages"), (dict(v_pages=_z(3, 1, 128, 64)), "v_pages"),
                      (dict(cu_seqlens=_z(4, dtype=I32)), "cu_seqlens"), (dict(out=_z(5, 4, 128)), "out"),
                      (dict(counts=_z(units - 1, dtype=I32)), "counts"), (dict(skip_mask=_z(units * 4 - 1, dtype=torch.uint8)), "skip_mask"),
                      (dict(), "CUDA tensor")):
        with pytest.raises((ValueError, TypeError), match=match):
            ss.chunk_paged(**{**args, **kw})


def test_pages_helpers_refuse():
    state = dict(page_refs=_z(8, dtype=I32), page_table=_z(3, 4, dtype=I32), seq_lens=_z(3, dtype=I32))
    pools, one = [_z(8, 16)], _z(1, dtype=I32)
    with pytest.raises(ValueError, match="seq_lens"):
        ss.pages_free(**{**state, "seq_lens": _z(4, dtype=I32)}, rows=one)
    with pytest.raises(ValueError, match="rows"):
        ss.pages_reserve(**state, add=one, rows=_z(2, dtype=I32))
    with pytest.raises(ValueError, match="4 entries for 3 rows"):
        ss.pages_reserve(**state, add=_z(4, dtype=I32))
    for bad in ([_z(7, 16)], [_z(8, 16), _z(8, 32)], [_z(16, 8).t()]):
        with pytest.raises(ValueError, match=r"pools\["):
            ss.pages_fork(bad, **state, src_rows=one, dst_rows=one)
    with pytest.raises(ValueError, match="dst_rows"):
        ss.pages_fork(pools, **state, src_rows=one, dst_rows=_z(2, dtype=I32))
    with pytest.raises(ValueError, match="no pools"):
        ss.pages_copy([], one, one)
    with pytest.raises(ValueError, match="out_table"):
        ss.pages_compact(pools, **state, out_table=_z(3, 5, dtype=I32))
    for call in (lambda: ss.pages_free(**state, rows=one), lambda: ss.pages_compact(pools, **state),
                 lambda: ss.pages_copy(pools, one, one), lambda: ss.pages_reserve(**state, add=one)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


@pytest.mark.parametrize("kw,expect", [
    (dict(B=1, out_strides=(1024, 128, 128)), "INVALID_ARG"),      # heads and tokens on the same rows
    (dict(out_strides=(1024, 256, 192)), "INVALID_ARG"),           # ... partly
    (dict(out_strides=(1000, 128, 256)), "INVALID_ARG"),           # a batch inside the reach of 4 tokens, 1024
    (dict(out_strides=(1 << 62, 1 << 61, 1 << 62)), "INVALID_ARG"),  # (the reach passes 64 bits)
    (dict(H=(1 << 30) + 1), "UNSUPPORTED"), (dict(B=1 << 16, L=1 << 16), "UNSUPPORTED"),
])
def test_rope_rejects_overlap_and_counts(capi, kw, expect):
    args = dict(x=FAKE, out=2 * FAKE, B=2, H=2, L=4, d=128, positions=FAKE, inv_freq=FAKE, rot_dim=128, stream=0)
    if "out_strides" not in kw:
        args["x_strides"] = (0, 0, 0)
    assert capi.ss_rope(**{**args, **kw}) == getattr(capi, "SS_ERR_" + expect)


@pytest.mark.parametrize("kw,expect", [
    (dict(q_out_strides=(128, 128)), "INVALID_ARG"), (dict(q_out_strides=(1000, 128)), "INVALID_ARG"),
    (dict(q_out=3 * FAKE), "INVALID_ARG"), (dict(q_out=4 * FAKE), "INVALID_ARG"), (dict(q_out_strides=(1024, -128)), "INVALID_ARG"),
    (dict(T=(1 << 30) + 1), "UNSUPPORTED"), (dict(Hkv=1 << 30), "UNSUPPORTED"),
    (dict(T=0, q=None, q_out=None, k=None, v=None, v_pages=None), "OK"),
])
def test_append_rejects_overlap_and_counts(capi, kw, expect):
    args = dict(q=FAKE, q_out=2 * FAKE, k=3 * FAKE, v=4 * FAKE, T=5, B=2, Hq=8, Hkv=2, d=128, cu_seqlens=FAKE, seq_lens=FAKE,
                inv_freq=FAKE, rot_dim=128, k_pages=FAKE, v_pages=FAKE, page_table=FAKE, num_pages=4, max_pages=4, stream=0)
    assert capi.ss_rope_append_paged(**{**args, **kw}) == getattr(capi, "SS_OK" if expect == "OK" else "SS_ERR_" + expect)


def test_a_step_without_tokens_needs_no_rows(capi):
    """The empty tensors of a step of no tokens have null addresses."""
    assert capi.ss_attn_chunk_paged(q=None, k_pages=FAKE, v_pages=FAKE, page_table=FAKE, cu_seqlens=FAKE, seq_lens=FAKE, o=None,
                                    T=0, B=2, Hq=8, Hkv=2, num_pages=4, max_pages=64, d=128, scale=0.1, causal=True,
                                    lambda_a=0.0, num_kv_splits=4, stream=0) == capi.SS_OK


def test_chunk_helper_refuses_its_queries_as_output():
    q = _z(5, 4, 64)
    with pytest.raises(ValueError, match="overlaps q"):
        ss.chunk_paged(q, _z(3, 2, 128, 64), _z(3, 2, 128, 64), _z(2, 4, dtype=I32), _z(3, dtype=I32), _z(2, dtype=I32),
                       scale=0.1, out=q)


@pytest.mark.parametrize("q", [
    _z(1, 4, 64).expand(5, 4, 64),                      # one row for all tokens
    _z(2000).as_strided((5, 4, 64), (128, 64, 1)),      # a token's last heads are the next one's first
    _z(2000).as_strided((5, 1, 64), (8, 64, 1)),
])
def test_chunk_helper_refuses_queries_whose_tokens_overlap(q):
    """A token stride of 0 means contiguous rows to the entry point, which would read behind such a tensor."""
    with pytest.raises(ValueError, match="tokens overlap"):
        ss.chunk_paged(q, _z(3, 1, 128, 64), _z(3, 1, 128, 64), _z(2, 4, dtype=I32), _z(3, dtype=I32), _z(2, dtype=I32), scale=0.1)


def test_chunk_helper_takes_one_token_of_any_stride():
    with pytest.raises(ValueError, match="CUDA tensor"):  # (the last check)
        ss.chunk_paged(_z(2000).as_strided((1, 4, 64), (0, 64, 1)), _z(3, 1, 128, 64), _z(3, 1, 128, 64), _z(2, 4, dtype=I32),
                       _z(3, dtype=I32), _z(2, dtype=I32), scale=0.1)


def test_append_ex_rejects_like_append(capi):
    args = dict(q=FAKE, q_out=2 * FAKE, k=3 * FAKE, v=4 * FAKE, T=5, B=2, Hq=8, Hkv=2, d=128, cu_seqlens=FAKE, seq_lens=FAKE,
                inv_freq=FAKE, rot_dim=128, k_pages=FAKE, v_pages=FAKE, page_table=FAKE, num_pages=4, max_pages=4, stream=0)
    for kw in (dict(refused=FAKE + 2), dict(k=None), dict(q_out=3 * FAKE), dict(max_pages=0)):
        assert capi.ss_rope_append_paged_ex(**{**args, **kw}) == capi.SS_ERR_INVALID_ARG
    assert capi.ss_rope_append_paged_ex(**{**args, "T": 0, "refused": FAKE}) == capi.SS_OK


def test_append_helper_refuses_other_results():
    args = dict(q=None, k=_z(5, 2, 64), v=_z(5, 2, 64), k_pages=_z(3, 2, 128, 64), v_pages=_z(3, 2, 128, 64),
                page_table=_z(2, 4, dtype=I32), cu_seqlens=_z(3, dtype=I32), seq_lens=_z(2, dtype=I32), inv_freq=FREQ)
    for refused, match in ((_z(1), "refused: element type"), (_z(2, dtype=I32), "refused: expected shape"), (0, "refused: expected a torch")):
        with pytest.raises((ValueError, TypeError), match=match):
            ss.rope_append_paged(**args, refused=refused)


# Calls with nothing to refuse but the missing GPU (their addresses are not memory).
without_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="only without a GPU")


@without_gpu
def test_chunk_refuses_outputs_on_its_inputs(capi):
    """o on q's other rows, or in a pool; rows that lie between q's are apart from them."""
    T, Hq, Hkv, d, pages = 5, 8, 2, 128, 4
    far, row, pool = 64 * FAKE, Hq * d, pages * Hkv * 128 * d
    args = dict(q=far, k_pages=2 * far, v_pages=3 * far, page_table=FAKE, cu_seqlens=FAKE, seq_lens=FAKE, o=4 * far, T=T, B=2, Hq=Hq,
                Hkv=Hkv, num_pages=pages, max_pages=64, d=d, scale=0.1, causal=True, lambda_a=0.0, num_kv_splits=1, stream=0)
    bad, fine = capi.SS_ERR_INVALID_ARG, capi.ss_attn_chunk_paged(**args)  # (without a GPU: SS_ERR_UNSUPPORTED or SS_ERR_CUDA)
    assert fine not in (bad, capi.SS_OK)
    for kw, want in ((dict(o=far), bad), (dict(o=far + 2 * row), bad), (dict(o=far - 16), bad), (dict(o=far + 2 * T * row), fine),
                     (dict(o=far - 2 * T * row), fine), (dict(o=2 * far + 2 * pool - 16), bad), (dict(o=2 * far + 2 * pool), fine),
                     (dict(o=3 * far - 16), bad), (dict(o=far + 2 * row, T=1), fine),
                     (dict(o=far + 2 * row, T=2, q_token_stride=3 * row), fine),     # both rows of o between q's two
                     (dict(o=far + 2 * row + 16, T=2, q_token_stride=3 * row), bad)):
        assert capi.ss_attn_chunk_paged(**{**args, **kw}) == want, kw


def test_chunk_helper_refuses_outputs_on_its_inputs():
    buf = _z(6, 4, 64)
    pool = _z(3, 2, 128, 64)
    args = dict(k_pages=pool, v_pages=pool.clone(), page_table=_z(2, 4, dtype=I32), cu_seqlens=_z(3, dtype=I32),
                seq_lens=_z(2, dtype=I32), scale=0.1)
    for q, out, match in ((buf[:-1], buf[1:], "overlaps q"), (buf[1:], buf[:-1], "overlaps q"), (buf[:5], pool.view(-1, 4, 64)[7:12], "overlaps k_pages"),
                          (buf[:2], buf[2:4], "CUDA tensor"), (buf[:0], buf[:0], "CUDA tensor"),
                          (buf[::3], buf[1:3], "CUDA tensor")):
        with pytest.raises(ValueError, match=match):
            ss.chunk_paged(q, out=out, **args)


def test_overlap_of_strided_tensors():
    """The test of shared elements against their sets, on random views of one buffer."""
    import random

    from block_sparse_attention_sm_gb300.cache import _meet

    r, buf = random.Random(0), _z(1 << 15)
    alike = wrong = 0
    for _ in range(4000):
        d, views = r.choice([1, 2, 8, 64]), []
        h = d * r.choice([1, 1, 2, 3]) + r.choice([0, 0, 1])
        t = h * r.randint(1, 6) + r.choice([0, 0, 5])
        for _ in range(2):
            shape = (r.randint(1, 5), r.randint(1, 4), d)
            strides = r.choice([(t, h, 1), (t, h, 1), (h, t, 1), (0, h, 1)])
            reach = sum(s * (n - 1) for s, n in zip(strides, shape)) + 1
            views.append(buf.as_strided(shape, strides, r.randint(0, min(buf.numel() - reach, 3 * t))))
        sets = []
        for v in views:
            at = torch.zeros(1, dtype=torch.long) + v.storage_offset()
            for s, n in zip(v.stride(), v.shape):
                at = (at[:, None] + s * torch.arange(n)).flatten()
            sets.append(set(at.tolist()))
        want, got = bool(sets[0] & sets[1]), _meet(*views)
        assert got or not want                     # never calls shared elements apart
        alike += 1
        wrong += got and not want                  # (views of different strides may be refused)
        if views[0].stride() == views[1].stride() and views[0].stride()[0] >= views[0].stride()[1] * 4 and views[0].stride()[1] >= d:
            assert got == want
    assert wrong < alike // 20


@without_gpu
@pytest.mark.parametrize("v", [True, False])
def test_append_refuses_overlapping_memory(capi, v):
    """q_out and the pools against every input and each other; parts of one projection are apart."""
    T, Hq, Hkv, d, pages = 5, 8, 2, 128, 4
    far, pool = 64 * FAKE, pages * Hkv * 128 * d * 2
    wide = (Hq + 2 * Hkv) * d  # entries of a token's row: q, k and v heads
    tok = (wide, d)
    args = dict(q=far, q_out=2 * far, k=far + 2 * Hq * d, v=far + 2 * (Hq + Hkv) * d if v else None, T=T, B=2, Hq=Hq, Hkv=Hkv, d=d,
                cu_seqlens=FAKE, seq_lens=FAKE, inv_freq=FAKE, rot_dim=128, k_pages=3 * far, v_pages=4 * far if v else None,
                page_table=FAKE, num_pages=pages, max_pages=4, stream=0, q_strides=tok, k_strides=tok, v_strides=tok)
    bad, fine = capi.SS_ERR_INVALID_ARG, capi.ss_rope_append_paged(**args)
    assert fine not in (bad, capi.SS_OK)
    for kw, want in ((dict(q_out=far, q_out_strides=tok), fine),                                   # in place
                     (dict(q_out=far + 2 * d, q_out_strides=tok), bad),                            # one head on
                     (dict(q_out=far + 2 * (Hq - 1) * d, q_out_strides=tok), bad),                 # on q, k and v
                     (dict(q_out=far + 2 * (Hkv + Hq) * d, q_out_strides=tok), bad),               # on v, and the next token's q
                     (dict(q_out=far + 2 * T * wide, q_out_strides=tok), fine),
                     (dict(q_out=far + 2 * Hq * d, q_out_strides=(wide, d), Hq=Hkv), bad),           # on k
                     (dict(q_out=far + 2 * (Hq + Hkv) * d, q_out_strides=(wide, d), Hq=Hkv), bad if v else fine),  # on v
                     (dict(q_out=far + 2 * wide - 2), bad),
                     (dict(q_out=3 * far + pool - 2), bad), (dict(q_out=3 * far + pool), fine),
                     (dict(q_out=4 * far), bad if v else fine),
                     (dict(k=3 * far + pool - 2), bad), (dict(k=3 * far - 2 * T * wide), fine),
                     (dict(k_pages=far + 32), bad), (dict(k_pages=far - pool), fine), (dict(k_pages=far - pool + 16), bad)) + (
                     ((dict(v=3 * far), bad), (dict(v=4 * far), bad), (dict(v_pages=3 * far), bad), (dict(v_pages=3 * far + pool), fine),
                      (dict(v_pages=far), bad)) if v else ()):
        assert capi.ss_rope_append_paged(**{**args, **kw}) == want, kw


def test_rope_helper_takes_rows_between_its_inputs():
    """Views of one tensor without a shared element are apart; the same memory is in place whatever an axis of one is called."""
    pos = _z(5, dtype=I32)
    proj, whole = _z(5, 8, 64), _z(2, 3, 10, 64)
    one = _z(1, 3, 5, 64)
    for x, out in ((proj[:, :3], proj[:, 3:6]), (whole[:, :, 0::2], whole[:, :, 1::2]), (whole[:, :, :5], whole[:, :, 5:]),
                   (proj[:, :3], proj[:, :3]), (one, one.as_strided(one.shape, (7, 320, 64, 1))), (_z(5, 8, 128)[..., :64], proj)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            ss.rope(x, pos, FREQ, out=out)
    both = _z(5, 2, 128)
    with pytest.raises(ValueError, match="CUDA tensor"):  # the rows' halves
        ss.rope(both[..., :64], pos, FREQ, out=both[..., 64:])
    for x, out in ((proj[:, :3], proj[:, 2:5]), (whole[:, :, :5], whole[:, :, 4:9]), (whole[:, :, 0::2], whole[:, :, :5]),
                   (both[..., :64], both[..., 32:96])):
        with pytest.raises(ValueError, match="overlaps its input"):
            ss.rope(x, pos, FREQ, out=out)


@without_gpu
def test_rope_refuses_overlapping_memory(capi):
    """The C entry point on the random views of one buffer that the helper is tested with."""
    import random

    from block_sparse_attention_sm_gb300.cache import _meet

    args = dict(d=64, positions=FAKE, inv_freq=FAKE, rot_dim=64, stream=0)
    fine = capi.ss_rope(FAKE, 2 * FAKE, 1, 1, 1, **args)
    assert fine not in (capi.SS_ERR_INVALID_ARG, capi.SS_OK)
    r, buf, met = random.Random(1), _z(1 << 16), 0
    for _ in range(2000):
        B, H, L = r.randint(1, 3), r.randint(1, 4), r.randint(1, 5)
        h = 64 * r.choice([1, 1, 2, 3])
        t = h * H * r.choice([1, 1, 2]) + r.choice([0, 64])
        strides = r.choice([(t * L, h, t), (t * L * 2, h, t)])
        xs = r.choice([strides, strides, (0, h, t), (t * L, 64, t)])
        reach = lambda s: sum(a * (n - 1) for a, n in zip(s, (B, H, L))) + 64  # noqa: E731
        x = buf.as_strided((B, H, L, 64), (*xs, 1), 2048 + r.randint(0, 3) * 64 + r.choice([0, 0, 8]))
        o = buf.as_strided((B, H, L, 64), (*strides, 1), 2048 + r.randint(-1, 3) * r.choice([64, h, t]))
        assert max(reach(xs), reach(strides)) < (1 << 16) - 8192  # (inside the buffer)
        want = _meet(o, x) and not (o.data_ptr() == x.data_ptr() and all(a == b for a, b, n in zip(xs, strides, (B, H, L)) if n > 1))
        if o.data_ptr() == x.data_ptr() and any(a != b for a, b, n in zip(xs, strides, (B, H, L)) if n > 1):
            want = True
        got = capi.ss_rope(x, o, B, H, L, x_strides=xs, out_strides=strides, **args)
        assert got == (capi.SS_ERR_INVALID_ARG if want else fine), (B, H, L, xs, strides, x.storage_offset(), o.storage_offset())
        met += want
    assert 400 < met < 1600


@without_gpu
def test_pages_refuse_overlapping_arrays(capi):
    """What a call writes lies apart from everything else it is given."""
    pages, rows, width, n, page_bytes = 40, 6, 5, 3, 256
    at = {x: (i + 1) * 16 * FAKE for i, x in enumerate(("refs", "table", "lens", "ws", "result", "a", "b", "out_refs", "out_table"))}
    size = dict(refs=4 * pages, table=4 * rows * width, lens=4 * rows, result=4, a=4 * n, b=4 * n, out_refs=4 * pages, out_table=4 * rows * width)
    size["ws"] = capi.ss_pages_workspace_size(pages, rows, n)
    pool, pool_bytes = 100 * 16 * FAKE, pages * page_bytes

    def call(name, x, pools):
        state = dict(page_refs=x["refs"], num_pages=pages, page_table=x["table"], num_rows=rows, max_pages=width, seq_lens=x["lens"])
        ws = dict(workspace=x["ws"], workspace_bytes=size["ws"], stream=0)
        if name == "reserve":
            return capi.ss_pages_reserve(**state, rows=x["a"], add=x["b"], n=n, result=x["result"], **ws)
        if name == "free":
            return capi.ss_pages_free(**state, rows=x["a"], n=n, stream=0)
        if name == "fork":
            return capi.ss_pages_fork(pools, page_bytes, **state, src_rows=x["a"], dst_rows=x["b"], n=n, result=x["result"], **ws)
        if name == "copy":
            return capi.ss_pages_copy(pools, page_bytes, pages, x["a"], x["b"], n, result=x["result"], **ws)
        return capi.ss_pages_compact(pools, page_bytes, **state, out_refs=x["out_refs"], out_table=x["out_table"], live=x["result"], **ws)

    written = dict(reserve=("refs", "table", "lens", "result", "ws"), free=("refs", "table", "lens"),
                   fork=("refs", "table", "lens", "result", "ws"), copy=("result", "ws"),
                   compact=("out_refs", "out_table", "result", "ws"))
    read = dict(reserve=("a", "b"), free=("a",), fork=("a", "b"), copy=("a", "b"), compact=("refs", "table", "lens"))
    apart = [pool, pool + 3 * pool_bytes, pool + pool_bytes]  # (not in order)
    bad = capi.SS_ERR_INVALID_ARG
    for name in written:
        fine = call(name, at, apart)
        assert fine not in (bad, capi.SS_OK, capi.SS_ERR_WORKSPACE)
        assert call(name, at, apart + apart[:1]) == fine  # a pool listed twice
        size["ws"] = capi.ss_pages_workspace_size(pages, 0 if name == "copy" else rows, 0 if name == "compact" else n)
        names = written[name] + read[name]
        for w in written[name]:
            for other in names:
                if other == w or {w, other} in ({"out_refs", "refs"}, {"out_table", "table"}):
                    continue
                base = at[other] + (size[other] - 1) // 16 * 16  # its last word(s)
                assert call(name, {**at, w: base}, apart) == bad, (name, w, other)
        for r in read[name]:
            if name in ("reserve", "fork", "copy"):
                assert call(name, {**at, "a": at["b"]}, apart) == fine  # both are read only
        if name == "compact":
            assert call(name, {**at, "out_refs": at["refs"], "out_table": at["table"]}, apart) == fine
            assert call(name, {**at, "out_refs": None, "out_table": None, "result": None}, apart) == fine
            assert call(name, {**at, "out_refs": at["refs"] + 16}, apart) == bad
            assert call(name, {**at, "out_table": at["table"] + 16}, apart) == bad
        if name in ("fork", "copy", "compact"):
            for w in names:
                assert call(name, {**at, w: pool + pool_bytes - 16}, apart) == bad, (name, w)
                assert call(name, {**at, w: pool + 2 * pool_bytes}, apart) == fine
            for pools in ([pool, pool + 16], [pool + 16, pool], [pool, pool + 2 * pool_bytes, pool + pool_bytes - 16],
                          [pool + pool_bytes, pool + pool_bytes, pool + 16]):
                assert call(name, at, pools) == bad


def test_rope_refuses_what_it_cannot_record():
    x, pos = _z(2, 3, 5, 64).requires_grad_(True), _z(5, dtype=I32)
    with pytest.raises(ValueError, match="out: not where a gradient"):
        ss.rope(x, pos, FREQ, out=_z(2, 3, 5, 64))
    with pytest.raises(ValueError, match="out: not where a gradient"):
        ss.rope(x, pos, FREQ, out=x)
    with pytest.raises(ValueError, match="frequencies"):
        ss.rope(_z(2, 3, 5, 64), pos, FREQ.clone().requires_grad_(True))
    for kw, match in ((dict(), "CUDA tensor"), (dict(positions=_z(4, dtype=I32)), "expected shape"), (dict(rot_offset=2), "entries")):
        with pytest.raises(ValueError, match=match):  # the other checks are as they were
            ss.rope(**{**dict(x=x, positions=pos, inv_freq=FREQ), **kw})
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA tensor"):
        ss.rope(x, pos, FREQ, out=x)


def test_chunk_workspace_bound(capi):
    """What the bound promises, by trying the smaller steps; smaller steps do need more than larger ones."""
    size, bound = capi.ss_attn_chunk_paged_workspace_size, capi.ss_attn_chunk_paged_workspace_bound
    assert [size(T, 1, 32, 8, 256, 128, 8) for T in (2048, 256)] == [0, 0]
    assert size(64, 1, 32, 8, 256, 128, 8) < size(63, 1, 32, 8, 256, 128, 8) <= bound(2048, 32, 8, 256, 128, 8)
    for T, Hq, Hkv, pages, splits in ((1, 1, 1, 1, 1), (5, 4, 1, 41, 7), (700, 8, 2, 64, 3), (700, 8, 2, 64, 1), (900, 32, 8, 256, 8),
                                      (300, 3, 1, 9999, 1000), (2000, 128, 1, 100, 2 ** 31 - 1), (9000, 1, 1, 80, 50), (50, 40, 40, 64, 4)):
        most = max(size(t, 1, Hq, Hkv, pages, 64, splits) for t in range(1, T + 1))
        assert bound(T, Hq, Hkv, pages, 64, splits) == most
        for t in {1, T // 3 + 1, T}:
            for b in (1, 2, 7, 80):
                for p in {1, pages // 2 + 1, pages}:
                    for s in {1, splits // 2 + 1, splits}:
                        assert size(t, b, Hq, Hkv, p, 64, s) <= most
    assert bound(0, 8, 2, 64, 128, 3) == 0 and bound(10, 1, 2, 64, 128, 3) == 0 and bound(10, 258, 2, 64, 128, 3) == 0
    ws, n = ss.chunk_paged_workspace(2048, 1, 32, 8, 256, 128, 8, "cpu")
    assert n == bound(2048, 32, 8, 256, 128, 8) and ws.numel() == n


@without_gpu
def test_sizes_beyond_64_bits_are_compared(capi):
    """Pools of more bytes than 64 bits count reach everything behind them; nothing wraps round."""
    far = 1 << 40
    state = dict(page_refs=far, num_pages=1 << 30, page_table=2 * far, num_rows=4, max_pages=4, seq_lens=3 * far)
    ws = dict(workspace=4 * far, workspace_bytes=1 << 40, stream=0)
    lists = dict(src_rows=5 * far, dst_rows=6 * far, n=2)
    assert capi.ss_pages_fork([FAKE], 1 << 34, **state, **ws, **lists) == capi.SS_ERR_INVALID_ARG     # (2^64 bytes a pool)
    assert capi.ss_pages_fork([7 * far], 1 << 34, **state, **ws, **lists) not in (capi.SS_OK, capi.SS_ERR_INVALID_ARG)
    assert capi.ss_pages_fork([7 * far, 8 * far], 1 << 34, **state, **ws, **lists) == capi.SS_ERR_INVALID_ARG
    args = dict(q=None, q_out=None, k=2 * far, v=None, T=5, B=2, Hq=8, Hkv=1 << 20, d=1 << 16, cu_seqlens=FAKE, seq_lens=FAKE, inv_freq=FAKE,
                rot_dim=128, k_pages=far, v_pages=None, page_table=FAKE, num_pages=1 << 30, max_pages=4, stream=0)
    assert capi.ss_rope_append_paged(**args) == capi.SS_ERR_INVALID_ARG                               # (2^74 bytes)
    assert capi.ss_rope_append_paged(**{**args, "k": FAKE, "k_pages": 1 << 60}) not in (capi.SS_OK, capi.SS_ERR_INVALID_ARG)
