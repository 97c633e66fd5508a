"""What the calls over shared pages, the record of weights and eviction refuse before any launch (CPU)."""
import pytest
import torch

import block_sparse_attention_sm_gb300 as ss
from block_sparse_attention_sm_gb300 import capi as _capi

BF, I32, F32 = torch.bfloat16, torch.int32, torch.float32
FAKE = 1 << 20  # a 16-byte-aligned non-null address; never dereferenced here
APART = [FAKE + (k << 44) for k in range(16)]  # arrays that lie apart


@pytest.fixture(scope="module")
def capi():
    ss.build()
    _capi.load()
    return _capi


def status(capi, name):
    return getattr(capi, "SS_ERR_" + name)


# ------------------------------------------------------------------------------ the plan


@pytest.mark.parametrize("kw,expect", [
    (dict(page_table=0), "INVALID_ARG"), (dict(seq_lens=0), "INVALID_ARG"), (dict(plan=0), "INVALID_ARG"), (dict(B=0), "INVALID_ARG"),
    (dict(max_pages=0), "INVALID_ARG"), (dict(max_pages=1 << 24), "INVALID_ARG"), (dict(plan=APART[2] + 2), "INVALID_ARG"),
    (dict(page_table=APART[0] + 1), "INVALID_ARG"), (dict(B=8193, plan_bytes=1 << 30), "UNSUPPORTED"), (dict(plan_bytes=64), "WORKSPACE"),
    (dict(plan=APART[0] + 8), "INVALID_ARG"), (dict(plan=APART[1]), "INVALID_ARG"),
])
def test_plan_rejects(capi, kw, expect):
    args = dict(page_table=APART[0], seq_lens=APART[1], B=4, max_pages=8, plan=APART[2], plan_bytes=1 << 20, stream=0)
    assert capi.ss_prefix_plan(**{**args, **kw}) == status(capi, expect)


def test_plan_sizes(capi):
    assert capi.ss_prefix_plan_size(0) == capi.ss_prefix_plan_size(8193) == 0
    sizes = [capi.ss_prefix_plan_size(b) for b in range(1, 200)]
    assert all(b > a > 0 for a, b in zip(sizes, sizes[1:])) and all(x % 4 == 0 for x in sizes)


# ---------------------------------------------------------------------------- the decode

DECODE = dict(q=APART[0], k_pages=APART[1], v_pages=APART[2], page_table=APART[3], seq_lens=APART[4], plan=APART[5], o=APART[6],
              weights=APART[7], B=4, Hq=8, Hkv=2, num_pages=16, max_pages=8, d=128, scale=0.1, workspace=APART[8],
              workspace_bytes=1 << 40, stream=0)


@pytest.mark.parametrize("kw,expect", [
    *[({k: 0}, "INVALID_ARG") for k in ("q", "k_pages", "v_pages", "page_table", "seq_lens", "o", "B", "Hq", "Hkv", "num_pages", "max_pages")],
    *[({k: DECODE[k] + 8}, "INVALID_ARG") for k in ("q", "k_pages", "v_pages", "o", "weights")],
    *[({k: DECODE[k] + 2}, "INVALID_ARG") for k in ("page_table", "seq_lens", "plan")],
    (dict(Hq=9), "INVALID_ARG"), (dict(scale=0.0), "INVALID_ARG"), (dict(scale=-1.0), "INVALID_ARG"), (dict(scale=float("nan")), "INVALID_ARG"),
    (dict(scale=float("inf")), "INVALID_ARG"), (dict(d=96), "UNSUPPORTED"), (dict(d=192), "UNSUPPORTED"), (dict(Hq=258, Hkv=2), "UNSUPPORTED"),
    (dict(q_token_stride=1016), "INVALID_ARG"), (dict(q_token_stride=1028), "INVALID_ARG"), (dict(q_token_stride=1 << 38), "INVALID_ARG"),
    (dict(q_token_stride=-1024), "INVALID_ARG"), (dict(max_pages=1 << 24), "INVALID_ARG"), (dict(num_pages=1 << 30, Hkv=4), "INVALID_ARG"),
    (dict(B=8193), "UNSUPPORTED"), (dict(B=32769, plan=0), "UNSUPPORTED"), (dict(max_pages=(1 << 23) + 1), "UNSUPPORTED"),
    (dict(workspace=0), "WORKSPACE"), (dict(workspace=APART[8] + 8), "WORKSPACE"), (dict(workspace_bytes=1000), "WORKSPACE"),
    *[(dict(o=DECODE[k]), "INVALID_ARG") for k in ("q", "k_pages", "v_pages", "page_table", "seq_lens", "plan", "weights", "workspace")],
    *[(dict(weights=DECODE[k]), "INVALID_ARG") for k in ("q", "k_pages", "v_pages", "page_table", "plan", "workspace")],
    (dict(workspace=APART[1] + 4096), "INVALID_ARG"),
])
def test_decode_rejects(capi, kw, expect):
    assert capi.ss_attn_decode_shared(**{**DECODE, **kw}) == status(capi, expect)


def test_decode_accepts_up_to_the_device(capi):
    """Without a GPU what is left to refuse is the device."""
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    fine = {status(capi, "UNSUPPORTED"), status(capi, "CUDA")}
    for kw in ({}, dict(plan=None, weights=None), dict(q_token_stride=1536), dict(B=8192), dict(B=32768, plan=None), dict(max_pages=1 << 23), dict(Hq=256),
               dict(B=1, q_token_stride=8), dict(d=64)):
        assert capi.ss_attn_decode_shared(**{**DECODE, **kw}) in fine, kw


def test_decode_workspace_grows_with_the_step(capi):
    size = lambda B=4, pages=8, plan=1, w=0: capi.ss_attn_decode_shared_workspace_size(B, 32, 8, pages, 128, plan, w)  # noqa: E731
    assert size() > size(plan=0) > 0 and size(w=1) > size()
    for plan in (0, 1):
        for w in (0, 1):
            last = 0
            for B in (1, 2, 3, 7, 64, 500, 8000):
                at = 0
                for pages in (1, 2, 3, 20, 64, 400):
                    n = size(B, pages, plan, w)
                    assert n >= at and n >= (last if pages == 400 else 0)
                    at = n
                last = at
    assert capi.ss_attn_decode_shared_workspace_size(0, 8, 2, 4, 128, 1, 1) == 0
    assert capi.ss_attn_decode_shared_workspace_size(1, 1, 2, 4, 128, 1, 1) == 0


# ---------------------------------------------------------------------------- key weights

KEYS = dict(q=APART[0], k_pages=APART[1], page_table=APART[2], cu_seqlens=APART[3], seq_lens=APART[4], weights=APART[5], T=40, B=4,
            Hq=8, Hkv=2, num_pages=16, max_pages=8, d=64, scale=0.1, causal=True, workspace=APART[6], workspace_bytes=1 << 40, stream=0)


@pytest.mark.parametrize("kw,expect", [
    *[({k: 0}, "INVALID_ARG") for k in ("q", "k_pages", "page_table", "cu_seqlens", "seq_lens", "weights", "B", "Hq", "Hkv", "num_pages", "max_pages")],
    *[({k: KEYS[k] + 8}, "INVALID_ARG") for k in ("q", "k_pages", "weights")],
    *[({k: KEYS[k] + 2}, "INVALID_ARG") for k in ("page_table", "cu_seqlens", "seq_lens")],
    (dict(T=-1), "INVALID_ARG"), (dict(Hq=7), "INVALID_ARG"), (dict(scale=0.0), "INVALID_ARG"), (dict(d=128 + 64), "UNSUPPORTED"),
    (dict(Hq=130, Hkv=1), "UNSUPPORTED"), (dict(q_token_stride=504), "INVALID_ARG"), (dict(q_token_stride=516), "INVALID_ARG"),
    (dict(T=0x7fffffff), "INVALID_ARG"), (dict(max_pages=1 << 24), "INVALID_ARG"), (dict(num_pages=1 << 30, Hkv=4), "INVALID_ARG"),
    (dict(B=1 << 30, max_pages=1 << 20), "INVALID_ARG"),
    (dict(workspace=0), "WORKSPACE"), (dict(workspace=APART[6] + 8), "WORKSPACE"), (dict(workspace_bytes=1000), "WORKSPACE"),
    *[(dict(weights=KEYS[k]), "INVALID_ARG") for k in ("q", "k_pages", "page_table", "cu_seqlens", "seq_lens", "workspace")],
    *[(dict(workspace=KEYS[k]), "INVALID_ARG") for k in ("q", "k_pages", "seq_lens")],
])
def test_key_weights_reject(capi, kw, expect):
    assert capi.ss_attn_key_weights(**{**KEYS, **kw}) == status(capi, expect)


def test_key_weights_without_tokens(capi):
    assert capi.ss_attn_key_weights(**{**KEYS, "T": 0, "q": 0, "workspace": 0}) == capi.SS_OK


def test_key_weights_workspace_grows_with_the_step(capi):
    for Hq, Hkv in ((8, 8), (32, 8), (100, 1)):
        last = 0
        for T in (1, 2, 40, 129, 5000):
            sizes = [capi.ss_attn_key_weights_workspace_size(T, B, Hq, Hkv) for B in (1, 2, 30, 400)]
            assert sizes == sorted(sizes) and sizes[0] > 0 and sizes[-1] >= last
            last = sizes[-1]


# -------------------------------------------------------------------------------- eviction

EVICT = dict(pools=APART[0:4], page_bytes=2 * 128 * 128, weights=APART[4:6], Hkv=2, page_refs=APART[6], num_pages=16, page_table=APART[7],
             num_rows=4, max_pages=8, seq_lens=APART[8], rows=APART[9], keep=APART[10], n=3, recent=8, result=APART[11],
             workspace=APART[12], workspace_bytes=1 << 40, stream=0)


@pytest.mark.parametrize("kw,expect", [
    *[({k: 0}, "INVALID_ARG") for k in ("page_refs", "num_pages", "page_table", "num_rows", "max_pages", "seq_lens", "keep", "Hkv", "page_bytes")],
    (dict(n=-1), "INVALID_ARG"), (dict(recent=-1), "INVALID_ARG"), (dict(rows=0, n=5), "INVALID_ARG"), (dict(pools=APART[0:3]), "INVALID_ARG"),
    (dict(pools=[]), "INVALID_ARG"), (dict(weights=[]), "INVALID_ARG"), (dict(pools=APART[0:1]), "INVALID_ARG"), (dict(page_bytes=2 * 128 * 8), "INVALID_ARG"),
    (dict(Hkv=3), "INVALID_ARG"), (dict(pools=[APART[0], APART[1], 0, APART[3]]), "INVALID_ARG"), (dict(weights=[APART[4], 0]), "INVALID_ARG"),
    (dict(weights=[APART[4], APART[5] + 4]), "INVALID_ARG"), (dict(pools=[APART[0]] * 4), "INVALID_ARG"), (dict(weights=[APART[4]] * 2), "INVALID_ARG"),
    (dict(weights=[APART[4], APART[4] + 4096]), "INVALID_ARG"), (dict(weights=[APART[4], APART[0]]), "INVALID_ARG"),
    (dict(out_weights=[APART[5], APART[13]]), "INVALID_ARG"), (dict(out_weights=[APART[13], APART[13]]), "INVALID_ARG"),
    (dict(out_weights=[APART[13], APART[7]]), "INVALID_ARG"), (dict(out_refs=APART[8]), "INVALID_ARG"), (dict(out_lens=APART[10]), "INVALID_ARG"),
    (dict(out_table=APART[6]), "INVALID_ARG"), (dict(out_table=APART[2]), "INVALID_ARG"), (dict(result=APART[8]), "INVALID_ARG"),
    (dict(rows=APART[8]), "INVALID_ARG"), (dict(keep=APART[8]), "INVALID_ARG"), (dict(keep=APART[10] + 2), "INVALID_ARG"),
    (dict(pools=[x << 1 for x in range(1 << 20, (1 << 20) + 16 * 65 * 8, 16 * 8)], weights=APART[4:5]), "UNSUPPORTED"),
    (dict(n=1 << 28, rows=APART[9]), "UNSUPPORTED"), (dict(workspace=0), "WORKSPACE"), (dict(workspace=APART[12] + 8), "WORKSPACE"),
    (dict(workspace_bytes=1000), "WORKSPACE"), (dict(workspace=APART[0]), "INVALID_ARG"), (dict(workspace=APART[4]), "INVALID_ARG"),
])
def test_evict_rejects(capi, kw, expect):
    assert capi.ss_pages_evict(**{**EVICT, **kw}) == status(capi, expect)


def test_evict_accepts_up_to_the_device(capi):
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    fine = {status(capi, "UNSUPPORTED"), status(capi, "CUDA")}
    for kw in ({}, dict(rows=None), dict(n=0, rows=None, keep=None), dict(out_weights=APART[4:6]), dict(out_weights=[APART[4], APART[13]]),
               dict(out_refs=APART[13], out_table=APART[14], out_lens=APART[15]), dict(pools=APART[0:2]), dict(result=None)):
        assert capi.ss_pages_evict(**{**EVICT, **kw}) in fine, kw


# --------------------------------------------------------------------------------- helpers


def _z(shape, dtype):
    return torch.zeros(shape, dtype=dtype)


def test_plan_helper_refuses():
    t, n = _z((3, 4), I32), _z(3, I32)
    for bad, what in (((t.long(), n), "page_table"), ((t[:, ::2], n), "page_table"), ((t, n[:2]), "seq_lens"), ((t, n.long()), "seq_lens")):
        with pytest.raises(ValueError, match=what):
            ss.prefix_plan(*bad)
    with pytest.raises(ValueError, match="out"):
        ss.prefix_plan(t, n, out=_z(5, I32))
    with pytest.raises(ValueError, match="8192"):
        ss.prefix_plan(_z((9000, 1), I32), _z(9000, I32))
    with pytest.raises(ValueError, match="CUDA"):
        ss.prefix_plan(t, n)


def test_decode_helper_refuses():
    q, kp, t, n = _z((3, 8, 128), BF), _z((6, 2, 128, 128), BF), _z((3, 4), I32), _z(3, I32)
    call = lambda q=q, kp=kp, vp=kp, t=t, n=n, plan=None, **kw: ss.decode_shared(q, kp, vp, t, n, plan, scale=0.1, **kw)  # noqa: E731
    wide = _z((3, 8, 256), BF)
    for kw, what in ((dict(q=q.float()), "q"), (dict(q=wide[..., ::2]), "q"), (dict(q=_z((3, 128, 8), BF).transpose(1, 2)), "q"),
                     (dict(q=q[:1].expand(3, 8, 128)), "overlap"), (dict(q=q[0]), "q"), (dict(kp=kp[:, :, :64]), "k_pages"),
                     (dict(kp=_z((6, 2, 128, 64), BF)), "k_pages"), (dict(vp=kp[:5]), "v_pages"), (dict(vp=kp.half()), "v_pages"),
                     (dict(t=t[:2]), "page_table"), (dict(t=t.long()), "page_table"), (dict(n=n[:2]), "seq_lens"),
                     (dict(plan=_z(7, I32)), "plan"), (dict(weights=_z((3, 2, 512), BF)), "weights"), (dict(weights=_z((3, 2, 511), F32)), "weights"),
                     (dict(weights=_z((3, 512, 2), F32).transpose(1, 2)), "weights"), (dict(out=_z((3, 8, 64), BF)), "out"),
                     (dict(out=wide[..., :128]), "out"), ({}, "CUDA")):
        with pytest.raises(ValueError, match=what):
            call(**kw)


def test_key_weights_helper_refuses():
    q, kp, t, cu, n, w = _z((9, 8, 64), BF), _z((6, 2, 128, 64), BF), _z((3, 4), I32), _z(4, I32), _z(3, I32), _z((3, 2, 512), F32)
    call = lambda q=q, kp=kp, t=t, cu=cu, n=n, w=w, **kw: ss.key_weights(q, kp, t, cu, n, w, scale=0.1, **kw)  # noqa: E731
    for kw, what in ((dict(q=q.half()), "q"), (dict(q=q[:1].expand(9, 8, 64)), "overlap"), (dict(kp=kp[..., :32]), "k_pages"),
                     (dict(t=t[0]), "page_table"), (dict(cu=cu[:3]), "cu_seqlens"), (dict(n=n[:1]), "seq_lens"), (dict(w=w[:2]), "weights"),
                     (dict(w=w.double()), "weights"), (dict(w=_z((3, 1, 512), F32).expand(3, 2, 512)), "weights"), ({}, "CUDA")):
        with pytest.raises(ValueError, match=what):
            call(**kw)


def test_evict_helper_refuses():
    pools, w = [_z((6, 2, 128, 64), BF) for _ in range(4)], [_z((3, 2, 512), F32) for _ in range(2)]
    refs, t, n, keep = _z(6, I32), _z((3, 4), I32), _z(3, I32), _z(3, I32)
    call = lambda pools=pools, w=w, refs=refs, t=t, n=n, keep=keep, **kw: ss.pages_evict(pools, w, refs, t, n, keep, **kw)  # noqa: E731
    for kw, what in ((dict(pools=pools[:3]), "layers"), (dict(w=[]), "layers"), (dict(pools=[]), "layers"), (dict(pools=pools[:3] + [pools[0][:5]]), r"pools\[3\]"),
                     (dict(pools=[_z((6, 4, 128, 32), BF)] * 2), r"pools\[0\]"), (dict(w=[w[0], w[1][:2]]), r"weights\[1\]"), (dict(w=[w[0].half(), w[1]]), r"weights\[0\]"),
                     (dict(out_weights=w[:1]), "out_weights"), (dict(out_weights=[w[0], _z((3, 2, 511), F32)]), r"out_weights\[1\]"),
                     (dict(keep=keep.long()), "keep"), (dict(keep=_z(4, I32)), "keep"), (dict(rows=_z(2, I32)), "rows"), (dict(out_refs=_z(5, I32)), "out_refs"),
                     (dict(out_table=t.long()), "out_table"), (dict(out_lens=_z(4, I32)), "out_lens"), (dict(result=_z(2, I32)), "result"), ({}, "CUDA")):
        with pytest.raises(ValueError, match=what):
            call(**kw)
