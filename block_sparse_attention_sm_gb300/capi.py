"""ctypes binding of libssattn (include/ssattn.h): same names, marshalling only.

Every ``ss_*`` function here forwards to the C entry point of the same name.
Tensor arguments may be torch tensors (their ``data_ptr()`` is passed) or
plain integers (device addresses).  ``stream`` defaults to torch's current
CUDA stream.  Nothing here computes: if the shared library is missing the
import of a function fails loudly -- there is no fallback path.
"""
from __future__ import annotations

import array
import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libssattn.so")

SS_OK, SS_ERR_INVALID_ARG, SS_ERR_UNSUPPORTED, SS_ERR_CUDA, SS_ERR_TIMEOUT, SS_ERR_WORKSPACE = range(6)
SS_PREFILL, SS_DECODE, SS_MLA_DECODE, SS_MLA_PREFILL = 0, 1, 2, 3
SS_ROPE_PLAIN, SS_ROPE_LINEAR, SS_ROPE_BASE, SS_ROPE_YARN, SS_ROPE_WAVELENGTH = range(5)

EXPORTS = (
    "ss_attn_prefill", "ss_attn_prefill_ex", "ss_attn_mla_prefill", "ss_attn_mla_prefill_ex",
    "ss_attn_decode_workspace_size", "ss_attn_decode",
    "ss_attn_decode_ex", "ss_attn_decode_noalloc", "ss_decode_static_scratch_bytes",
    "ss_attn_decode_paged",
    "ss_attn_mla_decode_workspace_size", "ss_attn_mla_decode", "ss_attn_mla_decode_ex",
    "ss_attn_mla_decode_paged",
    "ss_calibrate", "ss_fit_factor", "ss_lambda", "ss_status_string", "ss_stream_status",
    "ss_rope", "ss_rope_append_paged", "ss_rope_append_paged_ex", "ss_rope_frequencies",
    "ss_attn_chunk_paged", "ss_attn_chunk_paged_units", "ss_attn_chunk_paged_workspace_size",
    "ss_attn_chunk_paged_workspace_bound", "ss_pages_workspace_size", "ss_pages_reserve", "ss_pages_free", "ss_pages_fork",
    "ss_pages_copy", "ss_pages_compact",
)


class SSError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {ss_status_string(status)} (status {status})")


class ss_debug_opts(ctypes.Structure):
    _fields_ = [("skip_mask", ctypes.c_void_p), ("vote_margin", ctypes.c_void_p),
                ("count_only", ctypes.c_int), ("fault_inject", ctypes.c_int),
                ("vote_chunk_tiles", ctypes.c_int), ("prefill_kernel", ctypes.c_int)]


class ss_problem(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("B", ctypes.c_int), ("Hq", ctypes.c_int),
                ("Hkv", ctypes.c_int), ("Lq", ctypes.c_int), ("Lk", ctypes.c_int),
                ("d", ctypes.c_int), ("scale", ctypes.c_float), ("causal", ctypes.c_int),
                ("num_kv_splits", ctypes.c_int), ("skip_counts", ctypes.c_void_p),
                ("stream", ctypes.c_void_p), ("fault_inject", ctypes.c_int)]


_lib = None


def load() -> ctypes.CDLL:
    """Load libssattn.so (built by ``block_sparse_attention_sm_gb300.builder``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it first "
                           "(python -m block_sparse_attention_sm_gb300.builder)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, F, U = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    pre = [P, P, P, P, I, I, I, I, I, I, F, I, F, P]
    lib.ss_attn_prefill.argtypes = pre + [P]
    lib.ss_attn_prefill_ex.argtypes = pre + [ctypes.POINTER(ss_debug_opts), P]
    mpre = [P, P, P, P, I, I, I, I, I, I, I, F, I, F, P]
    lib.ss_attn_mla_prefill.argtypes = mpre + [P]
    lib.ss_attn_mla_prefill_ex.argtypes = mpre + [ctypes.POINTER(ss_debug_opts), P]
    dec = [P, P, P, P, I, I, I, I, I, F, F, I, P, P, U]
    lib.ss_attn_decode.argtypes = dec + [P]
    lib.ss_attn_decode_ex.argtypes = dec + [ctypes.POINTER(ss_debug_opts), P]
    lib.ss_attn_decode_noalloc.argtypes = [P, P, P, P, I, I, I, I, I, F, F, I, P, P]
    lib.ss_decode_static_scratch_bytes.argtypes = []
    lib.ss_decode_static_scratch_bytes.restype = U
    lib.ss_attn_decode_paged.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, F, F, I, P, P, U,
                                         ctypes.POINTER(ss_debug_opts), P]
    lib.ss_attn_decode_workspace_size.argtypes = [I, I, I, I]
    lib.ss_attn_decode_workspace_size.restype = U
    mla = [P, P, P, I, I, I, I, I, F, F, I, P, P, U]
    lib.ss_attn_mla_decode.argtypes = mla + [P]
    lib.ss_attn_mla_decode_ex.argtypes = mla + [ctypes.POINTER(ss_debug_opts), P]
    lib.ss_attn_mla_decode_paged.argtypes = [P, P, P, P, P, I, I, I, I, I, I, F, F, I, P, P, U,
                                             ctypes.POINTER(ss_debug_opts), P]
    lib.ss_attn_mla_decode_workspace_size.argtypes = [I, I, I, I]
    lib.ss_attn_mla_decode_workspace_size.restype = U
    lib.ss_calibrate.argtypes = [ctypes.POINTER(ss_problem), F, ctypes.POINTER(F), ctypes.POINTER(F)]
    lib.ss_fit_factor.argtypes = [ctypes.POINTER(F), ctypes.POINTER(F), I, ctypes.POINTER(F),
                                  ctypes.POINTER(F)]
    lib.ss_lambda.argtypes = [F, F, F, I]
    lib.ss_lambda.restype = F
    lib.ss_status_string.argtypes = [I]
    lib.ss_status_string.restype = ctypes.c_char_p
    lib.ss_stream_status.argtypes = [P]
    I64, D = ctypes.c_int64, ctypes.c_double
    lib.ss_rope.argtypes = [P, P, I, I, I, I] + [I64] * 6 + [P, I64, P, I, I, I, I, F, P]
    append = [P] * 4 + [I64] * 8 + [I] * 5 + [P] * 4 + [I, I, I, F, P, P, P, I, I]
    lib.ss_rope_append_paged.argtypes = append + [P]
    lib.ss_rope_append_paged_ex.argtypes = append + [P, P]
    lib.ss_rope_frequencies.argtypes = [P, I, D, I, D, I, D, D, ctypes.POINTER(F)]
    lib.ss_attn_chunk_paged.argtypes = [P, I64, P, P, P, P, P, P, I, I, I, I, I, I, I, F, I, F, I, P, P,
                                        U, ctypes.POINTER(ss_debug_opts), P]
    lib.ss_attn_chunk_paged_units.argtypes = [I, I, I, I]
    lib.ss_attn_chunk_paged_workspace_size.argtypes = [I] * 7
    lib.ss_attn_chunk_paged_workspace_bound.argtypes = [I] * 6
    lib.ss_pages_workspace_size.argtypes = [I, I, I]
    for name in ("ss_attn_chunk_paged_units", "ss_attn_chunk_paged_workspace_size",
                 "ss_attn_chunk_paged_workspace_bound", "ss_pages_workspace_size"):
        getattr(lib, name).restype = U
    state = [P, I, P, I, I, P]
    lib.ss_pages_reserve.argtypes = state + [P, P, I, P, P, U, P]
    lib.ss_pages_free.argtypes = state + [P, I, P]
    lib.ss_pages_fork.argtypes = [P, I, U] + state + [P, P, I, P, P, U, P]
    lib.ss_pages_copy.argtypes = [P, I, U, I, P, P, I, P, P, U, P]
    lib.ss_pages_compact.argtypes = [P, I, U] + state + [P, P, P, P, U, P]
    for name in ("ss_attn_prefill", "ss_attn_prefill_ex", "ss_attn_mla_prefill",
                 "ss_attn_mla_prefill_ex", "ss_attn_decode", "ss_attn_decode_ex",
                 "ss_attn_decode_noalloc", "ss_attn_decode_paged", "ss_attn_mla_decode",
                 "ss_attn_mla_decode_ex", "ss_attn_mla_decode_paged", "ss_calibrate",
                 "ss_fit_factor", "ss_stream_status", "ss_rope", "ss_rope_append_paged",
                 "ss_rope_append_paged_ex", "ss_rope_frequencies", "ss_attn_chunk_paged", "ss_pages_reserve", "ss_pages_free",
                 "ss_pages_fork", "ss_pages_copy", "ss_pages_compact"):
        getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch

        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dbg(skip_mask=None, vote_margin=None, count_only=False, fault_inject=0, vote_chunk_tiles=0,
         prefill_kernel=0):
    return ss_debug_opts(_ptr(skip_mask), _ptr(vote_margin), int(bool(count_only)),
                         int(fault_inject), int(vote_chunk_tiles), int(prefill_kernel))


def ss_status_string(status: int) -> str:
    return load().ss_status_string(int(status)).decode()


def ss_attn_prefill(q, k, v, o, B, Hq, Hkv, Lq, Lk, d, scale, causal, lam, skip_counts=None,
                    stream=None) -> int:
    return load().ss_attn_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, Hq, Hkv, Lq, Lk, d,
                                  float(scale), int(bool(causal)), float(lam), _ptr(skip_counts),
                                  _stream(stream))


def ss_attn_prefill_ex(q, k, v, o, B, Hq, Hkv, Lq, Lk, d, scale, causal, lam, skip_counts=None,
                       skip_mask=None, vote_margin=None, count_only=False, stream=None,
                       vote_chunk_tiles=0, prefill_kernel=0) -> int:
    dbg = _dbg(skip_mask, vote_margin, count_only, vote_chunk_tiles=vote_chunk_tiles,
               prefill_kernel=prefill_kernel)
    return load().ss_attn_prefill_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, Hq, Hkv, Lq, Lk, d,
                                     float(scale), int(bool(causal)), float(lam),
                                     _ptr(skip_counts), ctypes.byref(dbg), _stream(stream))


def ss_attn_mla_prefill(q, k, v, o, B, Hq, Hkv, Lq, Lk, d_qk, d_v, scale, causal, lam,
                        skip_counts=None, stream=None) -> int:
    """Latent-attention prefill: q/k rows d_qk wide, v/o rows d_v wide."""
    return load().ss_attn_mla_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, Hq, Hkv, Lq, Lk,
                                      d_qk, d_v, float(scale), int(bool(causal)), float(lam),
                                      _ptr(skip_counts), _stream(stream))


def ss_attn_mla_prefill_ex(q, k, v, o, B, Hq, Hkv, Lq, Lk, d_qk, d_v, scale, causal, lam,
                           skip_counts=None, skip_mask=None, vote_margin=None, count_only=False,
                           stream=None) -> int:
    dbg = _dbg(skip_mask, vote_margin, count_only)
    return load().ss_attn_mla_prefill_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, Hq, Hkv, Lq, Lk,
                                         d_qk, d_v, float(scale), int(bool(causal)), float(lam),
                                         _ptr(skip_counts), ctypes.byref(dbg), _stream(stream))


def ss_attn_decode_workspace_size(B, Hq, d, num_kv_splits) -> int:
    return int(load().ss_attn_decode_workspace_size(B, Hq, d, num_kv_splits))


def ss_attn_decode(q, k_cache, v_cache, o, B, Hq, Hkv, Lk, d, scale, lam, num_kv_splits,
                   skip_counts=None, workspace=None, workspace_bytes=0, stream=None) -> int:
    return load().ss_attn_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(o), B, Hq, Hkv, Lk,
                                 d, float(scale), float(lam), int(num_kv_splits),
                                 _ptr(skip_counts), _ptr(workspace), int(workspace_bytes),
                                 _stream(stream))


def ss_attn_decode_ex(q, k_cache, v_cache, o, B, Hq, Hkv, Lk, d, scale, lam, num_kv_splits,
                      skip_counts=None, workspace=None, workspace_bytes=0, skip_mask=None,
                      vote_margin=None, count_only=False, stream=None, fault_inject=0) -> int:
    dbg = _dbg(skip_mask, vote_margin, count_only, fault_inject)
    return load().ss_attn_decode_ex(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(o), B, Hq, Hkv,
                                    Lk, d, float(scale), float(lam), int(num_kv_splits),
                                    _ptr(skip_counts), _ptr(workspace), int(workspace_bytes),
                                    ctypes.byref(dbg), _stream(stream))


def ss_attn_decode_noalloc(q, k_cache, v_cache, o, B, Hq, Hkv, Lk, d, scale, lam, num_kv_splits,
                           skip_counts=None, stream=None) -> int:
    """Decode without a workspace (partials in the library's static device array)."""
    return load().ss_attn_decode_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(o), B, Hq,
                                         Hkv, Lk, d, float(scale), float(lam), int(num_kv_splits),
                                         _ptr(skip_counts), _stream(stream))


def ss_attn_decode_paged(q, k_pages, v_pages, page_table, seq_lens, o, B, Hq, Hkv, num_pages,
                         max_pages, d, scale, lambda_a, num_kv_splits, skip_counts=None,
                         workspace=None, workspace_bytes=0, skip_mask=None, vote_margin=None,
                         count_only=False, stream=None) -> int:
    """Decode over a paged, variable-length KV cache (pages of 128 keys)."""
    dbg = _dbg(skip_mask, vote_margin, count_only)
    return load().ss_attn_decode_paged(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(page_table),
                                       _ptr(seq_lens), _ptr(o), B, Hq, Hkv, num_pages, max_pages,
                                       d, float(scale), float(lambda_a), int(num_kv_splits),
                                       _ptr(skip_counts), _ptr(workspace), int(workspace_bytes),
                                       ctypes.byref(dbg), _stream(stream))


SS_DECODE_STATIC_SCRATCH_BYTES = 16 << 20  # the header's value; test_abi checks the library's


def ss_decode_static_scratch_bytes() -> int:
    """Size of ss_attn_decode_noalloc's built-in array in the loaded library."""
    return int(load().ss_decode_static_scratch_bytes())


def ss_attn_mla_decode_workspace_size(B, Hq, d_latent, num_kv_splits) -> int:
    return int(load().ss_attn_mla_decode_workspace_size(B, Hq, d_latent, num_kv_splits))


def ss_attn_mla_decode(q, kv, o, B, Hq, Lk, d_latent, d_rope, scale, lam, num_kv_splits,
                       skip_counts=None, workspace=None, workspace_bytes=0, stream=None) -> int:
    """Latent-attention decode: q [B,Hq,dk], one latent cache kv [B,Lk,dk]."""
    return load().ss_attn_mla_decode(_ptr(q), _ptr(kv), _ptr(o), B, Hq, Lk, d_latent, d_rope,
                                     float(scale), float(lam), int(num_kv_splits),
                                     _ptr(skip_counts), _ptr(workspace), int(workspace_bytes),
                                     _stream(stream))


def ss_attn_mla_decode_ex(q, kv, o, B, Hq, Lk, d_latent, d_rope, scale, lam, num_kv_splits,
                          skip_counts=None, workspace=None, workspace_bytes=0, skip_mask=None,
                          vote_margin=None, count_only=False, stream=None) -> int:
    dbg = _dbg(skip_mask, vote_margin, count_only)
    return load().ss_attn_mla_decode_ex(_ptr(q), _ptr(kv), _ptr(o), B, Hq, Lk, d_latent, d_rope,
                                        float(scale), float(lam), int(num_kv_splits),
                                        _ptr(skip_counts), _ptr(workspace), int(workspace_bytes),
                                        ctypes.byref(dbg), _stream(stream))


def ss_calibrate(problem: ss_problem, target_sparsity: float):
    """Returns (status, a, achieved_sparsity)."""
    a = ctypes.c_float()
    ach = ctypes.c_float()
    st = load().ss_calibrate(ctypes.byref(problem), float(target_sparsity), ctypes.byref(a),
                             ctypes.byref(ach))
    return st, a.value, ach.value


def ss_fit_factor(s, a):
    """Least squares ln a = ln A + B s; returns (status, A, B)."""
    n = len(s)
    S = (ctypes.c_float * n)(*map(float, s))
    Av = (ctypes.c_float * n)(*map(float, a))
    A = ctypes.c_float()
    Bv = ctypes.c_float()
    st = load().ss_fit_factor(S, Av, n, ctypes.byref(A), ctypes.byref(Bv))
    return st, A.value, Bv.value


def ss_lambda(A, B, s, L) -> float:
    return float(load().ss_lambda(float(A), float(B), float(s), int(L)))


def ss_stream_status(stream=None) -> int:
    return load().ss_stream_status(_stream(stream))


def ss_attn_mla_decode_paged(q, kv_pages, page_table, seq_lens, o, B, Hq, num_pages, max_pages,
                             d_latent, d_rope, scale, lambda_a, num_kv_splits, skip_counts=None,
                             workspace=None, workspace_bytes=0, skip_mask=None, vote_margin=None,
                             count_only=False, stream=None) -> int:
    """Latent-attention decode over a paged latent cache (pages of 128 rows)."""
    dbg = _dbg(skip_mask, vote_margin, count_only)
    return load().ss_attn_mla_decode_paged(_ptr(q), _ptr(kv_pages), _ptr(page_table),
                                           _ptr(seq_lens), _ptr(o), B, Hq, num_pages, max_pages,
                                           d_latent, d_rope, float(scale), float(lambda_a),
                                           int(num_kv_splits), _ptr(skip_counts), _ptr(workspace),
                                           int(workspace_bytes), ctypes.byref(dbg),
                                           _stream(stream))


def _addresses(pools):
    """Host array of the pools' device addresses (kept alive by the caller's reference)."""
    return array.array("Q", [_ptr(p) or 0 for p in pools])


def ss_rope(x, out, B, H, L, d, positions, inv_freq, rot_dim, x_strides=None, out_strides=None,
            position_stride=0, rot_offset=0, interleaved=False, inverse=False, attn_factor=1.0,
            stream=None) -> int:
    """Rotary positions of x [B,H,L,d] into out; strides (batch, head, token), None: contiguous."""
    dense = (H * L * d, L * d, d)
    return (_lib or load()).ss_rope(
        _ptr(x), _ptr(out), B, H, L, d, *(x_strides or dense), *(out_strides or dense), _ptr(positions),
        position_stride, _ptr(inv_freq), rot_dim, rot_offset, bool(interleaved), bool(inverse), attn_factor,
        _stream(stream))


def ss_rope_append_paged(q, q_out, k, v, T, B, Hq, Hkv, d, cu_seqlens, seq_lens, inv_freq, rot_dim,
                         k_pages, v_pages, page_table, num_pages, max_pages, positions=None,
                         q_strides=None, q_out_strides=None, k_strides=None, v_strides=None,
                         rot_offset=0, interleaved=False, attn_factor=1.0, stream=None) -> int:
    """Rotary positions of a step's new tokens and the write of their keys and values into pages;
    strides (token, head), None: contiguous."""
    q_dense, k_dense = (Hq * d, d), (Hkv * d, d)
    return (_lib or load()).ss_rope_append_paged(
        _ptr(q), _ptr(q_out), _ptr(k), _ptr(v), *(q_strides or q_dense), *(q_out_strides or q_dense),
        *(k_strides or k_dense), *(v_strides or k_dense), T, B, Hq, Hkv, d, _ptr(cu_seqlens), _ptr(seq_lens),
        _ptr(positions), _ptr(inv_freq), rot_dim, rot_offset, bool(interleaved), attn_factor, _ptr(k_pages),
        _ptr(v_pages), _ptr(page_table), num_pages, max_pages, _stream(stream))


def ss_rope_append_paged_ex(q, q_out, k, v, T, B, Hq, Hkv, d, cu_seqlens, seq_lens, inv_freq, rot_dim,
                            k_pages, v_pages, page_table, num_pages, max_pages, positions=None,
                            q_strides=None, q_out_strides=None, k_strides=None, v_strides=None,
                            rot_offset=0, interleaved=False, attn_factor=1.0, refused=None, stream=None) -> int:
    """ss_rope_append_paged that does nothing where the device int32 ``refused`` is not 0."""
    q_dense, k_dense = (Hq * d, d), (Hkv * d, d)
    return (_lib or load()).ss_rope_append_paged_ex(
        _ptr(q), _ptr(q_out), _ptr(k), _ptr(v), *(q_strides or q_dense), *(q_out_strides or q_dense),
        *(k_strides or k_dense), *(v_strides or k_dense), T, B, Hq, Hkv, d, _ptr(cu_seqlens), _ptr(seq_lens),
        _ptr(positions), _ptr(inv_freq), rot_dim, rot_offset, bool(interleaved), attn_factor, _ptr(k_pages),
        _ptr(v_pages), _ptr(page_table), num_pages, max_pages, _ptr(refused), _stream(stream))


def ss_rope_frequencies(rot_dim, base=10000.0, scaling=SS_ROPE_PLAIN, factor=1.0, original_length=0,
                        lo=0.0, hi=0.0):
    """Returns (status, list of rot_dim / 2 frequencies, attn_factor)."""
    n = max(1, int(rot_dim) // 2)
    out = (ctypes.c_double * n)()
    f = ctypes.c_float()
    st = load().ss_rope_frequencies(out, int(rot_dim), float(base), int(scaling), float(factor),
                                    int(original_length), float(lo), float(hi), ctypes.byref(f))
    return st, list(out), f.value


def ss_attn_chunk_paged_units(T, B, Hq, Hkv) -> int:
    return int((_lib or load()).ss_attn_chunk_paged_units(T, B, Hq, Hkv))


def ss_attn_chunk_paged_workspace_size(T, B, Hq, Hkv, max_pages, d, num_kv_splits) -> int:
    return int((_lib or load()).ss_attn_chunk_paged_workspace_size(T, B, Hq, Hkv, max_pages, d, num_kv_splits))


def ss_attn_chunk_paged_workspace_bound(T, Hq, Hkv, max_pages, d, num_kv_splits) -> int:
    return int((_lib or load()).ss_attn_chunk_paged_workspace_bound(T, Hq, Hkv, max_pages, d, num_kv_splits))


def ss_attn_chunk_paged(q, k_pages, v_pages, page_table, cu_seqlens, seq_lens, o, T, B, Hq, Hkv,
                        num_pages, max_pages, d, scale, causal, lambda_a, num_kv_splits,
                        skip_counts=None, workspace=None, workspace_bytes=0, q_token_stride=0,
                        skip_mask=None, vote_margin=None, stream=None) -> int:
    """Attention of a step's packed new tokens over the paged cache."""
    dbg = None
    if skip_mask is not None or vote_margin is not None:
        dbg = ctypes.byref(_dbg(skip_mask, vote_margin))
    return (_lib or load()).ss_attn_chunk_paged(
        _ptr(q), q_token_stride, _ptr(k_pages), _ptr(v_pages), _ptr(page_table), _ptr(cu_seqlens),
        _ptr(seq_lens), _ptr(o), T, B, Hq, Hkv, num_pages, max_pages, d, scale, bool(causal), lambda_a,
        num_kv_splits, _ptr(skip_counts), _ptr(workspace), workspace_bytes, dbg, _stream(stream))


def ss_pages_workspace_size(num_pages, num_rows, n) -> int:
    return int((_lib or load()).ss_pages_workspace_size(num_pages, num_rows, n))


def ss_pages_reserve(page_refs, num_pages, page_table, num_rows, max_pages, seq_lens, rows, add, n,
                     result=None, workspace=None, workspace_bytes=0, stream=None) -> int:
    return (_lib or load()).ss_pages_reserve(_ptr(page_refs), num_pages, _ptr(page_table), num_rows, max_pages,
                                   _ptr(seq_lens), _ptr(rows), _ptr(add), n, _ptr(result),
                                   _ptr(workspace), workspace_bytes, _stream(stream))


def ss_pages_free(page_refs, num_pages, page_table, num_rows, max_pages, seq_lens, rows, n,
                  stream=None) -> int:
    return (_lib or load()).ss_pages_free(_ptr(page_refs), num_pages, _ptr(page_table), num_rows, max_pages,
                                _ptr(seq_lens), _ptr(rows), n, _stream(stream))


def ss_pages_fork(pools, page_bytes, page_refs, num_pages, page_table, num_rows, max_pages, seq_lens,
                  src_rows, dst_rows, n, result=None, workspace=None, workspace_bytes=0,
                  stream=None) -> int:
    return (_lib or load()).ss_pages_fork((a := _addresses(pools)).buffer_info()[0], len(a), page_bytes, _ptr(page_refs),
                                num_pages, _ptr(page_table), num_rows, max_pages, _ptr(seq_lens),
                                _ptr(src_rows), _ptr(dst_rows), n, _ptr(result), _ptr(workspace),
                                workspace_bytes, _stream(stream))


def ss_pages_copy(pools, page_bytes, num_pages, src, dst, n, result=None, workspace=None,
                  workspace_bytes=0, stream=None) -> int:
    return (_lib or load()).ss_pages_copy((a := _addresses(pools)).buffer_info()[0], len(a), page_bytes, num_pages, _ptr(src),
                                _ptr(dst), n, _ptr(result), _ptr(workspace), workspace_bytes,
                                _stream(stream))


def ss_pages_compact(pools, page_bytes, page_refs, num_pages, page_table, num_rows, max_pages, seq_lens,
                     out_refs=None, out_table=None, live=None, workspace=None, workspace_bytes=0,
                     stream=None) -> int:
    return (_lib or load()).ss_pages_compact((a := _addresses(pools)).buffer_info()[0], len(a), page_bytes, _ptr(page_refs),
                                   num_pages, _ptr(page_table), num_rows, max_pages, _ptr(seq_lens),
                                   _ptr(out_refs), _ptr(out_table), _ptr(live), _ptr(workspace),
                                   workspace_bytes, _stream(stream))
