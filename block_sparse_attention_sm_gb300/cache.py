"""Helpers around the paged key/value cache: rotary positions, the write of new
tokens, attention of a chunk of new tokens, and the pages' bookkeeping.

As the helpers of the package itself: they check the tensors, allocate outputs
and workspaces with torch and forward to the entry points of ``libssattn``.
A call runs on the device of its tensors, on ``stream`` (default: that
device's current stream); what it allocates belongs to that stream.
"""
from __future__ import annotations

import contextlib

import torch

from . import capi
from .capi import SSError

_BF16, _I32, _F64 = torch.bfloat16, torch.int32, torch.float64
_SCALINGS = {None: capi.SS_ROPE_PLAIN, "none": capi.SS_ROPE_PLAIN, "linear": capi.SS_ROPE_LINEAR,
             "base": capi.SS_ROPE_BASE, "yarn": capi.SS_ROPE_YARN,
             "wavelength": capi.SS_ROPE_WAVELENGTH}


def _check(st: int, what: str):
    if st != capi.SS_OK:
        raise SSError(st, what)


def _dense(name, t, dtype, ndim=None, shape=None):
    """A contiguous tensor argument of this type, rank or shape."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: element type must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name}: expected {ndim} dimensions, got shape {tuple(t.shape)}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def _rows(name, t, ndim):
    """A bf16 tensor argument whose rows (innermost axis) are contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype != _BF16:
        raise ValueError(f"{name}: element type must be {_BF16}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name}: expected {ndim} dimensions, got shape {tuple(t.shape)}")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: the last axis must be contiguous")


def _writable(name, t):
    """Its elements lie at places of their own (the axes, by stride, do not overlap)."""
    reach = 1
    for stride, size in sorted((st, n) for st, n in zip(t.stride(), t.shape) if n > 1):
        if stride < reach:
            raise ValueError(f"{name}: its rows overlap (strides {t.stride()})")
        reach = stride * (size - 1) + reach
    return t


class _Launch:
    """Device and stream of a call: ``handle`` for the library; entered, torch
    allocates on that stream and the device is current."""

    __slots__ = ("handle", "_stack")

    def __init__(self, stream, *tensors):
        dev = None
        for name, t in tensors:
            if t is None:
                continue
            if not t.is_cuda:
                raise ValueError(f"{name}: must be a CUDA tensor, got device {t.device}")
            if dev is None:
                dev = t.device
            elif t.device != dev:
                raise ValueError(f"tensors on several devices: {dev}, {name} on {t.device}")
        contexts = []
        if torch.cuda.current_device() != dev.index:
            contexts.append(torch.cuda.device(dev))
        if stream is None:
            self.handle = torch._C._cuda_getCurrentRawStream(dev.index)
        else:
            if isinstance(stream, int):
                stream = torch.cuda.ExternalStream(stream, device=dev) if stream else torch.cuda.default_stream(dev)
            elif stream.device != dev:
                raise ValueError(f"stream of {stream.device}, tensors on {dev}")
            self.handle = stream.cuda_stream
            contexts.append(torch.cuda.stream(stream))
        self._stack = None
        if contexts:
            self._stack = contextlib.ExitStack()
            self._contexts(contexts)

    def _contexts(self, contexts):
        for c in contexts:
            self._stack.enter_context(c)

    def __enter__(self):
        return self.handle

    def __exit__(self, *exc):
        if self._stack is not None:
            self._stack.close()
        return False


def rope_frequencies(rot_dim: int, base: float = 10000.0, *, scaling: str | None = None, factor: float = 1.0,
                     original_length: int = 8192, lo: float = 1.0, hi: float | None = None, device="cuda"):
    """(inv_freq, attn_factor) for :func:`rope` and :func:`rope_append_paged`.

    inv_freq: float64 [rot_dim / 2] on ``device``, radians per position.
    ``scaling`` stretches positions for contexts ``factor`` times
    ``original_length``: None, "linear", "base", "yarn" (pairs above ``hi``
    turns over the original length kept, below ``lo`` divided; hi 32) or
    "wavelength" (the same ends, ramp in turns; hi 4)."""
    if scaling not in _SCALINGS:
        raise ValueError(f"rope_frequencies: unknown scaling {scaling!r}")
    if hi is None:
        hi = 32.0 if scaling == "yarn" else 4.0
    st, w, f = capi.ss_rope_frequencies(rot_dim, base, _SCALINGS[scaling], factor, original_length, lo, hi)
    _check(st, "ss_rope_frequencies")
    return torch.tensor(w, dtype=_F64, device=device), f


def rope(x, positions, inv_freq, *, rot_offset: int = 0, interleaved: bool = False, inverse: bool = False,
         attn_factor: float = 1.0, out=None, stream=None):
    """Rotary positions of the rows of x; returns ``out`` (``x`` itself: in place).

    x: bf16 CUDA, [B,H,L,d] with int32 ``positions`` [L] or [B,L], or [T,H,d]
    (packed tokens, or one decoded token a sequence) with [T]; any strides with
    a contiguous last axis.  inv_freq: float64 [rot_dim / 2]; entries
    [rot_offset, rot_offset + rot_dim) turn, the others are copied.
    ``inverse``: the transposed rotation; the gradient of ``rope`` with respect
    to x is ``rope(grad, ..., inverse=True)`` with the same other arguments."""
    if not isinstance(x, torch.Tensor) or x.dim() not in (3, 4):
        raise ValueError("rope expects x [B,H,L,d] or [T,H,d]")
    packed = x.dim() == 3
    _rows("x", x, x.dim())
    _dense("inv_freq", inv_freq, _F64, ndim=1)
    d, rot = x.shape[-1], 2 * inv_freq.shape[0]
    if packed:
        L, H, _ = x.shape
        B = 1
        _dense("positions", positions, _I32, shape=(L,))
        pos_stride = 0
    else:
        B, H, L, _ = x.shape
        _dense("positions", positions, _I32)
        if positions.shape == (L,):
            pos_stride = 0
        elif positions.shape == (B, L):
            pos_stride = L
        else:
            raise ValueError(f"positions: expected shape {(L,)} or {(B, L)}, got {tuple(positions.shape)}")
    if rot < 2 or rot_offset < 0 or rot_offset + rot > d:
        raise ValueError(f"rope: entries [{rot_offset}, {rot_offset + rot}) of rows of {d}")
    if out is not None:
        _rows("out", out, x.dim())
        if out.shape != x.shape:
            raise ValueError(f"out: expected shape {tuple(x.shape)}, got {tuple(out.shape)}")
        if out is not x:
            _no_overlap("out", out, x)
        _writable("out", out)
    with _Launch(stream, ("x", x), ("positions", positions), ("inv_freq", inv_freq), ("out", out)) as handle:
        o = out if out is not None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
        xs, os_ = x.stride(), o.stride()
        if packed:
            xs, os_ = (0, xs[1], xs[0]), (0, os_[1], os_[0])
        st = capi.ss_rope(x, o, B, H, L, d, positions, inv_freq, rot, xs[:3], os_[:3], pos_stride, rot_offset,
                          interleaved, inverse, attn_factor, handle)
    _check(st, "ss_rope")
    return o


def _no_overlap(name, t, x):
    """t is x's memory exactly, or apart from it."""
    a0, b0 = t.data_ptr(), x.data_ptr()
    if a0 == b0 and t.stride() == x.stride():
        return
    a1, b1 = (p.data_ptr() + 2 * (1 + sum((n - 1) * s for n, s in zip(p.shape, p.stride()))) for p in (t, x))
    if t.numel() and a0 < b1 and b0 < a1 and t.untyped_storage().data_ptr() == x.untyped_storage().data_ptr():
        raise ValueError(f"{name}: overlaps its input (only the same memory, in place, is allowed)")


def _batch(T, page_table, cu_seqlens, seq_lens):
    """Sequences and table width of a packed step."""
    _dense("page_table", page_table, _I32, ndim=2)
    B, max_pages = page_table.shape
    _dense("cu_seqlens", cu_seqlens, _I32, shape=(B + 1,))
    _dense("seq_lens", seq_lens, _I32, shape=(B,))
    return B, max_pages


def rope_append_paged(q, k, v, k_pages, v_pages, page_table, cu_seqlens, seq_lens, inv_freq=None, *,
                      positions=None, rot_offset: int = 0, interleaved: bool = False, attn_factor: float = 1.0,
                      out=None, stream=None):
    """Rotates a step's packed new tokens and writes their keys and values into the cache.

    q [T,Hq,d] (or None), k and v [T,Hkv,d] (v None: one row per token, as the
    latent cache) bf16 CUDA, any strides with a contiguous last axis (so parts
    of one projection); k_pages, v_pages [num_pages,Hkv,128,d] (v None: also
    [num_pages,128,d]).  New token i of sequence b's n_b, rows
    cu_seqlens[b] .. of the step, is key seq_lens[b] - n_b + i (seq_lens
    include the new tokens) and takes that as its position unless
    ``positions`` int32 [T] says otherwise.  inv_freq None: no rotation.
    Returns the rotated q (``out``; ``out=q``: in place), rows behind the last
    sequence left as they were, or None without q."""
    _rows("k", k, 3)
    T, Hkv, d = k.shape
    if q is not None:
        _rows("q", q, 3)
        if q.shape[0] != T or q.shape[2] != d:
            raise ValueError("rope_append_paged expects q [T,Hq,d] and k [T,Hkv,d]")
    B, max_pages = _batch(T, page_table, cu_seqlens, seq_lens)
    latent = v is None and isinstance(k_pages, torch.Tensor) and k_pages.dim() == 3
    if latent and Hkv != 1:
        raise ValueError("k_pages [num_pages,128,d] hold one head")
    _dense("k_pages", k_pages, _BF16, ndim=3 if latent else 4)
    if k_pages.shape[1:] != ((128, d) if latent else (Hkv, 128, d)):
        raise ValueError(f"k_pages: expected [num_pages, {Hkv}, 128, {d}], got {tuple(k_pages.shape)}")
    if (v is None) != (v_pages is None):
        raise ValueError("v and v_pages are given together")
    if v is not None:
        _rows("v", v, 3)
        if v.shape != k.shape:
            raise ValueError(f"v: expected shape {tuple(k.shape)}, got {tuple(v.shape)}")
        _dense("v_pages", v_pages, _BF16, shape=k_pages.shape)
    rot = 0
    if inv_freq is not None:
        _dense("inv_freq", inv_freq, _F64, ndim=1)
        rot = 2 * inv_freq.shape[0]
        if rot_offset < 0 or rot_offset + rot > d:
            raise ValueError(f"rope: entries [{rot_offset}, {rot_offset + rot}) of rows of {d}")
    if positions is not None:
        _dense("positions", positions, _I32, shape=(T,))
    if out is not None:
        if q is None:
            raise ValueError("out without q")
        _rows("out", out, 3)
        if out.shape != q.shape:
            raise ValueError(f"out: expected shape {tuple(q.shape)}, got {tuple(out.shape)}")
        if out is not q:
            _no_overlap("out", out, q)
        _writable("out", out)
    with _Launch(stream, ("k", k), ("q", q), ("v", v), ("k_pages", k_pages), ("v_pages", v_pages),
                 ("page_table", page_table), ("cu_seqlens", cu_seqlens), ("seq_lens", seq_lens),
                 ("inv_freq", inv_freq), ("positions", positions), ("out", out)) as handle:
        o = out
        if q is not None and o is None:
            o = torch.empty(q.shape, dtype=_BF16, device=q.device)
        st = capi.ss_rope_append_paged(
            q, o, k, v, T, B, q.shape[1] if q is not None else 0, Hkv, d, cu_seqlens, seq_lens, inv_freq, rot,
            k_pages, v_pages, page_table, k_pages.shape[0], max_pages, positions,
            q.stride()[:2] if q is not None else None, o.stride()[:2] if o is not None else None,
            k.stride()[:2], v.stride()[:2] if v is not None else None, rot_offset, interleaved, attn_factor,
            handle)
    _check(st, "ss_rope_append_paged")
    return o


def chunk_paged_workspace(T, Hq, d, num_kv_splits, device):
    n = capi.ss_attn_chunk_paged_workspace_size(T, Hq, d, num_kv_splits)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device), n


def chunk_paged(q, k_pages, v_pages, page_table, cu_seqlens, seq_lens, *, scale: float, causal: bool = True,
                lambda_a: float = 0.0, num_kv_splits: int = 1, counts=None, out=None, workspace=None,
                skip_mask=None, vote_margin=None, stream=None):
    """Attention of a step's packed new tokens over the paged cache, with the skip test.

    q [T,Hq,d] bf16 CUDA (heads contiguous within a token; the tokens' stride
    a multiple of 8), k_pages / v_pages [num_pages,Hkv,128,d], page_table int32
    [B,max_pages], cu_seqlens int32 [B+1], seq_lens int32 [B] (keys per
    sequence, the new ones included).  Causal: new token i of sequence b sees
    keys up to L_b - n_b + i; otherwise all L_b (cross attention).  lambda_a:
    the a of lambda_b = min(1, a / L_b), 0 keeps every tile.  ``counts``
    (capi.ss_attn_chunk_paged_units entries) receives the skipped tiles per
    unit, ``skip_mask`` / ``vote_margin`` [units][max_pages] the debug outputs.
    Returns o [T,Hq,d]; rows behind the last sequence are left as they were."""
    _rows("q", q, 3)
    T, Hq, d = q.shape
    if Hq > 1 and q.stride(1) != d:
        raise ValueError("q: the heads of a token must be contiguous")
    B, max_pages = _batch(T, page_table, cu_seqlens, seq_lens)
    _dense("k_pages", k_pages, _BF16, ndim=4)
    num_pages, Hkv, page, dk = k_pages.shape
    if page != 128 or dk != d:
        raise ValueError(f"k_pages: expected [num_pages, Hkv, 128, {d}], got {tuple(k_pages.shape)}")
    _dense("v_pages", v_pages, _BF16, shape=k_pages.shape)
    units = None
    for name, t, dtype in (("counts", counts, _I32), ("skip_mask", skip_mask, torch.uint8),
                           ("vote_margin", vote_margin, torch.float32)):
        if t is not None:
            _dense(name, t, torch.uint32 if name == "counts" and t.dtype == torch.uint32 else dtype)
            units = capi.ss_attn_chunk_paged_units(T, B, Hq, Hkv, num_kv_splits) if units is None else units
            need = units * (1 if name == "counts" else max_pages)
            if t.numel() < need:
                raise ValueError(f"{name}: needs at least {need} elements, has {t.numel()}")
    if out is not None:
        _dense("out", out, _BF16, shape=q.shape)
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace: must be contiguous")
    with _Launch(stream, ("q", q), ("k_pages", k_pages), ("v_pages", v_pages), ("page_table", page_table),
                 ("cu_seqlens", cu_seqlens), ("seq_lens", seq_lens), ("out", out), ("counts", counts),
                 ("workspace", workspace), ("skip_mask", skip_mask), ("vote_margin", vote_margin)) as handle:
        o = out if out is not None else torch.empty(q.shape, dtype=_BF16, device=q.device)
        nbytes = 0
        if workspace is not None:
            nbytes = workspace.numel() * workspace.element_size()
        elif num_kv_splits > 1:
            workspace, nbytes = chunk_paged_workspace(T, Hq, d, num_kv_splits, q.device)
        st = capi.ss_attn_chunk_paged(q, k_pages, v_pages, page_table, cu_seqlens, seq_lens, o, T, B, Hq, Hkv,
                                      num_pages, max_pages, d, scale, causal, lambda_a, num_kv_splits, counts,
                                      workspace, nbytes, q.stride(0) if T > 1 else 0, skip_mask, vote_margin,
                                      handle)
    _check(st, "ss_attn_chunk_paged")
    return o


def _state(page_refs, page_table, seq_lens):
    _dense("page_refs", page_refs, _I32, ndim=1)
    _dense("page_table", page_table, _I32, ndim=2)
    _dense("seq_lens", seq_lens, _I32, shape=page_table.shape[:1])
    return page_refs.shape[0], page_table.shape[0], page_table.shape[1]


def _pools(pools, num_pages):
    """Bytes of a page, the same in every pool [num_pages, ...]."""
    page_bytes = None
    for i, t in enumerate(pools):
        if not isinstance(t, torch.Tensor) or not t.is_contiguous() or t.dim() < 2:
            raise ValueError(f"pools[{i}]: expected a contiguous tensor [num_pages, ...]")
        n = t.element_size() * t[0].numel() if t.shape[0] else 0
        if t.shape[0] != num_pages or (page_bytes is not None and n != page_bytes):
            raise ValueError(f"pools[{i}]: expected {num_pages} pages of {page_bytes or n} bytes")
        page_bytes = n
    return page_bytes if page_bytes is not None else 16


def _list(name, t, n=None):
    _dense(name, t, _I32, ndim=1)
    if n is not None and t.shape[0] != n:
        raise ValueError(f"{name}: expected {n} entries, got {t.shape[0]}")
    return t.shape[0]


def _page_scratch(num_pages, num_rows, n, workspace, result, device):
    if workspace is None:
        nbytes = capi.ss_pages_workspace_size(num_pages, num_rows, n)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    else:
        if not workspace.is_contiguous():
            raise ValueError("workspace: must be contiguous")
        nbytes = workspace.numel() * workspace.element_size()
    if result is None:
        result = torch.empty(1, dtype=_I32, device=device)
    return workspace, nbytes, result


def pages_reserve(page_refs, page_table, seq_lens, add, *, rows=None, result=None, workspace=None, stream=None):
    """Sequences grow by ``add`` (int32 [n]) keys: row rows[i], or row i.

    They receive the lowest free pages of page_refs (int32 [num_pages], holders
    of each page, 0 free), in order; seq_lens is raised.  Returns ``result``,
    an int32 [1] on the device: 0, the number of pages that are missing, or -1
    for wrong arguments (then nothing has changed)."""
    num_pages, num_rows, max_pages = _state(page_refs, page_table, seq_lens)
    n = _list("add", add)
    if rows is not None:
        _list("rows", rows, n)
    elif n > num_rows:
        raise ValueError(f"add: {n} entries for {num_rows} rows")
    if result is not None:
        _dense("result", result, _I32, shape=(1,))
    with _Launch(stream, ("page_refs", page_refs), ("page_table", page_table), ("seq_lens", seq_lens),
                 ("add", add), ("rows", rows), ("result", result), ("workspace", workspace)) as handle:
        ws, nbytes, result = _page_scratch(num_pages, num_rows, n, workspace, result, page_refs.device)
        st = capi.ss_pages_reserve(page_refs, num_pages, page_table, num_rows, max_pages, seq_lens, rows, add, n,
                                   result, ws, nbytes, handle)
    _check(st, "ss_pages_reserve")
    return result


def pages_free(page_refs, page_table, seq_lens, rows, *, stream=None):
    """The sequences of the listed rows (int32 [n]) end; their pages lose a holder."""
    num_pages, num_rows, max_pages = _state(page_refs, page_table, seq_lens)
    n = _list("rows", rows)
    with _Launch(stream, ("page_refs", page_refs), ("page_table", page_table), ("seq_lens", seq_lens),
                 ("rows", rows)) as handle:
        st = capi.ss_pages_free(page_refs, num_pages, page_table, num_rows, max_pages, seq_lens, rows, n, handle)
    _check(st, "ss_pages_free")


def pages_fork(pools, page_refs, page_table, seq_lens, src_rows, dst_rows, *, result=None, workspace=None,
               stream=None):
    """Unused rows dst_rows become copies of the sequences src_rows (int32 [n] each).

    Full pages are shared; a last page that is not full is copied, in each of
    ``pools`` (contiguous [num_pages, ...] tensors of any type: every layer's
    key and value pages).  Returns ``result`` as :func:`pages_reserve`."""
    num_pages, num_rows, max_pages = _state(page_refs, page_table, seq_lens)
    page_bytes = _pools(pools, num_pages)
    n = _list("src_rows", src_rows)
    _list("dst_rows", dst_rows, n)
    if result is not None:
        _dense("result", result, _I32, shape=(1,))
    with _Launch(stream, ("page_refs", page_refs), ("page_table", page_table), ("seq_lens", seq_lens),
                 ("src_rows", src_rows), ("dst_rows", dst_rows), ("result", result), ("workspace", workspace),
                 *(("pools", t) for t in pools)) as handle:
        ws, nbytes, result = _page_scratch(num_pages, num_rows, n, workspace, result, page_refs.device)
        st = capi.ss_pages_fork(pools, page_bytes, page_refs, num_pages, page_table, num_rows, max_pages, seq_lens,
                                src_rows, dst_rows, n, result, ws, nbytes, handle)
    _check(st, "ss_pages_fork")
    return result


def pages_copy(pools, src, dst, *, result=None, workspace=None, stream=None):
    """Copies page src[i] over page dst[i] (int32 [n] each) in each of ``pools``;
    returns ``result``: 0, or -1 where a page is outside the pools, a
    destination listed twice or also a source (then nothing is copied)."""
    if len(pools) == 0:
        raise ValueError("pages_copy: no pools")
    num_pages = pools[0].shape[0]
    page_bytes = _pools(pools, num_pages)
    n = _list("src", src)
    _list("dst", dst, n)
    if result is not None:
        _dense("result", result, _I32, shape=(1,))
    with _Launch(stream, ("src", src), ("dst", dst), ("result", result), ("workspace", workspace),
                 *(("pools", t) for t in pools)) as handle:
        ws, nbytes, result = _page_scratch(num_pages, 0, n, workspace, result, src.device)
        st = capi.ss_pages_copy(pools, page_bytes, num_pages, src, dst, n, result, ws, nbytes, handle)
    _check(st, "ss_pages_copy")
    return result


def pages_compact(pools, page_refs, page_table, seq_lens, *, out_refs=None, out_table=None, live=None,
                  workspace=None, stream=None):
    """Moves the pages in use to the front of every pool.

    The new counts and table go to ``out_refs`` / ``out_table`` (default: in
    place).  Returns ``live``, an int32 [1] on the device: the number of pages
    in use, which are then the pages [0, live)."""
    num_pages, num_rows, max_pages = _state(page_refs, page_table, seq_lens)
    page_bytes = _pools(pools, num_pages)
    if out_refs is not None:
        _dense("out_refs", out_refs, _I32, shape=page_refs.shape)
    if out_table is not None:
        _dense("out_table", out_table, _I32, shape=page_table.shape)
    if live is not None:
        _dense("live", live, _I32, shape=(1,))
    with _Launch(stream, ("page_refs", page_refs), ("page_table", page_table), ("seq_lens", seq_lens),
                 ("out_refs", out_refs), ("out_table", out_table), ("live", live), ("workspace", workspace),
                 *(("pools", t) for t in pools)) as handle:
        ws, nbytes, live = _page_scratch(num_pages, num_rows, 0, workspace, live, page_refs.device)
        st = capi.ss_pages_compact(pools, page_bytes, page_refs, num_pages, page_table, num_rows, max_pages,
                                   seq_lens, out_refs, out_table, live, ws, nbytes, handle)
    _check(st, "ss_pages_compact")
    return live
