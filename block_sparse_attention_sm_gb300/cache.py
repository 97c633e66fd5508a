"""Helpers around the paged key/value cache: rotary positions, the write of new
tokens, attention of a chunk of new tokens, decode over shared pages, the record
of attention weights and eviction by it, and the pages' bookkeeping.

As the helpers of the package itself: they check the tensors, allocate outputs
and workspaces with torch and forward to the entry points of ``libssattn``.
A call runs on the device of its tensors, on ``stream`` (default: that
device's current stream); what it allocates belongs to that stream.
"""
from __future__ import annotations

import array
import contextlib
import functools

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
    if t.dtype is not dtype:
        raise ValueError(f"{name}: element type must be {dtype}, got {t.dtype}")
    if ndim is not None and t.ndim != ndim:
        raise ValueError(f"{name}: expected {ndim} dimensions, got shape {tuple(t.shape)}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def _rows(name, t, ndim):
    """Shape and strides of a bf16 tensor argument whose rows (innermost axis) are contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype is not _BF16:
        raise ValueError(f"{name}: element type must be {_BF16}, got {t.dtype}")
    shape, strides = t.shape, t.stride()
    if len(shape) != ndim:
        raise ValueError(f"{name}: expected {ndim} dimensions, got shape {tuple(shape)}")
    if strides[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name}: the last axis must be contiguous")
    return shape, strides


def _writable(name, t):
    """Its elements lie at places of their own (the axes, by stride, do not overlap)."""
    reach = 1
    for stride, size in sorted((st, n) for st, n in zip(t.stride(), t.shape) if n > 1):
        if stride < reach:
            raise ValueError(f"{name}: its rows overlap (strides {t.stride()})")
        reach = stride * (size - 1) + reach
    return t


def _on(stream, names, *tensors):
    """Device and stream of a call: (stream handle, context to make it in).

    All tensors must be on one CUDA device (``names``: theirs, or a function
    that gives them).  Inside the context that device is current and torch
    allocates on that stream; where both are so already there is nothing to enter."""
    dev = None
    for t in tensors:
        if t is not None:
            d = t.get_device()
            if d != dev:
                if d < 0 or dev is not None:
                    name = (names if isinstance(names, str) else names()).split()[[t is u for u in tensors].index(True)]
                    raise ValueError(f"{name}: must be a CUDA tensor, got device {t.device}" if d < 0 else
                                     f"tensors on several devices: {name} on {t.device}, others on cuda:{dev}")
                dev = d
    if stream is None and torch._C._cuda_getDevice() == dev:  # (a tensor on a GPU: CUDA is initialised)
        return torch._C._cuda_getCurrentRawStream(dev), _HERE
    if isinstance(stream, int):
        device = torch.device("cuda", dev)
        stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
    elif stream is None:
        stream = torch.cuda.current_stream(dev)
    elif stream.device.index != dev:
        raise ValueError(f"stream of {stream.device}, tensors on cuda:{dev}")
    stack = contextlib.ExitStack()
    stack.enter_context(torch.cuda.device(dev))
    stack.enter_context(torch.cuda.stream(stream))
    return stream.cuda_stream, stack


_HERE = contextlib.nullcontext()


def _written(out):
    """A graph that has saved ``out`` learns that a kernel has changed it (as of torch's own in-place functions)."""
    torch.autograd.graph.increment_version(out)


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
    to x is ``rope(grad, ..., inverse=True)`` with the same other arguments.
    Where gradients are recorded and x requires one, the result is part of the
    graph and its backward pass is that call; ``out`` and frequencies that
    require a gradient are refused there."""
    if not isinstance(x, torch.Tensor) or x.ndim not in (3, 4):
        raise ValueError("rope expects x [B,H,L,d] or [T,H,d]")
    packed = x.ndim == 3
    shape, xs = _rows("x", x, x.ndim)
    _dense("inv_freq", inv_freq, _F64, 1)
    if packed:
        L, H, d = shape
        B, pos_stride = 1, 0
        _dense("positions", positions, _I32, None, (L,))
    else:
        B, H, L, d = shape
        _dense("positions", positions, _I32)
        if positions.shape == (L,):
            pos_stride = 0
        elif positions.shape == (B, L):
            pos_stride = L
        else:
            raise ValueError(f"positions: expected shape {(L,)} or {(B, L)}, got {tuple(positions.shape)}")
    rot = 2 * inv_freq.shape[0]
    if rot < 2 or rot_offset < 0 or rot_offset + rot > d:
        raise ValueError(f"rope: entries [{rot_offset}, {rot_offset + rot}) of rows of {d}")
    given = out is not None
    if (x.requires_grad or inv_freq.requires_grad or given and out.requires_grad) and torch.is_grad_enabled():
        return _recorded(x, positions, inv_freq, rot_offset, interleaved, inverse, attn_factor, out, stream)
    if given:
        _output("out", out, x, shape)
    handle, context = _on(stream, "x positions inv_freq out", x, positions, inv_freq, out)
    with context:
        if out is None:
            out = torch.empty(shape, dtype=_BF16, device=x.device)
        if packed:
            xt, xh, _ = xs
            ot, oh, _ = out.stride()
            xb = ob = 0
        else:
            xb, xh, xt, _ = xs
            ob, oh, ot, _ = out.stride()
        st = (capi._lib or capi.load()).ss_rope(
            x.data_ptr(), out.data_ptr(), B, H, L, d, xb, xh, xt, ob, oh, ot, positions.data_ptr(), pos_stride,
            inv_freq.data_ptr(), rot, rot_offset, bool(interleaved), bool(inverse), attn_factor, handle)
    if st:
        raise SSError(st, "ss_rope")
    if given:
        _written(out)
    return out


class _Rope(torch.autograd.Function):
    """rope as a node of the graph: linear in x, its transpose is the inverse rotation."""

    @staticmethod
    def forward(ctx, x, positions, inv_freq, options):
        ctx.save_for_backward(positions, inv_freq)
        ctx.options = options
        return rope(x, positions, inv_freq, **options)

    @staticmethod
    def backward(ctx, grad):
        options = dict(ctx.options, inverse=not ctx.options["inverse"])
        if grad.stride(-1) != 1:  # (a broadcast gradient, as that of a sum)
            grad = grad.contiguous()
        return _Rope.apply(grad, *ctx.saved_tensors, options), None, None, None


def _recorded(x, positions, inv_freq, rot_offset, interleaved, inverse, attn_factor, out, stream):
    """rope while gradients are recorded for x; the node belongs to the call's stream."""
    if out is not None:
        raise ValueError("out: not where a gradient of the rotation is recorded")
    if inv_freq.requires_grad:
        raise ValueError("inv_freq: the rotation has no gradient with respect to its frequencies")
    options = dict(rot_offset=rot_offset, interleaved=interleaved, inverse=inverse, attn_factor=attn_factor)
    with _HERE if stream is None else _on(stream, "x", x)[1]:
        return _Rope.apply(x, positions, inv_freq, options)


def _output(name, out, x, shape):
    """``out`` for the rows of x: x itself, or memory of its own."""
    if _rows(name, out, len(shape))[0] != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(out.shape)}")
    if out is not x:
        _no_overlap(name, out, x)
    _writable(name, out)


def _no_overlap(name, t, x):
    """t is x's memory exactly, or apart from it (rows of t may lie between rows of x)."""
    if t.data_ptr() == x.data_ptr() and all(a == b for a, b, n in zip(t.stride(), x.stride(), t.shape) if n > 1):
        return
    if _meet(t, x):
        raise ValueError(f"{name}: overlaps its input (only the same memory, in place, is allowed)")


def _meet(a, b):
    """Whether two bf16 tensors share elements.  Axis by axis from the largest stride: only those index
    differences k matter at which what is left of both comes together.  Exact where the strides are the same
    (parts of one tensor); where more than a few k remain it answers True."""
    def walk(gap, x, y):  # gap: from b's first element to a's
        ex, ey = (1 + sum(s * (n - 1) for s, n in z) for z in (x, y))
        if gap >= ey or gap + ex <= 0:
            return False
        if not x and not y:
            return True
        s, nx, ny = max(z[0][0] for z in (x, y) if z), 1, 1
        if x and x[0][0] == s:
            (_, nx), x, ex = x[0], x[1:], ex - s * (x[0][1] - 1)
        if y and y[0][0] == s:
            (_, ny), y, ey = y[0], y[1:], ey - s * (y[0][1] - 1)
        lo, hi = max(1 - ny, (-ex - gap) // s + 1), min(nx - 1, (ey - gap - 1) // s)
        return hi - lo >= 4 or any(walk(gap + k * s, x, y) for k in range(lo, hi + 1))

    axes = [sorted(((s, n) for s, n in zip(t.stride(), t.shape) if n > 1 and s), reverse=True) for t in (a, b)]
    return a.numel() > 0 and b.numel() > 0 and walk((a.data_ptr() - b.data_ptr()) // 2, *axes)


def _batch(page_table, cu_seqlens, seq_lens):
    """Sequences and table width of a packed step."""
    _dense("page_table", page_table, _I32, 2)
    B, max_pages = page_table.shape
    _dense("cu_seqlens", cu_seqlens, _I32, None, (B + 1,))
    _dense("seq_lens", seq_lens, _I32, None, (B,))
    return B, max_pages


def rope_append_paged(q, k, v, k_pages, v_pages, page_table, cu_seqlens, seq_lens, inv_freq=None, *,
                      positions=None, rot_offset: int = 0, interleaved: bool = False, attn_factor: float = 1.0,
                      out=None, refused=None, stream=None):
    """Rotates a step's packed new tokens and writes their keys and values into the cache.

    q [T,Hq,d] (or None), k and v [T,Hkv,d] (v None: one row per token, as the
    latent cache) bf16 CUDA, any strides with a contiguous last axis (so parts
    of one projection); k_pages, v_pages [num_pages,Hkv,128,d] (v None: also
    [num_pages,128,d]).  New token i of sequence b's n_b, rows
    cu_seqlens[b] .. of the step, is key seq_lens[b] - n_b + i (seq_lens
    include the new tokens) and takes that as its position unless
    ``positions`` int32 [T] says otherwise.  inv_freq None: no rotation.
    ``refused`` (int32 [1] on the device): what :func:`pages_reserve` returned
    for this step; where it is not 0 the call does nothing (the lengths then do
    not include the new tokens, which would overwrite the newest cached ones).
    Returns the rotated q (``out``; ``out=q``: in place), rows behind the last
    sequence left as they were, or None without q.  A serving call: it records
    no gradients (:func:`rope` does)."""
    (T, Hkv, d), ks = _rows("k", k, 3)
    Hq, qs, os_, vs = 0, (0, 0), (0, 0), (0, 0)
    if q is not None:
        q_shape, qs = _rows("q", q, 3)
        Hq = q_shape[1]
        if q_shape[0] != T or q_shape[2] != d:
            raise ValueError("rope_append_paged expects q [T,Hq,d] and k [T,Hkv,d]")
    B, max_pages = _batch(page_table, cu_seqlens, seq_lens)
    latent = v is None and isinstance(k_pages, torch.Tensor) and k_pages.ndim == 3
    if latent and Hkv != 1:
        raise ValueError("k_pages [num_pages,128,d] hold one head")
    _dense("k_pages", k_pages, _BF16, 3 if latent else 4)
    pool = k_pages.shape
    if pool[1:] != ((128, d) if latent else (Hkv, 128, d)):
        raise ValueError(f"k_pages: expected [num_pages, {Hkv}, 128, {d}], got {tuple(pool)}")
    if (v is None) != (v_pages is None):
        raise ValueError("v and v_pages are given together")
    if v is not None:
        v_shape, vs = _rows("v", v, 3)
        if v_shape != (T, Hkv, d):
            raise ValueError(f"v: expected shape {(T, Hkv, d)}, got {tuple(v_shape)}")
        _dense("v_pages", v_pages, _BF16, None, pool)
    rot = 0
    if inv_freq is not None:
        _dense("inv_freq", inv_freq, _F64, 1)
        rot = 2 * inv_freq.shape[0]
        if rot_offset < 0 or rot_offset + rot > d:
            raise ValueError(f"rope: entries [{rot_offset}, {rot_offset + rot}) of rows of {d}")
    if positions is not None:
        _dense("positions", positions, _I32, None, (T,))
    if out is not None:
        if q is None:
            raise ValueError("out without q")
        _output("out", out, q, q_shape)
    if refused is not None:
        _dense("refused", refused, _I32, None, (1,))
    handle, context = _on(stream, "k q v k_pages v_pages page_table cu_seqlens seq_lens inv_freq positions out refused", k, q, v,
                          k_pages, v_pages, page_table, cu_seqlens, seq_lens, inv_freq, positions, out, refused)
    with context:
        o = out
        if q is not None:
            if o is None:
                o = torch.empty(q_shape, dtype=_BF16, device=q.device)
            os_ = o.stride()
        st = (capi._lib or capi.load()).ss_rope_append_paged_ex(
            q.data_ptr() if q is not None else None, o.data_ptr() if q is not None else None, k.data_ptr(),
            v.data_ptr() if v is not None else None, qs[0], qs[1], os_[0], os_[1], ks[0], ks[1], vs[0], vs[1], T, B, Hq,
            Hkv, d, cu_seqlens.data_ptr(), seq_lens.data_ptr(), positions.data_ptr() if positions is not None else None,
            inv_freq.data_ptr() if rot else None, rot, rot_offset, bool(interleaved), attn_factor, k_pages.data_ptr(),
            v_pages.data_ptr() if v is not None else None, page_table.data_ptr(), pool[0], max_pages,
            refused.data_ptr() if refused is not None else None, handle)
    if st:
        raise SSError(st, "ss_rope_append_paged")
    if out is not None:
        _written(out)
    return o


def chunk_paged_workspace(T, B, Hq, Hkv, max_pages, d, num_kv_splits, device):
    """(workspace, its bytes) that serves every :func:`chunk_paged` call of up to these sizes.

    (A call alone may need less, and a smaller step more than a larger one.)"""
    n = capi.ss_attn_chunk_paged_workspace_bound(T, Hq, Hkv, max_pages, d, num_kv_splits)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device), n


def chunk_paged(q, k_pages, v_pages, page_table, cu_seqlens, seq_lens, *, scale: float, causal: bool = True,
                lambda_a: float = 0.0, num_kv_splits: int = 1, counts=None, out=None, workspace=None,
                skip_mask=None, vote_margin=None, stream=None):
    """Attention of a step's packed new tokens over the paged cache, with the skip test.

    q [T,Hq,d] bf16 CUDA (heads contiguous within a token; the tokens' stride
    a multiple of 8, at least Hq * d: not broadcast), k_pages / v_pages [num_pages,Hkv,128,d], page_table int32
    [B,max_pages], cu_seqlens int32 [B+1], seq_lens int32 [B] (keys per
    sequence, the new ones included).  Causal: new token i of sequence b sees
    keys up to L_b - n_b + i; otherwise all L_b (cross attention).  lambda_a:
    the a of lambda_b = min(1, a / L_b), 0 keeps every tile.  ``counts``
    (capi.ss_attn_chunk_paged_units entries) receives the skipped tiles per
    unit, ``skip_mask`` / ``vote_margin`` [units][max_pages] the debug outputs.
    Returns o [T,Hq,d]; rows behind the last sequence are left as they were."""
    shape, qs = _rows("q", q, 3)
    T, Hq, d = shape
    if Hq > 1 and qs[1] != d:
        raise ValueError("q: the heads of a token must be contiguous")
    if T > 1 and qs[0] < Hq * d:  # (a stride of 0, of a broadcast row, would mean contiguous rows to the entry point)
        raise ValueError(f"q: its tokens overlap (stride {qs[0]}, rows of {Hq * d})")
    B, max_pages = _batch(page_table, cu_seqlens, seq_lens)
    _dense("k_pages", k_pages, _BF16, 4)
    pool = k_pages.shape
    num_pages, Hkv, page, dk = pool
    if page != 128 or dk != d:
        raise ValueError(f"k_pages: expected [num_pages, Hkv, 128, {d}], got {tuple(pool)}")
    _dense("v_pages", v_pages, _BF16, None, pool)
    if counts is not None or skip_mask is not None or vote_margin is not None:
        units = capi.ss_attn_chunk_paged_units(T, B, Hq, Hkv)
        for name, t, dtype, need in (("counts", counts, _I32, units), ("skip_mask", skip_mask, torch.uint8, units * max_pages),
                                     ("vote_margin", vote_margin, torch.float32, units * max_pages)):
            if t is not None:
                _dense(name, t, torch.uint32 if dtype is _I32 and t.dtype is torch.uint32 else dtype)
                if t.numel() < need:
                    raise ValueError(f"{name}: needs at least {need} elements, has {t.numel()}")
    if out is not None:
        _dense("out", out, _BF16, None, shape)
        start = out.data_ptr()
        for name, t, reach in (("q", q, (T - 1) * qs[0] + Hq * d), ("k_pages", k_pages, k_pages.numel()),
                               ("v_pages", v_pages, v_pages.numel())):
            at = t.data_ptr()
            if T > 0 and start < at + 2 * reach and at < start + 2 * out.numel() and _meet(out, t):
                raise ValueError(f"out: overlaps {name} (which other clusters read while this one writes)")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace: must be contiguous")
    handle, context = _on(stream, "q k_pages v_pages page_table cu_seqlens seq_lens out counts workspace skip_mask vote_margin",
                          q, k_pages, v_pages, page_table, cu_seqlens, seq_lens, out, counts, workspace, skip_mask,
                          vote_margin)
    with context:
        o = out if out is not None else torch.empty(shape, dtype=_BF16, device=q.device)
        nbytes = 0
        if workspace is not None:
            nbytes = workspace.numel() * workspace.element_size()
        elif num_kv_splits > 1:
            nbytes = capi.ss_attn_chunk_paged_workspace_size(T, B, Hq, Hkv, max_pages, d, num_kv_splits)
            workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
        st = capi.ss_attn_chunk_paged(q, k_pages, v_pages, page_table, cu_seqlens, seq_lens, o, T, B, Hq, Hkv,
                                      num_pages, max_pages, d, scale, causal, lambda_a, num_kv_splits, counts,
                                      workspace, nbytes, qs[0] if T > 1 else 0, skip_mask, vote_margin, handle)
    _check(st, "ss_attn_chunk_paged")
    if out is not None:
        _written(out)
    return o


def prefix_plan(page_table, seq_lens, *, out=None, stream=None):
    """What the sequences of a batch share, for :func:`decode_shared`: an int32 tensor on the device.

    page_table int32 [B,max_pages], seq_lens int32 [B] (B up to 8192).
    Sequences share the pages that their tables name alike from the first on
    and that are full in both (as after :func:`pages_fork`), in any grouping
    and on several levels.  The plan holds as long as these pages stay where
    they are: over steps that append keys, but not across a fork, free,
    eviction or compaction, nor where a sequence becomes shorter than the pages
    it shares (a rollback behind them is fine); then it is made anew.  Its
    time grows with the square of the sequences that begin alike (64: 11 us,
    1024: 0.7 ms, 8192: 42 ms), so keep the plan of a large batch."""
    _dense("page_table", page_table, _I32, 2)
    B, max_pages = page_table.shape
    _dense("seq_lens", seq_lens, _I32, None, (B,))
    lib = capi._lib or capi.load()
    words = _need("ss_prefix_plan_size", B) // 4
    if words == 0:
        raise ValueError(f"prefix_plan: {B} sequences (1 to 8192)")
    if out is not None:
        _dense("out", out, _I32, None, (words,))
    handle, context = _on(stream, "page_table seq_lens out", page_table, seq_lens, out)
    with context:
        if out is None:
            out = torch.empty(words, dtype=_I32, device=page_table.device)
        st = lib.ss_prefix_plan(page_table.data_ptr(), seq_lens.data_ptr(), B, max_pages, out.data_ptr(), 4 * words, handle)
    if st:
        raise SSError(st, "ss_prefix_plan")
    return out


def _recorded_weights(name, t, B, Hkv, max_pages):
    _dense(name, t, torch.float32, None, (B, Hkv, max_pages * 128))


@functools.lru_cache(maxsize=4096)
def _need(call, *sizes):
    """Bytes that a call's workspace takes: a function of its sizes alone, and a call of its own to ask for."""
    return getattr(capi._lib or capi.load(), call)(*sizes)


def _scratch(workspace, device, call, *sizes):
    """(workspace, its bytes), made where it is not given."""
    if workspace is None:
        need = _need(call, *sizes)
        return torch.empty(max(need, 16), dtype=torch.uint8, device=device), need
    if not workspace.is_contiguous():
        raise ValueError("workspace: must be contiguous")
    return workspace, workspace.numel() * workspace.element_size()


def _tokens(q):
    """Shape and token stride of queries [T,Hq,d] whose heads are contiguous within a token."""
    shape, qs = _rows("q", q, 3)
    T, Hq, d = shape
    if Hq > 1 and qs[1] != d:
        raise ValueError("q: the heads of a token must be contiguous")
    if T > 1 and qs[0] < Hq * d:  # (a stride of 0, of a broadcast row, would mean contiguous rows to the entry point)
        raise ValueError(f"q: its tokens overlap (stride {qs[0]}, rows of {Hq * d})")
    return shape, qs[0] if T > 1 else 0


def _pages_of(k_pages, d):
    _dense("k_pages", k_pages, _BF16, 4)
    num_pages, Hkv, page, dk = k_pages.shape
    if page != 128 or dk != d:
        raise ValueError(f"k_pages: expected [num_pages, Hkv, 128, {d}], got {tuple(k_pages.shape)}")
    return num_pages, Hkv


def decode_shared_workspace(B, Hq, Hkv, max_pages, d, device, *, plan=True, weights=False):
    """A workspace that serves every :func:`decode_shared` call of up to B sequences and max_pages pages each.

    With ``weights`` it holds the scores: 512 * B * Hq * max_pages bytes, however long the sequences are."""
    n = capi.ss_attn_decode_shared_workspace_size(B, Hq, Hkv, max_pages, d, plan, weights)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def decode_shared(q, k_pages, v_pages, page_table, seq_lens, plan=None, *, scale: float, weights=None, out=None,
                  workspace=None, stream=None):
    """Attention of one new token a sequence over the paged cache, pages that sequences share read once for all.

    q [B,Hq,d] bf16 CUDA (heads contiguous within a token), k_pages / v_pages
    [num_pages,Hkv,128,d], page_table int32 [B,max_pages], seq_lens int32 [B]
    (the new key included).  ``plan``: what :func:`prefix_plan` found; None:
    nothing is shared.  Every key counts (no skip test).  ``weights`` float32
    [B,Hkv,max_pages*128]: each key's softmax weight, summed over the query
    heads of its KV head, is added to it (:func:`pages_evict` chooses by it);
    cells behind a sequence's end are left as they are (the call's workspace then
    takes 512 * B * Hq * max_pages bytes: make one for all layers with
    :func:`decode_shared_workspace`).  A sequence without keys
    gives zeros.  Returns o [B,Hq,d].  A serving call: it records no gradients."""
    (B, Hq, d), stride = _tokens(q)
    _dense("page_table", page_table, _I32, 2)
    max_pages = page_table.shape[1]
    if page_table.shape[0] != B:
        raise ValueError(f"page_table: expected {B} rows, got {page_table.shape[0]}")
    _dense("seq_lens", seq_lens, _I32, None, (B,))
    num_pages, Hkv = _pages_of(k_pages, d)
    _dense("v_pages", v_pages, _BF16, None, k_pages.shape)
    lib = capi._lib or capi.load()
    if plan is not None:
        _dense("plan", plan, _I32, None, (_need("ss_prefix_plan_size", B) // 4,))
    if weights is not None:
        _recorded_weights("weights", weights, B, Hkv, max_pages)
    if out is not None:
        _dense("out", out, _BF16, None, q.shape)
    handle, context = _on(stream, "q k_pages v_pages page_table seq_lens plan weights out workspace", q, k_pages, v_pages,
                          page_table, seq_lens, plan, weights, out, workspace)
    with context:
        o = out if out is not None else torch.empty((B, Hq, d), dtype=_BF16, device=q.device)
        if B == 0:
            return o
        ws, nbytes = _scratch(workspace, q.device, "ss_attn_decode_shared_workspace_size", B, Hq, Hkv, max_pages, d,
                              plan is not None, weights is not None)
        st = lib.ss_attn_decode_shared(
            q.data_ptr(), stride, k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(),
            plan.data_ptr() if plan is not None else None, o.data_ptr(), weights.data_ptr() if weights is not None else None,
            B, Hq, Hkv, num_pages, max_pages, d, scale, ws.data_ptr(), nbytes, handle)
    if st:
        raise SSError(st, "ss_attn_decode_shared")
    if out is not None:
        _written(out)
    if weights is not None:
        _written(weights)
    return o


def key_weights(q, k_pages, page_table, cu_seqlens, seq_lens, weights, *, scale: float, causal: bool = True,
                workspace=None, stream=None):
    """Adds to ``weights`` the attention weight that each cached key receives from a step's packed new tokens.

    q [T,Hq,d] bf16 CUDA (heads contiguous within a token; a prompt's tokens, or
    only its last ones), k_pages [num_pages,Hkv,128,d], page_table int32
    [B,max_pages], cu_seqlens int32 [B+1], seq_lens int32 [B] (keys, the new
    tokens' included), weights float32 [B,Hkv,max_pages*128]: cell k of
    sequence b and KV head h gains the softmax weights of key k, summed over
    the sequence's new tokens and the query heads of h.  Causal: new token i of
    n sees keys up to L - n + i, otherwise all.  The attention's output is not
    computed.  Returns ``weights``."""
    (T, Hq, d), stride = _tokens(q)
    B, max_pages = _batch(page_table, cu_seqlens, seq_lens)
    num_pages, Hkv = _pages_of(k_pages, d)
    _recorded_weights("weights", weights, B, Hkv, max_pages)
    handle, context = _on(stream, "q k_pages page_table cu_seqlens seq_lens weights workspace", q, k_pages, page_table,
                          cu_seqlens, seq_lens, weights, workspace)
    with context:
        lib = capi._lib or capi.load()
        ws, nbytes = _scratch(workspace, q.device, "ss_attn_key_weights_workspace_size", T, B, Hq, Hkv)
        st = lib.ss_attn_key_weights(
            q.data_ptr(), stride, k_pages.data_ptr(), page_table.data_ptr(), cu_seqlens.data_ptr(), seq_lens.data_ptr(),
            weights.data_ptr(), T, B, Hq, Hkv, num_pages, max_pages, d, scale, bool(causal), ws.data_ptr(), nbytes, handle)
    if st:
        raise SSError(st, "ss_attn_key_weights")
    _written(weights)
    return weights


def _state(page_refs, page_table, seq_lens):
    _dense("page_refs", page_refs, _I32, 1)
    _dense("page_table", page_table, _I32, 2)
    rows, max_pages = page_table.shape
    _dense("seq_lens", seq_lens, _I32, None, (rows,))
    return page_refs.shape[0], rows, max_pages


def _pools(pools, num_pages):
    """Bytes of a page, the same in every pool [num_pages, ...]."""
    shape = dtype = None
    whole = 16 * num_pages
    for i, t in enumerate(pools):
        if not isinstance(t, torch.Tensor) or not t.is_contiguous():
            raise ValueError(f"pools[{i}]: expected a contiguous tensor [num_pages, ...]")
        if t.shape != shape or t.dtype is not dtype:
            n = t.numel() * t.element_size()
            if t.ndim < 2 or t.shape[0] != num_pages or (shape is not None and n != whole):
                raise ValueError(f"pools[{i}]: expected {num_pages} pages of "
                                 f"{(n if shape is None else whole) // max(1, num_pages)} bytes")
            shape, dtype, whole = t.shape, t.dtype, n
    return whole // max(1, num_pages)


def _list(name, t, n=None):
    _dense(name, t, _I32, 1)
    size = t.shape[0]
    if n is not None and size != n:
        raise ValueError(f"{name}: expected {n} entries, got {size}")
    return size


def _page_scratch(num_pages, num_rows, n, workspace, result, device):
    """(workspace, its bytes, result), made where they are not given."""
    if workspace is not None:
        if not workspace.is_contiguous():
            raise ValueError("workspace: must be contiguous")
        nbytes = workspace.numel() * workspace.element_size()
        return workspace, nbytes, torch.empty(1, dtype=_I32, device=device) if result is None else result
    nbytes = (capi._lib or capi.load()).ss_pages_workspace_size(num_pages, num_rows, n)
    return (torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes,
            torch.empty(1, dtype=_I32, device=device) if result is None else result)


def pages_reserve(page_refs, page_table, seq_lens, add, *, rows=None, result=None, workspace=None, stream=None):
    """Sequences grow by ``add`` (int32 [n]) keys: row rows[i], or row i.

    They receive the lowest free pages of page_refs (int32 [num_pages], holders
    of each page, 0 free), in order; seq_lens is raised.  Returns ``result``,
    an int32 [1] on the device: 0, the number of pages that are missing, or -1
    for wrong arguments (then nothing has changed, the lengths neither: give it
    to :func:`rope_append_paged` as ``refused``)."""
    num_pages, num_rows, max_pages = _state(page_refs, page_table, seq_lens)
    n = _list("add", add)
    if rows is not None:
        _list("rows", rows, n)
    elif n > num_rows:
        raise ValueError(f"add: {n} entries for {num_rows} rows")
    if result is not None:
        _dense("result", result, _I32, shape=(1,))
    handle, context = _on(stream, "page_refs page_table seq_lens add rows result workspace", page_refs, page_table, seq_lens,
                          add, rows, result, workspace)
    with context:
        ws, nbytes, result = _page_scratch(num_pages, num_rows, n, workspace, result, page_refs.device)
        st = capi.ss_pages_reserve(page_refs, num_pages, page_table, num_rows, max_pages, seq_lens, rows, add, n,
                                   result, ws, nbytes, handle)
    _check(st, "ss_pages_reserve")
    return result


def pages_free(page_refs, page_table, seq_lens, rows, *, stream=None):
    """The sequences of the listed rows (int32 [n]) end; their pages lose a holder."""
    num_pages, num_rows, max_pages = _state(page_refs, page_table, seq_lens)
    n = _list("rows", rows)
    handle, context = _on(stream, "page_refs page_table seq_lens rows", page_refs, page_table, seq_lens, rows)
    with context:
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
    handle, context = _on(stream, "page_refs page_table seq_lens src_rows dst_rows result workspace" + " pool" * len(pools),
                          page_refs, page_table, seq_lens, src_rows, dst_rows, result, workspace, *pools)
    with context:
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
    handle, context = _on(stream, "src dst result workspace" + " pool" * len(pools), src, dst, result, workspace, *pools)
    with context:
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
    handle, context = _on(stream, "page_refs page_table seq_lens out_refs out_table live workspace" + " pool" * len(pools),
                          page_refs, page_table, seq_lens, out_refs, out_table, live, workspace, *pools)
    with context:
        ws, nbytes, live = _page_scratch(num_pages, num_rows, 0, workspace, live, page_refs.device)
        st = capi.ss_pages_compact(pools, page_bytes, page_refs, num_pages, page_table, num_rows, max_pages,
                                   seq_lens, out_refs, out_table, live, ws, nbytes, handle)
    _check(st, "ss_pages_compact")
    return live


def pages_evict(pools, weights, page_refs, page_table, seq_lens, keep, *, rows=None, recent: int = 0, out_weights=None,
                out_refs=None, out_table=None, out_lens=None, result=None, workspace=None, stream=None):
    """Cuts sequences back to ``keep`` (int32 [n]) keys: row rows[i], or row i.

    ``pools``: each layer's in turn (its key and value pages; equally many a
    layer), contiguous [num_pages,Hkv,128,...]; ``weights``: a float32
    [num_rows,Hkv,max_pages*128] tensor a layer, as :func:`decode_shared` and
    :func:`key_weights` add them up.  Every KV head of every layer keeps the
    ``recent`` newest keys and, of the older ones, those of largest weight (of
    equal ones the first; NaN is below every number), in their order, at the
    front of the sequence's pages.  Weights move along, the cells behind the kept
    keys become 0.  Pages that become free lose a holder; a kept page that other
    sequences hold too is replaced by a free one.  Sequences of ``keep`` keys or
    fewer stay as they are.  Keys hold the positions that they were rotated at:
    later tokens need ``positions`` of their own.  ``out_refs``, ``out_table``,
    ``out_lens`` and ``out_weights`` (a list; listed rows only) receive the new
    state (default: in place); pools are always changed in place.  Returns
    ``result``, an int32 [1] on the device: 0, the number of free pages that are
    missing, or -1 for wrong arguments (then nothing has changed)."""
    num_pages, num_rows, max_pages = _state(page_refs, page_table, seq_lens)
    if len(weights) == 0 or len(pools) == 0 or len(pools) % len(weights):
        raise ValueError(f"pages_evict: {len(pools)} pools for {len(weights)} layers of weights")
    if out_weights is not None and len(out_weights) != len(weights):
        raise ValueError(f"out_weights: expected {len(weights)} tensors, got {len(out_weights)}")
    page_bytes = _pools(pools, num_pages)
    Hkv = weights[0].shape[1] if isinstance(weights[0], torch.Tensor) and weights[0].ndim == 3 else 0
    shape = (num_rows, Hkv, max_pages * 128)
    for some in (weights, out_weights) if out_weights is not None else (weights,):
        for t in some:
            if not isinstance(t, torch.Tensor) or t.dtype is not torch.float32 or t.shape != shape or not t.is_contiguous():
                i = [x is t for x in some].index(True)
                _dense(f"{'weights' if some is weights else 'out_weights'}[{i}]", t, torch.float32, 3, shape)
    want = (Hkv, 128)
    for t in pools:
        at = t.shape
        if at[1:3] != want and not (len(at) == 3 and Hkv == 1 and at[1] == 128):
            i = [x is t for x in pools].index(True)
            raise ValueError(f"pools[{i}]: expected [num_pages, {Hkv}, 128, ...], got {tuple(t.shape)}")
    n = _list("keep", keep)
    if rows is not None:
        _list("rows", rows, n)
    elif n > num_rows:
        raise ValueError(f"keep: {n} entries for {num_rows} rows")
    for name, t, like in (("out_refs", out_refs, page_refs), ("out_table", out_table, page_table), ("out_lens", out_lens, seq_lens)):
        if t is not None:
            _dense(name, t, _I32, None, like.shape)
    if result is not None:
        _dense("result", result, _I32, shape=(1,))
    moved = weights if out_weights is None else out_weights
    handle, context = _on(stream, lambda: "page_refs page_table seq_lens keep rows out_refs out_table out_lens result workspace" +
                          " pool" * len(pools) + " weights" * len(weights) + " out_weights" * len(moved), page_refs, page_table,
                          seq_lens, keep, rows, out_refs, out_table, out_lens, result, workspace, *pools, *weights, *moved)
    with context:
        lib = capi._lib or capi.load()
        ws, nbytes = _scratch(workspace, page_refs.device, "ss_pages_evict_workspace_size", num_pages, num_rows, max_pages, n,
                              Hkv, len(weights), len(pools))
        if result is None:
            result = torch.empty(1, dtype=_I32, device=page_refs.device)
        at, of = array.array("Q", [t.data_ptr() for t in pools]), array.array("Q", [t.data_ptr() for t in weights])
        to = array.array("Q", [t.data_ptr() for t in moved])
        st = lib.ss_pages_evict(
            at.buffer_info()[0], len(at), page_bytes, of.buffer_info()[0], len(of), Hkv, page_refs.data_ptr(), num_pages,
            page_table.data_ptr(), num_rows, max_pages, seq_lens.data_ptr(), rows.data_ptr() if rows is not None else None,
            keep.data_ptr(), n, recent, to.buffer_info()[0], out_refs.data_ptr() if out_refs is not None else None,
            out_table.data_ptr() if out_table is not None else None, out_lens.data_ptr() if out_lens is not None else None,
            result.data_ptr(), ws.data_ptr(), nbytes, handle)
    if st:
        raise SSError(st, "ss_pages_evict")
    _written(moved)
    return result
