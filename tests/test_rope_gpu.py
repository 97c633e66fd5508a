"""Rotary positions, alone and with the cache write, against 64-bit arithmetic (GPU)."""
import decimal
import math

import numpy as np
import pytest
import torch

from _serving import (PAGE, assert_rounded, fill_pool, offsets, random_tables, rotate, rotate_tolerance, tiles)

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    import block_sparse_attention_sm_gb300 as ss

    ss.build()
    assert torch.cuda.is_available()


def _x(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(BF)


def _freq(rot, base=10000.0):
    return torch.tensor([base ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64)


SHAPES = [
    # B, H, L, d, rot, off
    (1, 1, 1, 64, 64, 0),
    (2, 3, 5, 128, 128, 0),
    (1, 32, 7, 128, 64, 0),      # the first half of the head turns
    (3, 2, 130, 64, 32, 32),     # the second
    (1, 16, 33, 192, 64, 128),   # latent prefill rows
    (2, 1, 129, 576, 64, 512),   # latent cache rows
    (2, 5, 9, 80, 24, 8),        # 12 pairs: single entries
    (1, 3, 4, 33, 10, 7),        # odd width and place
    (1, 2, 3, 2, 2, 0),
    (1, 70, 2, 256, 256, 0),
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_rope(shape, interleaved, inverse):
    import block_sparse_attention_sm_gb300 as ss

    B, H, L, d, rot, off = shape
    x = _x((B, H, L, d), 1)
    pos = torch.randint(0, 1 << 20, (B, L), generator=torch.Generator().manual_seed(2), dtype=torch.int32)
    pos[0, 0] = 0
    w, f = _freq(rot), 1.25
    out = ss.rope(x.cuda(), pos.cuda(), w.cuda(), rot_offset=off, interleaved=interleaved, inverse=inverse,
                  attn_factor=f)
    want = rotate(x, pos[:, None], w, f, off, interleaved, inverse)
    assert_rounded(out.cpu(), want, rotate_tolerance(x, w, f, off, interleaved))
    assert torch.equal(out.cpu()[..., :off], x[..., :off])
    assert torch.equal(out.cpu()[..., off + rot:], x[..., off + rot:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_packed_strided_and_in_place(interleaved):
    """[T,H,d] rows inside a wider projection; a row of positions shared by the batch; in place; empty."""
    import block_sparse_attention_sm_gb300 as ss

    T, Hq, Hkv, d = 37, 6, 2, 128
    w = _freq(d).cuda()
    proj = _x((T, Hq + 2 * Hkv, d), 3)
    pos = torch.arange(T, dtype=torch.int32) * 911
    dev = proj.cuda()
    q = dev[:, :Hq]
    want = rotate(proj[:, :Hq], pos[:, None], w.cpu(), 1.0, 0, interleaved)
    tol = rotate_tolerance(proj[:, :Hq], w.cpu(), 1.0, 0, interleaved)
    out = ss.rope(q, pos.cuda(), w, interleaved=interleaved)
    assert out.is_contiguous()
    assert_rounded(out.cpu(), want, tol)
    same = ss.rope(q, pos.cuda(), w, interleaved=interleaved, out=q)
    assert same.data_ptr() == dev.data_ptr()
    assert torch.equal(dev[:, :Hq].cpu(), out.cpu())
    assert torch.equal(dev[:, Hq:].cpu(), proj[:, Hq:])  # the rows' other heads are as they were
    # heads 8 bytes off the 16-byte grid take single entries: the same results
    odd = torch.empty(T, Hq * d + 4, dtype=BF, device="cuda")[:, 4:].unflatten(1, (Hq, d))
    odd.copy_(proj[:, :Hq])
    assert torch.equal(ss.rope(odd, pos.cuda(), w, interleaved=interleaved).cpu(), out.cpu())
    # one head broadcast over the batch
    wide = proj[:, :1].cuda().transpose(0, 1)[None].expand(3, 1, T, d)
    got = ss.rope(wide, pos.cuda(), w, interleaved=interleaved)
    for b in range(3):
        assert torch.equal(got[b, 0].cpu(), out[:, 0].cpu())
    for empty in (torch.empty(0, 3, d), torch.empty(5, 0, d)):
        e = empty.to(BF).cuda()
        assert ss.rope(e, torch.zeros(e.shape[0], dtype=torch.int32, device="cuda"), w).shape == e.shape


def test_rope_far_positions_are_exact():
    """Angles up to position 2^31 - 1 (and negative ones) against 60-digit arithmetic."""
    import block_sparse_attention_sm_gb300 as ss

    decimal.getcontext().prec = 60
    two_pi = 2 * decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
    rot = 128
    w = _freq(rot, 500000.0)
    pos = [0, 1, -1, 131071, 10 ** 6 + 7, (1 << 24) + 1, (1 << 31) - 1, -(1 << 31)]
    x = torch.zeros(len(pos), 1, rot, dtype=BF)
    x[:, :, :rot // 2] = 1.0  # a = 1, b = 0: the outputs are cos and sin
    out = ss.rope(x.cuda(), torch.tensor(pos, dtype=torch.int32, device="cuda"), w.cuda()).cpu().double()
    for i, p in enumerate(pos):
        for j in range(rot // 2):
            t = float((decimal.Decimal(p) * decimal.Decimal(float(w[j]))) % two_pi)
            for got, want in ((out[i, 0, j], math.cos(t)), (out[i, 0, rot // 2 + j], math.sin(t))):
                assert abs(float(got) - want) <= abs(want) * 2.0 ** -8 + 1e-6, (p, j, float(got), want)


def test_rope_gradient():
    """rope(g, inverse) is the gradient: against differences of the 64-bit rotation, and <g, R x> = <R' g, x>."""
    import block_sparse_attention_sm_gb300 as ss

    B, H, L, d, rot, off, f = 1, 2, 6, 64, 32, 16, 1.5
    x, g = _x((B, H, L, d), 5), _x((B, H, L, d), 6)
    pos, w = torch.arange(L, dtype=torch.int32) * 333, _freq(rot)
    grad = ss.rope(g.cuda(), pos.cuda(), w.cuda(), rot_offset=off, inverse=True, attn_factor=f).cpu().double()
    eps = 2.0 ** -10
    value = lambda z: (rotate(z, pos, w, f, off, False) * g.double()).sum()  # noqa: E731
    tol = rotate_tolerance(g, w, f, off, False)
    for i in np.random.default_rng(0).integers(0, x.numel(), 40):
        e = torch.zeros(x.numel(), dtype=torch.float64)
        e[i] = eps
        diff = float(value(x.double() + e.view_as(x)) - value(x.double() - e.view_as(x))) / (2 * eps)
        got = float(grad.flatten()[i])  # the value is linear in x: the difference is exact to ~1e-11
        assert abs(got - diff) <= float(tol.flatten()[i]) + (abs(diff) + 1e-6) * 2.0 ** -8 + 1e-9


def test_rope_of_a_batch_larger_than_one_wave():
    import block_sparse_attention_sm_gb300 as ss

    x = torch.randn(2, 8, 4097, 128, device="cuda", dtype=BF)
    pos = torch.arange(4097, dtype=torch.int32, device="cuda")
    w = _freq(128).cuda()
    out = ss.rope(x, pos, w)
    for l in (0, 1, 2048, 4096):
        want = rotate(x[:, :, l].cpu(), pos[l].cpu(), w.cpu(), 1.0, 0, False)
        assert_rounded(out[:, :, l].cpu(), want, rotate_tolerance(x[:, :, l].cpu(), w.cpu(), 1.0, 0, False))


APPEND = [
    # Hq, Hkv, d, rot, off, new tokens, lengths after them
    (4, 2, 128, 128, 0, [1, 1, 1], [1, 128, 129]),
    (8, 1, 64, 32, 0, [5, 0, 130, 1], [5, 77, 400, 256]),
    (3, 3, 64, 24, 8, [7, 300, 2], [200, 300, 2]),        # single entries
    (16, 1, 576, 64, 512, [3, 1, 0, 129], [140, 64, 0, 129]),  # latent rows
    (32, 8, 128, 128, 0, [1] * 40, list(range(1, 41))),
    (1, 1, 576, 10, 3, [2, 9], [2, 500]),                 # 576-wide rows in single entries
    (2, 2, 128, 0, 0, [4, 140], [130, 140]),              # no rotation
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", APPEND)
def test_append(case, interleaved):
    import block_sparse_attention_sm_gb300 as ss

    Hq, Hkv, d, rot, off, n, L = case
    rng = np.random.default_rng(4)
    latent = d == 576
    pad = 3  # rows behind the last sequence
    T = sum(n) + pad
    q, k, v = _x((T, Hq, d), 1), _x((T, Hkv, d), 2), _x((T, Hkv, d), 3)
    table, pages = random_tables(L, 2, rng)
    old_k, old_v = _x((pages, Hkv, PAGE, d), 7), _x((pages, Hkv, PAGE, d), 8)
    w = _freq(rot) if rot else torch.empty(0, dtype=torch.float64)
    cu = offsets(n)
    seq = np.repeat(np.arange(len(n)), n)
    pos = torch.tensor([L[b] - n[b] + i for b in range(len(n)) for i in range(n[b])], dtype=torch.int64)
    kp, vp = old_k.cuda(), old_v.cuda()
    if latent:
        kp = kp[:, 0].contiguous()
    out = torch.full((T, Hq, d), 9.0, dtype=BF, device="cuda")
    # q, k and v as parts of one projection
    proj = torch.cat([q, k, v], 1).cuda()
    qd, kd, vd = proj.split([Hq, Hkv, Hkv], 1)
    got = ss.rope_append_paged(qd, kd, None if latent else vd, kp, None if latent else vp, table.cuda(), cu.cuda(),
                               torch.tensor(L, dtype=torch.int32, device="cuda"), w.cuda() if rot else None,
                               rot_offset=off, interleaved=interleaved, attn_factor=1.5, out=out)
    assert got is out
    real = T - pad
    f = 1.5
    assert_rounded(out[:real].cpu(), rotate(q[:real], pos[:, None], w, f, off, interleaved),
                   rotate_tolerance(q[:real], w, f, off, interleaved))
    assert (out[real:] == 9.0).all()
    want_k, want_v = old_k.double(), old_v.double()
    tol = torch.zeros_like(want_k)
    page, row = table[seq, pos.numpy() // PAGE].long(), pos % PAGE
    want_k[page, :, row] = rotate(k[:real], pos[:, None], w, f, off, interleaved)
    tol[page, :, row] = rotate_tolerance(k[:real], w, f, off, interleaved)
    want_v[page, :, row] = v[:real].double()
    kp = kp[:, None] if latent else kp
    written = torch.zeros_like(want_k, dtype=torch.bool)
    written[page, :, row] = True
    assert_rounded(kp.cpu(), want_k, tol)
    assert torch.equal(kp.cpu()[~written], old_k[~written])
    if not latent:
        assert torch.equal(vp.cpu().double(), want_v)


def test_append_keys_without_a_page_and_given_positions():
    """Places outside the table or the pool are not written; positions override the angle, not the place."""
    import block_sparse_attention_sm_gb300 as ss

    d, pages = 64, 3
    w = _freq(d)
    # sequence 0: its second page does not exist; 1: shorter than its new tokens; 2: longer than the table
    n, L = [200, 5, 2], [200, 3, 300]
    table = torch.tensor([[0, 99], [1, -1], [2, 2]], dtype=torch.int32)
    T = sum(n)
    k, v = _x((T, 1, d), 1), _x((T, 1, d), 2)
    pos = torch.randint(0, 5000, (T,), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    old = _x((pages, 1, PAGE, d), 3)
    kp, vp = old.cuda(), old.cuda()
    none = ss.rope_append_paged(None, k.cuda(), v.cuda(), kp, vp, table.cuda(), offsets(n).cuda(),
                                torch.tensor(L, dtype=torch.int32, device="cuda"), w.cuda(), positions=pos.cuda())
    assert none is None
    want, want_v, tol = old.double(), old.clone(), torch.zeros(old.shape, dtype=torch.float64)
    turned, t = rotate(k, pos[:, None], w, 1.0, 0, False), rotate_tolerance(k, w, 1.0, 0, False)
    for i in range(128):  # of sequence 0, the first page
        want[0, 0, i], tol[0, 0, i], want_v[0, 0, i] = turned[i, 0], t[i, 0], v[i, 0]
    for i in range(2, 5):  # of sequence 1, keys 0 .. 2 (its first two tokens lie before key 0)
        want[1, 0, i - 2], tol[1, 0, i - 2], want_v[1, 0, i - 2] = turned[200 + i, 0], t[200 + i, 0], v[200 + i, 0]
    assert_rounded(kp.cpu(), want, tol)
    assert torch.equal(vp.cpu(), want_v)


def test_append_refuses_outputs_on_its_inputs():
    import block_sparse_attention_sm_gb300 as ss

    T, Hq, Hkv, d = 6, 2, 2, 64
    proj = _x((T, Hq + 2 * Hkv, d), 1).cuda()
    q, k, v = proj.split([Hq, Hkv, Hkv], 1)
    pool = torch.zeros(3, Hkv, PAGE, d, dtype=BF, device="cuda")
    table, cu = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"), offsets([T]).cuda()
    lens, w = torch.tensor([T], dtype=torch.int32, device="cuda"), _freq(d).cuda()
    before = proj.clone()
    for out, vp in ((k, pool.clone()), (v, pool.clone()), (pool.view(-1, Hq, d)[5:5 + T], pool.clone()), (None, pool)):
        with pytest.raises((ss.SSError, ValueError)):
            ss.rope_append_paged(q, k, v, pool, vp, table, cu, lens, w, out=out)
    torch.cuda.synchronize()
    assert torch.equal(proj, before) and not pool.any()


def test_rope_into_the_rows_between():
    """From the first heads of a projection into the next ones, and from the even tokens into the odd ones."""
    import block_sparse_attention_sm_gb300 as ss

    T, H, d = 9, 3, 128
    w, pos = _freq(d).cuda(), torch.arange(T, dtype=torch.int32, device="cuda") * 77
    proj = _x((T, 2 * H + 1, d), 5).cuda()
    want = ss.rope(proj[:, :H].contiguous(), pos, w)
    got = ss.rope(proj[:, :H], pos, w, out=proj[:, H:2 * H])
    assert got.data_ptr() == proj[:, H:].data_ptr() and torch.equal(got, want)
    x = _x((2, H, 2 * T, d), 6).cuda()
    old, want = x.clone(), ss.rope(x[:, :, 0::2].contiguous(), pos, w)
    ss.rope(x[:, :, 0::2], pos, w, out=x[:, :, 1::2])
    assert torch.equal(x[:, :, 1::2], want) and torch.equal(x[:, :, 0::2], old[:, :, 0::2])


@pytest.mark.parametrize("case", [
    # shape, rot, off, interleaved, inverse, factor
    ((2, 3, 7, 64), 64, 0, False, False, 1.0),
    ((1, 2, 33, 192), 64, 128, True, False, 1.5),
    ((9, 4, 80), 24, 8, False, True, 1.25),       # packed, single entries
])
def test_rope_is_recorded(case):
    """The graph's gradients are the formula's, R' g: of a first and a second backward pass."""
    import block_sparse_attention_sm_gb300 as ss

    shape, rot, off, inter, inv, f = case
    L = shape[-2] if len(shape) == 4 else shape[0]
    x, g = _x(shape, 5).cuda().requires_grad_(True), _x(shape, 6).cuda()
    pos, w = (torch.arange(L, dtype=torch.int32) * 333).cuda(), _freq(rot).cuda()
    kw = dict(rot_offset=off, interleaved=inter, inverse=inv, attn_factor=f)
    at = pos.cpu()[:, None] if len(shape) == 3 else pos.cpu()
    plain = lambda t, i: rotate(t.cpu(), at, w.cpu(), f, off, inter, i)  # noqa: E731
    tol = lambda t: rotate_tolerance(t.cpu(), w.cpu(), f, off, inter)  # noqa: E731
    y = ss.rope(x, pos, w, **kw)
    assert y.requires_grad
    with torch.no_grad():
        same = ss.rope(x, pos, w, **kw)
    assert torch.equal(y, same) and not same.requires_grad
    assert_rounded(y.detach().cpu(), plain(x.detach(), inv), tol(x.detach()))
    v = g.clone().requires_grad_(True)
    grad, = torch.autograd.grad(y, x, v, create_graph=True)
    assert_rounded(grad.detach().cpu(), plain(g, not inv), tol(g))
    # <h, R' v> differentiated by v is R h
    h = _x(shape, 7).cuda()
    second, = torch.autograd.grad(grad, v, h)
    assert_rounded(second.cpu(), plain(h, inv), tol(h))
    # differences of the 64-bit rotation, in some entries
    for i in np.random.default_rng(0).integers(0, x.numel(), 12):
        e = torch.zeros(x.numel(), dtype=torch.float64)
        e[i] = 2.0 ** -10
        moved = [(plain(x.detach().double().cpu() + s * e.view(shape), inv) * g.cpu().double()).sum() for s in (1, -1)]
        diff = float(moved[0] - moved[1]) / 2.0 ** -9
        assert abs(float(grad.detach().flatten()[i]) - diff) <= float(tol(g).flatten()[i]) + (abs(diff) + 1e-6) * 2.0 ** -8 + 1e-9


def test_rope_gradients_of_broadcast_and_strided_inputs():
    """A head shared by the batch, heads of a projection, the broadcast gradient of a sum, another stream."""
    import block_sparse_attention_sm_gb300 as ss

    T, H, d = 12, 3, 64
    w, pos = _freq(d).cuda(), torch.arange(T, dtype=torch.int32, device="cuda") * 11
    proj = _x((T, H + 2, d), 8).cuda().requires_grad_(True)
    ss.rope(proj[:, :H], pos, w).sum().backward()
    ones = torch.ones(T, H, d, dtype=BF)
    want = rotate(ones, pos.cpu()[:, None], w.cpu(), 1.0, 0, False, True)
    assert_rounded(proj.grad[:, :H].cpu(), want, rotate_tolerance(ones, w.cpu(), 1.0, 0, False))
    assert not proj.grad[:, H:].any()
    one = _x((1, 1, T, d), 9).cuda().requires_grad_(True)
    g = _x((4, 1, T, d), 10).cuda()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    y = ss.rope(one.expand(4, 1, T, d), pos, w, stream=stream)
    torch.cuda.current_stream().wait_stream(stream)
    y.backward(g)
    torch.cuda.synchronize()
    parts = rotate(g.cpu(), pos.cpu(), w.cpu(), 1.0, 0, False, True)
    # four gradients, each rounded, summed in bf16: three more roundings of sums of at most sum |part|
    tol = (4 * 2.0 ** -8) * parts.abs().sum(0, keepdim=True) + rotate_tolerance(g.cpu(), w.cpu(), 1.0, 0, False).sum(0, keepdim=True)
    assert ((one.grad.cpu().double() - parts.sum(0, keepdim=True)).abs() <= tol + 1e-40).all()


def test_rope_in_place_is_seen_by_the_graph():
    """A tensor that a graph has saved and that is rotated in place after that is an error of the backward pass."""
    import block_sparse_attention_sm_gb300 as ss

    w, pos = _freq(64).cuda(), torch.arange(4, dtype=torch.int32, device="cuda")
    x, scale = _x((4, 2, 64), 3).cuda(), torch.ones(64, dtype=BF, device="cuda", requires_grad=True)
    y = (x * scale).sum()
    ss.rope(x, pos, w, out=x)
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        y.backward()
    with torch.inference_mode():
        z = x.clone()
        assert ss.rope(z, pos, w, out=z) is z


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_frequencies_of_any_size(interleaved):
    """Just below 2 the angle is exact at any position; beyond, off by |p w| 2^-63 turns; NaN where there is none."""
    import block_sparse_attention_sm_gb300 as ss

    decimal.getcontext().prec = 80
    two_pi = 2 * decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
    bad = [math.inf, -math.inf, math.nan, 2.0 ** 64, -1e30, 1.7e308]
    good = [math.nextafter(2.0, 0), -1.999, 2.0, -3.75, 1000.1, 1e6, -1e12, 1e-300, 5e-324, 0.0]
    w = torch.tensor(good + bad, dtype=torch.float64)
    n, d = len(w), 2 * len(w)
    pos = [0, 1, -3, 40, 131071, (1 << 31) - 1, -(1 << 31)]
    x = torch.zeros(len(pos), 1, d + 8, dtype=BF)
    a, b = (slice(0, d, 2), slice(1, d, 2)) if interleaved else (slice(0, n), slice(n, d))
    x[:, :, a] = 1.0
    x[:, :, d:] = 3.0
    out = ss.rope(x.cuda(), torch.tensor(pos, dtype=torch.int32, device="cuda"), w.cuda(), interleaved=interleaved).cpu().double()
    c, s = out[:, 0, a], out[:, 0, b]
    assert c[:, len(good):].isnan().all() and s[:, len(good):].isnan().all() and (out[:, :, d:] == 3).all()
    for i, p in enumerate(pos):
        for j, f in enumerate(good):
            t = float((decimal.Decimal(p) * decimal.Decimal(f)) % two_pi)
            off = 1e-6 + 2 * math.pi * abs(p * f) * 2.0 ** -63
            for got, want in ((c[i, j], math.cos(t)), (s[i, j], math.sin(t))):
                assert abs(float(got) - want) <= off + (abs(want) + off) * 2.0 ** -8, (p, f, float(got), want)
