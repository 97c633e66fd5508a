"""The serving operators around the paged key/value cache, as measured work.

Four families of calls, each with the inputs that a serving (or training) step has in hand:

* ``rope``    rotary positions of query or key rows, and the gradient of that rotation;
* ``append``  rotary positions of a step's new tokens together with the write of their keys and
              values into the cache's pages;
* ``chunk``   attention of the step's new tokens over the paged cache (causal), or over an
              encoder's cached states (not causal), with or without the skip test;
* ``fork`` / ``compact``  the cache's pages: sequences freed and forked, live pages moved to the
              front of the pools.

Every case is a dict of plain values; lengths of a batch are drawn from the case's own ``mix``, so
that the work of a case does not depend on the seed of its values.
"""
import math
import random

import torch

own = False

PAGE = 128  # keys per page


# ------------------------------------------------------------------------------------ the cases


def listed():
    return [
        # One decode step of 64 sequences: the query heads' rows inside the fused projection.
        dict(name="rope_decode_64", op="rope", layout="thd", B=1, H=32, L=64, extra=16, d=128, rot=128, off=0,
             interleaved=False, inverse=False, scaling="none", factor=1.0, far=32768),
        # Training on 16K tokens, latent-attention rows: the gradient of the rotation of the last
        # 64 of 192 entries, adjacent pairs, positions stretched eightfold.
        dict(name="rope_grad_latent_16k", op="rope", layout="bhld", B=1, H=16, L=16384, extra=0, d=192, rot=64, off=128,
             interleaved=True, inverse=True, scaling="yarn", factor=8.0, far=131072),
        # One decode step of 64 sequences: queries and keys rotated, one key and value row each
        # written to the cache.
        dict(name="append_decode_64", op="append", B=64, n_min=1, n_max=1, L_min=8192, L_max=32768, Hq=32, Hkv=8, d=128,
             rot=128, off=0, latent=False, interleaved=False, scaling="wavelength", factor=8.0, mix=1),
        # Four prompts' chunks of about 2K tokens.
        dict(name="append_chunk_4x2k", op="append", B=4, n_min=1800, n_max=2048, L_min=30000, L_max=32768, Hq=32, Hkv=8,
             d=128, rot=128, off=0, latent=False, interleaved=False, scaling="none", factor=1.0, mix=2),
        # Five drafted tokens of eight sequences are verified against short contexts.
        dict(name="chunk_verify_8x5", op="chunk", B=8, n_min=5, n_max=5, L_min=1500, L_max=2600, long_share=1.0, Hq=32, Hkv=8,
             d=128, causal=True, a=0.0, splits=4, hot=0.1, mix=3),
        # A mixed step: most sequences decode one token, some bring a piece of their prompt.
        dict(name="chunk_mixed_48", op="chunk", B=48, n_min=33, n_max=700, L_min=700, L_max=9000, long_share=0.25, Hq=32, Hkv=8,
             d=128, causal=True, a=16.0, splits=2, hot=0.1, mix=4),
        # Chunked prefill: 2K new tokens of four sequences over 32K keys, every tile kept.
        dict(name="chunk_2k_on_32k", op="chunk", B=4, n_min=2048, n_max=2048, L_min=32768, L_max=32768, long_share=1.0, Hq=32,
             Hkv=8, d=128, causal=True, a=0.0, splits=1, hot=0.1, mix=5),
        # The same with the skip test at a threshold that drops most tiles without weight.
        dict(name="chunk_2k_on_32k_skip", op="chunk", B=4, n_min=2048, n_max=2048, L_min=32768, L_max=32768, long_share=1.0,
             Hq=32, Hkv=8, d=128, causal=True, a=16.0, splits=1, hot=0.1, mix=5),
        # Decoder tokens of ten sequences attend to their encoder's states (64-wide heads).
        dict(name="chunk_cross_d64", op="chunk", B=10, n_min=130, n_max=448, L_min=700, L_max=1500, long_share=1.0, Hq=16, Hkv=16,
             d=64, causal=False, a=0.0, splits=1, hot=0.1, mix=6),
        # Two prompts sampled four ways each, one layer.
        dict(name="pages_fork_small", op="fork", parents=2, children=8, L_min=300, L_max=900, pools=2, pages=96, Hkv=2, d=64, mix=7),
        # Four long prompts branch into 32 sequences, eight layers' keys and values.
        dict(name="pages_fork_layers", op="fork", parents=4, children=32, L_min=3000, L_max=6000, pools=16, pages=512, Hkv=8, d=128,
             mix=8),
        # Requests have ended all over the pools of four layers: live pages move to the front.
        dict(name="pages_compact", op="compact", rows=96, L_min=100, L_max=1500, pools=8, pages=1500, Hkv=8, d=128, mix=9),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "chunk", "chunk", "fork", "compact"])
    mix = rng.randrange(1 << 30)
    if op == "rope":
        d = rng.choice([64, 128, 192, 576, 8 * rng.randint(2, 32)])
        rot = rng.choice([d if d <= 256 else 64, max(2, 2 * rng.randint(1, min(d, 256) // 2)), 64 if d >= 64 else d])
        L, H = _log(rng, 1, 16384), _log(rng, 1, 48)
        layout = rng.choice(["thd", "bhld"])
        return dict(op=op, layout=layout, B=1 if layout == "thd" else rng.randint(1, max(1, min(8, 16384 // L))), H=H, L=L,
                    extra=rng.choice([0, 0, 2, 16]), d=d, rot=rot, off=rng.choice([0, d - rot]), interleaved=rng.random() < 0.5,
                    inverse=rng.random() < 0.3, scaling=rng.choice(["none", "linear", "yarn", "wavelength"]), factor=rng.choice([2.0, 8.0, 32.0]),
                    far=_log(rng, 1024, 1 << 20))
    B = _log(rng, 1, 64)
    if op == "append":
        latent = rng.random() < 0.3
        Hkv = 1 if latent else rng.choice([1, 2, 4, 8])
        d = 576 if latent else rng.choice([64, 128])
        n_max = max(1, min(_log(rng, 1, 2048), 8192 // B))
        L_max = max(n_max, _log(rng, 256, 32768))
        rot = 64 if latent else rng.choice([d, d // 2, 24])
        return dict(op=op, B=B, n_min=rng.randint(1, n_max), n_max=n_max, L_min=rng.randint(n_max, L_max), L_max=L_max,
                    Hq=Hkv * rng.choice([1, 3, 4, 8]) if not latent else rng.choice([16, 32]), Hkv=Hkv, d=d, rot=rot, off=512 if latent else 0,
                    latent=latent, interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "yarn", "wavelength"]),
                    factor=rng.choice([2.0, 8.0]), mix=mix)
    if op == "chunk":
        G, Hkv = rng.choice([1, 1, 2, 3, 4, 4, 5, 7, 8, 16]), rng.choice([1, 2, 4, 8])
        n_max = max(1, min(_log(rng, 1, 2048), 8192 // B))
        L_max = max(n_max, min(_log(rng, 128, 32768), 131072 // B))
        a = rng.choice([0.0, 0.0, 4.0, 16.0])
        return dict(op=op, B=B, n_min=rng.randint(1, n_max), n_max=n_max, L_min=rng.randint(n_max, L_max), L_max=L_max,
                    long_share=rng.choice([1.0, 0.3]), Hq=G * Hkv, Hkv=Hkv, d=rng.choice([64, 128, 128]), causal=rng.random() < 0.8, a=a,
                    splits=rng.choice([1, 1, 2, 3, 8]), hot=rng.choice([0.05, 0.2]), mix=mix)
    Hkv, d = rng.choice([(8, 128), (4, 128), (2, 64), (1, 128)])
    pools = 2 * _log(rng, 1, 8)
    if op == "fork":
        parents, L_max = _log(rng, 1, 4), _log(rng, 64, 4096)
        children = parents * _log(rng, 1, 8)
        pages = (parents + children) * -(-L_max // PAGE) + rng.randint(children + 1, children + 64)
        pages = min(pages, 640)  # the parents, and the children's own last pages, always fit
        return dict(op=op, parents=parents, children=children, L_min=rng.randint(1, L_max), L_max=L_max, pools=pools, pages=pages, Hkv=Hkv,
                    d=d, mix=mix)
    rows, L_max = _log(rng, 1, 96), _log(rng, 64, 1500)
    pages = min(1500, max(rows * -(-L_max // PAGE) + 1, _log(rng, 64, 1500)))
    return dict(op=op, rows=rows, L_min=rng.randint(1, L_max), L_max=L_max, pools=min(pools, 8), pages=pages, Hkv=Hkv, d=d, mix=mix)


# --------------------------------------------------------------------------- what a batch looks like


def _lengths(case):
    """(new tokens, keys in all) of each sequence of a step."""
    r = random.Random(case["mix"])
    n, L = [], []
    for _ in range(case["B"]):
        chunk = r.random() < case.get("long_share", 1.0)
        n.append(r.randint(case["n_min"], case["n_max"]) if chunk else 1)
        L.append(max(n[-1] if case.get("causal", True) else 1, r.randint(case["L_min"], case["L_max"])))
    return n, L


def _tiles(L):
    return -(-L // PAGE)


def _fork_lengths(case):
    r = random.Random(case["mix"])
    return [r.randint(case["L_min"], case["L_max"]) for _ in range(case["parents"])]


def _old_children(case):
    """Lengths of the sequences that the forked ones take the place of: what of the pool the parents leave, less one page a child."""
    r = random.Random(case["mix"] + 1)
    room = case["pages"] - sum(_tiles(x) for x in _fork_lengths(case)) - case["children"]
    each = max(0, room // case["children"])
    return [r.randint(0, min(case["L_max"], each * PAGE)) for _ in range(case["children"])]


def _compact_lengths(case):
    r = random.Random(case["mix"])
    lens, left = [], case["pages"] - 1
    for _ in range(case["rows"]):
        L = min(r.randint(case["L_min"], case["L_max"]) if r.random() < 0.8 else 0, left * PAGE)
        lens.append(L)
        left -= _tiles(L)
    return lens


def _live_pages(case):
    """The pages in use, in ascending order: scattered over the pool."""
    used = sum(_tiles(x) for x in _compact_lengths(case))
    return sorted(random.Random(case["mix"] + 2).sample(range(case["pages"]), used))


def _page_bytes(case):
    return 2 * case["Hkv"] * PAGE * case["d"]


def work(case):
    op = case["op"]
    if op == "rope":
        rows = case["B"] * case["H"] * case["L"]
        return {"bytes": 2 * 2 * rows * case["d"] + 4 * case["B"] * case["L"], "flops": 3 * rows * case["rot"]}
    if op == "append":
        n, _ = _lengths(case)
        T, kv = sum(n), 1 if case["latent"] else 2
        return {"bytes": 2 * 2 * T * case["d"] * (case["Hq"] + kv * case["Hkv"]) + 8 * case["B"] + 4 * T,
                "flops": 3 * T * case["rot"] * (case["Hq"] + case["Hkv"])}
    if op == "chunk":
        n, L = _lengths(case)
        pairs = sum(x * y - (x * (x - 1) // 2 if case["causal"] else 0) for x, y in zip(n, L))
        kept = 1.0 if case["a"] == 0 else case["hot"]
        return {"bytes": int(2 * 2 * sum(n) * case["Hq"] * case["d"] + 2 * (1 + kept) * sum(L) * case["Hkv"] * case["d"]),
                "flops": int(2 * (1 + kept) * pairs * case["Hq"] * case["d"])}
    if op == "fork":
        L = _fork_lengths(case)
        each = case["children"] // case["parents"]
        copies = sum(each for x in L if x % PAGE)
        return {"bytes": 2 * copies * case["pools"] * _page_bytes(case) + 8 * each * sum(_tiles(x) for x in L) + 4 * case["pages"], "flops": 0}
    live = _live_pages(case)
    moves = sum(p >= len(live) for p in live)
    return {"bytes": 2 * moves * case["pools"] * _page_bytes(case) + 8 * case["pages"] + 8 * len(live), "flops": 0}


# ------------------------------------------------------------------------------------ the inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _frequencies(rot, scaling, factor, base=500000.0, original=8192):
    """(radians per position of each pair, factor of the cosines and sines), in 64 bits."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":  # between beta_fast = 32 and beta_slow = 1 turns over the original length
        lo, hi = [rot * math.log(original / (t * 2 * math.pi)) / (2 * math.log(base)) for t in (32.0, 1.0)]
        lo, hi = max(0.0, math.floor(lo)), min(rot - 1.0, math.ceil(hi))
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0
    if scaling == "wavelength":  # kept above 4 turns over the original length, divided below 1
        s = ((original * f / (2 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return f * s + f / factor * (1 - s), 1.0
    return f, 1.0


def _paged(L, spare, r):
    """A page table over shuffled pages: (table, number of pages)."""
    need = sum(_tiles(x) for x in L)
    pages = need + spare
    order = list(range(pages))
    r.shuffle(order)
    width = max(1, max(_tiles(x) for x in L))
    table, at = [], 0
    for x in L:
        table.append(order[at:at + _tiles(x)] + [-1] * (width - _tiles(x)))
        at += _tiles(x)
    return table, pages


def _prepare_rope(case, g):
    B, H, L, d = case["B"], case["H"], case["L"], case["d"]
    f, factor = _frequencies(case["rot"], case["scaling"], case["factor"])
    if case["layout"] == "thd":  # heads inside the rows of a wider projection, a position a row
        x = _normal((L, H + case["extra"], d), g)[:, :H]
        pos = torch.randint(0, case["far"], (L,), generator=g, device="cuda", dtype=torch.int32)
    else:
        x = _normal((B, H, L + case["extra"], d), g)[:, :, :L]
        pos = torch.randint(0, case["far"], (B, 1), generator=g, device="cuda", dtype=torch.int32) + torch.arange(L, device="cuda", dtype=torch.int32)
    return dict(x=x, pos=pos.contiguous(), inv_freq=f.cuda(), factor=factor)


def _prepare_append(case, g, r):
    n, L = _lengths(case)
    T, Hq, Hkv, d = sum(n), case["Hq"], case["Hkv"], case["d"]
    table, pages = _paged(L, 4, r)
    f, factor = _frequencies(case["rot"], case["scaling"], case["factor"])
    if case["latent"]:
        q, k, v = _normal((T, Hq, d), g), _normal((T, 1, d), g), None
    else:  # one fused projection
        q, k, v = _normal((T, Hq + 2 * Hkv, d), g).split([Hq, Hkv, Hkv], dim=1)
    kp = _normal((pages, Hkv, PAGE, d), g)
    return dict(q=q, k=k, v=v, kp=kp, vp=None if case["latent"] else _normal((pages, Hkv, PAGE, d), g), table=_ints(table),
                cu=_ints([sum(n[:i]) for i in range(len(n) + 1)]), lens=_ints(L), inv_freq=f.cuda(), factor=factor)


def _prepare_chunk(case, g, r):
    n, L = _lengths(case)
    T, Hq, Hkv, d = sum(n), case["Hq"], case["Hkv"], case["d"]
    table, pages = _paged(L, 4, r)
    # The softmax's weight lies on few keys: queries and the keys of some tiles share a direction.
    u = torch.nn.functional.normalize(torch.randn((Hkv, d), generator=g, device="cuda"), dim=-1)
    q = (torch.randn((T, Hkv, Hq // Hkv, d), generator=g, device="cuda") + 12.0 * u[:, None]).to(torch.bfloat16).view(T, Hq, d)
    hot = (torch.rand((pages, Hkv, 1, 1), generator=g, device="cuda") < case["hot"])
    hot[[row[0] for row in table]] = True  # the first keys of a sequence
    kp = _normal((pages, Hkv, PAGE, d), g) + (hot * 12.0 * u[:, None]).to(torch.bfloat16)
    return dict(q=q, kp=kp, vp=_normal((pages, Hkv, PAGE, d), g), table=_ints(table), cu=_ints([sum(n[:i]) for i in range(len(n) + 1)]),
                lens=_ints(L), n=n, L=L)


def _prepare_fork(case, g, r):
    parents, children = case["parents"], case["children"]
    lens = _fork_lengths(case) + _old_children(case)
    width = max(1, max(_tiles(x) for x in lens))
    order = list(range(case["pages"]))
    r.shuffle(order)
    table, refs, at = [], [0] * case["pages"], 0
    for x in lens:
        own_pages = order[at:at + _tiles(x)]
        at += _tiles(x)
        table.append(own_pages + [-1] * (width - len(own_pages)))
        for p in own_pages:
            refs[p] = 1
    src = [i * parents // children for i in range(children)]
    pools = _normal((case["pools"], case["pages"], case["Hkv"], PAGE, case["d"]), g)
    return dict(pools=pools, each=list(pools), refs=_ints(refs), table=_ints(table), lens=_ints(lens), src=_ints(src),
                dst=_ints(list(range(parents, parents + children))))


def _prepare_compact(case, g, r):
    lens, live = _compact_lengths(case), _live_pages(case)
    moves = sum(p >= len(live) for p in live)
    order = list(live)
    r.shuffle(order)
    width = max(1, max(_tiles(x) for x in lens))
    table, at = [], 0
    for x in lens:
        table.append(order[at:at + _tiles(x)] + [-1] * (width - _tiles(x)))
        at += _tiles(x)
    refs = [0] * case["pages"]
    for p in live:
        refs[p] = 1
    pools = _normal((case["pools"], case["pages"], case["Hkv"], PAGE, case["d"]), g)
    table = _ints(table)
    return dict(pools=pools, each=list(pools), refs=_ints(refs), table=table, lens=_ints(lens), moves=moves, new_refs=torch.empty_like(_ints(refs)),
                new_table=torch.empty_like(table))


def prepare(case, seed):
    g, r = _gen(seed), random.Random(seed)
    op = case["op"]
    if op == "rope":
        state = _prepare_rope(case, g)
    elif op == "append":
        state = _prepare_append(case, g, r)
    elif op == "chunk":
        state = _prepare_chunk(case, g, r)
    elif op == "fork":
        state = _prepare_fork(case, g, r)
    else:
        state = _prepare_compact(case, g, r)
    state["case"] = dict(case)
    return state


# -------------------------------------------------------------------------- the plain forms (32 bits)


def _rotate(x, pos, inv_freq, factor, rot, off, interleaved, inverse):
    """x [..., d] rotated by the angles of its positions; pos broadcasts against x's leading axes. Angles of far positions are formed in 64 bits."""
    angle = pos.double()[..., None] * inv_freq
    c, s = (factor * torch.cos(angle)).float(), (factor * torch.sin(angle)).float()
    s = -s if inverse else s
    y = x.float().clone()
    part = y[..., off:off + rot]
    if interleaved:
        a, b = part[..., 0::2].clone(), part[..., 1::2].clone()
        part[..., 0::2], part[..., 1::2] = a * c - b * s, b * c + a * s
    else:
        a, b = part[..., :rot // 2].clone(), part[..., rot // 2:].clone()
        part[..., :rot // 2], part[..., rot // 2:] = a * c - b * s, b * c + a * s
    return y.to(x.dtype)


def _plain_rope(s, case):
    pos = s["pos"][:, None] if case["layout"] == "thd" else s["pos"][:, None, :]
    return _rotate(s["x"], pos, s["inv_freq"], s["factor"], case["rot"], case["off"], case["interleaved"], case["inverse"])


def _token_places(cu, lens, T):
    """Sequence of each new token, its place among the sequence's new tokens, and its position."""
    t = torch.arange(T, device="cuda")
    seq = torch.searchsorted(cu, t.int(), right=True) - 1
    i = t - cu[seq]
    return seq, i, lens[seq] - (cu[seq + 1] - cu[seq]) + i


def _plain_append(s, case):
    seq, _, pos = _token_places(s["cu"], s["lens"], s["q"].shape[0])
    turn = (s["inv_freq"], s["factor"], case["rot"], case["off"], case["interleaved"], False)
    q = _rotate(s["q"], pos[:, None], *turn)
    page = s["table"][seq, pos // PAGE].long()
    s["kp"][page, :, pos % PAGE] = _rotate(s["k"], pos[:, None], *turn)
    if s["vp"] is None:
        return q, s["kp"]
    s["vp"][page, :, pos % PAGE] = s["v"]
    return q, s["kp"], s["vp"]


def _kept(S, lens, case):
    """The skip test: which of the tiles of S [B, heads, n, G, tiles, 128] the blocks of 128 // G tokens keep."""
    B, heads, n, G, nT, _ = S.shape
    top = S.amax(-1)
    # each split of a sequence's tiles starts its own running maximum: a padded [splits, tiles of a split] layout
    per = ((lens + PAGE - 1) // PAGE + case["splits"] - 1) // case["splits"]
    per = per.clamp_min(1).long().view(B, 1, 1, 1, 1)
    s, i = torch.arange(case["splits"], device="cuda").view(1, 1, 1, 1, -1, 1), torch.arange(nT, device="cuda")
    at = s * per[..., None] + i
    fine = (i < per[..., None]) & (at < nT)
    size = (B, heads, n, G, case["splits"], nT)
    laid = torch.gather(top, 4, at.clamp_max(nT - 1).expand(B, heads, n, G, -1, -1).reshape(B, heads, n, G, -1)).view(size)
    run = torch.cummax(laid.masked_fill(~fine, -math.inf), dim=-1).values
    run = torch.cat([torch.full_like(run[..., :1], -math.inf), run[..., :-1]], dim=-1)
    before = torch.gather(run.view(B, heads, n, G, -1), 4, ((i // per).clamp_max(case["splits"] - 1) * nT + i % per).expand(B, heads, n, G, nT))
    c = torch.where(top == -math.inf, -math.inf, torch.where(before == -math.inf, math.inf, top - before))
    tokens = PAGE // G
    c = torch.nn.functional.pad(c.permute(0, 1, 4, 3, 2), (0, -n % tokens), value=-math.inf)
    c = c.view(B, heads, nT, G, -1, tokens).amax((3, 5))  # the vote: every row of the block
    lam = (case["a"] / lens.clamp_min(1)).clamp_max(1.0).view(B, 1, 1, 1)
    keep = ~(c < torch.log(lam))
    return keep.repeat_interleave(tokens, dim=3)[..., :n].permute(0, 1, 3, 2)[:, :, :, None, :, None]


def _attend(q, kp, vp, table, first, new, lens, n, case):
    """Attention of a padded batch of sequences, n new tokens each at most: [B, n, Hq, d]. first, new, lens: of each sequence, on the GPU."""
    T, Hq, d = q.shape
    Hkv, (B, nT) = case["Hkv"], table.shape
    G = Hq // Hkv
    t, key = torch.arange(n, device="cuda"), torch.arange(nT * PAGE, device="cuda")
    last = (lens - new)[:, None] + t if case["causal"] else (lens - 1)[:, None].expand(B, n)
    last = torch.minimum(last, lens[:, None] - 1).masked_fill(t >= new[:, None], -1)
    hidden = (key > last[..., None])[:, None, :, None]  # [B, 1, n, 1, keys]
    rows = (first[:, None] + t).clamp_max(T - 1)
    qs = q.view(T, Hkv, G, d)[rows].permute(0, 2, 1, 3, 4)  # [B, Hkv, n, G, d]
    out = torch.empty((B, Hkv, n, G, d), device="cuda")
    step = max(1, min(Hkv, (1 << 31) // max(1, B * n * G * nT * PAGE)))
    for h in range(0, Hkv, step):  # as many heads at a time as leave the scores room
        part = slice(h, h + step)
        k = kp[:, part][table].permute(0, 2, 1, 3, 4).float().reshape(B, -1, nT * PAGE, d)
        S = torch.matmul(qs[:, part].float().reshape(B, -1, n * G, d), k.transpose(-1, -2)) / math.sqrt(d)
        S = S.view(B, -1, n, G, nT * PAGE).masked_fill_(hidden, -math.inf)
        if case["a"] > 0:
            S = S.view(B, -1, n, G, nT, PAGE)
            S = S.masked_fill_(~_kept(S, lens, case), -math.inf).view(B, -1, n, G, nT * PAGE)
        top = S.amax(-1, keepdim=True)
        P = S.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
        v = vp[:, part][table].permute(0, 2, 1, 3, 4).float().reshape(B, -1, nT * PAGE, d)
        total = P.sum(-1, keepdim=True)
        O = torch.matmul(P.view(B, -1, n * G, nT * PAGE), v).view(B, -1, n, G, d)
        out[:, part] = torch.where(total > 0, O / total, 0.0)
    return out.permute(0, 2, 1, 3, 4).reshape(B, n, Hq, d)


def _plain_chunk(s, case):
    q, cu, lens, table = s["q"], s["cu"], s["lens"], s["table"].clamp_min(0).long()
    n, L = s["n"], s["L"]  # the same lengths, as the scheduler has them on the host
    if len(n) * max(n) * table.shape[1] <= 4 * sum(x * _tiles(y) for x, y in zip(n, L)):
        O = _attend(q, s["kp"], s["vp"], table, cu[:-1], cu[1:] - cu[:-1], lens, max(n), case)
        seq, i, _ = _token_places(cu, lens, q.shape[0])
        return O[seq, i].to(q.dtype)
    out, at = torch.empty_like(q), 0
    for b, (x, y) in enumerate(zip(n, L)):  # too ragged to pad: one sequence after the other
        one = slice(b, b + 1)
        out[at:at + x] = _attend(q, s["kp"], s["vp"], table[one, :_tiles(y)], cu[one], cu[b + 1:b + 2] - cu[one], lens[one], x, case)[0]
        at += x
    return out


def _plain_fork(s):
    refs, table, lens, dst, src = s["refs"], s["table"], s["lens"], s["dst"].long(), s["src"].long()
    j = torch.arange(table.shape[1], device="cuda")
    # free the sequences whose places are taken
    used = (j < ((lens[dst] + PAGE - 1) // PAGE)[:, None])
    refs.index_add_(0, table[dst].clamp_min(0).reshape(-1).long(), -used.reshape(-1).int())
    # whole pages are shared; a last page that is not full is copied into the lowest free page
    L = lens[src]
    full, partial = (L // PAGE)[:, None], (L % PAGE > 0)
    free = torch.sort((refs > 0).to(torch.uint8), stable=True).indices
    fresh = free[(torch.cumsum(partial, 0) - 1).clamp_min(0)]
    old = table[src, torch.where(partial, L // PAGE, 0)].clamp_min(0).long()
    table[dst] = torch.where(j < full, table[src], torch.where((j == full) & partial[:, None], fresh[:, None].int(), -1))
    refs.index_add_(0, table[src].clamp_min(0).reshape(-1).long(), (j < full).reshape(-1).int())
    refs.index_add_(0, fresh, partial.int())
    lens[dst] = L
    to = torch.where(partial, fresh, old)
    s["pools"][:, to] = s["pools"][:, old]
    return s["pools"], refs, table, lens


def _plain_compact(s):
    refs, table, lens = s["refs"], s["table"], s["lens"]
    N, moves = refs.shape[0], s["moves"]
    live, p = refs > 0, torch.arange(refs.shape[0], device="cuda")
    count = live.sum()
    holes = torch.sort(torch.where(~live & (p < count), p, N)).values[:moves]
    movers = torch.sort(torch.where(live & (p >= count), p, -1), descending=True).values[:moves]
    s["pools"][:, holes] = s["pools"][:, movers]
    s["new_refs"].copy_(torch.where(p < count, refs, 0))
    s["new_refs"][holes] = refs[movers]
    to = p.int()
    to[movers] = holes.int()
    used = torch.arange(table.shape[1], device="cuda") < ((lens + PAGE - 1) // PAGE)[:, None]
    s["new_table"].copy_(torch.where(used, to[table.clamp_min(0).long()], -1))
    return s["pools"], s["new_refs"], s["new_table"], count.int()


# -------------------------------------------------------------------------------------- one pass


def _own_run(s, case):
    import block_sparse_attention_sm_gb300 as ss

    op = case["op"]
    if op == "rope":
        return ss.rope(s["x"], s["pos"], s["inv_freq"], rot_offset=case["off"], interleaved=case["interleaved"], inverse=case["inverse"],
                       attn_factor=s["factor"])
    if op == "append":
        q = ss.rope_append_paged(s["q"], s["k"], s["v"], s["kp"], s["vp"], s["table"], s["cu"], s["lens"], s["inv_freq"],
                                 rot_offset=case["off"], interleaved=case["interleaved"], attn_factor=s["factor"])
        return (q, s["kp"]) if s["vp"] is None else (q, s["kp"], s["vp"])
    if op == "chunk":
        return ss.chunk_paged(s["q"], s["kp"], s["vp"], s["table"], s["cu"], s["lens"], scale=1.0 / math.sqrt(case["d"]),
                              causal=case["causal"], lambda_a=case["a"], num_kv_splits=case["splits"])
    if op == "fork":
        ss.pages_free(s["refs"], s["table"], s["lens"], s["dst"])
        ss.pages_fork(s["each"], s["refs"], s["table"], s["lens"], s["src"], s["dst"])
        return s["pools"], s["refs"], s["table"], s["lens"]
    live = ss.pages_compact(s["each"], s["refs"], s["table"], s["lens"], out_refs=s["new_refs"], out_table=s["new_table"])
    return s["pools"], s["new_refs"], s["new_table"], live.view(())


def run(state):
    case = state["case"]
    if own:
        return _own_run(state, case)
    op = case["op"]
    if op == "rope":
        return _plain_rope(state, case)
    if op == "append":
        return _plain_append(state, case)
    if op == "chunk":
        return _plain_chunk(state, case)
    if op == "fork":
        return _plain_fork(state)
    return _plain_compact(state)


# ------------------------------------------------------------------------- the definitions in 64 bits


def _exact_turn(x, pos, inv_freq, factor, case, inverse):
    """Each pair (a, b) as the complex number a + ib, times factor * exp(+-i * angle)."""
    rot, off = case["rot"], case["off"]
    y = x.double()
    z = y[..., off:off + rot]
    pair = torch.stack([z[..., 0::2], z[..., 1::2]], -1) if case["interleaved"] else torch.stack([z[..., :rot // 2], z[..., rot // 2:]], -1)
    angle = pos.double()[..., None] * inv_freq.double()
    turned = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * torch.polar(torch.full_like(angle, factor), -angle if inverse else angle))
    turned = turned.flatten(-2) if case["interleaved"] else torch.cat([turned[..., 0], turned[..., 1]], -1)
    return torch.cat([y[..., :off], turned, y[..., off + rot:]], -1)


def _exact_append(s, case):
    cu, lens, table = s["cu"].tolist(), s["lens"].tolist(), s["table"].tolist()
    where = [(lens[b] - (cu[b + 1] - cu[b]) + i, b) for b in range(case["B"]) for i in range(cu[b + 1] - cu[b])]
    pos = torch.tensor([p for p, _ in where], device="cuda")
    page = torch.tensor([table[b][p // PAGE] for p, b in where], device="cuda")
    q, k = [_exact_turn(s[x], pos[:, None], s["inv_freq"], s["factor"], case, False) for x in ("q", "k")]
    kp = s["kp"].double()
    kp[page, :, pos % PAGE] = k
    if s["vp"] is None:
        return q, kp
    vp = s["vp"].double()
    vp[page, :, pos % PAGE] = s["v"].double()
    return q, kp, vp


def _exact_chunk(s, case):
    """One sequence after the other, one tile of keys after the other: the running maximum, sum and output of every row, the vote of every block."""
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    G, tokens = Hq // Hkv, PAGE // (Hq // Hkv)
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        n, L = cu[b + 1] - cu[b], lens[b]
        q = s["q"][cu[b]:cu[b + 1]].double().view(n, Hkv, G, d).permute(1, 0, 2, 3).reshape(Hkv, n * G, d)
        place = torch.arange(n, device="cuda").repeat_interleave(G)
        block = place // tokens
        sees = place + (L - n) if case["causal"] else torch.full_like(place, L - 1)
        per = -(-_tiles(L) // case["splits"])
        bound = math.log(min(1.0, case["a"] / L)) if case["a"] > 0 else -math.inf
        none = torch.full((Hkv, n * G), -math.inf, dtype=torch.float64, device="cuda")
        top, since, l, o = none.clone(), none.clone(), torch.zeros_like(none), torch.zeros_like(q)
        for j in range(_tiles(L)):
            if j % per == 0:
                since = none.clone()  # the vote's maximum: of this split only
            keys = torch.arange(j * PAGE, min(L, (j + 1) * PAGE), device="cuda")
            page = s["table"][b, j].long()
            S = q @ s["kp"][page, :, :len(keys)].double().transpose(1, 2) / math.sqrt(d)
            S = S.masked_fill(keys > sees[:, None], -math.inf)
            m = S.amax(-1)
            votes = torch.where(m == -math.inf, -math.inf, torch.where(since == -math.inf, math.inf, m - since))
            c = torch.full((Hkv, int(block[-1]) + 1), -math.inf, dtype=torch.float64, device="cuda")
            c = c.scatter_reduce(1, block.expand(Hkv, -1), votes, "amax")
            keep = (~(c < bound) if case["a"] > 0 else torch.ones_like(c, dtype=torch.bool))[:, block] & (m > -math.inf)
            since = torch.maximum(since, m)
            higher = torch.where(keep, torch.maximum(top, m), top)
            P = torch.where(keep[..., None], torch.exp(S - higher.masked_fill(higher == -math.inf, 0.0)[..., None]), 0.0)
            shrink = torch.where(top == -math.inf, 0.0, torch.exp(top - higher))
            l = l * shrink + P.sum(-1)
            o = o * shrink[..., None] + P @ s["vp"][page, :, :len(keys)].double()
            top = higher
        o = torch.where(l[..., None] > 0, o / l[..., None], 0.0)
        out[cu[b]:cu[b + 1]] = o.view(Hkv, n, G, d).permute(1, 0, 2, 3).reshape(n, Hq, d)
    return out


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None  # copies and whole numbers
    s = prepare(case, seed)
    if case["op"] == "rope":
        pos = s["pos"][:, None] if case["layout"] == "thd" else s["pos"][:, None, :]
        return _exact_turn(s["x"], pos, s["inv_freq"], s["factor"], case, case["inverse"])
    if case["op"] == "append":
        return _exact_append(s, case)
    if work(dict(case, a=0.0))["flops"] > 6e12:
        return None
    return _exact_chunk(s, case)
