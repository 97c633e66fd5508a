"""Operators around a paged cache that many sequences share or that is kept short, as measured work.

* ``shared``  one decode step of a batch whose sequences share pages (a long prompt forked many ways,
              a system prompt with documents behind it): the plan of what is shared, then the
              attention of each layer, every shared page read once for all its sequences;
* ``weigh``   one decode step that also adds each key's attention weight to the sequence's record of
              it (with or without shared pages);
* ``window``  the same record for the tokens of a prompt, or of its last window: how much weight
              each cached key receives from them, without the attention's output;
* ``evict``   the cache is cut back to the keys of largest accumulated weight and the newest ones,
              every head of every layer choosing its own, and the pages that became free are given back.

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
        # A prompt of 2K tokens answered eight ways: the first steps of sampling, where latency counts.
        dict(name="shared_8_on_2k", op="shared", B=8, groups=1, root_min=2000, root_max=2100, doc_min=0, doc_max=0, own_min=1,
             own_max=200, Hq=32, Hkv=8, d=128, layers=1, hot=0.1, mix=1),
        # 64 requests behind one prompt of 32K tokens (a code base, a book), four layers.
        dict(name="shared_64_on_32k", op="shared", B=64, groups=1, root_min=32768, root_max=32768, doc_min=0, doc_max=0, own_min=100,
             own_max=900, Hq=32, Hkv=8, d=128, layers=4, hot=0.1, mix=2),
        # A system prompt for all, six documents, eight questions to each: two levels of sharing.
        dict(name="shared_tree_48", op="shared", B=48, groups=6, root_min=3000, root_max=4000, doc_min=4000, doc_max=9000, own_min=1,
             own_max=700, Hq=16, Hkv=2, d=64, layers=2, hot=0.1, mix=3),
        # A small batch's decode step with the record of weights.
        dict(name="weigh_8", op="weigh", B=8, groups=0, root_min=0, root_max=0, doc_min=0, doc_max=0, own_min=130, own_max=2500, Hq=32,
             Hkv=8, d=128, layers=1, hot=0.1, mix=4),
        # A full batch of long sequences, each on its own.
        dict(name="weigh_64x32k", op="weigh", B=64, groups=0, root_min=0, root_max=0, doc_min=0, doc_max=0, own_min=30000,
             own_max=32768, Hq=32, Hkv=8, d=128, layers=1, hot=0.1, mix=5),
        # 24 sequences forked from a prompt of 8K tokens, each with a record of its own.
        dict(name="weigh_shared_24", op="weigh", B=24, groups=1, root_min=8000, root_max=8300, doc_min=0, doc_max=0, own_min=1,
             own_max=1000, Hq=28, Hkv=4, d=128, layers=1, hot=0.1, mix=6),
        # Short prompts' last tokens, narrow heads, one query head for each key head.
        dict(name="window_3x17", op="window", B=3, n_min=5, n_max=17, L_min=300, L_max=900, Hq=8, Hkv=8, d=64, hot=0.1, mix=7),
        # The last 32 tokens of sixteen long prompts choose which of their keys will be kept.
        dict(name="window_16x32", op="window", B=16, n_min=32, n_max=32, L_min=4000, L_max=16000, Hq=32, Hkv=8, d=128, hot=0.1,
             mix=8),
        # Two whole prompts of about 8K tokens.
        dict(name="window_prompts_8k", op="window", B=2, n_min=7000, n_max=8192, L_min=8192, L_max=8192, Hq=32, Hkv=8, d=128,
             hot=0.1, mix=9),
        # Four short sequences of a small model, one layer.
        dict(name="evict_4x900", op="evict", rows=4, L_min=500, L_max=900, keep_min=300, keep_max=448, recent=32, layers=1, Hkv=2,
             d=64, shared=0, mix=10),
        # Sixteen long prompts are cut to 4K keys in four layers.
        dict(name="evict_16x12k", op="evict", rows=16, L_min=8000, L_max=12000, keep_min=4000, keep_max=4096, recent=256, layers=4,
             Hkv=8, d=128, shared=0, mix=11),
        # Sequences that were forked from one prompt part from it: pages that others hold are not written.
        dict(name="evict_forked_12", op="evict", rows=12, L_min=3000, L_max=5000, keep_min=1000, keep_max=2000, recent=128, layers=2,
             Hkv=8, d=128, shared=2500, mix=12),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["shared", "shared", "weigh", "window", "evict"])
    mix = rng.randrange(1 << 30)
    Hkv = rng.choice([1, 2, 4, 8])
    if op == "evict":
        L_max = _log(rng, 40, 12000)
        rows = max(1, min(_log(rng, 1, 16), 120000 // L_max))
        keep_max = rng.randint(1, L_max)
        return dict(op=op, rows=rows, L_min=rng.randint(max(1, L_max // 2), L_max), L_max=L_max, keep_min=rng.randint(1, keep_max), keep_max=keep_max,
                    recent=rng.choice([0, 1, 32, 256]), layers=_log(rng, 1, 4), Hkv=Hkv, d=rng.choice([64, 128]),
                    shared=rng.choice([0, 0, L_max // 3]), mix=mix)
    G, d, hot = rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 16]), rng.choice([64, 128, 128]), rng.choice([0.05, 0.2])
    if op == "window":
        B = _log(rng, 1, 16)
        n_max = max(1, min(_log(rng, 1, 8192), 8192 // B))
        L_max = max(n_max, min(_log(rng, 64, 16000), 64000 // B, max(64, (1 << 25) // (B * n_max))))
        return dict(op=op, B=B, n_min=rng.randint(1, n_max), n_max=n_max, L_min=rng.randint(n_max, L_max), L_max=L_max, Hq=min(64, G * Hkv) // Hkv * Hkv,
                    Hkv=Hkv, d=d, hot=hot, mix=mix)
    B = _log(rng, 1, 64)
    own_max = _log(rng, 1, 4096)
    shares = op == "shared" or rng.random() < 0.5
    root = _log(rng, 64, 32768) if shares else 0
    doc = rng.choice([0, _log(rng, 64, 8192)]) if shares else 0
    if not shares:
        own_max = max(1, min(_log(rng, 1, 32768), (1 << 20) // B))
    return dict(op=op, B=B, groups=0 if not shares else rng.choice([1, 1, min(B, 3), min(B, 6)]), root_min=root, root_max=root, doc_min=doc // 2, doc_max=doc,
                own_min=rng.randint(1, own_max), own_max=own_max, Hq=min(64, G * Hkv) // Hkv * Hkv, Hkv=Hkv, d=d, layers=1, hot=hot, mix=mix)


# --------------------------------------------------------------------------- what a batch looks like


def _tiles(L):
    return -(-L // PAGE)


def _tree(case):
    """(length, group, keys shared by all, keys shared by the group too) of each sequence of a decode step."""
    r = random.Random(case["mix"])
    root = r.randint(case["root_min"], case["root_max"])
    docs = [r.randint(case["doc_min"], case["doc_max"]) for _ in range(max(1, case["groups"]))]
    seqs = []
    for b in range(case["B"]):
        g = b * len(docs) // case["B"]
        seqs.append((root + docs[g] + r.randint(case["own_min"], case["own_max"]), g, root, root + docs[g]))
    r.shuffle(seqs)  # requests come in any order
    return seqs


def _distinct_keys(case):
    """Keys that a step reads once: whole pages that sequences share are counted once."""
    seen, total = set(), 0
    for L, g, root, doc in _tree(case):
        a, b = (root // PAGE * PAGE, doc // PAGE * PAGE) if case["groups"] else (0, 0)
        for name, n in ((("root",), a), (("doc", g), b - a)):
            if name not in seen:
                seen.add(name)
                total += n
        total += L - b
    return total


def _lengths(case):
    """(new tokens, keys in all) of each sequence of a window."""
    r = random.Random(case["mix"])
    n = [r.randint(case["n_min"], case["n_max"]) for _ in range(case["B"])]
    return n, [max(x, r.randint(case["L_min"], case["L_max"])) if case["n_max"] < case["L_min"] else x for x in n]


def _evicted(case):
    """(keys, keys to keep) of each sequence that is cut back."""
    r = random.Random(case["mix"])
    return [(r.randint(case["L_min"], case["L_max"]), r.randint(case["keep_min"], case["keep_max"])) for _ in range(case["rows"])]


def work(case):
    op, Hkv, d = case["op"], case["Hkv"], case["d"]
    if op in ("shared", "weigh"):
        seqs = _tree(case)
        keys = sum(s[0] for s in seqs)
        bytes_ = 2 * 2 * case["B"] * case["Hq"] * d + 2 * 2 * _distinct_keys(case) * Hkv * d
        if op == "weigh":
            bytes_ += 2 * 4 * keys * Hkv
        return {"bytes": case["layers"] * bytes_, "flops": case["layers"] * 4 * keys * case["Hq"] * d}
    if op == "window":
        n, L = _lengths(case)
        pairs = sum(x * y - x * (x - 1) // 2 for x, y in zip(n, L))
        return {"bytes": 2 * sum(n) * case["Hq"] * d + sum(L) * Hkv * (2 * d + 2 * 4), "flops": 2 * pairs * case["Hq"] * d}
    b = 0
    for L, keep in _evicted(case):
        if L > keep:  # the weights read, the kept ones written, the kept rows of keys and values moved
            b += 4 * L + 4 * keep + 2 * 2 * 2 * keep * d
    return {"bytes": case["layers"] * Hkv * b, "flops": 0}


# ------------------------------------------------------------------------------------ the inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _queries_and_pools(case, T, pages, first, g):
    """Queries, keys and values whose softmax has its weight on few keys: queries and the keys of some pages share a direction."""
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    u = torch.nn.functional.normalize(torch.randn((Hkv, d), generator=g, device="cuda"), dim=-1)
    q = (torch.randn((T, Hkv, Hq // Hkv, d), generator=g, device="cuda") + 8.0 * u[:, None]).to(torch.bfloat16).view(T, Hq, d)
    hot = (torch.rand((pages, Hkv, 1, 1), generator=g, device="cuda") < case["hot"])
    hot[first] = True  # the first keys of a sequence
    kp = _normal((pages, Hkv, PAGE, d), g) + (hot * 8.0 * u[:, None]).to(torch.bfloat16)
    return q, kp, _normal((pages, Hkv, PAGE, d), g)


def _pages_in_order(r, n):
    order = list(range(n))
    r.shuffle(order)
    return iter(order)


def _prepare_decode(case, g, r):
    seqs = _tree(case)
    width = max(_tiles(s[0]) for s in seqs)
    pages = _tiles(_distinct_keys(case)) + 2 * case["B"] + 8
    fresh, shared, table = _pages_in_order(r, pages), {}, []
    for L, group, root, doc in seqs:
        row = []
        for j in range(_tiles(L)):
            name = ("root", j) if j < root // PAGE else ("doc", group, j) if j < doc // PAGE else None
            if not case["groups"] or name is None:
                row.append(next(fresh))
            else:
                if name not in shared:
                    shared[name] = next(fresh)
                row.append(shared[name])
        table.append(row + [-1] * (width - len(row)))
    layers = [_queries_and_pools(case, case["B"], pages, [row[0] for row in table], g) for _ in range(case["layers"])]
    state = dict(layers=layers, table=_ints(table), lens=_ints([s[0] for s in seqs]))
    if case["op"] == "weigh":  # what earlier steps have left: few keys with much of it
        state["weights"] = [torch.rand((case["B"], case["Hkv"], width * PAGE), generator=g, device="cuda").pow_(8) for _ in range(case["layers"])]
    return state


def _prepare_window(case, g, r):
    n, L = _lengths(case)
    width = max(_tiles(x) for x in L)
    pages = sum(_tiles(x) for x in L) + 4
    fresh = _pages_in_order(r, pages)
    table = [[next(fresh) for _ in range(_tiles(x))] + [-1] * (width - _tiles(x)) for x in L]
    q, kp, _ = _queries_and_pools(case, sum(n), pages, [row[0] for row in table], g)
    return dict(q=q, kp=kp, table=_ints(table), cu=_ints([sum(n[:i]) for i in range(len(n) + 1)]), lens=_ints(L), n=n, L=L,
                weights=torch.zeros((case["B"], case["Hkv"], width * PAGE), device="cuda"))


def _prepare_evict(case, g, r):
    seqs = _evicted(case)
    shared = case["shared"] // PAGE  # pages at the front that all sequences hold
    width = max(_tiles(L) for L, _ in seqs)
    pages = shared + sum(_tiles(L) + (_tiles(min(L, keep)) if shared else 0) for L, keep in seqs) + 8
    fresh = _pages_in_order(r, pages)
    front = [next(fresh) for _ in range(shared)]
    table, refs = [], [0] * pages
    for L, _ in seqs:
        mine = front[:L // PAGE]
        mine = mine + [next(fresh) for _ in range(_tiles(L) - len(mine))]
        for p in mine:
            refs[p] += 1
        table.append(mine + [-1] * (width - len(mine)))
    shape = (case["layers"], case["rows"], case["Hkv"], width * PAGE)
    # accumulated weights: a few keys have most, sinks and all others little, whole ones among them (ties)
    weights = torch.rand(shape, generator=g, device="cuda").pow_(8) * 100.0
    weights = torch.where(torch.rand(shape, generator=g, device="cuda") < 0.2, weights.round(), weights)
    pools = _normal((case["layers"], 2, pages, case["Hkv"], PAGE, case["d"]), g)
    state = dict(pools=pools, weights=weights, refs=_ints(refs), table=_ints(table), lens=_ints([L for L, _ in seqs]),
                 keep=_ints([keep for _, keep in seqs]), most=max(min(L, keep) for L, keep in seqs))
    # a user's lists of tensors, and the buffers that take turns with the state's
    state["each"] = [pools[i, j] for i in range(case["layers"]) for j in range(2)]
    state["each_weights"] = list(weights)
    state["new"] = dict(weights=torch.zeros_like(weights), refs=torch.zeros_like(state["refs"]), table=torch.full_like(state["table"], -1),
                        lens=torch.zeros_like(state["lens"]))
    state["new_each"] = list(state["new"]["weights"])
    return state


def prepare(case, seed):
    g, r = _gen(seed), random.Random(seed)
    op = case["op"]
    state = _prepare_evict(case, g, r) if op == "evict" else _prepare_window(case, g, r) if op == "window" else _prepare_decode(case, g, r)
    state["case"] = dict(case)
    return state


# -------------------------------------------------------------------------- the plain forms (32 bits)


def _plain_decode(q, kp, vp, table, lens, weights, case):
    """One layer: the output, and what each key received, added to `weights` (nullable)."""
    (B, Hq, d), Hkv, nT = q.shape, case["Hkv"], table.shape[1]
    G = Hq // Hkv
    hidden = (torch.arange(nT * PAGE, device="cuda") >= lens[:, None])[:, None, None]
    out = torch.empty((B, Hkv, G, d), device="cuda")
    step = max(1, min(Hkv, (1 << 32) // (B * nT * PAGE * d)))
    for h in range(0, Hkv, step):  # as many heads at a time as leave their keys room
        part = slice(h, h + step)
        k = kp[:, part][table].permute(0, 2, 1, 3, 4).float().reshape(B, -1, nT * PAGE, d)
        S = torch.matmul(q.view(B, Hkv, G, d)[:, part].float(), k.transpose(-1, -2)) / math.sqrt(d)
        del k
        S = S.masked_fill_(hidden, -math.inf)
        P = S.sub_(S.amax(-1, keepdim=True)).exp_()
        P = P.div_(P.sum(-1, keepdim=True))
        v = vp[:, part][table].permute(0, 2, 1, 3, 4).float().reshape(B, -1, nT * PAGE, d)
        out[:, part] = torch.matmul(P, v)
        del v
        if weights is not None:
            weights[:, part] += P.sum(2)
    return out.view(B, Hq, d).to(q.dtype)


def _plain_step(s, case):
    table = s["table"].clamp_min(0).long()
    weights = s.get("weights", [None] * case["layers"])
    out = [_plain_decode(q, kp, vp, table, s["lens"], w, case) for (q, kp, vp), w in zip(s["layers"], weights)]
    return (out, s["weights"]) if case["op"] == "weigh" else out


def _plain_window(s, case):
    q, cu, weights = s["q"], s["cu"], s["weights"]
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    at = 0
    for b, (n, L) in enumerate(zip(s["n"], s["L"])):  # the same lengths, as the scheduler has them on the host
        pages, nK = s["table"][b, :_tiles(L)].long(), _tiles(L) * PAGE
        hidden = torch.arange(nK, device="cuda") > torch.arange(L - n, L, device="cuda")[:, None, None]
        rows = q[at:at + n].view(n, Hkv, Hq // Hkv, d).float()
        step = max(1, min(Hkv, (1 << 31) // (n * (Hq // Hkv) * nK)))
        for h in range(0, Hkv, step):
            k = s["kp"][pages, h:h + step].transpose(0, 1).float().reshape(-1, nK, d)
            S = torch.einsum("nhgd,hkd->hngk", rows[:, h:h + step], k) / math.sqrt(d)
            S = S.masked_fill_(hidden, -math.inf)
            P = S.sub_(S.amax(-1, keepdim=True)).exp_()
            total = P.sum(-1, keepdim=True)
            weights[b, h:h + step, :nK] += torch.einsum("hngk,hngk->hk", P, (1.0 / total).expand_as(P))
            del S, P
        at += n
    return weights


def _plain_evict(s, case):
    refs, table, lens, new = s["refs"], s["table"], s["lens"], s["new"]
    rows, width = table.shape
    keep = torch.minimum(s["keep"], lens)
    cut = lens > keep
    place = torch.arange(width * PAGE, device="cuda")
    # the keys of largest weight among the older ones, and the newest; the lowest of equal ones first
    newest = torch.clamp(keep, max=case["recent"])
    rank = torch.where(place >= (lens - newest)[:, None], math.inf, 0.0)[:, None] + s["weights"]
    rank = rank.masked_fill((place >= lens[:, None])[:, None], -math.inf)
    best = torch.sort(rank, dim=-1, descending=True, stable=True).indices
    chosen = torch.zeros(best.shape, dtype=torch.bool, device="cuda").scatter_(-1, best, (place < keep[:, None])[:, None].expand(best.shape))
    source = torch.sort(torch.where(chosen, place, width * PAGE), dim=-1).values[..., :s["most"]]
    # entries behind a sequence's kept keys repeat its last one
    j = torch.minimum(place[:s["most"]], keep[:, None] - 1)  # [rows, most]
    source = torch.gather(source, -1, j[:, None].expand(source.shape))
    # pages that others hold too are not written: the lowest free pages take their place
    tile = torch.arange(width, device="cuda")
    left = (tile < ((keep + PAGE - 1) // PAGE)[:, None])
    used = (tile < ((lens + PAGE - 1) // PAGE)[:, None])
    held = table.clamp_min(0).long()
    moved = left & cut[:, None] & (refs[held] > 1)
    free = torch.sort((refs > 0).to(torch.uint8), stable=True).indices
    fresh = free[(torch.cumsum(moved.reshape(-1), 0) - 1).clamp_min(0)].view(rows, width)
    to = torch.where(moved, fresh, held)
    new["table"].copy_(torch.where(left, to, -1))
    new["lens"].copy_(keep)
    new["refs"].copy_(refs)
    new["refs"].index_add_(0, held.reshape(-1), -(used & (moved | ~left)).reshape(-1).int())
    new["refs"].index_add_(0, fresh.reshape(-1), moved.reshape(-1).int())
    # rows of keys and values, and their weights
    h = torch.arange(case["Hkv"], device="cuda")[:, None]
    b = torch.arange(rows, device="cuda")[:, None, None]
    page, at = to[b, (j // PAGE)[:, None].expand(rows, case["Hkv"], -1)], (j % PAGE)[:, None].expand(rows, case["Hkv"], -1)
    for i in range(case["layers"]):
        pool, src = s["pools"][i], source[i]
        pool[:, page, h, at] = pool[:, held[b, src // PAGE], h, src % PAGE]
    w = torch.gather(s["weights"], -1, source)
    new["weights"].zero_()
    new["weights"][..., :s["most"]] = torch.where((place[:s["most"]] < keep[:, None])[:, None], w, 0.0)
    return s["pools"], new["weights"], new["refs"], new["table"], new["lens"]


# -------------------------------------------------------------------------------------- one pass


def _own_run(s, case):
    import block_sparse_attention_sm_gb300 as ss

    op, scale = case["op"], 1.0 / math.sqrt(case["d"])
    if op in ("shared", "weigh"):
        plan = ss.prefix_plan(s["table"], s["lens"]) if case["groups"] else None
        weights = s.get("weights", [None] * case["layers"])
        out = [ss.decode_shared(q, kp, vp, s["table"], s["lens"], plan, scale=scale, weights=w) for (q, kp, vp), w in zip(s["layers"], weights)]
        return (out, s["weights"]) if op == "weigh" else out
    if op == "window":
        return ss.key_weights(s["q"], s["kp"], s["table"], s["cu"], s["lens"], s["weights"], scale=scale)
    new = s["new"]
    ss.pages_evict(s["each"], s["each_weights"], s["refs"], s["table"], s["lens"], s["keep"], recent=case["recent"],
                   out_weights=s["new_each"], out_refs=new["refs"], out_table=new["table"], out_lens=new["lens"])
    return s["pools"], new["weights"], new["refs"], new["table"], new["lens"]


def run(state):
    case = state["case"]
    if own:
        return _own_run(state, case)
    op = case["op"]
    if op in ("shared", "weigh"):
        return _plain_step(state, case)
    if op == "window":
        return _plain_window(state, case)
    return _plain_evict(state, case)


# ------------------------------------------------------------------------- the definitions in 64 bits


def _exact_softmax(q, kp, pages, L, sees):
    """Softmax weights [Hkv, n, G, L] of the rows q [n, Hq, d] over a sequence's keys; row i sees keys up to sees[i]."""
    Hkv, d = kp.shape[1], kp.shape[3]
    k = torch.cat([kp[p, :, :min(PAGE, L - i * PAGE)] for i, p in enumerate(pages)], dim=1).double()
    x = torch.einsum("nhgd,hkd->hngk", q.double().view(len(q), Hkv, -1, d), k) * d ** -0.5
    x = torch.where(torch.arange(L, device="cuda") > sees[:, None, None], -math.inf, x)
    return torch.exp(x - torch.logsumexp(x, -1, keepdim=True))


def _exact_step(s, case):
    outs, table = [], s["table"].tolist()
    for i, (q, kp, vp) in enumerate(s["layers"]):
        o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
        if case["op"] == "weigh":
            s["weights"][i] = s["weights"][i].double()
        for b, L in enumerate(s["lens"].tolist()):
            pages = table[b][:_tiles(L)]
            p = _exact_softmax(q[b:b + 1], kp, pages, L, torch.tensor([L - 1], device="cuda"))
            v = torch.cat([vp[x, :, :min(PAGE, L - j * PAGE)] for j, x in enumerate(pages)], dim=1).double()
            o[b] = torch.einsum("hngk,hkd->nhgd", p, v).reshape(o[b].shape)
            if case["op"] == "weigh":
                s["weights"][i][b, :, :L] += p.sum((1, 2))
        outs.append(o)
    return (outs, s["weights"]) if case["op"] == "weigh" else outs


def _exact_window(s, case):
    weights, cu = s["weights"].double(), s["cu"].tolist()
    for b, L in enumerate(s["lens"].tolist()):
        n = cu[b + 1] - cu[b]
        pages = s["table"][b, :_tiles(L)].tolist()
        for i in range(0, n, 256):
            m = min(256, n - i)
            p = _exact_softmax(s["q"][cu[b] + i:cu[b] + i + m], s["kp"], pages, L, torch.arange(L - n + i, L - n + i + m, device="cuda"))
            weights[b, :, :L] += p.sum((1, 2))
    return weights


def _exact_evict(s, case):
    """One sequence, layer and head after the other: the keys in the order of their rank, then the kept ones in the order of their places."""
    refs, old = s["refs"].tolist(), s["table"].tolist()
    table, lens, counts = [list(row) for row in old], s["lens"].tolist(), list(refs)
    free = (p for p, held in enumerate(refs) if held == 0)
    for b, keep in enumerate(s["keep"].tolist()):
        if lens[b] <= keep:
            continue
        for j in range(_tiles(lens[b])):
            if j >= _tiles(keep) or refs[old[b][j]] > 1:
                counts[old[b][j]] -= 1
                table[b][j] = -1
                if j < _tiles(keep):
                    table[b][j] = next(free)
                    counts[table[b][j]] = 1
        table[b][_tiles(lens[b]):] = [-1] * (len(table[b]) - _tiles(lens[b]))
    pools, weights = s["pools"].double(), torch.zeros_like(s["weights"], dtype=torch.float64)
    for b, keep in enumerate(s["keep"].tolist()):
        L, keep = lens[b], min(keep, lens[b])
        was = torch.tensor(old[b], device="cuda")
        now = torch.tensor(table[b], device="cuda")
        j = torch.arange(keep, device="cuda")
        for i in range(case["layers"]):
            for h in range(case["Hkv"]):
                w = s["weights"][i, b, h, :L].double()
                recent = min(case["recent"], keep)
                order = torch.sort(-w[:L - recent], stable=True).indices[:keep - recent]
                kept = torch.cat([torch.sort(order).values, torch.arange(L - recent, L, device="cuda")])
                weights[i, b, h, :keep] = w[kept]
                pools[i][:, now[j // PAGE], h, j % PAGE] = s["pools"][i][:, was[kept // PAGE], h, kept % PAGE].double()
        lens[b] = keep
    return pools, weights, _ints(counts), _ints(table), _ints(lens)


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_evict(s, case) if case["op"] == "evict" else _exact_window(s, case) if case["op"] == "window" else _exact_step(s, case)
