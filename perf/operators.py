"""The operators of the paged key-value cache, as measured calls: attention of one new token over
the cache (`attention`), and what keeps the cache: writing new tokens' keys and values (`append`),
growing and shrinking sequences with copy on write (`resize`), sharing a sequence's pages with a
new one (`fork`) and moving the pages in use to the front of the pool (`compact`).

A case is a dict of plain values.  Lengths, head counts and page counts follow from the case
alone; the values, and which page of the pool holds what, follow from the seed.  `run` with
`own = False` computes the operator in elementary torch operations in 32 bits; with `own = True`
it calls the library.

The cache.  k_pages, v_pages [P, page, Hkv, d], or [P, Hkv, page, d] where head_major; token t of
sequence s lies in slot t % page of page page_table[s, t // page]; ref[p] counts the sequences
that hold page p (0: free).
"""
import math
import zlib

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------
# cases


def listed():
    return [
        # one user's stream at 4K of context, 24 query and 8 key-value heads: pure latency
        dict(name="attention-1x4k", op="attention", dtype="bf16", B=1, Hkv=8, G=3, d=128, page=16,
             lo=4096, hi=4096, empty=0, window=0, head_major=False, lse=False),
        # a serving batch: ragged lengths, four idle slots
        dict(name="attention-64-ragged", op="attention", dtype="bf16", B=64, Hkv=8, G=3, d=128,
             page=16, lo=200, hi=32768, empty=4, window=0, head_major=False, lse=False),
        # two documents of half a million tokens, with the log-sum-exp for joining over GPUs
        dict(name="attention-2x512k", op="attention", dtype="bf16", B=2, Hkv=8, G=3, d=128,
             page=64, lo=524288, hi=524288, empty=0, window=0, head_major=True, lse=True),
        # fp32 heads of 64, a window of 1000 tokens over a ragged batch
        dict(name="attention-f32-window", op="attention", dtype="f32", B=48, Hkv=4, G=4, d=64,
             page=32, lo=1, hi=7001, empty=1, window=1000, head_major=False, lse=False),
        # one decode step of 256 slots, nine of them idle
        dict(name="append-step", op="append", dtype="bf16", B=256, Hkv=8, d=128, page=16, lo=1,
             hi=1, empty=9, start=1500, packed=False, head_major=False),
        # prompts of 37 requests behind cached prefixes
        dict(name="append-prompts", op="append", dtype="bf16", B=37, Hkv=8, d=128, page=16, lo=50,
             hi=32768, empty=2, start=700, packed=True, head_major=False),
        # one decode step: every slot grows by a token, some sit on a page shared by a beam
        dict(name="resize-step", op="resize", dtype="bf16", S=256, Hkv=8, d=128, page=16, P=20000,
             lo=100, hi=2000, beam=4, kind="step", head_major=False),
        # requests come and go on a large pool of narrow pages
        dict(name="resize-churn", op="resize", dtype="bf16", S=1000, Hkv=1, d=64, page=16,
             P=786433, lo=100, hi=20000, beam=2, kind="churn", head_major=False),
        # four beams out of each of sixteen short prompts
        dict(name="fork-beams", op="fork", S=96, n=64, parents=16, page=16, P=4096, lo=300,
             hi=1200),
        # 512 requests on four cached documents
        dict(name="fork-documents", op="fork", S=600, n=512, parents=4, page=16, P=65537,
             lo=100000, hi=131072),
        # a small pool after a burst
        dict(name="compact-small", op="compact", dtype="bf16", S=40, Hkv=8, d=128, page=16,
             P=1500, live=300, head_major=False),
        # a pool of 65536 pages, half of them in use
        dict(name="compact-large", op="compact", dtype="bf16", S=300, Hkv=8, d=128, page=16,
             P=65536, live=32000, head_major=True),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread evenly over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention"] * 5 + ["append"] * 2 + ["resize"] * 2 + ["fork", "compact"])
    page = rng.choice([8, 16, 32, 64, 128])
    heads = dict(dtype=rng.choice(["bf16", "bf16", "f32"]), Hkv=rng.choice([1, 2, 3, 4, 8, 16]),
                 d=rng.choice([64, 128]), head_major=rng.random() < 0.4)
    row = heads["Hkv"] * heads["d"]
    if op == "attention":
        B = _log(rng, 1, 300)
        # at most 2^21 tokens and 2^30 elements of keys
        hi = _log(rng, 1, max(1, min(2 ** 21, 2 ** 30 // row) // B))
        return dict(op=op, **heads, G=rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16, 24]), B=B, page=page,
                    lo=_log(rng, 1, hi), hi=hi, empty=rng.choice([0, 0, B // 7]),
                    window=rng.choice([0, 0, _log(rng, 1, 5000)]), lse=rng.random() < 0.3)
    if op == "append":
        packed = rng.random() < 0.6
        B = _log(rng, 1, 600)
        hi = _log(rng, 1, max(1, min(2 ** 19, 2 ** 28 // row) // B)) if packed else 1
        return dict(op=op, **heads, B=B, page=page, lo=_log(rng, 1, hi), hi=hi,
                    empty=rng.choice([0, B // 9]), start=_log(rng, 1, 2000), packed=packed)
    S = _log(rng, 2, 1500)
    if op == "resize":
        hi = _log(rng, 20, max(20, min(40000, 2 ** 20 // S)))
        held = S * (hi // page + 1)
        extra = _log(rng, 100, 100000)
        P = max(S, min(held + extra + S * (4096 // page + 2), 2 ** 30 // (row * page)))
        return dict(op=op, **heads, S=S, page=page, P=P, lo=max(1, hi // rng.choice([1, 3, 20])),
                    hi=hi, beam=rng.choice([1, 2, 5]), kind=rng.choice(["step", "churn"]))
    if op == "fork":
        parents = rng.randint(1, max(1, S // 4))
        n = rng.randint(1, S - parents)
        hi = _log(rng, 2, max(2, min(200000, 2 ** 24 // S)))
        return dict(op=op, S=S, n=n, parents=parents, page=page,
                    P=parents * (hi // page + 2) + rng.randint(1, 50000),
                    lo=max(1, hi // rng.choice([1, 4])), hi=hi)
    P = _log(rng, 16, max(16, min(200000, 2 ** 29 // (row * page))))
    return dict(op=op, **heads, S=min(S, P), page=page, P=P, live=rng.randint(1, P))


# ---------------------------------------------------------------------------------------------
# what follows from the case alone


def _shape_rng(case):
    text = repr(sorted((k, v) for k, v in case.items() if k != "name"))
    return np.random.default_rng(zlib.crc32(text.encode()))


def _lengths(rng, n, lo, hi, empty=0):
    """n lengths spread over lo .. hi evenly in their logarithm, `empty` of them zero."""
    x = np.exp(rng.uniform(np.log(lo), np.log(hi + 1), n)).astype(np.int64).clip(lo, hi)
    x[rng.permutation(n)[:empty]] = 0
    return x


def _attention_lengths(case):
    return _lengths(_shape_rng(case), case["B"], case["lo"], case["hi"], case["empty"])


def _append_lengths(case):
    """(new tokens, position of the first) of each sequence."""
    rng = _shape_rng(case)
    new = _lengths(rng, case["B"], case["lo"], case["hi"], case["empty"])
    return new, rng.integers(0, case["start"] + 1, case["B"])


def _resize_plan(case):
    """(lengths, changes, first row of the beam that each row belongs to)."""
    rng = _shape_rng(case)
    S, page = case["S"], case["page"]
    first = np.arange(S)
    # the first quarter of the rows: beams, whose rows share all their pages
    n = max(1, S // 4 // case["beam"]) * case["beam"]
    if n <= S:
        first[:n] = np.arange(n) // case["beam"] * case["beam"]
    lens = _lengths(rng, S, case["lo"], case["hi"])
    budget = case["P"] * 3 // 4                      # pages that may be in use at the start
    pages = (lens + page - 1) // page
    pages[first != np.arange(S)] = 0
    lens[np.cumsum(pages) > budget] = 0
    lens = lens[first]
    delta = np.ones(S, np.int64)
    delta[rng.random(S) < 0.05] = 0
    if case["kind"] == "churn":
        what = rng.random(S)
        delta = np.where(what < 0.3, -lens, delta)                             # retired
        delta = np.where((what >= 0.3) & (what < 0.6), rng.integers(1, 4097, S), delta)
        delta = np.where(what > 0.9, -rng.integers(1, 9, S), delta)            # drafts taken back
    return lens, delta, first


def _fork_plan(case):
    """(lengths, source rows, rows they are forked to)."""
    rng = _shape_rng(case)
    lens = np.zeros(case["S"], np.int64)
    rows = rng.permutation(case["S"])
    parents, children = rows[:case["parents"]], rows[case["parents"]:case["parents"] + case["n"]]
    lens[parents] = _lengths(rng, case["parents"], case["lo"], case["hi"])
    return lens, parents[rng.integers(0, case["parents"], case["n"])], children


def _compact_lengths(case):
    """Lengths that hold `live` pages between them."""
    rng = _shape_rng(case)
    S = case["S"]
    pages = rng.multinomial(case["live"], np.full(S, 1.0 / S))
    return np.maximum(pages * case["page"] - rng.integers(0, case["page"], S), 0) * (pages > 0)


# ---------------------------------------------------------------------------------------------
# inputs


def _pool(case, P, gen):
    a, b = (case["Hkv"], case["page"]) if case["head_major"] else (case["page"], case["Hkv"])
    mk = lambda: torch.randn((P, a, b, case["d"]), generator=gen, device="cuda",  # noqa: E731
                             dtype=DTYPES[case["dtype"]])
    return mk(), mk()


def _table(rng, lens, page, P, width, first=None):
    """A page table whose rows hold pages taken at random from the pool; rows of one beam
    (`first`) hold the same ones."""
    S = len(lens)
    n = (lens + page - 1) // page
    mine = n.copy()
    if first is not None:
        mine[first != np.arange(S)] = 0
    ids = rng.permutation(P)[:mine.sum()]
    table = np.full((S, width), -1, np.int32)
    table[np.arange(width) < mine[:, None]] = ids
    if first is not None:
        table = table[first]
    ref = np.bincount(table[table >= 0], minlength=P).astype(np.int32)
    return table, ref


def _dev(x, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(x)).to("cuda", dtype)


def _meta(lens, ref, table):
    """Lengths, counts and page table in one buffer, so that a pass can start from a copy."""
    flat = np.concatenate([lens.astype(np.int32), ref, table.reshape(-1)])
    return dict(meta=_dev(flat), S=len(lens), P=len(ref), width=table.shape[1])


def _views(st):
    m = st["meta"].clone()
    S, P = st["S"], st["P"]
    return m[:S], m[S:S + P], m[S + P:].view(S, st["width"])


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator("cuda").manual_seed(seed)
    op, page = case["op"], case["page"]
    st = dict(case=case)
    if op == "attention":
        lens = _attention_lengths(case)
        pages = (lens + page - 1) // page
        P, width = int(pages.sum()) + 3, int(pages.max()) + 2
        table, _ = _table(rng, lens, page, P, width)
        k, v = _pool(case, P, gen)
        q = torch.randn((case["B"], case["Hkv"] * case["G"], case["d"]), generator=gen,
                        device="cuda", dtype=DTYPES[case["dtype"]])
        return dict(st, q=q, lens=_dev(lens), table=_dev(table), k_pages=k, v_pages=v)
    if op == "append":
        new, start = _append_lengths(case)
        pages = (start + new + page - 1) // page
        P, width = int(pages.sum()) + 3, int(pages.max()) + 2
        table, _ = _table(rng, start + new, page, P, width)
        k_pages, v_pages = _pool(case, P, gen)
        T = int(new.sum()) if case["packed"] else case["B"]
        mk = lambda: torch.randn((T, case["Hkv"], case["d"]), generator=gen,  # noqa: E731
                                 device="cuda", dtype=DTYPES[case["dtype"]])
        cu = _dev(np.concatenate([[0], np.cumsum(new)])) if case["packed"] else None
        return dict(st, k=mk(), v=mk(), pos=_dev(np.where(new > 0, start, -1)), cu=cu,
                    table=_dev(table), k_pages=k_pages, v_pages=v_pages)
    P = case["P"]
    if op == "resize":
        lens, delta, first = _resize_plan(case)
        width = int(max(0, (np.maximum(lens, lens + delta)).max()) // page) + 2
        table, ref = _table(rng, lens, page, P, width, first)
        k, v = _pool(case, P, gen)
        return dict(st, **_meta(lens, ref, table), delta=_dev(delta), k_pages=k, v_pages=v)
    if op == "fork":
        lens, src, dst = _fork_plan(case)
        table, ref = _table(rng, lens, page, P, int(lens.max()) // page + 2)
        return dict(st, **_meta(lens, ref, table), src=_dev(src), dst=_dev(dst))
    lens = _compact_lengths(case)
    table, ref = _table(rng, lens, page, P, int(lens.max()) // page + 2)
    k, v = _pool(case, P, gen)
    return dict(st, **_meta(lens, ref, table), k_pages=k, v_pages=v)


# ---------------------------------------------------------------------------------------------
# one pass


def run(st):
    return globals()["_own_" + st["case"]["op"] if own else "_plain_" + st["case"]["op"]](st)


def _own_attention(st):
    import gated_retention_linear_b200 as G
    c = st["case"]
    o, lse = G.gret_paged_attention_decode(
        st["q"], st["lens"], st["table"], st["k_pages"], st["v_pages"], window=c["window"],
        head_major=c["head_major"], lse=True if c["lse"] else None)
    return (o, lse) if c["lse"] else o


def _own_append(st):
    import gated_retention_linear_b200 as G
    G.gret_paged_append(st["k"], st["v"], st["pos"], st["table"], st["k_pages"], st["v_pages"],
                        cu_seqlens=st["cu"], head_major=st["case"]["head_major"])
    return st["k_pages"], st["v_pages"]


def _own_resize(st):
    import gated_retention_linear_b200 as G
    lens, ref, table = _views(st)
    pos = G.gret_paged_resize(st["delta"], lens, table, ref, st["k_pages"], st["v_pages"],
                              head_major=st["case"]["head_major"])
    return pos, lens, ref, table, st["k_pages"], st["v_pages"]


def _own_fork(st):
    import gated_retention_linear_b200 as G
    lens, ref, table = _views(st)
    G.gret_paged_fork(st["src"], st["dst"], lens, table, ref, page_size=st["case"]["page"])
    return lens, ref, table


def _own_compact(st):
    import gated_retention_linear_b200 as G
    lens, ref, table = _views(st)
    n_live = G.gret_paged_compact(lens, table, ref, st["k_pages"], st["v_pages"],
                                  head_major=st["case"]["head_major"])
    return n_live, ref, table, st["k_pages"], st["v_pages"]


def _tokens_first(pages, head_major):
    """The pool as [P, page, Hkv, d]."""
    return pages.transpose(1, 2) if head_major else pages


def _plain_attention(st):
    c = st["case"]
    q, lens, table = st["q"], st["lens"].long(), st["table"]
    B, Hkv, G, d, page = c["B"], c["Hkv"], c["G"], c["d"], c["page"]
    t = torch.arange(table.shape[1] * page, device=q.device)
    seen = t < lens[:, None]                                                     # [B, T]
    if c["window"]:
        seen &= t >= lens[:, None] - c["window"]
    ids = table.clamp(min=0).long()

    def tokens(pages):                                                           # [B, Hkv, T, d]
        x = _tokens_first(pages, c["head_major"])[ids].reshape(B, -1, Hkv, d)
        return x.transpose(1, 2).float()

    s = q.float().view(B, Hkv, G, d) @ tokens(st["k_pages"]).transpose(2, 3) * d ** -0.5
    s = s.masked_fill(~seen[:, None, None], -math.inf)                           # [B, Hkv, G, T]
    m = s.amax(-1, keepdim=True)
    m = torch.where(lens.view(B, 1, 1, 1) > 0, m, torch.zeros_like(m))
    p = torch.exp(s - m)
    z = p.sum(-1, keepdim=True)
    o = p @ tokens(st["v_pages"]).masked_fill(~seen[:, None, :, None], 0.0) / z
    o = torch.where(lens.view(B, 1, 1, 1) > 0, o, torch.zeros_like(o))
    o = o.reshape(B, Hkv * G, d).to(q.dtype)
    return (o, (m + torch.log(z)).reshape(B, Hkv * G)) if c["lse"] else o


def _plain_append(st):
    c = st["case"]
    k, v, pos, table, page = st["k"], st["v"], st["pos"].long(), st["table"], c["page"]
    i = torch.arange(k.shape[0], device=k.device)
    if st["cu"] is None:
        b, at, keep = i, pos, pos >= 0
    else:
        b = torch.searchsorted(st["cu"], i, right=True) - 1
        at, keep = pos[b] + i - st["cu"][b], pos[b] >= 0
    b, at, k, v = b[keep], at[keep], k[keep], v[keep]
    ids = table[b, at // page].long()
    _tokens_first(st["k_pages"], c["head_major"])[ids, at % page] = k
    _tokens_first(st["v_pages"], c["head_major"])[ids, at % page] = v
    return st["k_pages"], st["v_pages"]


def _plain_resize(st):
    c = st["case"]
    lens, ref, table = _views(st)
    page, (S, width) = c["page"], table.shape
    n0 = lens.long()
    n1 = (n0 + st["delta"]).clamp(min=0)
    c0, c1 = (n0 + page - 1) // page, (n1 + page - 1) // page
    last = table.gather(1, (c0 - 1).clamp(min=0)[:, None])[:, 0].long()
    grow = n1 > n0
    fits = n1 <= width * page
    cow = grow & fits & (n0 % page > 0) & (ref[last.clamp(min=0)] > 1)
    need = torch.where(grow & fits, c1 - c0 + cow, torch.zeros_like(c0))
    upto = need.cumsum(0)
    free = (ref == 0).nonzero()[:, 0]
    done = grow & fits & ((need == 0) | (upto <= free.numel()))
    cow &= done
    # the lowest free pages, row by row
    j = torch.arange(width, device=lens.device)
    lo = c0 - cow.long()
    new = done[:, None] & (j >= lo[:, None]) & (j < c1[:, None])
    gone = (n1 < n0)[:, None] & (j >= c1[:, None]) & (j < c0[:, None])
    dropped = table[gone].long()
    rows = cow.nonzero()[:, 0]
    table[new] = free[:new.sum()].int()
    table[gone] = -1
    ref[table[new].long()] = 1
    ref.index_add_(0, dropped, torch.full_like(dropped, -1, dtype=torch.int32))
    ref.index_add_(0, last[rows], torch.full_like(rows, -1, dtype=torch.int32))
    # copy on write: the rows in use of a shared last page
    to = table[rows, lo[rows]].long()
    used = (torch.arange(page, device=lens.device) < (n0 % page)[rows, None])[:, :, None, None]
    for_k, for_v = (_tokens_first(st[x], c["head_major"]) for x in ("k_pages", "v_pages"))
    for_k[to] = torch.where(used, for_k[last[rows]], for_k[to])
    for_v[to] = torch.where(used, for_v[last[rows]], for_v[to])
    pos = torch.where(done, n0, torch.full_like(n0, -1)).int()
    lens.copy_(torch.where(done | (n1 < n0), n1, n0))
    return pos, lens, ref, table, st["k_pages"], st["v_pages"]


def _plain_fork(st):
    lens, ref, table = _views(st)
    src, dst, page = st["src"].long(), st["dst"].long(), st["case"]["page"]
    held = torch.arange(table.shape[1], device=lens.device) < \
        ((lens[src].long() + page - 1) // page)[:, None]
    rows = table[src]
    ids = rows[held].long()
    ref.index_add_(0, ids, torch.ones_like(ids, dtype=torch.int32))
    table[dst] = torch.where(held, rows, table[dst])
    lens[dst] = lens[src]
    return lens, ref, table


def _plain_compact(st):
    c = st["case"]
    lens, ref, table = _views(st)
    i = torch.arange(ref.numel(), device=ref.device)
    live = ref > 0
    n_live = live.sum()
    frm, to = (live & (i >= n_live)).nonzero()[:, 0], (~live & (i < n_live)).nonzero()[:, 0]
    st["k_pages"][to] = st["k_pages"][frm]
    st["v_pages"][to] = st["v_pages"][frm]
    ref[to] = ref[frm]
    ref[frm] = 0
    where = i.clone()
    where[frm] = to
    held = torch.arange(table.shape[1], device=lens.device) < \
        ((lens.long() + c["page"] - 1) // c["page"])[:, None]
    table.copy_(torch.where(held, where[table.clamp(min=0).long()].int(), table))
    return n_live.int().view(1), ref, table, st["k_pages"], st["v_pages"]


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    op, page = case["op"], case["page"]
    es = 2 if case.get("dtype") == "bf16" else 4
    row = 2 * case.get("Hkv", 0) * case.get("d", 0) * es             # a token's key and value
    if op == "attention":
        lens = _attention_lengths(case)
        n = np.minimum(lens, case["window"]) if case["window"] else lens
        Hq = case["Hkv"] * case["G"]
        pages = (lens + page - 1) // page - (lens - n) // page
        out = case["B"] * Hq * (2 * case["d"] * es + (4 if case["lse"] else 0))
        return dict(bytes=int(n.sum()) * row + int(pages.sum()) * 4 + case["B"] * 4 + out,
                    flops=4 * int(n.sum()) * Hq * case["d"])
    if op == "append":
        new, _ = _append_lengths(case)
        return dict(bytes=int(new.sum()) * (2 * row) + 8 * case["B"], flops=0)
    if op == "resize":
        lens, delta, first = _resize_plan(case)
        n1 = np.maximum(lens + delta, 0)
        c0, c1 = (lens + page - 1) // page, (n1 + page - 1) // page
        beams = np.bincount(first, minlength=case["S"])[first]
        cow = (n1 > lens) & (lens % page > 0) & (beams > 1)
        taken, dropped = np.maximum(c1 - c0, 0).sum() + cow.sum(), np.maximum(c0 - c1, 0).sum()
        return dict(bytes=int(4 * case["P"] + 16 * case["S"] + 8 * taken + 16 * dropped
                              + 2 * row * (lens % page)[cow].sum()), flops=0)
    if op == "fork":
        lens, src, _ = _fork_plan(case)
        held = (lens[src] + page - 1) // page
        # the parents' entries read once and the children's written; the counts read and written
        once = (lens + page - 1) // page
        return dict(bytes=int(4 * once.sum() + 4 * held.sum() + 8 * once[np.unique(src)].sum()
                              + 12 * case["n"]), flops=0)
    # which pages move follows from the seed; on average the share of pages in use that lie past
    # the front of the pool
    moved = int(case["live"] * (1 - case["live"] / case["P"]))
    return dict(bytes=4 * case["P"] + 8 * case["live"] + 2 * moved * (page * row + 4), flops=0)


# ---------------------------------------------------------------------------------------------
# the definitions, in 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    return globals()["_exact_" + case["op"]](case, st)


def _slots(st, case, s, a, b):
    """Tokens a .. b-1 of sequence s as (page, slot) index tensors."""
    t = torch.arange(a, b, device="cuda")
    return st["table"][s].long()[t // case["page"]], t % case["page"]


def _exact_attention(case, st):
    B, Hkv, G, d = (case[x] for x in ("B", "Hkv", "G", "d"))
    o = torch.zeros((B, Hkv * G, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hkv * G), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_attention_lengths(case).tolist()):
        if n == 0:
            continue
        pg, sl = _slots(st, case, b, max(0, n - case["window"]) if case["window"] else 0, n)
        for h in range(Hkv):
            at = (pg, h, sl) if case["head_major"] else (pg, sl, h)
            w = st["q"][b, h * G:(h + 1) * G].double() @ st["k_pages"][at].double().T / math.sqrt(d)
            lse[b, h * G:(h + 1) * G] = torch.logsumexp(w, 1)
            o[b, h * G:(h + 1) * G] = torch.softmax(w, 1) @ st["v_pages"][at].double()
    return (o, lse) if case["lse"] else o


def _exact_append(case, st):
    new, start = _append_lengths(case)
    i = 0
    for b, n in enumerate(new.tolist()):
        if n:
            src = slice(i, i + n) if case["packed"] else slice(b, b + 1)
            pg, sl = _slots(st, case, b, int(start[b]), int(start[b]) + n)
            for pool, x in ((st["k_pages"], st["k"]), (st["v_pages"], st["v"])):
                if case["head_major"]:
                    pool[pg, :, sl] = x[src]
                else:
                    pool[pg, sl] = x[src]
        i += n
    return st["k_pages"], st["v_pages"]


def _host(st):
    m = st["meta"].cpu().numpy()
    S, P = st["S"], st["P"]
    return m[:S].copy(), m[S:S + P].copy(), m[S + P:].reshape(S, st["width"]).copy()


def _exact_resize(case, st):
    lens, ref, table = _host(st)
    page, width, delta = case["page"], st["width"], st["delta"].cpu().numpy()
    was, free, got = ref.copy(), np.flatnonzero(ref == 0), 0
    pos = np.full(len(lens), -1, np.int32)
    asked = 0
    for s in range(len(lens)):
        n0 = int(lens[s])
        n1 = max(0, n0 + int(delta[s]))
        c0, c1 = -(-n0 // page), -(-n1 // page)
        if n1 < n0:
            np.subtract.at(ref, table[s, c1:c0], 1)
            table[s, c1:c0] = -1
            lens[s] = n1
        elif n1 > n0 and n1 <= width * page:
            copy = n0 % page > 0 and was[table[s, c0 - 1]] > 1
            need = c1 - c0 + copy
            asked += need
            if need and asked > len(free):
                continue
            if copy:
                old, new = int(table[s, c0 - 1]), int(free[got])
                ref[old] -= 1
                for x in ("k_pages", "v_pages"):
                    if case["head_major"]:
                        st[x][new, :, :n0 % page] = st[x][old, :, :n0 % page]
                    else:
                        st[x][new, :n0 % page] = st[x][old, :n0 % page]
            table[s, c0 - copy:c1] = free[got:got + need]
            ref[free[got:got + need]] = 1
            got += need
            pos[s], lens[s] = n0, n1
    return pos, lens, ref, table, st["k_pages"], st["v_pages"]


def _exact_fork(case, st):
    lens, ref, table = _host(st)
    for a, b in zip(st["src"].tolist(), st["dst"].tolist()):
        n = -(-int(lens[a]) // case["page"])
        table[b, :n] = table[a, :n]
        np.add.at(ref, table[a, :n], 1)
        lens[b] = lens[a]
    return lens, ref, table


def _exact_compact(case, st):
    lens, ref, table = _host(st)
    n_live = int((ref > 0).sum())
    frm = [p for p in range(n_live, len(ref)) if ref[p] > 0]
    to = [p for p in range(n_live) if ref[p] == 0]
    where = np.arange(len(ref), dtype=np.int32)
    where[frm] = to
    ref[to], ref[frm] = ref[frm], 0
    for s in range(len(lens)):
        n = -(-int(lens[s]) // case["page"])
        table[s, :n] = where[table[s, :n]]
    f, t = (torch.tensor(x, dtype=torch.int64, device="cuda") for x in (frm, to))
    for x in ("k_pages", "v_pages"):
        st[x].index_copy_(0, t, st[x].index_select(0, f))
    return np.array([n_live], np.int32), ref, table, st["k_pages"], st["v_pages"]
