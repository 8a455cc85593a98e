"""The paged key-value cache at the sizes where its kernels change their ways: many rows that copy at
once, pages of several copy steps, page counts at every alignment, forks with counts added once or
one by one, every number of query rows a pass, sequences in one part and in hundreds, and calls
queued without a wait in between."""
import numpy as np
import pytest
import torch

from paged_model import Cache, attention
from parity import bf16_half_ulp
from test_paged_gpu import BF16, F32, Dev, check, filled, i32, lib, queries, resize

pytestmark = pytest.mark.gpu


# -------------------------------------------------------------------------------- attention


@pytest.mark.parametrize("dtype,d,G", [
    (BF16, 64, 1), (BF16, 64, 8), (BF16, 64, 15), (BF16, 64, 16), (BF16, 64, 17), (BF16, 64, 24),
    (BF16, 128, 8), (BF16, 128, 12), (BF16, 128, 17), (BF16, 128, 24), (BF16, 128, 25),
    (BF16, 128, 32), (BF16, 128, 48),
    (F32, 64, 4), (F32, 64, 5), (F32, 64, 8), (F32, 64, 12), (F32, 64, 16), (F32, 64, 17),
    (F32, 128, 4), (F32, 128, 7), (F32, 128, 9), (F32, 128, 13), (F32, 128, 16), (F32, 128, 24),
])
def test_attention_group_sizes(dtype, d, G):
    """Every number of rows a block works on, as many as it holds, one more, and several passes; two
    kv heads, so that groups lie side by side; sequences that end in one block and ones that do not."""
    lens = [1, 700, 33, 0, 95, 2500]
    c = filled(lens, 16, 2, d, dtype, seed=G + d)
    dev, q = Dev(c), queries(len(lens), 2 * G, d, dtype, seed=G)
    o, lse = dev.decode(q)
    check(c, q, o, lse)
    o, lse = dev.decode(q, window=90)
    check(c, q, o, lse, 90)
    assert int(dev.status) == 0


@pytest.mark.parametrize("dtype,d,G,n", [
    (BF16, 128, 1, 9473), (BF16, 128, 20, 9500), (BF16, 64, 3, 20001), (F32, 64, 2, 9472),
    (F32, 128, 16, 9600), (BF16, 128, 3, 31), (BF16, 128, 3, 33), (BF16, 64, 9, 9471),
])
def test_attention_one_pair_over_all_blocks(dtype, d, G, n):
    """One sequence with one kv head: up to 296 parts (and, with few keys, blocks without any)."""
    c = filled([n], 32, 1, d, dtype, seed=n)
    dev, q = Dev(c), queries(1, G, d, dtype, seed=n)
    o, lse = dev.decode(q)
    check(c, q, o, lse)


@pytest.mark.parametrize("seed", range(6))
def test_attention_borders(seed):
    """Lengths around the borders of tiles, units and blocks, many pairs a block and pairs that end
    with a block, in batches of every density."""
    rng = np.random.default_rng(seed)
    B = [1, 3, 20, 70, 130, 300][seed]
    near = np.array([1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 96, 127, 128, 129, 0, 512])
    lens = rng.choice(near, B) + (rng.random(B) < 0.1) * rng.integers(0, 900, B)
    H, G, d = [(8, 3, 128), (3, 8, 64), (4, 1, 128), (1, 5, 64), (2, 12, 128), (1, 2, 64)][seed]
    dtype = F32 if seed in (2, 5) else BF16
    c = filled(lens.tolist(), [16, 8, 32, 1, 16, 64][seed], H, d, dtype, seed=40 + seed)
    dev, q = Dev(c, seed % 2 == 1), queries(B, H * G, d, dtype, seed)
    o, lse = dev.decode(q)
    check(c, q, o, lse)


@pytest.mark.parametrize("dtype,H,G,d,page,hm,window", [
    (BF16, 8, 3, 128, 16, False, 0), (BF16, 4, 8, 64, 8, True, 0), (BF16, 3, 16, 64, 32, False, 30),
    (BF16, 5, 24, 64, 16, False, 0), (BF16, 6, 1, 128, 1, True, 100), (F32, 4, 4, 128, 16, False, 0),
    (F32, 3, 7, 128, 8, True, 0), (F32, 4, 12, 64, 16, False, 50), (F32, 3, 20, 64, 64, False, 0),
    (BF16, 3, 12, 128, 16, False, 0), (F32, 3, 16, 128, 16, False, 0), (BF16, 4, 40, 64, 16, True, 0),
])
def test_attention_many_short_pairs(dtype, H, G, d, page, hm, window):
    """Hundreds of short sequences, of every length around what a warp takes on by itself, among
    empty ones and long ones; then few short ones among many long, and only short ones."""
    rng = np.random.default_rng(H * G + d)
    tile = (32 if d == 64 else 16) // (2 if dtype == F32 else 1)
    most = 8 * tile
    near = np.array([1, 2, tile - 1, tile, tile + 1, 3 * tile + 1, most - 1, most, most + 1, most + 7])
    for mix in range(3):
        B = 330
        lens = rng.choice(near if mix < 2 else near[:8], B)
        if mix == 0:
            lens[rng.random(B) < 0.1] = 0
            lens[rng.permutation(B)[:5]] = rng.integers(500, 3000, 5)
        if mix == 1:
            lens[rng.random(B) < 0.8] = most + 5
        c = filled(lens.tolist(), page, H, d, dtype, seed=70 + mix)
        dev, q = Dev(c, hm), queries(B, H * G, d, dtype, mix)
        o, lse = dev.decode(q, window=window)
        check(c, q, o, lse, window)
        again, _ = dev.decode(q, window=window)
        assert torch.equal(o, again) and int(dev.status) == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_short_pairs_bad_pages(dtype):
    """Bad pages and lengths in sequences that single warps work on: left out and reported."""
    G = lib()
    c = filled([20] * 300, 8, 2, 64, dtype, seed=80)
    dev, q = Dev(c), queries(300, 6, 64, dtype, 80)
    dev.table[7, 1], dev.table[250, 2] = -1, len(c.ref)
    dev.table[9, 0], dev.lens[9] = 10 ** 9, 8          # no key left
    dev.lens[100] = -4
    status = dev.status
    o, lse = dev.decode(q)
    assert G.gret_paged_status(status) == G.GRET_PAGED_BAD_PAGE | G.GRET_PAGED_BAD_LENGTH
    same = [s for s in range(300) if s not in (7, 9, 100, 250)]
    check(c, q, o, lse, rows=same)
    assert (o[100] == 0).all() and (lse[100] == -float("inf")).all()
    assert torch.isnan(o[9]).all() and (lse[9] == -float("inf")).all()
    for s, keep in ((7, np.r_[0:8, 16:20]), (250, np.r_[0:16])):
        k, v = c.tokens(s, 0, 20)
        ro, rl, eo, el = attention(q[s].cpu(), k[keep], v[keep], 64 ** -0.5)
        half = torch.from_numpy(bf16_half_ulp(ro.numpy()) * 2) if dtype == BF16 \
            else ro.abs() * 2.0 ** -24
        assert ((o[s].cpu().double() - ro).abs() <= eo + half).all()
        assert ((lse[s].cpu().double() - rl).abs() <= el).all()


# -------------------------------------------------------------------------------- upkeep


@pytest.mark.parametrize("dtype,S,beam,H,d,page,hm", [
    (BF16, 256, 4, 8, 128, 16, False), (BF16, 700, 5, 3, 64, 16, True), (F32, 300, 2, 2, 128, 32, True),
    (F32, 520, 40, 1, 16, 64, False), (BF16, 40, 3, 5, 48, 128, False),
])
def test_resize_many_copies(dtype, S, beam, H, d, page, hm):
    """Hundreds of rows leave shared pages of several copy steps in one call, beside rows that do
    not grow; and once more, when the copies are nobody else's."""
    rng = np.random.default_rng(S)
    lens = np.repeat(rng.integers(1, 3 * page, -(-S // beam)), beam)[:S]
    lens[rng.random(S) < 0.1] = 0                     # idle rows among them
    first = np.arange(S) // beam * beam
    lens[first[lens[first] == 0]] = 0
    lens = np.where(lens[first] == 0, 0, lens)
    parents = np.where(first == np.arange(S), lens, 0)
    c = filled(parents.tolist(), page, H, d, dtype, seed=S, spare=3 * S)
    c.table = np.concatenate([c.table, np.full((S, 2), -1, np.int32)], 1)
    c.W += 2
    for s in np.flatnonzero((first != np.arange(S)) & (lens > 0)):
        n = c.pages(lens[s])
        c.table[s], c.lens[s] = c.table[first[s]], lens[s]
        c.ref[c.table[s, :n]] += 1
    dev = Dev(c, hm)
    delta = np.where(rng.random(S) < 0.8, rng.integers(0, page + 2, S), -rng.integers(1, page, S))
    resize(dev, c, delta)
    resize(dev, c, np.ones(S, int))


@pytest.mark.parametrize("off", range(4))
@pytest.mark.parametrize("P", [1, 2, 3, 5, 127, 4095, 16387, 600000])
def test_pool_alignments(off, P):
    """ref at each place within 16 bytes, pools whose last pages do not fill a load."""
    rng = np.random.default_rng(P + off)
    S = 4
    c = Cache(S=S, W=min(P, 3000) + 1, P=P, page=1, H=1, d=8, dtype=BF16)
    taken = rng.random(P) < 0.3
    c.ref[taken] = 1                                  # held by nobody in the table
    dev = Dev(c)
    wide = torch.full((P + 8,), 0, dtype=torch.int32, device="cuda")      # zeros around: free, if read
    dev.ref = wide[off:off + P]
    dev.ref.copy_(i32(c.ref))
    free = min(int((~taken).sum()), 3000)             # of it, what a row's table holds
    resize(dev, c, [free // 7, 0, free // 5, free // 3])
    resize(dev, c, [-(free // 9), free // 11, 0, -free])
    n = lib().gret_paged_compact(dev.lens, dev.table, dev.ref, dev.k, dev.v, status=dev.status)
    assert int(n) == c.compact()
    dev.same_as(c)
    assert int(wide[:off].sum()) == 0 and int(wide[off + P:].sum()) == 0 and int(dev.status) == 0


@pytest.mark.parametrize("parents,children,pages", [
    (1, 1, 5000), (2, 3, 9000), (3, 40, 4097), (2, 1300, 120), (5, 60, 2000), (4, 64, 76),
    (4, 600, 4000), (1, 1, 9000),
])
def test_fork_kinds(parents, children, pages):
    """Few long rows, many short ones, and pairs that are refused among those that share a source."""
    rng = np.random.default_rng(pages)
    S = parents + children + 3
    c = Cache(S=S, W=pages, P=2 * parents * pages, page=4, H=1, d=8, dtype=F32)
    ids = rng.permutation(len(c.ref))
    for s in range(parents):
        c.lens[s] = rng.integers(pages * 2, pages * 4 + 1)
        n = c.pages(c.lens[s])
        c.table[s, :n] = ids[s * pages:s * pages + n]
        if s:                                         # a prefix shared by all parents
            c.table[s, :n // 3] = c.table[0, :n // 3] if n // 3 <= c.pages(c.lens[0]) else ids[:n // 3]
    np.add.at(c.ref, c.table[c.table >= 0], 1)
    c.lens[S - 1] = 1                                 # not empty, and holds a page of its own
    c.table[S - 1, 0] = ids[-1]
    c.ref[ids[-1]] += 1
    dev = Dev(c)
    src = rng.integers(0, parents, children + 4)
    dst = np.concatenate([parents + rng.permutation(children), [S - 1, parents, S, 0 if parents > 2 else -1]])
    order = rng.permutation(children + 4)
    src, dst = src[order], dst[order]
    seen, ok = set(), []
    for i, (s, t) in enumerate(zip(src, dst)):
        ok.append(0 <= t < S and c.lens[t] == 0 and t not in seen and s not in dst)
        seen.add(t)
    lib().gret_paged_fork(i32(src), i32(dst), dev.lens, dev.table, dev.ref, 4, status=dev.status)
    for s, t in zip(src[ok], dst[ok]):
        n = c.pages(c.lens[s])
        c.table[t, :n], c.lens[t] = c.table[s, :n], c.lens[s]
        c.ref[c.table[s, :n]] += 1
    assert not all(ok) and any(ok)
    dev.same_as(c)
    assert lib().gret_paged_status(dev.status) == lib().GRET_PAGED_BAD_ROW


@pytest.mark.parametrize("dtype,H,d,T", [
    (BF16, 8, 128, 9471), (BF16, 8, 128, 9473), (F32, 3, 24, 30001), (BF16, 1, 8, 80000),
    (F32, 2, 64, 1),
])
def test_append_token_counts(dtype, H, d, T):
    """One token a warp and several, with the last warp's not all there; rows cut at random, empty
    ones among them, from inputs that are parts of wider ones."""
    rng = np.random.default_rng(T)
    S, page = 50, 16
    cu = np.sort(np.concatenate([[3 % T, T], rng.integers(3 % T, T + 1, S - 1)]))
    new = np.diff(cu)
    start = rng.integers(0, 40, S)
    c = Cache(S, int((start + new).max()) // page + 2, int(((start + new) // page + 1).sum()), page, H,
              d, dtype)
    at = 0
    for s in range(S):
        n = c.pages(start[s] + new[s])
        c.table[s, :n] = np.arange(at, at + n)
        at += n
    dev = Dev(c)
    kv = torch.randn((T, 2, H, d)).to(dtype)
    pos = np.where(rng.random(S) < 0.1, -1, start)
    for s in range(S):
        if pos[s] >= 0:
            t = pos[s] + np.arange(new[s])
            pg, sl = torch.from_numpy(c.table[s, t // page]).long(), torch.from_numpy(t % page)
            c.k[pg, sl], c.v[pg, sl] = kv[cu[s]:cu[s + 1], 0], kv[cu[s]:cu[s + 1], 1]
    both = kv.cuda()
    lib().gret_paged_append(both[:, 0], both[:, 1], i32(pos), dev.table, dev.k, dev.v,
                            cu_seqlens=i32(cu), status=dev.status)
    dev.same_as(c)
    assert int(dev.status) == 0


# -------------------------------------------------------------------------------- together


def test_queued_calls():
    """Sixty steps of resize, append, fork, compact and attention queued behind one another, each
    call's outputs the next one's inputs, with nothing waited for before the end; on the current
    stream and on one that is given."""
    G = lib()
    S, H, d, page = 40, 2, 64, 8
    for side in (None, torch.cuda.Stream()):
        rng = np.random.default_rng(50)
        c = filled([50, 0, 9] + [0] * (S - 3), page, H, d, BF16, seed=50, spare=400)
        c.table = np.concatenate([c.table, np.full((S, 12), -1, np.int32)], 1)
        c.W += 12
        dev = Dev(c)
        steps = []
        for step in range(60):
            delta = np.where(c.lens > 0, 1, 0)
            if step % 5 == 4:
                delta[rng.integers(0, S, 3)] = -2 ** 31
            if step % 5 == 1:
                delta[0] = 1                          # a new sequence, if the row is idle
            pos, refused = c.resize(delta)
            assert refused == []
            k, v = (torch.randn((S, H, d)).to(BF16) for _ in range(2))
            for s in np.flatnonzero(pos >= 0):
                c.append(s, pos[s], k[s:s + 1], v[s:s + 1])
            src, dst = rng.integers(0, S, 4), rng.integers(0, S, 4)
            c.fork(src.tolist(), dst.tolist())
            if step % 9 == 8:
                c.compact()
            steps.append((i32(delta), k.cuda(), v.cuda(), i32(src), i32(dst), step % 9 == 8))
        q = queries(S, 6, d, BF16, 50)
        torch.cuda.synchronize()
        outs = []
        for delta, k, v, src, dst, compact in steps:
            pos = G.gret_paged_resize(delta, dev.lens, dev.table, dev.ref, dev.k, dev.v, stream=side)
            G.gret_paged_append(k, v, pos, dev.table, dev.k, dev.v, stream=side)
            if side is None:
                del pos                               # its memory may go to the next call
            G.gret_paged_fork(src, dst, dev.lens, dev.table, dev.ref, page, stream=side)
            if compact:
                G.gret_paged_compact(dev.lens, dev.table, dev.ref, dev.k, dev.v, stream=side)
            outs.append(G.gret_paged_attention_decode(q, dev.lens, dev.table, dev.k, dev.v, lse=True,
                                                      stream=side))
        torch.cuda.synchronize()
        dev.same_as(c)
        check(c, q, *outs[-1])


def test_binding_scope():
    """What the binding refuses on a GPU, and that a stream given does not stay current."""
    G = lib()
    c = filled([20], 16, 1, 64, BF16, seed=60)
    dev, q = Dev(c), queries(1, 2, 64, BF16, 60)
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    torch.cuda.synchronize()
    o, none = G.gret_paged_attention_decode(q, dev.lens, dev.table, dev.k, dev.v, stream=side)
    assert none is None and torch.cuda.current_stream() == here
    side.synchronize()
    lse = torch.zeros((1, 2), device="cuda")
    dec = G.gret_paged_attention_decode
    for error, f in [
        (TypeError, lambda: dec(q, dev.lens, dev.table, dev.k, dev.v, stream=3)),
        (TypeError, lambda: dec(q, None, dev.table, dev.k, dev.v)),
        (TypeError, lambda: dec(q, dev.lens, dev.table, dev.k, dev.v, window=1.5)),
        (ValueError, lambda: dec(q, dev.lens, dev.table, dev.k, dev.v, window=2 ** 31)),
        (ValueError, lambda: dec(q, dev.lens.repeat(2), dev.table, dev.k, dev.v)),
        (ValueError, lambda: dec(q, dev.lens, dev.table, dev.k, dev.v, lse=lse[0])),
        (ValueError, lambda: dec(q, dev.lens, dev.table, dev.k, dev.v, lse=lse.cpu())),
        (ValueError, lambda: dec(q, dev.lens, dev.table, dev.k, dev.v, status=dev.ref[:2])),
        (ValueError, lambda: dec(q.transpose(0, 1), dev.lens.repeat(2), dev.table, dev.k, dev.v)),
        (ValueError, lambda: G.gret_paged_resize(dev.lens.long(), dev.lens, dev.table, dev.ref, dev.k,
                                                 dev.v)),
        (ValueError, lambda: G.gret_paged_fork(dev.lens, dev.lens, dev.lens, dev.table, dev.ref, 2 ** 40)),
        (G.GretError, lambda: G.gret_paged_fork(dev.lens, dev.lens, dev.lens, dev.table, dev.ref, 24)),
        (G.GretError, lambda: dec(q, dev.lens, dev.table, dev.k, dev.v, scale=float("inf"))),
    ]:
        with pytest.raises(error):
            f()
    dev.same_as(c)
    o2, got = dec(q, dev.lens, dev.table, dev.k, dev.v, scale=1, lse=lse)   # an integer scale
    assert got is lse
    check(c, q, o2, lse, scale=1)
    check(c, q, o, G.gret_paged_attention_decode(q, dev.lens, dev.table, dev.k, dev.v, lse=True)[1])


@pytest.mark.parametrize("dtype,B,H,G,d", [
    (BF16, 3, 2, 3, 128), (BF16, 250, 4, 5, 64), (F32, 7, 1, 13, 64), (F32, 300, 3, 2, 128),
])
def test_attention_writes_its_outputs_only(dtype, B, H, G, d):
    """o, lse and the workspace lie between bytes that stay as they are, and every value is set."""
    rng = np.random.default_rng(B)
    c = filled(rng.integers(0, 90, B).tolist() + [2000], 16, H, d, dtype, seed=90)
    B += 1
    dev, q = Dev(c), queries(B, H * G, d, dtype, 90)
    need = lib().gret_paged_attention_workspace_size(dtype, H * G, H, d)
    sizes = [q.numel() * q.element_size(), 4 * B * H * G, need]
    bufs = [torch.full((n + 512,), 0x7b, dtype=torch.uint8, device="cuda") for n in sizes]
    o, lse, ws = (b[256:256 + n] for b, n in zip(bufs, sizes))
    o, lse = o.view(dtype).view(q.shape), lse.view(torch.float32).view(B, H * G)
    lib().gret_paged_attention_decode(q, dev.lens, dev.table, dev.k, dev.v, o=o, lse=lse,
                                      workspace=ws)
    check(c, q, o, lse)
    for b, n in zip(bufs, sizes):
        assert (b[:256] == 0x7b).all() and (b[256 + n:] == 0x7b).all()


def test_two_streams_at_once():
    """Decode attention of two caches on two streams, calls of both in flight together, each with its
    own workspace: the outputs are those of one call at a time."""
    G = lib()
    rng = np.random.default_rng(91)
    sets = []
    for seed, (B, H, G_, d, dtype) in enumerate([(300, 4, 3, 128, BF16), (6, 2, 8, 64, F32)]):
        c = filled(rng.integers(1, 120 if B > 99 else 3000, B).tolist(), 16, H, d, dtype, seed=seed)
        dev, q = Dev(c), queries(B, H * G_, d, dtype, seed)
        sets.append((dev, q, dev.decode(q), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(30):
        for i, (dev, q, _, stream) in enumerate(sets):
            outs[i].append(G.gret_paged_attention_decode(q, dev.lens, dev.table, dev.k, dev.v,
                                                         lse=True, stream=stream))
    torch.cuda.synchronize()
    for (_, _, (o, lse), _), many in zip(sets, outs):
        assert all(torch.equal(o, x) and torch.equal(lse, y) for x, y in many)


@pytest.mark.parametrize("P", [500, 140000])
def test_captured_upkeep(P):
    """Resize, fork and compact captured once and replayed on a cache that comes, goes and runs full,
    with the lists of what to do written between the replays."""
    G = lib()
    rng = np.random.default_rng(P)
    S, page, W = 30, 4, 60 if P < 1000 else 5000
    c = Cache(S, W, P, page, 1, 8, BF16, fill=0.0)
    dev = Dev(c)
    delta, pos, src, dst = (i32(np.zeros(n)) for n in (S, S, 4, 4))
    n_live = i32([0])
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda")
          for n in (G.gret_paged_resize_workspace_size(S), G.gret_paged_compact_workspace_size(P))]

    def step():
        G.gret_paged_resize(delta, dev.lens, dev.table, dev.ref, dev.k, dev.v, pos=pos,
                            workspace=ws[0])
        G.gret_paged_fork(src, dst, dev.lens, dev.table, dev.ref, page)
        G.gret_paged_compact(dev.lens, dev.table, dev.ref, dev.k, dev.v, n_live=n_live,
                             workspace=ws[1])

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()                                       # nothing to do: loads the kernels
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    big = 200 if P < 1000 else 15000
    for _ in range(25):
        d = np.where(rng.random(S) < 0.5, rng.integers(-big, big, S), 1)
        s, t = rng.integers(0, S, 4), rng.integers(0, S, 4)
        for x, y in ((delta, d), (src, s), (dst, t)):
            x.copy_(i32(y))
        graph.replay()
        rpos, _ = c.resize(d)
        c.fork(s.tolist(), t.tolist())
        n = c.compact()
        assert np.array_equal(pos.cpu().numpy(), rpos) and int(n_live) == n
        dev.same_as(c)


def test_attention_neighbouring_heads_of_64():
    """Heads of 64 dimensions that lie next to one another: what is not finite in one does not reach
    the other, whichever it is; and pools where they lie apart, or further apart than they are wide."""
    G = lib()
    for H, G_ in ((2, 3), (4, 8), (6, 1)):
        c = filled([100, 3, 2000], 16, H, 64, BF16, seed=95)
        c.v[c.table[0, 2], 5, 0, 7] = float("inf")
        c.v[c.table[2, 9], 1, 1, 63] = float("nan")
        q = queries(3, H * G_, 64, BF16, 95)
        k1 = c.k.clone()
        k1[c.table[0, 1], 3, 1] = float("inf")            # head 1: scores of +-inf or NaN
        dev = Dev(c)
        o, lse = G.gret_paged_attention_decode(q, dev.lens, dev.table, k1.cuda(), dev.v, lse=True)
        assert (o[0, :G_, 7] == float("inf")).all() and torch.isnan(o[2, G_:2 * G_, 63]).all()
        odd = torch.zeros_like(o, dtype=torch.bool)
        odd[0, :G_, 7] = odd[2, G_:2 * G_, 63] = odd[0, G_:2 * G_] = True
        assert torch.isfinite(o[~odd]).all()
        assert torch.isfinite(lse[1:]).all() and torch.isfinite(lse[0, :G_]).all()
    c = filled([700, 0, 33, 64], 16, 4, 64, BF16, seed=96)
    dev, q = Dev(c), queries(4, 20, 64, BF16, 96)
    o, lse = dev.decode(q)
    check(c, q, o, lse)
    for wide in ((16, 4, 128), (16, 4, 64), (20, 6, 72)):
        kw, vw = (torch.full((len(c.ref),) + wide, float("nan"), dtype=BF16, device="cuda")
                  for _ in range(2))
        kw, vw = kw[:, :16, :4, :64], vw[:, :16, :4, :64]
        kw.copy_(dev.k)
        vw.copy_(dev.v)
        o, lse = G.gret_paged_attention_decode(q, dev.lens, dev.table, kw, vw, lse=True)
        check(c, q, o, lse)
