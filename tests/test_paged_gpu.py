"""GPU tests of the paged key-value cache against plain models (paged_model.py): attention of one
new token against 64-bit softmax with a derived error bound, the cache's upkeep exactly."""
import numpy as np
import pytest
import torch

from paged_model import Cache, attention
from parity import bf16_half_ulp

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def lib():
    import gated_retention_linear_b200 as G
    return G


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Dev:
    """A model's cache on the GPU."""

    def __init__(self, c, head_major=False):
        self.hm = head_major
        put = lambda x: (x.transpose(1, 2) if head_major else x).contiguous().cuda()  # noqa: E731
        self.k, self.v = put(c.k), put(c.v)
        self.lens, self.table, self.ref = i32(c.lens), i32(c.table), i32(c.ref)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def same_as(self, c):
        tok = lambda x: (x.transpose(1, 2) if self.hm else x).cpu()  # noqa: E731
        bits = lambda x: x.contiguous().view(torch.uint8)  # noqa: E731  (NaN compare equal)
        assert np.array_equal(self.lens.cpu().numpy(), c.lens)
        assert np.array_equal(self.table.cpu().numpy(), c.table)
        assert np.array_equal(self.ref.cpu().numpy(), c.ref)
        assert torch.equal(bits(tok(self.k)), bits(c.k))
        assert torch.equal(bits(tok(self.v)), bits(c.v))

    def decode(self, q, **kw):
        return lib().gret_paged_attention_decode(q, self.lens, self.table, self.k, self.v,
                                                 head_major=self.hm, status=self.status, lse=True,
                                                 **kw)


def filled(lens, page, H, d, dtype, seed, spare=3, shuffle=True):
    """A cache whose rows hold `lens` random tokens on pages in random order; NaN elsewhere."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    n = [-(-x // page) for x in lens]
    c = Cache(len(lens), max(n) + 1, sum(n) + spare, page, H, d, dtype)
    ids = rng.permutation(len(c.ref)) if shuffle else np.arange(len(c.ref))
    at = 0
    for s, x in enumerate(lens):
        c.lens[s] = x
        c.table[s, :n[s]] = ids[at:at + n[s]]
        at += n[s]
        c.append(s, 0, torch.randn((x, H, d), generator=gen).to(dtype),
                 torch.randn((x, H, d), generator=gen).to(dtype))
    c.ref[ids[:at]] = 1
    return c


def check(c, q, o, lse, window=0, scale=None, rows=None):
    """o and lse of every sequence against the definition, within its bound."""
    d = q.shape[2]
    o, lse, qc = o.cpu(), lse.cpu(), q.cpu()
    for s in range(len(c.lens)) if rows is None else rows:
        n = int(c.lens[s])
        k, v = c.tokens(s, max(0, n - window) if window else 0, n)
        ro, rl, eo, el = attention(qc[s], k, v, d ** -0.5 if scale is None else scale)
        got = o[s].double()
        lim = eo.numpy() + (bf16_half_ulp(np.maximum(ro.abs().numpy(), got.abs().numpy()))
                            if o.dtype == BF16 else ro.abs().numpy() * 2.0 ** -24)
        off = (got - ro).abs().numpy()
        assert (off <= lim).all(), (s, n, float((off - lim).max()))
        if n == 0:
            assert (lse[s] == -float("inf")).all() and (o[s] == 0).all()
        else:
            assert ((lse[s].double() - rl).abs() <= el).all(), (s, n)


def queries(B, Hq, d, dtype, seed, size=1.0):
    gen = torch.Generator().manual_seed(seed + 1000)
    return (torch.randn((B, Hq, d), generator=gen) * size).to(dtype).cuda()


# -------------------------------------------------------------------------------- attention


@pytest.mark.parametrize("dtype,d,H,G,page,lens,window,hm", [
    (BF16, 128, 8, 3, 16, [1, 15, 16, 17, 63, 64, 65, 0, 300], 0, False),
    (BF16, 128, 1, 1, 1, [5, 1, 0, 70], 0, False),              # pages of one token
    (BF16, 64, 3, 8, 8, [129, 31, 1000, 2], 0, True),
    (BF16, 128, 2, 9, 64, [200, 64, 128], 0, False),            # a second group of query rows
    (BF16, 64, 1, 16, 32, [777, 32], 0, False),
    (BF16, 128, 2, 24, 16, [333, 90], 0, True),
    (BF16, 128, 1, 33, 128, [500, 1], 0, False),
    (BF16, 64, 2, 71, 16, [100], 0, False),
    (BF16, 128, 4, 4, 1024, [1500, 1024, 3], 0, False),         # pages longer than a tile
    (BF16, 128, 2, 5, 16, [5000], 0, False),                    # one sequence over many blocks
    (BF16, 128, 2, 3, 16, [400, 99, 100, 101, 7, 0, 1000], 100, False),
    (BF16, 64, 2, 3, 32, [400, 1, 33], 1, True),                # window 1: o = v
    (BF16, 128, 2, 3, 8, [400, 4000], 10 ** 9, False),          # window past every length
    (F32, 64, 4, 4, 32, [1, 7, 64, 65, 0, 1000], 0, False),
    (F32, 128, 2, 3, 16, [500, 17], 0, True),
    (F32, 128, 1, 9, 1, [40], 0, False),
    (F32, 64, 1, 20, 128, [700, 130], 64, False),
    (F32, 128, 8, 1, 16, [3000], 0, False),
])
def test_attention(dtype, d, H, G, page, lens, window, hm):
    c = filled(lens, page, H, d, dtype, seed=len(lens) + d + G)
    dev, q = Dev(c, hm), queries(len(lens), H * G, d, dtype, seed=G)
    o, lse = dev.decode(q, window=window)
    assert int(dev.status) == 0
    check(c, q, o, lse, window)
    o2, lse2 = dev.decode(q, window=window)                     # results do not depend on timing
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    o3, none = lib().gret_paged_attention_decode(q, dev.lens, dev.table, dev.k, dev.v,
                                                 window=window, head_major=hm)
    assert none is None and torch.equal(o, o3)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_large_and_equal_scores(dtype):
    """Scores of several hundred (only the running maximum keeps them finite), a scale of 0 (o is
    the mean of the values) and a negative scale."""
    c = filled([900, 64, 3], 16, 2, 64, dtype, seed=5)
    dev, q = Dev(c), queries(3, 6, 64, dtype, 5, size=40.0)
    for scale in (1.0, 0.0, -0.5):
        o, lse = dev.decode(q, scale=scale)
        check(c, q, o, lse, scale=scale)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F32, 64)])
def test_attention_infinite_scores(dtype, d):
    """Keys that give -inf weigh nothing, wherever they lie and however many there are; a row whose
    every score is -inf gives NaN, as a softmax of it does."""
    lens = [700, 40, 90]
    c = filled(lens, 16, 1, d, dtype, seed=6)
    q = queries(3, 3, d, dtype, 6).abs()
    rng = np.random.default_rng(6)
    gone = [np.r_[0:600], rng.permutation(40)[:39], np.r_[0:90]]
    for s, js in enumerate(gone):
        for j in js:
            c.k[c.table[s, j // 16], j % 16] = -float("inf")
    o, lse = Dev(c).decode(q)
    for s in (0, 1):
        keep = np.setdiff1d(np.arange(lens[s]), gone[s])
        k, v = c.tokens(s, 0, lens[s])
        ro, rl, eo, el = attention(q[s].cpu(), k[keep], v[keep], d ** -0.5)
        lim = eo + torch.from_numpy(bf16_half_ulp(ro.numpy()) * 2) if dtype == BF16 \
            else eo + ro.abs() * 2.0 ** -24
        assert ((o[s].cpu().double() - ro).abs() <= lim).all()
        assert ((lse[s].cpu().double() - rl).abs() <= el).all()
    assert torch.isnan(o[2]).all() and (lse[2] == -float("inf")).all()


def test_attention_values_not_finite():
    """An infinite value of a key with weight, and a NaN in a query, reach the rows they concern
    and no other."""
    c = filled([100, 100], 16, 2, 128, BF16, seed=8)
    c.v[c.table[0, 2], 5, 0, 7] = float("inf")
    q = queries(2, 4, 128, BF16, 8)
    q[1, 3, 0] = float("nan")
    o, lse = Dev(c).decode(q)
    assert (o[0, :2, 7] == float("inf")).all() and torch.isnan(o[1, 3]).all()
    o[0, :2, 7], q[1, 3, 0] = 0, 0
    assert torch.isfinite(o[0]).all() and torch.isfinite(o[1, :3]).all()
    assert torch.isfinite(lse[0]).all() and torch.isfinite(lse[1, :3]).all()


def test_attention_strides():
    """Keys and values interleaved in one pool, a page table that is a part of a wider one."""
    c = filled([200, 35, 0], 16, 3, 64, BF16, seed=9)
    both = torch.stack([c.k, c.v], 1).cuda()                    # [P, 2, page, H, d]
    wide = torch.full((3, 40), 77777, dtype=torch.int32, device="cuda")
    table = wide[:, 5:5 + c.W]
    table.copy_(i32(c.table))
    q = queries(3, 9, 64, BF16, 9)
    o, lse = lib().gret_paged_attention_decode(q, i32(c.lens), table, both[:, 0], both[:, 1],
                                               lse=True)
    check(c, q, o, lse)


@pytest.mark.parametrize("dtype,d", [(BF16, 64), (F32, 128)])
def test_attention_bad_pages_and_lengths(dtype, d):
    """Pages out of range are left out and reported; a length past the table is cut off there, a
    negative one is 0; pages before the window are not looked at."""
    G = lib()
    c = filled([100, 60, 47, 32], 16, 2, d, dtype, seed=10)
    W = c.W
    c.table[3, 2:] = c.table[0, 2:]                             # so that row 3 has W full pages
    k3 = [c.k.clone(), c.v.clone()]
    q = queries(4, 4, d, dtype, 10)
    dev = Dev(c)
    bad = dev.table.clone()
    bad[0, 1], bad[0, 4], bad[1, 0] = -1, len(c.ref), 2 ** 31 - 1
    lens = dev.lens.clone()
    lens[2] = -5
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = G.gret_paged_attention_decode(q, lens, bad, dev.k, dev.v, status=status, lse=True)
    assert G.gret_paged_status(status) == G.GRET_PAGED_BAD_PAGE | G.GRET_PAGED_BAD_LENGTH
    for s, keep in ((0, np.r_[0:16, 32:64, 80:100]), (1, np.r_[16:60])):
        k, v = c.tokens(s, 0, int(c.lens[s]))
        ro, _, eo, _ = attention(q[s].cpu(), k[keep], v[keep], d ** -0.5)
        half = torch.from_numpy(bf16_half_ulp(ro.numpy()) * 2) if dtype == BF16 \
            else ro.abs() * 2.0 ** -24
        assert ((o[s].cpu().double() - ro).abs() <= eo + half).all()
    assert (o[2] == 0).all() and (lse[2] == -float("inf")).all()
    # behind the window nothing is read
    status.zero_()
    bad = dev.table.clone()
    bad[0, :4], bad[1, :1] = -1, 10 ** 6                        # windows begin at 68 and 28
    lens = dev.lens.clone()
    lens[2:] = 0
    o, lse = G.gret_paged_attention_decode(q, lens, bad, dev.k, dev.v, window=32, status=status,
                                           lse=True)
    assert G.gret_paged_status(status) == 0
    check(c, q, o, lse, 32, rows=[0, 1])
    # a length past the table
    lens = torch.zeros_like(dev.lens)
    lens[0] = 10 ** 9
    row = dev.table.clone()
    row[0] = row[0, 0]
    full, _ = G.gret_paged_attention_decode(q, lens, row, dev.k, dev.v, status=status)
    lens[0] = W * 16
    assert G.gret_paged_status(status) == G.GRET_PAGED_BAD_LENGTH
    want, _ = G.gret_paged_attention_decode(q, lens, row, dev.k, dev.v)
    assert torch.equal(full, want)


def test_attention_far_offsets():
    """Pages past 2^32 bytes and 2^31 elements into the pool."""
    H, d, page, P = 8, 128, 64, 36000                           # 4.7 GB each
    k = torch.empty((P, page, H, d), dtype=BF16, device="cuda")
    v = torch.empty_like(k)
    c = filled([200, 100], page, H, d, BF16, seed=11, spare=0)
    far = np.array([P - 1, P - 7, 32768, 5, 35000, 32767])[:len(c.ref)]
    k[torch.from_numpy(far).cuda()] = c.k.cuda()
    v[torch.from_numpy(far).cuda()] = c.v.cuda()
    table = np.where(c.table >= 0, far[c.table], -1)
    q = queries(2, 24, d, BF16, 11)
    o, lse = lib().gret_paged_attention_decode(q, i32(c.lens), i32(table), k, v, lse=True)
    check(c, q, o, lse)


def test_attention_many_short_and_one_long():
    """600 short sequences around one long one: whole sequences, split ones and empty ones in the
    same call; more sequences than threads of a block."""
    rng = np.random.default_rng(12)
    lens = rng.integers(0, 40, 600)
    lens[300] = 30000
    lens[rng.permutation(600)[:200]] = 0
    c = filled(lens.tolist(), 16, 1, 64, BF16, seed=12)
    dev, q = Dev(c), queries(600, 2, 64, BF16, 12)
    o, lse = dev.decode(q)
    check(c, q, o, lse)


def test_attention_nothing_to_do():
    c = filled([0, 0], 16, 2, 64, BF16, seed=13)
    q = queries(2, 4, 64, BF16, 13)
    o, lse = Dev(c).decode(q)
    assert (o == 0).all() and (lse == -float("inf")).all()
    k = torch.zeros((1, 16, 2, 64), dtype=BF16, device="cuda")
    o, lse = lib().gret_paged_attention_decode(q[:0], i32([]), i32(np.zeros((0, 3))), k, k, lse=True)
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)


def test_attention_buffers_stream_and_refusals():
    """Given outputs and workspace are the ones used; a call on another stream runs there."""
    G = lib()
    c = filled([500, 20], 16, 2, 64, BF16, seed=14)
    dev, q = Dev(c), queries(2, 6, 64, BF16, 14)
    o, lse = torch.empty_like(q), torch.empty((2, 6), device="cuda")
    need = G.gret_paged_attention_workspace_size(BF16, 6, 2, 64)
    ws = torch.full((need + 256,), 0xff, dtype=torch.uint8, device="cuda")
    got = G.gret_paged_attention_decode(q, dev.lens, dev.table, dev.k, dev.v, o=o, lse=lse,
                                        workspace=ws[:need])
    assert got[0] is o and got[1] is lse and (ws[need:] == 0xff).all()
    check(c, q, o, lse)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    o2, _ = G.gret_paged_attention_decode(q, dev.lens, dev.table, dev.k, dev.v, stream=side)
    side.synchronize()
    assert torch.equal(o, o2)
    with pytest.raises(G.GretError):
        G.gret_paged_attention_decode(q, dev.lens, dev.table, dev.k, dev.v, workspace=ws[:64])
    with pytest.raises(G.GretError):
        G.gret_paged_attention_decode(q, dev.lens, dev.table, dev.k, dev.v, window=-1)
    with pytest.raises(ValueError):
        G.gret_paged_attention_decode(q, dev.lens.cpu(), dev.table, dev.k, dev.v)
    with pytest.raises(ValueError):
        G.gret_paged_attention_decode(q, dev.lens, dev.table, dev.k, dev.v, o=o[:1])


# -------------------------------------------------------------------------------- upkeep


@pytest.mark.parametrize("dtype,H,d,page,hm", [
    (BF16, 8, 128, 16, False), (BF16, 3, 64, 8, True), (F32, 1, 8, 4, False), (F32, 2, 128, 32, True),
    (BF16, 1, 64, 1, False),
])
def test_append_packed(dtype, H, d, page, hm):
    """Ragged prompts behind cached tokens, an empty one, a skipped one, tokens before the first
    sequence and behind the last; keys and values are parts of a wider buffer."""
    rng = np.random.default_rng(20)
    start = [0, 5, 33, 0, 16, 7]
    new = [40, 0, 17, 1, 100, 9]
    c = filled([a + b for a, b in zip(start, new)], page, H, d, dtype, seed=20)
    dev = Dev(c, hm)
    lead, tail = 3, 21
    cu = lead + np.concatenate([[0], np.cumsum(new)])
    T = int(cu[-1]) + tail
    qkv = torch.randn((T, 3 * H, d)).to(dtype)
    pos = np.array(start)
    pos[3] = -1
    for s in range(6):
        if pos[s] >= 0:
            c.append(s, pos[s], qkv[cu[s]:cu[s + 1], H:2 * H], qkv[cu[s]:cu[s + 1], 2 * H:])
    x = qkv.cuda()
    lib().gret_paged_append(x[:, H:2 * H], x[:, 2 * H:], i32(pos), dev.table, dev.k, dev.v,
                            cu_seqlens=i32(cu), head_major=hm, status=dev.status)
    dev.same_as(c)
    assert int(dev.status) == 0 and rng is not None


def test_append_one_token_each_and_bad_places():
    G = lib()
    c = filled([17, 1, 16, 40, 33], 16, 2, 64, BF16, seed=21)
    dev = Dev(c)
    W = c.W
    k, v = (torch.randn((5, 2, 64)).to(BF16) for _ in range(2))
    pos = [16, -1, 15, W * 16, 2 ** 31 - 1]                     # skipped: row 1; past the table: 3, 4
    for s in (0, 2):
        c.append(s, pos[s], k[s:s + 1], v[s:s + 1])
    G.gret_paged_append(k.cuda(), v.cuda(), i32(pos), dev.table, dev.k, dev.v, status=dev.status)
    dev.same_as(c)
    assert G.gret_paged_status(dev.status) == G.GRET_PAGED_BAD_LENGTH
    # entries that are no pages
    dev.status.zero_()
    bad = dev.table.clone()
    bad[0, 1], bad[2, 0] = -1, len(c.ref)
    G.gret_paged_append(k.cuda(), v.cuda(), i32([16, -1, 0, -1, -1]), bad, dev.k, dev.v,
                        status=dev.status)
    dev.same_as(c)
    assert G.gret_paged_status(dev.status) == G.GRET_PAGED_BAD_PAGE


def test_append_long():
    """More tokens than one wave of blocks takes, one sequence among many empty ones."""
    S, n, page = 300, 40000, 64
    lens = [0] * S
    lens[200] = n
    c = filled(lens, page, 1, 64, BF16, seed=22)
    dev = Dev(c)
    k, v = (torch.randn((n, 1, 64)).to(BF16) for _ in range(2))
    c.append(200, 0, k, v)
    cu = np.where(np.arange(S + 1) > 200, n, 0)
    lib().gret_paged_append(k.cuda(), v.cuda(), i32([0] * S), dev.table, dev.k, dev.v,
                            cu_seqlens=i32(cu))
    dev.same_as(c)


def resize(dev, c, delta, want_status=0):
    pos = lib().gret_paged_resize(i32(delta), dev.lens, dev.table, dev.ref, dev.k, dev.v,
                                  head_major=dev.hm, status=dev.status)
    rpos, refused = c.resize(delta)
    assert np.array_equal(pos.cpu().numpy(), rpos)
    dev.same_as(c)
    assert lib().gret_paged_status(dev.status) == want_status
    dev.status.zero_()
    return refused


@pytest.mark.parametrize("P", [1, 31, 32, 33, 1000, 8193, 70000])
def test_resize_pool_sizes(P):
    """The pool fills to the last page, refuses more, and takes pages back."""
    G = lib()
    c = Cache(S=5, W=P + 2, P=P, page=2, H=1, d=8, dtype=F32)
    dev = Dev(c)
    assert resize(dev, c, [1, 0, 0, 0, 0]) == []
    assert resize(dev, c, [0, 2 * P, 0, 0, 1], G.GRET_PAGED_NO_PAGES)[0] == 1
    if P > 1:
        assert resize(dev, c, [1, 2 * (P - 1), 0, 0, 0]) == []
    assert (c.ref == 1).all()
    assert resize(dev, c, [0, 0, 1, 0, 0], G.GRET_PAGED_NO_PAGES) == [2]
    assert resize(dev, c, [-2 ** 31, 0, 1, 0, 0], G.GRET_PAGED_NO_PAGES) == [2]   # from the next call on
    assert resize(dev, c, [0, -3, 1, 0, 0]) == []


def test_resize_rows_that_do_not_fit():
    """Greedy in row order: rows that need no page grow all the same; a row past the table is
    refused and asks for nothing; odd deltas."""
    G = lib()
    c = Cache(S=7, W=4, P=10, page=4, H=2, d=8, dtype=BF16)
    dev = Dev(c)
    resize(dev, c, [1, 2, 3, 4, 0, 0, 0])
    both = G.GRET_PAGED_TABLE_FULL | G.GRET_PAGED_NO_PAGES
    # 6 pages are free; rows 1, 2 and 3 ask for 2, 3 and 1 of them, row 5 for a seventh
    assert resize(dev, c, [3, 8, 12, 1, 17, 1, 0], both) == [4, 5]
    assert c.lens.tolist() == [4, 10, 15, 5, 0, 0, 0]
    # all 10 pages are held: row 2 stays within its last one, rows 5 and 6 find none
    assert resize(dev, c, [2 ** 31 - 1, -2 ** 31, 1, -4, -1, 4, 5], both) == [0, 5, 6]


def test_resize_copy_on_write():
    """Rows that share a partly filled page part when they grow, one or all at once; full shared
    pages stay shared; a row shrunk into a shared page gets its own copy when it grows again."""
    c = Cache(S=6, W=8, P=40, page=8, H=2, d=16, dtype=BF16)
    dev = Dev(c)
    resize(dev, c, [21, 16, 0, 0, 0, 0])
    for s, n in ((0, 21), (1, 16)):
        k, v = (torch.randn((n, 2, 16)).to(BF16) for _ in range(2))
        c.append(s, 0, k, v)
    dev = Dev(c)
    lib().gret_paged_fork(i32([0, 0, 1]), i32([2, 3, 4]), dev.lens, dev.table, dev.ref, 8)
    c.fork([0, 0, 1], [2, 3, 4])
    dev.same_as(c)
    resize(dev, c, [0, 0, 1, 0, 1, 0])           # row 2 leaves page 2; row 4 needs a new page only
    assert c.ref[c.table[0, 2]] == 2
    resize(dev, c, [1, 0, 0, 9, 0, 0])           # the last two leave at once: the page is free
    assert (c.ref >= 0).all() and c.ref[2] == 0
    resize(dev, c, [-13, 0, -22 + 3, 0, 0, 0])   # into shared pages
    resize(dev, c, [4, 0, 40, 0, 0, 30])
    resize(dev, c, [-100] * 6)
    assert (c.ref == 0).all() and (c.table == -1).all()


def test_resize_many_rows_and_large_pool():
    """16384 rows, the most a table may have; and a pool of a million pages."""
    rng = np.random.default_rng(23)
    for S, P in ((16384, 40000), (3, 1 << 20)):
        c = Cache(S=S, W=12, P=P, page=1, H=1, d=8, dtype=BF16)
        c.ref[rng.random(P) < 0.5] = 1               # held by nobody in the table
        dev = Dev(c)
        resize(dev, c, rng.integers(0, 3, S))
        # 20000 of 40000 pages are taken by nobody's rows, 16384 by the first call on average: the
        # second one runs out of pages
        refused = resize(dev, c, rng.integers(-3, 3, S), lib().GRET_PAGED_NO_PAGES if S > 3 else 0)
        assert bool(refused) == (S > 3)


def test_resize_bad_state():
    """Lengths that the table cannot hold, entries that are no pages and counts that are 0 already
    are reported and left alone."""
    G = lib()
    c = filled([10, 20, 30, 5], 8, 1, 8, F32, seed=24)
    dev = Dev(c)
    dev.lens[0], dev.lens[3] = -3, 10 ** 6
    dev.table[1, 2] = len(c.ref)
    dev.ref[int(c.table[2, 3])] = 0
    before = dev.table.clone()
    pos = G.gret_paged_resize(i32([5, -20, -30, -5]), dev.lens, dev.table, dev.ref, dev.k, dev.v,
                              status=dev.status)
    assert G.gret_paged_status(dev.status) == \
        G.GRET_PAGED_BAD_LENGTH | G.GRET_PAGED_BAD_PAGE | G.GRET_PAGED_BAD_COUNT
    assert pos.tolist() == [-1] * 4 and dev.lens.tolist() == [-3, 0, 0, 10 ** 6]
    assert torch.equal(dev.table[0], before[0]) and torch.equal(dev.table[3], before[3])
    ref = np.zeros(len(c.ref), int)
    ref[c.table[0, :2]] = 1
    ref[c.table[3, 0]] = ref[c.table[1, 2]] = 1       # the entry that named it is gone
    assert np.array_equal(dev.ref.cpu().numpy(), ref)


def test_fork():
    G = lib()
    lens = [100, 0, 0, 37, 0, 1, 0, 0, 0]
    c = filled(lens, 16, 1, 8, F32, seed=25)
    dev = Dev(c)
    src = [0, 3, 0, 0, 1, 5, 9, 3, 3, -1, 3, 0]
    dst = [1, 1, 3, 2, 4, 6, 7, -1, 8, 8, 3, 1]
    refused = c.fork(src, dst)
    G.gret_paged_fork(i32(src), i32(dst), dev.lens, dev.table, dev.ref, 16, status=dev.status)
    dev.same_as(c)
    assert G.gret_paged_status(dev.status) == G.GRET_PAGED_BAD_ROW and len(refused) > 5


def test_fork_many_children():
    """1500 children of three parents of up to 3000 pages."""
    c = filled([3000, 1, 2500] + [0] * 1500, 1, 1, 8, F32, seed=26, spare=0)
    dev = Dev(c)
    src = np.random.default_rng(26).integers(0, 3, 1500)
    dst = 3 + np.random.default_rng(27).permutation(1500)
    lib().gret_paged_fork(i32(src), i32(dst), dev.lens, dev.table, dev.ref, 1, status=dev.status)
    for s in range(3):                                # as Cache.fork, without its loops
        rows, n = dst[src == s], int(c.lens[s])
        c.table[rows, :n] = c.table[s, :n]
        c.lens[rows] = n
        c.ref[c.table[s, :n]] += len(rows)
    dev.same_as(c)
    assert int(dev.status) == 0


@pytest.mark.parametrize("dtype,P,page,H,d,share,hm", [
    (BF16, 200, 16, 8, 128, 0.5, False), (F32, 33, 4, 1, 8, 0.3, True), (BF16, 1, 8, 1, 64, 1.0, False),
    (BF16, 40, 8, 2, 64, 0.0, False), (F32, 64, 2, 3, 16, 1.0, True), (BF16, 9000, 1, 1, 8, 0.7, False),
    (BF16, 500, 8, 1, 64, 0.02, True),
])
def test_compact(dtype, P, page, H, d, share, hm):
    n = int(P * share)
    lens = [0] * 7
    for i in range(n):
        lens[i % 6] += page
    lens = [max(0, x - 1) if page > 1 else x for x in lens]
    n = sum(-(-x // page) for x in lens)
    c = filled(lens, page, H, d, dtype, seed=P, spare=P - n)
    dev = Dev(c, hm)
    c.fork([0], [6])
    lib().gret_paged_fork(i32([0]), i32([6]), dev.lens, dev.table, dev.ref, page)
    got = lib().gret_paged_compact(dev.lens, dev.table, dev.ref, dev.k, dev.v, head_major=hm,
                                   status=dev.status)
    assert int(got) == c.compact() == n
    dev.same_as(c)
    assert int(dev.status) == 0
    lib().gret_paged_compact(dev.lens, dev.table, dev.ref, dev.k, dev.v, head_major=hm)
    dev.same_as(c)                                    # nothing left to do


def test_compact_bad_state():
    G = lib()
    c = filled([40, 20], 8, 1, 8, F32, seed=28, spare=20)
    dev = Dev(c)
    dev.table[0, 1], dev.table[0, 2], dev.lens[1] = 10 ** 6, -7, 10 ** 6
    dev.ref.zero_()
    dev.ref[int(c.table[0, 0])] = 1
    before = dev.table.clone()
    n = G.gret_paged_compact(dev.lens, dev.table, dev.ref, dev.k, dev.v, status=dev.status)
    flags = G.gret_paged_status(dev.status)
    assert int(n) == 1 and int(dev.table[0, 0]) == 0
    assert flags & G.GRET_PAGED_BAD_PAGE and flags & G.GRET_PAGED_BAD_LENGTH
    before[0, 0] = 0
    assert torch.equal(dev.table, before)             # entries of free pages stay as they are


# -------------------------------------------------------------------------------- together


@pytest.mark.parametrize("dtype,H,G_,d,page,hm,seed", [
    (BF16, 8, 3, 128, 16, False, 1), (BF16, 2, 8, 64, 4, True, 2), (F32, 2, 2, 64, 8, False, 3),
])
def test_serving(dtype, H, G_, d, page, hm, seed):
    """Requests come, share prompts, grow token by token, are rolled back and leave, on a pool that
    runs full and is compacted: after every call the cache is the model's, every decode's output
    is within its bound."""
    G = lib()
    rng = np.random.default_rng(seed)
    S, P, W = 9, 60, 14
    c = Cache(S, W, P, page, H, d, dtype)
    dev, shared = Dev(c, hm), 0
    for step in range(40):
        delta = np.where(c.lens > 0, 1, 0)
        for s in range(S):
            x = rng.random()
            if c.lens[s] == 0 and x < 0.4:
                delta[s] = rng.integers(1, 6 * page)
            elif x < 0.05:
                delta[s] = -2 ** 31
            elif x < 0.15:
                delta[s] = -rng.integers(1, page + 2)
        pos = G.gret_paged_resize(i32(delta), dev.lens, dev.table, dev.ref, dev.k, dev.v,
                                  head_major=hm)
        rpos, _ = c.resize(delta)
        assert np.array_equal(pos.cpu().numpy(), rpos)
        new = np.where(rpos >= 0, c.lens - rpos, 0)
        cu = np.concatenate([[0], np.cumsum(new)])
        k, v = (torch.randn((int(cu[-1]), H, d)).to(dtype) for _ in range(2))
        for s in range(S):
            c.append(s, rpos[s], k[cu[s]:cu[s + 1]], v[cu[s]:cu[s + 1]])
        G.gret_paged_append(k.cuda(), v.cuda(), pos, dev.table, dev.k, dev.v, cu_seqlens=i32(cu),
                            head_major=hm)
        if step % 3 == 0:
            src = rng.integers(0, S, 3)
            dst = rng.integers(0, S, 3)
            G.gret_paged_fork(i32(src), i32(dst), dev.lens, dev.table, dev.ref, page)
            c.fork(src.tolist(), dst.tolist())
        if step % 7 == 6:
            n = G.gret_paged_compact(dev.lens, dev.table, dev.ref, dev.k, dev.v, head_major=hm)
            assert int(n) == c.compact()
        dev.same_as(c)
        q = queries(S, H * G_, d, dtype, step)
        w = (0, 10)[step % 2]
        o, lse = dev.decode(q, window=w)
        check(c, q, o, lse, w)
        shared = max(shared, int(c.ref.max()))
    assert shared > 1 and int(dev.status) == 0        # the story had pages that are shared


def test_captured_step():
    """A decode step (resize, append, attention) captured once and replayed on a cache that grows,
    beside a second graph that uses the same workspace; the replays equal uncaptured calls."""
    G = lib()
    H, d, page, S = 2, 64, 8, 4
    c = filled([30, 7, 0, 16], page, H, d, BF16, seed=30, spare=30)
    c.table = np.concatenate([c.table, np.full((S, 20), -1, np.int32)], 1)
    c.W += 20
    dev = Dev(c)
    delta = i32([1, 1, 0, 1])
    k, v = (torch.zeros((S, H, d), dtype=BF16, device="cuda") for _ in range(2))
    q = queries(S, 6, d, BF16, 30)
    o, o2 = torch.zeros_like(q), torch.zeros_like(q)
    pos = torch.zeros(S, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(G.gret_paged_attention_workspace_size(BF16, 6, H, d),
                         G.gret_paged_resize_workspace_size(S)), dtype=torch.uint8, device="cuda")

    def step():
        G.gret_paged_resize(delta, dev.lens, dev.table, dev.ref, dev.k, dev.v, pos=pos,
                            workspace=ws, status=dev.status)
        G.gret_paged_append(k, v, pos, dev.table, dev.k, dev.v, status=dev.status)
        G.gret_paged_attention_decode(q, dev.lens, dev.table, dev.k, dev.v, o=o, workspace=ws,
                                      status=dev.status)

    def narrow():
        G.gret_paged_attention_decode(q, dev.lens, dev.table, dev.k, dev.v, o=o2, workspace=ws,
                                      window=5)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        narrow()                                     # loads the kernels before the capture
    side.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    with torch.cuda.graph(graphs[0]):
        step()
    with torch.cuda.graph(graphs[1]):
        narrow()
    for t in range(20):
        kn, vn = (torch.randn((S, H, d)).to(BF16) for _ in range(2))
        k.copy_(kn)
        v.copy_(vn)
        graphs[0].replay()
        graphs[1].replay()
        rpos, _ = c.resize([1, 1, 0, 1])
        for s in (0, 1, 3):
            c.append(s, rpos[s], kn[s:s + 1], vn[s:s + 1])
        dev.same_as(c)
        for out, w in ((o, 0), (o2, 5)):
            want, lse = dev.decode(q, window=w)
            assert torch.equal(out, want)
            check(c, q, want, lse, w)
    assert int(dev.status) == 0
