"""What the upkeep of the paged cache reports, and leaves out, where a row holds a page that is none
or whose count says that nobody holds it."""
import numpy as np
import pytest
import torch

from test_paged_gpu import BF16, F32, Dev, filled, i32, lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("S", [5, 2000])
def test_resize_bad_last_page(S):
    """A row whose partly filled last page is no page, or is counted as free, is not grown and asks
    for nothing; one that does not write to such a page (it is full, or the row stays or shrinks) is
    not looked at.  The other rows get their pages."""
    G = lib()
    lens = ([10, 20, 30, 16, 5] * S)[:S]
    c = filled(lens, 8, 1, 8, F32, seed=31, spare=S + 9)
    c.table = np.concatenate([c.table, np.full((S, 1), -1, np.int32)], 1)
    c.W += 1
    last = lambda s: int(c.table[s, c.pages(lens[s]) - 1])  # noqa: E731
    delta = [7, 6, 5, 4, 0] + [1] * (S - 5)
    dev = Dev(c)
    dev.table[0, 1], dev.ref[last(1)], dev.ref[last(2)], dev.ref[last(3)] = -1, 0, -2, 0
    before = dev.ref.cpu().numpy()
    want_table = dev.table.cpu().numpy()
    pos = G.gret_paged_resize(i32(delta), dev.lens, dev.table, dev.ref, dev.k, dev.v,
                              status=dev.status)
    assert G.gret_paged_status(dev.status) == G.GRET_PAGED_BAD_PAGE | G.GRET_PAGED_BAD_COUNT
    assert pos[:5].tolist() == [-1, -1, -1, 16, -1]
    assert dev.lens[:5].tolist() == [10, 20, 30, 20, 5]
    # the free pages, those that rows 1 and 3 hold among them, in order
    free, got = np.flatnonzero(before == 0), 0
    for s in range(3, S):
        n0, n1 = lens[s], lens[s] + delta[s]
        for j in range(c.pages(n0), c.pages(n1)):
            want_table[s, j] = free[got]
            before[free[got]] = 1
            got += 1
    assert np.array_equal(dev.table.cpu().numpy(), want_table)
    assert np.array_equal(dev.ref.cpu().numpy(), before)
    assert (pos[5:] == i32(lens[5:])).all()


@pytest.mark.parametrize("pages,children", [(6, 3), (9000, 3), (3000, 1500)])
def test_fork_counts_page_that_counts_as_free(pages, children):
    """Forks that add one by one, few long rows, and many rows of one source."""
    G = lib()
    lens = [pages, pages] + [0] * children
    for bad in (True, False):
        c = filled(lens, 1, 1, 8, F32, seed=32, spare=1)
        dev = Dev(c)
        if bad:
            c.ref[c.table[0, pages // 2]] = 0
            dev.ref.copy_(i32(c.ref))
        dst = np.arange(2, 2 + children)
        src = np.zeros(children, np.int32)
        G.gret_paged_fork(i32(src), i32(dst), dev.lens, dev.table, dev.ref, 1, status=dev.status)
        c.table[dst] = c.table[0]
        c.lens[dst] = pages
        c.ref[c.table[0, :pages]] += children
        dev.same_as(c)
        assert G.gret_paged_status(dev.status) == (G.GRET_PAGED_BAD_COUNT if bad else 0)


@pytest.mark.parametrize("where", ["front", "behind", "both"])
def test_compact_held_page_that_counts_as_free(where):
    """Pages that a row holds and whose count is 0, below the pages in use afterwards and past them:
    reported; the entry stays, all else moves as if nobody held them."""
    G = lib()
    c = filled([64, 48, 40, 8], 8, 2, 8, BF16, seed=33, spare=20)
    L = int((c.ref > 0).sum()) - 1
    row, j = np.nonzero((c.table >= 0) & ((c.table < L - 1) if where == "front" else (c.table >= L)))
    held = [(int(row[0]), int(j[0]))]
    if where == "both":
        row, j = np.nonzero((c.table >= 0) & (c.table < L - 2))
        held.append((int(row[0]), int(j[0])))
    ids = [int(c.table[h]) for h in held]
    dev = Dev(c)
    for i in ids:
        dev.ref[i] = c.ref[i] = 0
    n = G.gret_paged_compact(dev.lens, dev.table, dev.ref, dev.k, dev.v, status=dev.status)
    assert G.gret_paged_status(dev.status) == G.GRET_PAGED_BAD_COUNT
    was = c.table.copy()
    assert int(n) == c.compact()
    for h, i in zip(held, ids):
        c.table[h] = i
    assert (c.table != was).any()
    dev.same_as(c)


def test_compact_sound_cache_reports_nothing():
    G = lib()
    c = filled([64, 0, 40, 8, 1], 8, 2, 8, BF16, seed=34, spare=40)
    dev = Dev(c)
    n = G.gret_paged_compact(dev.lens, dev.table, dev.ref, dev.k, dev.v, status=dev.status)
    assert int(n) == c.compact() and G.gret_paged_status(dev.status) == 0
    dev.same_as(c)
    assert torch.equal(torch.sort(dev.ref, descending=True).values, dev.ref)
