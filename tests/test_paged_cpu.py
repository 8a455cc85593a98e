"""Refusals of the paged-cache entry points, on the CPU: every argument error is found on the host
before anything is launched, so these calls touch no device.  Also the tests' own model of the
cache, on small cases worked out by hand."""
import numpy as np
import pytest
import torch

from paged_model import Cache, attention


def lib():
    import gated_retention_linear_b200 as G
    return G


POOL = dict(kp=1 << 20, vp=2 << 20, sp=16 * 8 * 128, st=8 * 128, sh=128, P=100, page=16, dtype=1)
TABLE = dict(table=4096, ts=64, mp=64)


def _attention(**kw):
    G = lib()
    a = dict(q=1024, lens=2048, **TABLE, **POOL, scale=0.088, window=0, B=4, Hq=24, Hkv=8, d=128,
             o=8192, lse=None, status=None, ws=1 << 16, wsb=1 << 40, stream=None)
    a.update(kw)
    return G._lib.gret_paged_attention_decode(*a.values())


@pytest.mark.parametrize("want,kw", [
    (0, dict(B=0)),
    (1, dict(scale=float("nan"))), (1, dict(scale=float("inf"))), (1, dict(window=-1)),
    (1, dict(Hq=20)),                         # not a multiple of Hkv
    (1, dict(Hq=0)), (1, dict(Hkv=0)), (1, dict(B=-1)), (1, dict(mp=0)), (1, dict(ts=63)),
    (1, dict(P=0)), (1, dict(page=0)), (1, dict(dtype=2)), (1, dict(st=-8)), (1, dict(q=None)),
    (1, dict(lens=None)), (1, dict(o=None)), (1, dict(kp=None)), (1, dict(table=None)),
    (1, dict(sp=1 << 62)),                    # the last page's address would not fit
    (2, dict(d=96)), (2, dict(d=256)), (2, dict(page=24)), (2, dict(page=2048)),
    (2, dict(B=16385)), (2, dict(mp=1 << 28, ts=1 << 28)),    # lengths past int32
    (3, dict(q=1032)), (3, dict(o=8200)), (3, dict(kp=(1 << 20) + 8)), (3, dict(st=1028)),
    (3, dict(lens=2050)), (3, dict(lse=4098)), (3, dict(status=4097)), (3, dict(table=4098)),
    (3, dict(ws=(1 << 16) + 8)),
    (4, dict(ws=None)), (4, dict(wsb=100)),
])
def test_attention_refusals(want, kw):
    assert _attention(**kw) == want


def test_attention_workspace_size():
    G = lib()
    need = G.gret_paged_attention_workspace_size(torch.bfloat16, 24, 8, 128)
    assert need > 0 and _attention(wsb=need - 1) == 4
    assert G.gret_paged_attention_workspace_size(torch.float32, 24, 8, 64) > 0
    assert G.gret_paged_attention_workspace_size(torch.float32, 24, 8, 96) == 0
    assert G.gret_paged_attention_workspace_size(torch.float32, 20, 8, 64) == 0


@pytest.mark.parametrize("want,kw", [
    (0, dict(T=0)), (0, dict(S=0)),
    (1, dict(T=-1)), (1, dict(cu=None)),      # one token a row needs T = S
    (1, dict(k=None)), (1, dict(pos=None)), (1, dict(kt=-8)), (1, dict(vt=1 << 61)),
    (2, dict(T=1 << 31)), (2, dict(page=48)), (2, dict(S=16385)),
    (3, dict(k=1032)), (3, dict(kt=1028)), (3, dict(vh=132)), (3, dict(d=129)), (3, dict(pos=2049)),
    (3, dict(cu=3074)), (3, dict(status=1025)),
])
def test_append_refusals(want, kw):
    G = lib()
    a = dict(k=1024, kt=1024, kh=128, v=2048, vt=1024, vh=128, T=77, cu=5120, pos=2048, S=4, **TABLE,
             **POOL, H=8, d=128, status=None, stream=None)
    a.update(kw)
    assert G._lib.gret_paged_append(*a.values()) == want


@pytest.mark.parametrize("want,kw", [
    (0, dict(S=0)),
    (1, dict(S=-1)), (1, dict(delta=None)), (1, dict(lens=None)), (1, dict(ref=None)),
    (1, dict(pos=None)), (1, dict(H=0)),
    (2, dict(S=16385)), (2, dict(P=(1 << 30) + 1)), (2, dict(page=12)),
    (3, dict(delta=1025)), (3, dict(ref=1026)), (3, dict(pos=1027)), (3, dict(vp=4 + (2 << 20))),
    (3, dict(ws=8200)), (4, dict(wsb=15)), (4, dict(ws=None)),
])
def test_resize_refusals(want, kw):
    G = lib()
    assert G.gret_paged_resize_workspace_size(4) == 16
    a = dict(delta=1024, lens=2048, S=4, **TABLE, ref=4096, **POOL, H=8, d=128, pos=5120, status=None,
             ws=8192, wsb=16, stream=None)
    a.update(kw)
    assert G._lib.gret_paged_resize(*a.values()) == want


@pytest.mark.parametrize("want,kw", [
    (0, dict(n=0)), (0, dict(S=0)),
    (1, dict(n=-1)), (1, dict(src=None)), (1, dict(dst=None)), (1, dict(lens=None)),
    (1, dict(ref=None)), (1, dict(P=0)), (1, dict(page=-16)),
    (2, dict(n=16385)), (2, dict(page=17)),
    (3, dict(src=1025)), (3, dict(ref=4098)),
])
def test_fork_refusals(want, kw):
    G = lib()
    a = dict(src=1024, dst=2048, n=2, lens=3076, S=4, **TABLE, ref=4096, P=100, page=16, status=None,
             stream=None)
    a.update(kw)
    assert G._lib.gret_paged_fork(*a.values()) == want


@pytest.mark.parametrize("want,kw", [
    (1, dict(lens=None)), (1, dict(ref=None)), (1, dict(n_live=None)), (1, dict(S=-1)),
    (2, dict(page=1025)), (3, dict(n_live=1026)), (3, dict(kp=8 + (1 << 20))), (3, dict(ws=8200)),
    (4, dict(ws=None)), (4, dict(wsb=1215)),
])
def test_compact_refusals(want, kw):
    G = lib()
    assert G.gret_paged_compact_workspace_size(100) == 1216      # 3 int32 a page and 4 more
    assert G.gret_paged_compact_workspace_size(0) == 0
    a = dict(lens=2048, S=4, **TABLE, ref=4096, **POOL, H=8, d=128, n_live=1024, status=None, ws=8192,
             wsb=1216, stream=None)
    a.update(kw)
    assert G._lib.gret_paged_compact(*a.values()) == want


def test_binding_refusals():
    """What the binding refuses before the library is called: tensors on the CPU among it."""
    G = lib()
    kp = torch.zeros((4, 16, 2, 64))
    q, lens = torch.zeros((3, 6, 64)), torch.zeros(3, dtype=torch.int32)
    table, ref = torch.zeros((3, 5), dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    dec = G.gret_paged_attention_decode
    bad = [
        lambda: dec(q, lens, table, kp, kp),                               # no GPU tensors
        lambda: dec(q.bfloat16(), lens, table, kp, kp),                    # q's dtype
        lambda: dec(q[..., :32], lens, table, kp, kp),                     # q's d
        lambda: dec(q, lens, table[:2], kp, kp),                           # rows of the table
        lambda: dec(q, lens, table.long(), kp, kp),
        lambda: dec(q, lens, table.t(), kp, kp),
        lambda: dec(q, lens, table, kp, kp[:2]),                           # pools differ
        lambda: dec(q, lens, table, kp, kp.transpose(1, 2).contiguous().transpose(1, 2)),
        lambda: dec(q, lens, table, kp[0], kp[0]),
        lambda: G.gret_paged_append(q[:, :2], q[:, :2], lens, table, kp, kp),
        lambda: G.gret_paged_append(q, q, lens, table, kp, kp),            # heads
        lambda: G.gret_paged_append(q[:, :2].bfloat16(), q[:, :2].bfloat16(), lens, table, kp, kp),
        lambda: G.gret_paged_resize(lens, lens, table, ref, kp, kp),
        lambda: G.gret_paged_fork(lens, lens, lens, table, ref, 16),
        lambda: G.gret_paged_compact(lens, table, ref, kp, kp),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):                                         # fp16 pool
        G.gret_paged_compact(lens, table, ref, kp.half(), kp.half())


def test_model_by_hand():
    c = Cache(S=4, W=3, P=6, page=4, H=1, d=2, dtype=torch.float32)
    pos, refused = c.resize([5, 0, 3, 0])
    assert pos.tolist() == [0, -1, 0, -1] and refused == []
    assert c.table[:, :2].tolist() == [[0, 1], [-1, -1], [2, -1], [-1, -1]]
    c.k[1, 0] = 7.0
    assert c.fork([0, 0, 2], [1, 1, 0]) == [0, 1, 2]     # row 0 is a destination; twice row 1
    assert c.fork([0, 2, 2], [1, 3, 3]) == [2]
    assert c.ref.tolist() == [2, 2, 2, 0, 0, 0] and c.lens.tolist() == [5, 5, 3, 3]
    # rows 0 and 1 part: each gets its own copy of page 1, which nobody holds any more
    pos, refused = c.resize([1, 1, -3, 0])
    assert pos.tolist() == [5, 5, -1, -1] and refused == []
    assert c.table.tolist() == [[0, 3, -1], [0, 4, -1], [-1, -1, -1], [2, -1, -1]]
    assert c.ref.tolist() == [2, 0, 1, 1, 1, 0] and c.k[3, 0, 0, 0] == c.k[4, 0, 0, 0] == 7.0
    assert c.compact() == 4
    assert c.ref.tolist() == [2, 1, 1, 1, 0, 0] and c.table[1].tolist() == [0, 1, -1]
    pos, refused = c.resize([12, 2, 9, 9])               # 2 pages free; row 1 stays in its page
    assert refused == [0, 2, 3] and pos.tolist() == [-1, 6, -1, -1]


def test_model_attention_by_hand():
    q = torch.tensor([[1.0, 0.0], [0.0, 2.0]])
    k = torch.tensor([[[np.log(3.0), 9.0]], [[0.0, 9.0]]])
    v = torch.tensor([[[4.0, 0.0]], [[0.0, 8.0]]])
    o, lse, eo, el = attention(q, k, v, 1.0)
    assert np.allclose(o, [[3.0, 2.0], [2.0, 4.0]], atol=1e-6)
    assert np.allclose(lse, [np.log(4.0), 18 + np.log(2.0)], atol=1e-6)
    assert (eo < 1e-3).all() and (el < 1e-3).all()
