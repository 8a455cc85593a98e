"""Calls of the paged cache queued behind one another, every one of their outputs looked at: a kernel
that starts before the one in front has ended, or a workspace that is used again too early, shows
in the call that it happens to and not in the last one alone."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from test_paged_gpu import BF16, F32, Dev, check, filled, i32, lib, queries
from test_paged_binding_cpu import KV_RULE, Q_RULE

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("dtype,H,G_,d,S", [(BF16, 2, 3, 64, 40), (BF16, 8, 3, 128, 90), (F32, 2, 5, 64, 40)])
def test_queued_calls_give_what_single_ones_do(dtype, H, G_, d, S, given):
    """Sixty steps of resize, append, fork, compact and attention, queued without a wait, on the
    current stream or on one that is given: positions, counts of pages, outputs and log-sum-exps of
    every step are bit for bit those of the same calls made one at a time, which agree with the
    definition step by step."""
    G = lib()
    page = 8
    rng = np.random.default_rng(51)
    c = filled([50, 0, 9] + [0] * (S - 3), page, H, d, dtype, seed=51, spare=11 * S)
    c.table = np.concatenate([c.table, np.full((S, 12), -1, np.int32)], 1)
    c.W += 12
    steps, q = [], queries(S, H * G_, d, dtype, 51)
    one, many = Dev(c), Dev(c)
    stream = torch.cuda.Stream() if given else None
    alone = []

    def calls(dev, step, stream=None):
        delta, k, v, src, dst, compact = step
        pos = G.gret_paged_resize(delta, dev.lens, dev.table, dev.ref, dev.k, dev.v, stream=stream)
        yield pos
        G.gret_paged_append(k, v, pos, dev.table, dev.k, dev.v, stream=stream)
        yield dev.lens
        G.gret_paged_fork(src, dst, dev.lens, dev.table, dev.ref, page, stream=stream)
        yield dev.lens
        if compact:
            yield G.gret_paged_compact(dev.lens, dev.table, dev.ref, dev.k, dev.v, stream=stream)
        yield from G.gret_paged_attention_decode(q, dev.lens, dev.table, dev.k, dev.v, lse=True,
                                                 stream=stream)

    for t in range(60):
        delta = np.where(c.lens > 0, 1, 0)
        if t % 5 == 4:
            delta[rng.integers(0, S, 3)] = -2 ** 31
        if t % 5 == 1:
            delta[0] = 1                              # a new sequence, if the row is idle
        k, v = (torch.randn((S, H, d)).to(dtype) for _ in range(2))
        src, dst = rng.integers(0, S, 4), rng.integers(0, S, 4)
        steps.append((i32(delta), k.cuda(), v.cuda(), i32(src), i32(dst), t % 9 == 8))
        outs = []
        for x in calls(one, steps[-1]):
            torch.cuda.synchronize()
            outs.append(x.clone())
        alone.append(outs)
        pos, refused = c.resize(delta)
        assert refused == [] and np.array_equal(outs[0].cpu().numpy(), pos)
        for s in np.flatnonzero(pos >= 0):
            c.append(s, pos[s], k[s:s + 1], v[s:s + 1])
        c.fork(src.tolist(), dst.tolist())
        if t % 9 == 8:
            assert int(outs[3]) == c.compact()
        one.same_as(c)
        check(c, q, *outs[-2:])
    torch.cuda.synchronize()
    kept = [[x for x in calls(many, s, stream) if x is not many.lens] for s in steps]
    torch.cuda.synchronize()
    many.same_as(c)
    for queued, outs in zip(kept, alone):
        outs = outs[:1] + outs[3:]                    # without the lengths
        assert len(queued) == len(outs)
        assert all(torch.equal(x, y) for x, y in zip(queued, outs))


def test_refusals_of_gpu_tensors():
    """What can only be refused once the device is known, told by its own message."""
    G = lib()
    c = filled([20, 9], 16, 2, 64, BF16, seed=61)
    dev, q = Dev(c), queries(2, 4, 64, BF16, 61)
    k = torch.zeros((2, 2, 64), dtype=BF16, device="cuda")
    P = c.ref.size

    def dec(q=q, lens=dev.lens, **kw):
        return G.gret_paged_attention_decode(q, lens, dev.table, dev.k, dev.v, **kw)

    def app(k=k, v=k, pos=dev.lens, **kw):
        return G.gret_paged_append(k, v, pos, dev.table, dev.k, dev.v, **kw)

    def res(delta=dev.lens, lens=dev.lens, ref=dev.ref, **kw):
        return G.gret_paged_resize(delta, lens, dev.table, ref, dev.k, dev.v, **kw)

    def fork(src=dev.lens, dst=dev.lens, lens=dev.lens, ref=dev.ref, **kw):
        return G.gret_paged_fork(src, dst, lens, dev.table, ref, 16, **kw)

    def comp(lens=dev.lens, ref=dev.ref, **kw):
        return G.gret_paged_compact(lens, dev.table, ref, dev.k, dev.v, **kw)

    two, wrong = r"must be contiguous int32 \[2\]", torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    for message, call in [
        ("seq_lens " + two, lambda: dec(lens=dev.lens.long())),
        ("seq_lens " + two, lambda: dec(lens=wrong[:2, 0])),
        ("seq_lens " + two, lambda: dec(lens=wrong[:1].t())),
        (r"status must be contiguous int32 \[1\]", lambda: dec(status=dev.lens)),
        ("o must be contiguous and of q's shape", lambda: dec(o=q[:1])),
        ("o must be contiguous and of q's shape", lambda: dec(o=q.float())),
        (r"lse must be contiguous float32 \[B, Hq\]", lambda: dec(lse=torch.zeros((4, 2), device="cuda"))),
        ("workspace must be contiguous", lambda: dec(workspace=wrong[:, :1])),
        (Q_RULE, lambda: dec(q=q[..., ::2])),
        ("pos " + two, lambda: app(pos=dev.lens.long())),
        (r"cu_seqlens must be contiguous int32 \[3\]", lambda: app(cu_seqlens=dev.lens)),
        (KV_RULE, lambda: app(v=k.float())),
        (r"status must be contiguous int32 \[1\]", lambda: app(status=dev.lens.float()[:1])),
        ("delta " + two, lambda: res(delta=dev.lens[:1])),
        ("delta " + two, lambda: res(delta=dev.lens.float())),
        (r"ref must be contiguous int32 \[%d\]" % P, lambda: res(ref=dev.ref[1:])),
        ("pos " + two, lambda: res(pos=wrong[:2, 0])),
        ("workspace must be contiguous", lambda: res(workspace=wrong[:, :1])),
        ("dst " + two, lambda: fork(dst=dev.lens[:1])),
        ("src " + two, lambda: fork(src=dev.lens.long())),
        (r"ref must be contiguous int32 \[%d\]" % P, lambda: comp(ref=dev.ref.repeat(2))),
        (r"n_live must be contiguous int32 \[1\]", lambda: comp(n_live=dev.lens)),
        ("on one device", lambda: dec(lens=dev.lens.cpu())),
        ("on one device", lambda: app(cu_seqlens=torch.zeros(3, dtype=torch.int32))),
        ("on one device", lambda: res(pos=torch.zeros(2, dtype=torch.int32))),
        ("on one device", lambda: fork(ref=dev.ref.cpu())),
        ("on one device", lambda: comp(n_live=torch.zeros(1, dtype=torch.int32))),
    ]:
        with pytest.raises(ValueError, match=message):
            call()
    with pytest.raises(G.GretError, match="INVALID_ARG"):
        res(delta=torch.ones_like(dev.lens), pos=dev.lens)
    dev.same_as(c)


@pytest.mark.parametrize("dtype,B,H,G_,d", [
    (BF16, 3, 2, 3, 128), (BF16, 250, 4, 5, 64), (BF16, 4, 1, 40, 128), (F32, 300, 3, 2, 128),
    (F32, 5, 2, 20, 64),
])
def test_attention_in_place(dtype, B, H, G_, d):
    """Outputs in the queries' place: no block reads a query after another has written there."""
    rng = np.random.default_rng(B)
    c = filled(rng.integers(0, 90, B).tolist() + [3000], 16, H, d, dtype, seed=92)
    dev, q = Dev(c), queries(B + 1, H * G_, d, dtype, 92)
    want, _ = dev.decode(q)
    o, _ = dev.decode(q, o=q)
    assert o is q and torch.equal(o, want)


FIRST_CALL = """
import torch
import gated_retention_linear_b200 as G
dev = "cuda"
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
P, page, W, S = %d, 4, 40, 20
kp, vp = (torch.zeros((P, page, 2, 64), dtype=torch.bfloat16, device=dev) for _ in range(2))
table, lens, ref = torch.full((S, W), -1, dtype=torch.int32, device=dev), i32([0] * S), i32([0] * P)
delta, src, dst = i32([9, 2] + [0] * (S - 2)), i32([0]), i32([3])
k, v = (torch.randn((11, 2, 64), device=dev).bfloat16() for _ in range(2))
q, cu = torch.randn((S, 6, 64), device=dev).bfloat16(), i32([0, 9] + [11] * (S - 1))
status, n_live = i32([0]), i32([0])
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    pos = G.gret_paged_resize(delta, lens, table, ref, kp, vp, status=status)
    G.gret_paged_append(k, v, pos, table, kp, vp, cu_seqlens=cu, status=status)
    G.gret_paged_fork(src, dst, lens, table, ref, page, status=status)
    G.gret_paged_compact(lens, table, ref, kp, vp, n_live=n_live, status=status)
    o, lse = G.gret_paged_attention_decode(q, lens, table, kp, vp, lse=True, status=status)
graph.replay()
torch.cuda.synchronize()
assert lens.tolist() == [9, 2, 0, 9] + [0] * (S - 4) and int(n_live) == 4 and int(status) == 0
assert pos[:3].tolist() == [0, 0, -1] and ref[:5].tolist() == [2, 2, 2, 1, 0]
for s, a, b in ((0, 0, 9), (1, 9, 11), (3, 0, 9)):
    w = torch.einsum("hgd,nhd->hgn", q[s].view(2, 3, 64).float(), k[a:b].float()) / 8
    want = torch.einsum("hgn,nhd->hgd", torch.softmax(w, 2), v[a:b].float()).reshape(6, 64)
    assert (o[s].float() - want).abs().max() < 0.03
    assert (lse[s] - torch.logsumexp(w, 2).reshape(6)).abs().max() < 1e-4
assert (o[2] == 0).all() and (lse[2] == -float("inf")).all()
"""


@pytest.mark.parametrize("P", [100, 140000])
def test_first_call_of_a_process_in_a_capture(P):
    """Nothing that a call does once a process or a device is out of place in a capture."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", FIRST_CALL % P], cwd=root, check=True, timeout=300)
