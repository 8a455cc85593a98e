"""The softmax weights of decode attention over the paged cache are held in 32 bits: on inputs whose
scores are (nearly) exact, what is left of the error is a few 2^-23, for bf16 pools as for fp32."""
import math

import numpy as np
import pytest
import torch

from paged_model import Cache
from parity import bf16_half_ulp
from test_paged_gpu import BF16, F32, Dev, lib, queries

pytestmark = pytest.mark.gpu


def placed(lens, k, v, page):
    """A cache of rows of `lens` tokens whose keys and values are the first of k, v [S, n, H, d]."""
    S, H, d = len(lens), k.shape[2], k.shape[3]
    c = Cache(S, max(lens) // page + 1, sum(-(-n // page) for n in lens), page, H, d, k.dtype)
    at = 0
    for s, n in enumerate(lens):
        m = c.pages(n)
        c.table[s, :m] = np.arange(at, at + m)
        at += m
        c.lens[s] = n
        for j in range(0, n, page):
            e = min(n, j + page)
            c.k[c.table[s, j // page], :e - j] = k[s, j:e]
            c.v[c.table[s, j // page], :e - j] = v[s, j:e]
    return c


@pytest.mark.parametrize("H,G,d,lens", [
    (2, 3, 128, [2, 64, 1024, 16384]), (2, 3, 64, [2, 64, 1024, 16384]), (1, 12, 64, [4, 512]),
    (1, 24, 128, [8, 4096]), (3, 1, 64, [2, 32]), (8, 3, 128, [2] * 200), (4, 8, 64, [16] * 200),
])
def test_mean_that_lies_between_two_values(H, G, d, lens):
    """Equal scores weigh every key 1.  The mean of as many 1 as 1 + 2^-7 lies midway between these
    two neighbours in bf16, and its sums are exact in 32 bits (at most 2^14 terms of 8 bits): it goes
    to the even one, 1.  A weight off by 2^-20 to the one side gives the other."""
    n = max(lens)
    v = torch.ones((len(lens), n, H, d))
    v[:, 1::2] += 2.0 ** -7
    v[..., 1::2] *= -1
    k = torch.zeros_like(v)
    c = placed(lens, k.to(BF16), v.to(BF16), 16)
    q = queries(len(lens), H * G, d, BF16, seed=1)
    o, lse = Dev(c).decode(q)
    want = torch.ones(d)
    want[1::2] = -1
    assert (o.cpu().float() == want).all()
    for s, x in enumerate(lens):
        assert (lse[s].cpu().double() - math.log(x)).abs().max() <= math.log(x) * 2.0 ** -22


@pytest.mark.parametrize("dtype,H,G,d,n", [
    (BF16, 4, 3, 128, 2), (BF16, 4, 8, 64, 2), (BF16, 3, 2, 64, 2), (BF16, 2, 12, 64, 2),
    (BF16, 2, 24, 128, 2), (BF16, 4, 3, 128, 4), (F32, 4, 4, 64, 4),
])
def test_weights_in_32_bits(dtype, H, G, d, n):
    """Scores that are one product each, at most S = 1 in size, and few keys.

    In units of u = 2^-23, relative to a weight: the factor scale log2(e) and its product with the
    score are rounded (u S), the difference to the maximum too (u S, of two scores), all of it for
    the score and for the maximum (together 4 u S at most); exp2 is off by 2 u.  A tensor core may cut
    off each of the n + 1 numbers that it adds up, of each of a weight's three parts: 3 (n + 1); the
    join's factors and the division add 3.  All of it counts twice, above and below the line.  (With
    weights rounded to 16 bits, up to 128 u of a weight come on top.)"""
    B, S = 400, 1.0
    gen = torch.Generator().manual_seed(n + d)
    k = torch.zeros((B, n, H, d))
    k[..., 0] = (torch.rand((B, n, H), generator=gen) * 2 - 1) * S
    k, v = k.to(dtype), torch.randn((B, n, H, d), generator=gen).to(dtype)
    c = placed([n] * B, k, v, 8)
    q = torch.zeros((B, H * G, d))
    q[..., 0] = 1 - torch.arange(G).repeat(H) / 64.0          # at most 1, exact in bf16
    q = q.to(dtype)
    o, _ = Dev(c).decode(q.cuda(), scale=1.0)
    s = (q[:, None, :, 0].double() * k[..., 0].double().repeat_interleave(G, 2))    # [B, n, H G]
    p = torch.softmax(s, 1)
    vv = v.double().repeat_interleave(G, 2)
    want = torch.einsum("bnh,bnhd->bhd", p, vv)
    lim = 2 * (4 * S + 2 + 3 * (n + 1) + 3) * 2.0 ** -23 * torch.einsum("bnh,bnhd->bhd", p, vv.abs())
    got = o.cpu().double()
    lim += torch.from_numpy(bf16_half_ulp(np.maximum(want.abs().numpy(), got.abs().numpy()))) \
        if dtype == BF16 else want.abs() * 2.0 ** -24
    over = (got - want).abs() - lim
    assert (over <= 0).all(), (int((over > 0).sum()), float(over.max()))


@pytest.mark.parametrize("d,H,G", [(128, 2, 3), (64, 2, 8), (64, 1, 24)])
def test_infinite_value_of_a_light_key(d, H, G):
    """An infinite value reaches the output however little its key weighs, down to what exp2 gives
    in 32 bits (2^-126); a key of weight 1 and one of a weight that three 8-bit parts just hold are
    among them.  Scores: one product, 8 times a key's first dimension."""
    ln2 = math.log(2)
    light = torch.tensor([0.0, -1.0, -7.25, -33.5, -60.0, -99.0, -108.0, -114.5, -120.0, -125.0])
    B = len(light)
    k = torch.zeros((B, 2, H, d))
    k[:, 1, :, 0] = light[:, None] * (ln2 / 8)
    v = torch.ones((B, 2, H, d))
    v[:, 1, :, 3], v[:, 1, :, 5] = float("inf"), -float("inf")
    c = placed([2] * B, k.to(BF16), v.to(BF16), 8)
    q = torch.zeros((B, H * G, d))
    q[..., 0] = 8
    o, lse = Dev(c).decode(q.to(BF16).cuda(), scale=1.0)
    o = o.cpu()
    assert (o[..., 3] == float("inf")).all() and (o[..., 5] == -float("inf")).all()
    o[..., 3] = o[..., 5] = 1
    assert (o == 1).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("H,G,d", [(1, 8, 128), (2, 8, 64), (1, 16, 64), (1, 24, 128)])
def test_long_sums_are_not_cut_off(H, G, d):
    """300 rows read the same 65536 keys, some 16000 a warp, whose values are all positive.  Sums that
    are rounded to 32 bits are off to either side, ones that are cut off all to one: 2048 steps that
    lose 2^-23 or so of what is summed up by then, half of the whole on average, make 1.1e-4.

    The outputs, 1 to 2, are rounded to multiples of 2^-7 and spread over several of them (scores
    that vary by 2.5 leave some hundred keys that count), so the mean of N errors has a deviation of
    2^-7 / sqrt(12 N); 6 of them are allowed, and 2^-21 for the arithmetic."""
    B, n, page = 300, 65536, 64
    gen = torch.Generator("cuda").manual_seed(G + d)
    k, v = (torch.randn((n // page, page, H, d), generator=gen, device="cuda") for _ in range(2))
    v = 1.5 + 0.29 * v.clamp(-1.7, 1.7)
    k, v = k.to(BF16), v.to(BF16)
    q = torch.randn((B, H * G, d), generator=gen, device="cuda") * 2.5
    q = q.to(BF16)
    table = torch.randperm(n // page, generator=gen, device="cuda").int().expand(B, -1).contiguous()
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    o, _ = lib().gret_paged_attention_decode(q, lens, table, k, v)
    off = 0.0
    for h in range(H):
        kk, vv = k[:, :, h].reshape(n, d).double(), v[:, :, h].reshape(n, d).double()
        for qh, oh in zip(q[:, h * G:(h + 1) * G].split(30), o[:, h * G:(h + 1) * G].split(30)):
            want = torch.softmax(qh.double() @ kk.T * d ** -0.5, -1) @ vv
            assert want.std() > 2.0 ** -7
            off += float((oh.double() - want).sum())
    assert abs(off / o.numel()) <= 6 * 2.0 ** -7 / math.sqrt(12 * o.numel()) + 2.0 ** -21
