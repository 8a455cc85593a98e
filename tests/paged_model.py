"""A plain model of the paged cache for the tests: lengths, page table and counts as numpy arrays,
keys and values as CPU tensors, one sequence at a time; and attention over it in 64 bits with a
bound on what a 32-bit kernel may be off."""
import numpy as np
import torch


class Cache:
    """lens [S], table [S, W], ref [P] int32; k, v [P, page, H, d] (tokens before heads)."""

    def __init__(self, S, W, P, page, H, d, dtype, fill=float("nan")):
        self.page, self.W = page, W
        self.lens = np.zeros(S, np.int32)
        self.table = np.full((S, W), -1, np.int32)
        self.ref = np.zeros(P, np.int32)
        self.k = torch.full((P, page, H, d), fill, dtype=dtype)
        self.v = torch.full((P, page, H, d), fill, dtype=dtype)

    def pages(self, n):
        return -(-int(n) // self.page)

    def resize(self, delta):
        """Returns (pos, refused rows)."""
        was, free = self.ref.copy(), np.flatnonzero(self.ref == 0)
        pos, refused, asked, got = np.full(len(self.lens), -1, np.int32), [], 0, 0
        for s, dl in enumerate(delta):
            n0 = int(self.lens[s])
            n1 = max(0, n0 + int(dl))
            c0, c1 = self.pages(n0), self.pages(n1)
            if n1 < n0:
                for j in range(c1, c0):
                    self.ref[self.table[s, j]] -= 1
                    self.table[s, j] = -1
                self.lens[s] = n1
            elif n1 > n0:
                if n1 > self.W * self.page:
                    refused.append(s)
                    continue
                old = int(self.table[s, c0 - 1]) if n0 % self.page else -1
                cow = old >= 0 and was[old] > 1
                need = c1 - c0 + cow
                asked += need
                if need and asked > len(free):
                    refused.append(s)
                    continue
                mine = free[got:got + need]
                got += need
                if cow:
                    self.ref[old] -= 1
                    for x in (self.k, self.v):
                        x[mine[0], :n0 % self.page] = x[old, :n0 % self.page]
                self.table[s, c0 - cow:c1] = mine
                self.ref[mine] = 1
                pos[s], self.lens[s] = n0, n1
        return pos, refused

    def append(self, s, pos, k, v):
        for i in range(k.shape[0]):
            p, t = divmod(int(pos) + i, self.page)
            self.k[self.table[s, p], t] = k[i]
            self.v[self.table[s, p], t] = v[i]

    def fork(self, src, dst):
        """Returns the refused pairs."""
        refused, was = [], self.lens.copy()
        S = len(was)
        for i, (s, d) in enumerate(zip(src, dst)):
            if not (0 <= s < S and 0 <= d < S) or s == d or d in list(dst[:i]) or s in list(dst) \
                    or was[d] != 0:
                refused.append(i)
                continue
            n = self.pages(was[s])
            self.table[d, :n] = self.table[s, :n]
            for j in range(n):
                self.ref[self.table[s, j]] += 1
            self.lens[d] = was[s]
        return refused

    def compact(self):
        n = int((self.ref > 0).sum())
        frm = [p for p in range(n, len(self.ref)) if self.ref[p] > 0]
        to = [p for p in range(n) if self.ref[p] == 0]
        where = np.arange(len(self.ref), dtype=np.int32)
        for f, t in zip(frm, to):
            self.k[t], self.v[t] = self.k[f], self.v[f]
            self.ref[t], self.ref[f], where[f] = self.ref[f], 0, t
        for s in range(len(self.lens)):
            c = self.pages(self.lens[s])
            self.table[s, :c] = where[self.table[s, :c]]
        return n

    def tokens(self, s, a, b):
        """Keys and values [b - a, H, d] of tokens a .. b-1 of sequence s."""
        t = np.arange(a, b)
        pg = torch.from_numpy(self.table[s, t // self.page].astype(np.int64))
        sl = torch.from_numpy(t % self.page)
        return self.k[pg, sl], self.v[pg, sl]


def attention(q, k, v, scale):
    """q [Hq, d], k, v [n, Hkv, d]: o [Hq, d] and lse [Hq] in 64 bits, and what each may be off in
    32 bits: `eo` the arithmetic error of o (its rounding to 16 bits comes on top), `el` of lse.

    A score is a sum of d products: d + 2 roundings (the products, the sums, the scaling), each at
    most 2^-23 of sum |q k| scale (2^-23, not 2^-24: tensor cores may cut off instead of round).  A
    weight e^(s - m) is then off by the error of s and of m, by exp2's 2^-21 and by 2^-16 for being
    fed to the tensor cores as two 16-bit parts; the sums over n keys add 2^-23 a step.  o is a
    ratio of two such sums, so the relative errors of the weights count twice, against sum p |v|."""
    if k.shape[0] == 0:
        z = torch.zeros(q.shape, dtype=torch.float64)
        return z, torch.full(q.shape[:1], -float("inf"), dtype=torch.float64), z, z[:, 0]
    G = q.shape[0] // k.shape[1]
    q, k, v = q.double(), k.double().repeat_interleave(G, 1), v.double().repeat_interleave(G, 1)
    n, d = k.shape[0], q.shape[1]
    s = torch.einsum("hd,nhd->hn", q, k) * scale
    size = torch.einsum("hd,nhd->hn", q.abs(), k.abs()).amax(1) * abs(scale)
    es = (d + 2) * 2.0 ** -23 * size
    w = 2 * es + 2.0 ** -21 + 2.0 ** -16 + n * 2.0 ** -23
    lse = torch.logsumexp(s, 1)
    p = torch.softmax(s, 1)
    o = torch.einsum("hn,nhd->hd", p, v)
    eo = 2 * w[:, None] * torch.einsum("hn,nhd->hd", p, v.abs())
    return o, lse, eo, w + lse.abs() * 2.0 ** -22
