"""Plain statements of the paged cache's calls for its tests: the page calls one
sequence and one page after another in Python, the attention in 64 bits."""
import math

import numpy as np
import torch


class PageModel:
    """Table, lengths and reference counts as plain lists."""

    def __init__(self, B, N, S, P):
        self.B, self.N, self.S, self.P, self.W = B, N, S, P, -(-N // S)
        self.table = [[-1] * self.W for _ in range(B)]
        self.lens = [0] * B
        self.refs = [0] * P
        self.head, self.pairs, self.grant = [0, 0, 0, P], [], [0] * B

    def _count(self, missing=0):
        live = sum(r > 0 for r in self.refs)
        self.head = [len(self.pairs), missing, live, self.P - live]

    def reserve(self, add):
        self.pairs, self.grant = [], [0] * self.B
        free = [i for i in range(self.P) if self.refs[i] == 0]
        refs, plan, need = list(self.refs), [], 0
        for b, a in enumerate(add):
            n = self.lens[b]
            if a <= 0 or n + a > self.N:
                continue
            have, want = -(-n // self.S), -(-(n + a) // self.S)
            cols = list(range(have, want))
            if n % self.S:
                page = self.table[b][have - 1]
                if not 0 <= page < self.P:
                    continue
                if refs[page] > 1:
                    refs[page] -= 1
                    cols = [have - 1] + cols
            plan.append((b, a, cols))
            need += len(cols)
        if need > len(free):
            self._count(need - len(free))
            return
        for b, a, cols in plan:
            for w in cols:
                page = free.pop(0)
                if self.table[b][w] >= 0:
                    self.pairs.append((self.table[b][w], page))
                    self.refs[self.table[b][w]] -= 1
                self.table[b][w], self.refs[page] = page, 1
            self.grant[b] = a
            self.lens[b] += a
        self._count()

    def fork(self, parent):
        old = self.table
        self.table = [list(old[p]) if 0 <= p < self.B else [-1] * self.W for p in parent]
        self.lens = [self.lens[p] if 0 <= p < self.B else 0 for p in parent]
        for sign, rows in ((1, self.table), (-1, old)):
            for row in rows:
                for x in row:
                    if x >= 0:
                        self.refs[x] += sign

    def free(self, seqs):
        for b in seqs:
            if 0 <= b < self.B:
                for w, x in enumerate(self.table[b]):
                    if x >= 0:
                        self.refs[x] -= 1
                    self.table[b][w] = -1
                self.lens[b] = 0

    def compact(self):
        L = sum(r > 0 for r in self.refs)
        self.pairs = list(zip([i for i in range(L, self.P) if self.refs[i] > 0],
                              [i for i in range(L) if self.refs[i] == 0]))
        for a, z in self.pairs:
            self.refs[z], self.refs[a] = self.refs[a], 0
        to = dict(self.pairs)
        self.table = [[to.get(x, x) for x in row] for row in self.table]
        self._count()


def free_bits(state, P):
    """The bitmap of free pages in a page state (numpy int32 words) as a list of bools."""
    at = -(-P // 4) * 4
    words = state[at:at + -(-P // 32)].view(np.uint32)
    return [bool((int(words[i // 32]) >> (i % 32)) & 1) for i in range(P)]


def attend64(q, K, V, table, lens, S, G):
    """o, lse and, for the tolerances, sum |q||k| / sqrt(d) and max |v| of each head; in 64 bits.
    Keys whose table entry lies outside the pool do not count."""
    B, Hq, d = q.shape
    P = K.shape[0]
    o = torch.zeros(B, Hq, d, dtype=torch.float64)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64)
    size = torch.zeros(B, Hq, 2, dtype=torch.float64)
    for b in range(B):
        pos = torch.arange(int(lens[b]))
        page = table[b].long()[pos // S] if len(pos) else pos
        ok = (page >= 0) & (page < P)
        pos, page = pos[ok], page[ok]
        if not len(pos):
            continue
        for h in range(Hq):
            k, v = K[page, h // G, pos % S].double(), V[page, h // G, pos % S].double()
            x = q[b, h].double()
            z = (k @ x) / math.sqrt(d)
            lse[b, h] = torch.logsumexp(z, 0)
            o[b, h] = torch.exp(z - lse[b, h]) @ v
            size[b, h, 0] = ((k.abs() @ x.abs()) / math.sqrt(d)).max()
            size[b, h, 1] = v.abs().max()
    return o, lse, size


def tolerances(o, lse, size, lens, d, dtype):
    """Largest errors of o and lse, from the roundings the kernels make.

    A logit is a sum of d products in 32 bits, scaled: at most (d + 4) roundings of
    2^-24 of sum |q||k| / sqrt(d). A probability then has that error, that of the
    exponential (2^-22, two units in the last place). Sums over n keys run in chains of
    at most n / 16 + 700 additions. Numerator and denominator both carry these, hence
    2 p. Where a probability enters the tensor cores it is in two bf16 parts: the first
    cut (below 2^-7 of it is left), the second rounded (2^-9 of that), 2^-16 in all; the
    denominator is summed in 32 bits and does not have it, so 2 * 2^-17 stands for it.
    The output is rounded once, by half of eps."""
    bf16 = dtype == torch.bfloat16
    chain = (torch.as_tensor(lens).double() / 16 + 700)[:, None]
    z = (d + 4) * 2.0 ** -24 * size[..., 0]
    p = z + 2.0 ** -22 + (2.0 ** -17 if bf16 else 0.0) + chain * 2.0 ** -24
    half = torch.finfo(dtype).eps / 2
    tol_o = half * o.abs() + (2 * p * size[..., 1])[..., None] * (1 + half)
    tol_lse = p + 2.0 ** -22 * (1 + lse.abs().nan_to_num(posinf=0.0))
    return tol_o, tol_lse
