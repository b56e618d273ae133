"""PagedCache on the GPU, used as its documentation allows: captured steps between forks,
calls right behind a fork, layers that take dense tokens and prompts and then sparse steps."""
import math
import random

import numpy as np
import pytest
import torch

from hierarchical_block_sparse_b200 import pisa
from tests.paged_ref import PageModel, attend64, tolerances

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
I32 = dict(dtype=torch.int32, device=DEV)


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("a CUDA device is required for the gpu-marked tests")
    pisa.load()


class Story:
    """What every sequence of a cache should hold: K and V rows of each layer, beside a page model."""

    def __init__(self, cache, layers):
        c = cache.cfg
        self.c, self.cache, self.layers = c, cache, layers
        self.dt = cache.K[0].dtype
        self.m = PageModel(c.B, c.N, cache.pages.S, cache.pages.P)
        self.rows = [self.empty() for _ in range(c.B)]

    def empty(self):
        return [torch.zeros(self.c.Hkv, 0, self.c.d, dtype=self.dt) for _ in range(2 * self.layers)]

    def add(self, b, new):
        self.rows[b] = [torch.cat([x, y], 1) for x, y in zip(self.rows[b], new)]

    def fork(self, parent):
        self.m.fork(parent)
        self.rows = [list(self.rows[p]) if 0 <= p < self.c.B else self.empty() for p in parent]

    def check(self):
        torch.cuda.synchronize()
        c, S = self.cache, self.cache.pages.S
        assert c.table.tolist() == self.m.table and c.lens.tolist() == self.m.lens
        assert c.state[:self.m.P].tolist() == self.m.refs
        table = c.table.cpu().long()
        for b in range(self.c.B):
            pos = torch.arange(self.m.lens[b])
            for i in range(self.layers):
                for j, pool in enumerate((c.K[i], c.V[i])):
                    got = pool[table[b][pos // S].to(DEV), :, (pos % S).to(DEV)].transpose(0, 1).cpu()
                    assert torch.equal(got, self.rows[b][2 * i + j]), (b, i, j)

    def check_dense(self, layer, q, o, lse, lens):
        c, G = self.cache, self.c.Hq // self.c.Hkv
        ro, rl, size = attend64(q, c.K[layer].cpu(), c.V[layer].cpu(), c.table.cpu(), torch.tensor(lens), c.pages.S, G)
        tol_o, tol_l = tolerances(ro, rl, size, lens, self.c.d, q.dtype)
        assert bool(((o.cpu().double() - ro).abs() <= tol_o).all())
        none = rl == -math.inf
        assert torch.equal(lse.cpu() == -math.inf, none)
        assert not bool(((lse.cpu().double() - rl).abs() > tol_l)[~none].any())

    def check_sparse(self, layer, q, idx, o):
        """Against the oracle's selection over the sequence's own rows (choices that are no tie), and 64 bits."""
        from oracle import oracle
        from tests.parity import TIE_BAND
        cfg, G, seen = self.c, self.c.Hq // self.c.Hkv, 0
        for b in range(cfg.B):
            n = self.m.lens[b]
            if n == 0:
                assert bool((idx[b] == -1).all()) and not bool(o[b].any())
                continue
            for h in range(cfg.Hkv):
                k, v = (self.rows[b][2 * layer + j][h] for j in range(2))
                Kh = oracle.to_f64(k)
                Ph = oracle.build_pyramid(Kh, cfg.C, N=n, N_layout=cfg.N)
                heads = oracle.to_f64(q[b, h * G:h * G + G])[None]
                want, gap = oracle.select_rows(heads, np.array([n - 1]), Kh, Ph, C=cfg.C, K=cfg.K, N=n, N_layout=cfg.N)
                got = [x for x in idx[b, h].tolist() if x >= 0]
                if gap[0] >= TIE_BAND:
                    seen += 1
                    assert got == [x for x in want[0].tolist() if x >= 0], (b, h)
                pos = torch.cat([torch.arange(i * cfg.C, min(i * cfg.C + cfg.C, n)) for i in got])
                for i in range(G):
                    x = q[b, h * G + i].double()
                    z = (k[pos].double() @ x) / math.sqrt(cfg.d)
                    ro = torch.softmax(z, 0) @ v[pos].double()
                    size = torch.tensor([float((k[pos].double().abs() @ x.abs()).max()) / math.sqrt(cfg.d), float(v[pos].abs().max())])
                    tol, _ = tolerances(ro[None, None], torch.zeros(1, 1), size[None, None], [cfg.K * cfg.C], cfg.d, q.dtype)
                    assert bool(((o[b, h * G + i].double() - ro).abs() <= tol[0, 0]).all()), (b, h, i)
        return seen


def _make(B, N, S, P, *, layers=1, C=16, K=4, Hkv=2, G=2, d=64, dtype=torch.bfloat16, sparse=True):
    cfg = pisa.make_cfg(B=B, Hq=Hkv * G, Hkv=Hkv, N=N, d=d, C=C, K=K, dtype=dtype)
    c = pisa.PagedCache(cfg, pisa.make_pages(S, P), layers=layers, sparse=sparse, device=DEV)
    for p in c.K + c.V:
        p.zero_()
    for p in c.pyr:   # a summary that was never written shows
        p.fill_(math.nan)
    return c, Story(c, layers)


# capacities: units of few tiles (one cluster each), and 4 times as many (shares of a list; rows by TMA, by single copies)
@pytest.mark.parametrize("N,S,dtype", [(512, 32, torch.bfloat16), (8192, 64, torch.bfloat16), (8192, 48, torch.bfloat16),
                                       (8192, 32, torch.float32)])
def test_captured_steps_go_on_across_forks(N, S, dtype):
    B, P = 5, 120
    g, r = torch.Generator().manual_seed(51), random.Random(52)
    c, story = _make(B, N, S, P, layers=2, dtype=dtype)
    Hkv, Hq, d = 2, 4, 64
    q = torch.zeros(B, Hq, d, dtype=dtype, device=DEV)
    new = [torch.zeros(B, Hkv, d, dtype=dtype, device=DEV) for _ in range(4)]
    o, o2, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(B, Hq, device=DEV)
    idx, one = torch.empty(B, Hkv, 4, **I32), torch.ones(B, **I32)
    first = [200, 31, 0, 77, 5]
    c.reserve(torch.tensor(first, **I32))
    story.m.reserve(first)
    prompt = [torch.randn(B, Hkv, 200, d, generator=g).to(dtype) for _ in range(4)]
    for layer in range(2):
        c.append(prompt[2 * layer].to(DEV), prompt[2 * layer + 1].to(DEV), layer)
        c.build_pyramid(layer)
    for b in range(B):
        story.add(b, [x[b, :, :first[b]] for x in prompt])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.reserve(one)
        c.attend(q, o, lse, new[0], new[1], 0)
        c.step(q, new[2], new[3], idx, o2, 1)
    story.check()
    seen = 0
    for turn in range(12):
        for t in [q] + new:
            t.copy_(torch.randn(t.shape, generator=g).to(dtype))
        graph.replay()
        story.m.reserve([1] * B)
        assert c.grant.tolist() == story.m.grant == [1] * B
        for b in range(B):
            story.add(b, [x[b].cpu()[:, None] for x in new])
        story.check()
        story.check_dense(0, q.cpu(), o, lse, story.m.lens)
        seen += story.check_sparse(1, q.cpu(), idx.cpu(), o2.cpu())
        if turn % 4 != 3:   # one, two and three forks between steps
            for _ in range(turn % 4 + 1):
                parent = [r.choice([b, r.randrange(B), r.randrange(B)]) for b in range(B)]
                c.fork(torch.tensor(parent, **I32))
                story.fork(parent)
            story.check()
        else:
            c.compact()
            story.m.compact()
    assert seen > 40


def test_counts_of_an_append_are_checked_and_may_be_longer():
    c, story = _make(2, 256, 16, 40)
    g = torch.Generator().manual_seed(63)
    c.reserve(torch.tensor([20, 30], **I32))
    story.m.reserve([20, 30])
    k, v = (torch.randn(2, 2, 30, 64, generator=g).bfloat16() for _ in range(2))
    for T in (1, 30):
        for bad in (torch.ones(2, dtype=torch.int64, device=DEV), torch.ones(1, **I32), torch.ones(2, dtype=torch.int32), torch.ones(4, **I32)[::2]):
            with pytest.raises(ValueError):
                c.append(k[:, :, :T].contiguous().to(DEV), v[:, :, :T].contiguous().to(DEV), count=bad)
    c.append(k.to(DEV), v.to(DEV), count=torch.tensor([20, 30, 7, 7], **I32))
    for b, n in enumerate((20, 30)):
        story.add(b, [k[b, :, :n], v[b, :, :n]])
    c.reserve(torch.ones(2, **I32))
    story.m.reserve([1, 1])
    k1, v1 = (torch.randn(2, 2, 64, generator=g).bfloat16() for _ in range(2))
    c.append(k1.to(DEV), v1.to(DEV), count=torch.tensor([1, 1, 0], **I32))
    for b in range(2):
        story.add(b, [k1[b][:, None], v1[b][:, None]])
    story.check()
    pyr = c.pyr[0].clone()
    c.build_pyramid()
    live = [(b, n) for b, n in enumerate(story.m.lens)]
    for b, n in live:   # level 1: means of at most 16 rows in 32 bits
        assert float((c.pyr[0][b, :, :-(-n // 16)] - pyr[b, :, :-(-n // 16)]).abs().max()) <= 16 * 2.0 ** -24 * 8


def test_a_captured_turn_with_its_fork_and_compaction():
    # everything of a beam step in one graph, replayed; eager calls in between
    B, N, S, P = 4, 512, 16, 130
    g, r = torch.Generator().manual_seed(59), random.Random(60)
    c, story = _make(B, N, S, P)
    lens = [50, 9, 17, 1]
    c.reserve(torch.tensor(lens, **I32))
    story.m.reserve(lens)
    k, v = (torch.randn(B, 2, 50, 64, generator=g).bfloat16() for _ in range(2))
    c.append(k.to(DEV), v.to(DEV))
    for b in range(B):
        story.add(b, [k[b, :, :lens[b]], v[b, :, :lens[b]]])
    parent, one = torch.arange(B, **I32), torch.ones(B, **I32)
    q, k1, v1 = (torch.zeros(B, h, 64, device=DEV).bfloat16() for h in (4, 2, 2))
    idx, o = torch.empty(B, 2, 4, **I32), torch.empty_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.fork(parent)
        c.compact()
        c.reserve(one)
        c.step(q, k1, v1, idx, o)
    story.check()
    for turn in range(8):
        p = [r.choice([b, r.randrange(B)]) for b in range(B)]
        parent.copy_(torch.tensor(p, dtype=torch.int32))
        for t in (q, k1, v1):
            t.copy_(torch.randn(t.shape, generator=g).bfloat16())
        graph.replay()
        story.fork(p)
        story.m.compact()
        story.m.reserve([1] * B)
        for b in range(B):
            story.add(b, [k1[b].cpu()[:, None], v1[b].cpu()[:, None]])
        story.check()
        story.check_sparse(0, q.cpu(), idx.cpu(), o.cpu())
        if turn == 4:
            c.free(torch.tensor([2], **I32))
            story.m.free([2])
            story.rows[2] = story.empty()


def test_nothing_is_in_hand_behind_a_fork():
    # rows may be written again once a reserve has given room: the forked rows' pages are shared
    c, story = _make(3, 256, 16, 60)
    g = torch.Generator().manual_seed(53)
    lens = [40, 5, 23]
    c.reserve(torch.tensor(lens, **I32))
    story.m.reserve(lens)
    k, v = (torch.randn(3, 2, 40, 64, generator=g).bfloat16() for _ in range(2))
    c.append(k.to(DEV), v.to(DEV))
    c.build_pyramid()
    for b in range(3):
        story.add(b, [k[b, :, :lens[b]], v[b, :, :lens[b]]])
    for parent in ([0, 0, 2], [1, 0, -1]):
        c.fork(torch.tensor(parent, **I32))
        story.fork(parent)
        before = [x.clone() for x in (c.K[0], c.V[0], c.pyr[0])]
        q, k1, v1 = (torch.randn(3, h, 64, generator=g).bfloat16().to(DEV) for h in (4, 2, 2))
        o, lse, idx = torch.ones(3, 4, 64, device=DEV).bfloat16(), torch.ones(3, 4, device=DEV), torch.zeros(3, 2, 4, **I32)
        c.step(q, k1, v1, idx, o)
        assert not o.any() and bool((idx == -1).all())
        o.fill_(1)
        c.attend(q, o, lse, k1, v1)
        assert not o.any() and bool((lse == -math.inf).all())
        c.append(k1, v1)
        c.append(torch.randn(3, 2, 50, 64, generator=g).bfloat16().to(DEV), torch.randn(3, 2, 50, 64, generator=g).bfloat16().to(DEV))
        story.check()
        for x, y in zip(before, (c.K[0], c.V[0], c.pyr[0])):
            assert torch.equal(x.float().nan_to_num(5.0), y.float().nan_to_num(5.0))
    c.reserve(torch.tensor([1, 0, 0], **I32))
    c.step(q, k1, v1, idx, o)
    assert bool((idx[0, :, 0] == 0).all()) and bool((idx[1:] == -1).all())


def test_freed_sequences_have_nothing_in_hand():
    # and those that go on keep their token
    c, story = _make(3, 256, 16, 60)
    g = torch.Generator().manual_seed(54)
    k, v = (torch.randn(3, 2, 30, 64, generator=g).bfloat16() for _ in range(2))
    c.reserve(torch.tensor([30, 20, 10], **I32))
    c.append(k.to(DEV), v.to(DEV))
    c.build_pyramid()
    c.reserve(torch.tensor([1, 1, 1], **I32))
    c.free(torch.tensor([0, 0, 7], **I32))
    before = [x.clone() for x in (c.K[0], c.V[0], c.pyr[0])]
    q, k1, v1 = (torch.randn(3, h, 64, generator=g).bfloat16().to(DEV) for h in (4, 2, 2))
    o, lse, idx = torch.ones(3, 4, 64, device=DEV).bfloat16(), torch.ones(3, 4, device=DEV), torch.zeros(3, 2, 4, **I32)
    c.step(q, k1, v1, idx, o)
    assert not o[0].any() and bool((idx[0] == -1).all()) and bool((idx[1:, :, 0] == 0).all())
    c.attend(q, o, lse, k1, v1)
    assert not o[0].any() and bool((lse[0] == -math.inf).all()) and bool((lse[1:] > -math.inf).all())
    c.append(k1, v1)
    changed = (c.K[0] != before[0]).any(-1).any(1).nonzero().tolist()
    assert sorted(changed) == sorted([[int(c.table[b, (n - 1) // 16]), (n - 1) % 16] for b, n in ((1, 21), (2, 11))])
    assert torch.equal(c.pyr[0][0].nan_to_num(5.0), before[2][0].nan_to_num(5.0))


@pytest.mark.parametrize("C,S,d,dtype", [(16, 48, 64, torch.float32), (64, 64, 128, torch.bfloat16), (7, 14, 64, torch.bfloat16)])
def test_one_token_s_summaries_are_the_contiguous_cache_s(C, S, d, dtype):
    B, Hkv, N = 6, 2, 700
    g = torch.Generator().manual_seed(56)
    cfg = pisa.make_cfg(B=B, Hq=Hkv, Hkv=Hkv, N=N, d=d, C=C, K=4, dtype=dtype)
    W = -(-N // S)
    pages = pisa.make_pages(S, B * W + 3)
    table = torch.randperm(B * W + 3, generator=g)[:B * W].view(B, W).int().to(DEV)
    n = torch.tensor([0, 1, C, 333, N - 3, C - 1], **I32)
    Kc, Vc = (torch.randn(B, Hkv, N, d, generator=g).to(dtype).to(DEV) for _ in range(2))
    Kp, Vp = (torch.zeros(B * W + 3, Hkv, S, d, dtype=dtype, device=DEV) for _ in range(2))
    pisa.pisa_paged_append(cfg, pages, Kc, Vc, n, n, table, Kp, Vp)
    pyr = torch.zeros(B, Hkv, pisa.pisa_pyramid_rows(cfg), d, device=DEV)
    pisa.pisa_build_pyramid_prefix(cfg, Kc, n, pyr)
    pyp = pyr.clone()
    for _ in range(3):
        k, v = (torch.randn(B, Hkv, d, generator=g).to(dtype).to(DEV) for _ in range(2))
        pisa.pisa_pyramid_append(cfg, Kc, Vc, pyr, k, v, n)
        n = n + 1
        pisa.pisa_paged_pyramid_append(cfg, pages, k, v, Kp, Vp, table, n, pyp)
        assert torch.equal(pyr, pyp)
    for b in range(B):
        pos = torch.arange(int(n[b]), device=DEV)
        for c, p in ((Kc, Kp), (Vc, Vp)):
            assert torch.equal(p[table[b].long()[pos // S], :, pos % S].transpose(0, 1), c[b, :, :int(n[b])])
    # no token, past the capacity, no page: untouched
    before = [x.clone() for x in (Kp, Vp, pyp)]
    table[3, (int(n[3]) - 1) // S] = pages.P
    pisa.pisa_paged_pyramid_append(cfg, pages, k, v, Kp, Vp, table, torch.tensor([0, -4, N + 1, int(n[3]), 0, 2 ** 31 - 1], **I32), pyp)
    for x, y in zip(before, (Kp, Vp, pyp)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("C,S,d,dtype", [(16, 32, 64, torch.float32), (64, 64, 128, torch.bfloat16)])
def test_summaries_count_absent_leaves_as_zero_keys(C, S, d, dtype):
    B, Hkv, N = 3, 2, 40 * C
    g = torch.Generator().manual_seed(58)
    cfg = pisa.make_cfg(B=B, Hq=Hkv, Hkv=Hkv, N=N, d=d, C=C, K=4, dtype=dtype)
    W = -(-N // S)
    P = B * W + 3
    table = torch.randperm(P, generator=g)[:B * W].view(B, W).int()
    K = torch.randn(P, Hkv, S, d, generator=g).to(dtype)
    lens = [33 * C + 5, 7 * C, 9]
    table[0, 3], table[0, 8], table[0, (lens[0] - 1) // S], table[1, 0], table[2] = -1, P, -2000000000, 10 ** 9, -1
    pyr = torch.full((B, Hkv, pisa.pisa_pyramid_rows(cfg), d), math.nan, device=DEV)
    pisa.pisa_paged_build_pyramid(cfg, pisa.make_pages(S, P), K.to(DEV), table.to(DEV), torch.tensor(lens, **I32), pyr)
    pyr = pyr.cpu().double()
    for b in range(B):
        pos = torch.arange(lens[b])
        page = table[b].long()[pos // S]
        x = K[page.clamp(0, P - 1), :, pos % S].double().masked_fill(((page < 0) | (page >= P))[:, None, None], 0.0).transpose(0, 1)
        x = torch.stack([x[:, i:i + C].mean(1) for i in range(0, lens[b], C)], 1)
        for level in range(1, pisa.pisa_num_levels(cfg) + 1):
            at = pisa.pisa_level_offset(cfg, level)
            got = pyr[b, :, at:at + x.shape[1]]
            # a mean of C rows in 32 bits, and a halving a level above: C + level roundings of 2^-24 of the largest key
            assert float((got - x).abs().max()) <= (C + level) * 2.0 ** -24 * 6, (b, level)
            x = torch.stack([x[:, i:i + 2].mean(1) for i in range(0, x.shape[1], 2)], 1)


def test_a_sparse_cache_of_pages_that_split_leaves_still_serves_densely():
    # there are no summaries to keep: append, attention and forks work, a step is refused
    c, story = _make(2, 256, 24, 40)
    g = torch.Generator().manual_seed(57)
    k, v = (torch.randn(2, 2, 30, 64, generator=g).bfloat16() for _ in range(2))
    c.reserve(torch.tensor([30, 7], **I32))
    story.m.reserve([30, 7])
    c.append(k.to(DEV), v.to(DEV))
    for b, n in enumerate((30, 7)):
        story.add(b, [k[b, :, :n], v[b, :, :n]])
    c.fork(torch.tensor([0, 0], **I32))
    story.fork([0, 0])
    c.reserve(torch.ones(2, **I32))
    story.m.reserve([1, 1])
    q, k1, v1 = (torch.randn(2, h, 64, generator=g).bfloat16() for h in (4, 2, 2))
    o, lse = torch.ones(2, 4, 64, device=DEV).bfloat16(), torch.ones(2, 4, device=DEV)
    c.attend(q.to(DEV), o, lse, k1.to(DEV), v1.to(DEV))
    for b in range(2):
        story.add(b, [k1[b][:, None], v1[b][:, None]])
    story.check()
    story.check_dense(0, q, o, lse, story.m.lens)
    with pytest.raises(pisa.PisaError) as e:
        c.step(q.to(DEV), k1.to(DEV), v1.to(DEV), torch.zeros(2, 2, 4, **I32), o)
    assert e.value.status == -2


@pytest.mark.parametrize("N,S,C,d,G,dtype", [(512, 32, 16, 64, 2, torch.bfloat16), (8192, 64, 32, 128, 4, torch.bfloat16),
                                             (4096, 48, 16, 64, 1, torch.float32)])
def test_a_layer_takes_dense_tokens_and_then_sparse_steps(N, S, C, d, G, dtype):
    """Short sequences are attended in full, longer ones sparsely: the summaries have to be there."""
    B, Hkv, K = 4, 2, 4
    g = torch.Generator().manual_seed(55)
    c, story = _make(B, N, S, 150, C=C, K=K, d=d, G=G, dtype=dtype)
    one = torch.ones(B, **I32)

    def rnd(*shape):
        return torch.randn(*shape, generator=g).to(dtype)

    def token(sparse):
        q, k, v = rnd(B, Hkv * G, d), rnd(B, Hkv, d), rnd(B, Hkv, d)
        grant = c.reserve(one).tolist()
        story.m.reserve([1] * B)
        for b in range(B):
            if grant[b]:
                story.add(b, [k[b][:, None], v[b][:, None]])
        o, lse, idx = torch.empty(B, Hkv * G, d, dtype=dtype, device=DEV), torch.empty(B, Hkv * G, device=DEV), torch.empty(B, Hkv, K, **I32)
        if sparse:
            c.step(q.to(DEV), k.to(DEV), v.to(DEV), idx, o)
        else:
            c.attend(q.to(DEV), o, lse, k.to(DEV), v.to(DEV))
        return q, idx, o, lse

    def prompt(add, T):
        k, v = rnd(B, Hkv, T, d), rnd(B, Hkv, T, d)
        c.reserve(torch.tensor(add, **I32))
        story.m.reserve(add)
        c.append(k.to(DEV), v.to(DEV))
        for b in range(B):
            story.add(b, [k[b, :, :add[b]], v[b, :, :add[b]]])

    seen = 0
    prompt([3 * C + 1, 0, 1, 9 * C], 9 * C)
    for _ in range(3):
        for _ in range(2 * C + 3):
            q, _, o, lse = token(False)
        story.check()
        story.check_dense(0, q, o, lse, story.m.lens)
        for _ in range(2):
            q, idx, o, _ = token(True)
            seen += story.check_sparse(0, q, idx.cpu(), o.cpu())
        # several rows behind what is there, by a count of the caller's; then a sparse step at once
        prompt([0, 5, 3 * C, 1], 3 * C)
        q, idx, o, _ = token(True)
        seen += story.check_sparse(0, q, idx.cpu(), o.cpu())
        # a token by append alone
        k, v = rnd(B, Hkv, d), rnd(B, Hkv, d)
        c.reserve(one)
        story.m.reserve([1] * B)
        c.append(k.to(DEV), v.to(DEV))
        for b in range(B):
            story.add(b, [k[b][:, None], v[b][:, None]])
        q, idx, o, _ = token(True)
        seen += story.check_sparse(0, q, idx.cpu(), o.cpu())
        story.check()
    assert seen > 40
