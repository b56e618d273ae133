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
