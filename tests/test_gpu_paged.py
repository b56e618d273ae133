"""The paged decode cache on the GPU: attention against 64 bits, the page calls
against a plain model, the sparse step against the contiguous cache's, and runs
of them together as a serving program makes them."""
import math
import random

import numpy as np
import pytest
import torch

from hierarchical_block_sparse_b200 import pisa
from tests.paged_ref import PageModel, attend64, free_bits, tolerances

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("a CUDA device is required for the gpu-marked tests")
    pisa.load()


def _cache(lens, *, Hkv, G, d, S, N, dtype, seed, spare=3, noise=1.0):
    """Pools with random pages; every pool row that is no token is NaN."""
    g = torch.Generator().manual_seed(seed)
    B, W = len(lens), -(-N // S)
    used = sum(-(-n // S) for n in lens)
    P = used + spare
    perm = torch.randperm(P, generator=g)
    table = torch.full((B, W), -1, dtype=torch.int32)
    K = torch.full((P, Hkv, S, d), math.nan)
    V = torch.full((P, Hkv, S, d), math.nan)
    at = 0
    for b, n in enumerate(lens):
        for w in range(-(-n // S)):
            page, rows = int(perm[at]), min(S, n - w * S)
            table[b, w] = page
            K[page, :, :rows] = torch.randn(Hkv, rows, d, generator=g) * noise
            V[page, :, :rows] = torch.randn(Hkv, rows, d, generator=g)
            at += 1
    q = torch.randn(B, Hkv * G, d, generator=g).to(dtype)
    cfg = pisa.make_cfg(B=B, Hq=Hkv * G, Hkv=Hkv, N=N, d=d, C=16, K=4, dtype=dtype)
    return cfg, pisa.make_pages(S, P), q, K.to(dtype), V.to(dtype), table, torch.tensor(lens, dtype=torch.int32)


def _attend(cfg, pages, q, K, V, table, lens, k_new=None, v_new=None, ws=None):
    to = [None if x is None else x.to(DEV) for x in (q, k_new, v_new, K, V, table, lens)]
    o = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    if ws is None:  # arbitrary contents
        ws = pisa.alloc_paged_workspace(cfg, pages, DEV).fill_(0xFF)
    pisa.pisa_paged_attn(cfg, pages, *to, o, lse, ws)
    torch.cuda.synchronize()
    return o.cpu(), lse.cpu(), to[3].cpu(), to[4].cpu()


def _check(o, lse, q, K, V, table, lens, S, G):
    ro, rl, size = attend64(q, K, V, table, lens, S, G)
    tol_o, tol_l = tolerances(ro, rl, size, lens.clamp(min=0), q.shape[-1], q.dtype)
    off = (o.double() - ro).abs() - tol_o
    assert not torch.isnan(o).any() and bool((off <= 0).all()), float(off.max())
    none = rl == -math.inf
    assert torch.equal(lse == -math.inf, none)
    off = ((lse.double() - rl).abs() - tol_l)[~none]
    assert off.numel() == 0 or float(off.max()) <= 0, float(off.max())


# (Hkv, G, d, S): head groups, both widths, pages that divide a tile, hold several and neither
SHAPES = [(8, 1, 128, 64), (2, 4, 128, 16), (2, 8, 64, 48), (1, 16, 128, 128), (3, 2, 64, 7), (2, 16, 64, 32), (1, 8, 128, 1)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("Hkv,G,d,S", SHAPES)
def test_attention_over_ragged_sequences(Hkv, G, d, S, dtype):
    lens = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 500, 0, 777, 1000]
    case = _cache(lens, Hkv=Hkv, G=G, d=d, S=S, N=1000, dtype=dtype, seed=1)
    o, lse, _, _ = _attend(*case)
    _check(o, lse, *case[2:], S, G)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,n,Hkv,G,d,S", [(1, 70000, 1, 2, 128, 64), (1, 33333, 2, 1, 64, 16), (300, 40, 2, 4, 64, 16),
                                           (40, 1200, 1, 16, 128, 32), (1, 1, 1, 1, 128, 64)])
def test_attention_split_and_joined(B, n, Hkv, G, d, S, dtype):
    # one long sequence cut into shares, and far more sequences than shares
    lens = [max(0, n - (b * 13) % (n + 1)) for b in range(B)]
    case = _cache(lens, Hkv=Hkv, G=G, d=d, S=S, N=n + 5, dtype=dtype, seed=2)
    o, lse, _, _ = _attend(*case)
    _check(o, lse, *case[2:], S, G)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_attention_of_large_logits(dtype):
    # keys 40 times as long: maxima move, most probabilities vanish
    case = _cache([2000, 1, 300], Hkv=2, G=4, d=128, S=64, N=2048, dtype=dtype, seed=3, noise=40.0)
    o, lse, _, _ = _attend(*case)
    _check(o, lse, *case[2:], 64, 4)


def test_attention_skips_absent_pages_and_clamps_lengths():
    cfg, pages, q, K, V, table, lens = _cache([640, 640, 200, 64], Hkv=2, G=2, d=64, S=32, N=640, dtype=torch.bfloat16, seed=4)
    table[0, 3], table[0, 7], table[0, 19] = -1, pages.P, -2000000000
    table[3] = -1            # a sequence without any page
    lens = torch.tensor([640, 10 ** 9, -5, 64], dtype=torch.int32)
    o, lse, _, _ = _attend(cfg, pages, q, K, V, table, lens)
    _check(o, lse, q, K, V, table, lens.clamp(0, 640), 32, 2)


def test_infinite_and_nan_keys_that_count():
    # as in the formula: a NaN logit or value spreads over its head, others are untouched
    cfg, pages, q, K, V, table, lens = _cache([100, 100], Hkv=2, G=2, d=64, S=16, N=128, dtype=torch.bfloat16, seed=5)
    K[int(table[0, 2]), 0, 3] = math.nan
    V[int(table[1, 1]), 1, 5, 9] = math.inf
    o, lse, _, _ = _attend(cfg, pages, q, K, V, table, lens)
    assert torch.isnan(o[0, :2]).all() and torch.isnan(lse[0, :2]).all()
    assert bool((o[1, 2:, 9] == math.inf).all()) and bool(torch.isfinite(o[1, 2:, :9]).all())
    ro, _, _ = attend64(q, K, V, table, lens, 16, 2)
    assert float((o[0, 2:].double() - ro[0, 2:]).abs().max()) < 2e-2 and float((o[1, :2].double() - ro[1, :2]).abs().max()) < 2e-2


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d,S", [(128, 64), (64, 24)])
def test_attention_with_the_token_appended_on_the_way(d, S, dtype):
    lens = [0, 1, S, S + 1, 640, 64, 65, 700]
    cfg, pages, q, K, V, table, n = _cache(lens, Hkv=2, G=4, d=d, S=S, N=704, dtype=dtype, seed=6)
    table[6, 64 // S] = -1  # no page for the token: not written, not counted
    g = torch.Generator().manual_seed(7)
    k_new, v_new = (torch.randn(len(lens), 2, d, generator=g).to(dtype) for _ in range(2))
    o, lse, K1, V1 = _attend(cfg, pages, q, K, V, table, n, k_new, v_new)
    Kd, Vd = K.to(DEV), V.to(DEV)
    one = torch.ones(len(lens), dtype=torch.int32, device=DEV)
    pisa.pisa_paged_append(cfg, pages, k_new.to(DEV), v_new.to(DEV), n.to(DEV), one, table.to(DEV), Kd, Vd)
    torch.cuda.synchronize()
    for a, b in ((K1, Kd.cpu()), (V1, Vd.cpu())):
        assert torch.equal(a.nan_to_num(5.0), b.nan_to_num(5.0))
    for b, x in enumerate(lens):
        if x and b != 6:
            assert torch.equal(K1[int(table[b, (x - 1) // S]), :, (x - 1) % S], k_new[b])
    o2, lse2, _, _ = _attend(cfg, pages, q, K1, V1, table, n)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    _check(o, lse, q, K1, V1, table, n, S, 4)


def test_a_length_past_the_capacity_appends_nothing():
    for S in (64, 24):   # rows by TMA, by single copies
        cfg, pages, q, K, V, table, n = _cache([640, 640], Hkv=2, G=2, d=128, S=S, N=640, dtype=torch.bfloat16, seed=16)
        k_new, v_new = torch.full((2, 2, 128), 9.0).bfloat16(), torch.full((2, 2, 128), 9.0).bfloat16()
        lens = torch.tensor([641, 640], dtype=torch.int32)
        o, lse, K1, V1 = _attend(cfg, pages, q, K, V, table, lens, k_new, v_new)
        page, row = table[:, 639 // S].long(), 639 % S
        assert torch.equal(K1[page[0], :, row], K[page[0], :, row]) and bool((K1[page[1], :, row] == 9).all())
        _check(o, lse, q, K1, V1, table, lens.clamp(max=640), S, 2)


@pytest.mark.parametrize("S,n,B", [(64, 5000, 3), (64, 200, 1), (24, 5000, 3)], ids=["tma", "cluster", "copies"])
def test_pools_past_32_bit_offsets(S, n, B):
    # 10 GB of keys, and as much of values: the pages in use lie at the end
    Hkv, G, d = 8, 2, 128
    P = 40_000_000 // (Hkv * S)
    cfg = pisa.make_cfg(B=B, Hq=Hkv * G, Hkv=Hkv, N=n, d=d, C=8, K=4)
    pages, W = pisa.make_pages(S, P), -(-n // S)
    K, V = (torch.empty(P, Hkv, S, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    assert K.numel() > 2 ** 32
    g = torch.Generator().manual_seed(17)
    table = (P - 1 - torch.randperm(B * W + 5, generator=g)[:B * W]).view(B, W).int().to(DEV)
    lens = torch.tensor([n - b for b in range(B)], dtype=torch.int32, device=DEV)
    k, v = (torch.randn(B, Hkv, n, d, generator=g).bfloat16() for _ in range(2))
    pisa.pisa_paged_append(cfg, pages, k.to(DEV), v.to(DEV), lens, lens, table, K, V)
    q = torch.randn(B, Hkv * G, d, generator=g).bfloat16()
    o, lse = torch.empty(B, Hkv * G, d, dtype=torch.bfloat16, device=DEV), torch.empty(B, Hkv * G, device=DEV)
    pisa.pisa_paged_attn(cfg, pages, q.to(DEV), None, None, K, V, table, lens, o, lse, pisa.alloc_paged_workspace(cfg, pages, DEV))
    small = [x.view(B, Hkv, n, 1, d).transpose(1, 2).reshape(B * n, Hkv, 1, d) for x in (k, v)]
    flat = torch.arange(B * n, dtype=torch.int32).view(B, n)
    _check(o.cpu(), lse.cpu(), q, *small, flat, lens.cpu(), 1, G)
    moves = torch.tensor([1, 0, 0, 0, int(table[0, 0]), P - 1 - (B * W + 10)], dtype=torch.int32, device=DEV)
    pisa.pisa_pages_copy(cfg, pages, moves, K, V)
    torch.cuda.synchronize()
    rows = min(S, n)
    assert torch.equal(K[int(moves[5]), :, :rows].cpu(), k[0, :, :rows]) and torch.equal(V[int(moves[5]), :, :rows].cpu(), v[0, :, :rows])


def test_two_calls_at_once():
    # two streams, a workspace each, one cache
    cfg, pages, q, K, V, table, lens = [x.to(DEV) if torch.is_tensor(x) else x for x in
                                        _cache([30000, 77, 5000], Hkv=2, G=4, d=128, S=64, N=30000, dtype=torch.bfloat16, seed=18)]
    ws = [pisa.alloc_paged_workspace(cfg, pages, DEV) for _ in range(2)]
    want = torch.empty_like(q)
    pisa.pisa_paged_attn(cfg, pages, q, None, None, K, V, table, lens, want, None, ws[0])
    outs = [[torch.empty_like(q) for _ in range(20)] for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(20):
        for s in range(2):
            with torch.cuda.stream(streams[s]):
                pisa.pisa_paged_attn(cfg, pages, q, None, None, K, V, table, lens, outs[s][i], None, ws[s])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for group in outs for o in group)


def test_attention_gives_equal_bits_and_leaves_its_inputs():
    case = _cache([5000, 3, 0, 900], Hkv=2, G=8, d=128, S=16, N=5000, dtype=torch.bfloat16, seed=8)
    first = _attend(*case)
    for _ in range(3):
        again = _attend(*case, ws=torch.randint(0, 255, (pisa.pisa_paged_workspace_bytes(*case[:2]),), dtype=torch.uint8, device=DEV))
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    assert torch.equal(first[2].nan_to_num(5.0), case[3].nan_to_num(5.0))


def test_attention_without_lse_and_on_another_stream():
    cfg, pages, q, K, V, table, lens = [x.to(DEV) if torch.is_tensor(x) else x for x in
                                        _cache([1000, 77], Hkv=2, G=2, d=128, S=64, N=1024, dtype=torch.bfloat16, seed=9)]
    ws = pisa.alloc_paged_workspace(cfg, pages, DEV)
    o, o2 = torch.empty_like(q), torch.empty_like(q)
    pisa.pisa_paged_attn(cfg, pages, q, None, None, K, V, table, lens, o, None, ws)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        pisa.pisa_paged_attn(cfg, pages, q, None, None, K, V, table, lens, o2, None, ws)
    st.synchronize()
    assert torch.equal(o, o2)


def test_captured_steps_follow_the_lengths_and_share_a_workspace():
    # two graphs with one workspace, replayed in turn while the sequences grow
    S, N, B = 16, 512, 3
    cfg = pisa.make_cfg(B=B, Hq=4, Hkv=2, N=N, d=64, C=16, K=4, dtype=torch.float32)
    c = pisa.PagedCache(cfg, pisa.make_pages(S, 100), sparse=False, device=DEV)
    g = torch.Generator().manual_seed(10)
    k0, v0 = (torch.randn(B, 2, 200, 64, generator=g).to(DEV) for _ in range(2))
    c.reserve(torch.tensor([200, 31, 1], dtype=torch.int32, device=DEV))
    c.append(k0, v0)
    q, k, v = torch.zeros(B, 4, 64, device=DEV), torch.zeros(B, 2, 64, device=DEV), torch.zeros(B, 2, 64, device=DEV)
    o, o2, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(B, 4, device=DEV)
    one = torch.ones(B, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    step, look = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(step):
        c.reserve(one)
        c.attend(q, o, lse, k, v)
    with torch.cuda.graph(look):
        c.attend(q, o2)
    assert c.lens.tolist() == [200, 31, 1]
    for i in range(40):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g))
        step.replay()
        look.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and c.lens.tolist() == [201 + i, 32 + i, 2 + i]
        if i % 13 == 0:
            _check(o.cpu(), lse.cpu(), q.cpu(), c.K[0].cpu(), c.V[0].cpu(), c.table.cpu(), c.lens.cpu(), S, 2)


# ---- page calls ----------------------------------------------------------------------------

class Both:
    """A cache's integers on the GPU beside the plain model."""

    def __init__(self, B, N, S, P):
        self.m = PageModel(B, N, S, P)
        self.cfg = pisa.make_cfg(B=B, Hq=2, Hkv=2, N=N, d=64, C=16, K=4, dtype=torch.float32)
        self.pages = pisa.make_pages(S, P)
        i32 = dict(dtype=torch.int32, device=DEV)
        self.state = torch.full((pisa.pisa_pages_state_words(self.pages),), 77, **i32)
        self.table, self.lens = torch.full((B, self.m.W), 5, **i32), torch.full((B,), 5, **i32)
        self.other = (torch.empty_like(self.table), torch.empty_like(self.lens))
        self.grant, self.moves = torch.full((B,), -9, **i32), torch.full((4 + 2 * max(B, P // 2),), -9, **i32)
        pisa.pisa_pages_init(self.cfg, self.pages, self.state, self.table, self.lens)

    def reserve(self, add):
        a = torch.tensor(add, dtype=torch.int32, device=DEV)
        pisa.pisa_pages_reserve(self.cfg, self.pages, a, self.state, self.table, self.lens, self.grant, self.moves)
        self.m.reserve(add)
        self.check(moves=True)
        assert self.grant.tolist() == self.m.grant

    def fork(self, parent):
        p = torch.tensor(parent, dtype=torch.int32, device=DEV)
        pisa.pisa_pages_fork(self.cfg, self.pages, p, self.state, self.table, self.lens, *self.other)
        (self.table, self.lens), self.other = self.other, (self.table, self.lens)
        self.m.fork(parent)
        self.check()

    def free(self, seqs):
        pisa.pisa_pages_free(self.cfg, self.pages, torch.tensor(seqs, dtype=torch.int32, device=DEV), self.state, self.table, self.lens)
        self.m.free(seqs)
        self.check()

    def compact(self):
        pisa.pisa_pages_compact(self.cfg, self.pages, self.state, self.table, self.moves)
        self.m.compact()
        self.check(moves=True)

    def check(self, moves=False):
        m, state = self.m, self.state.cpu().numpy()
        assert self.table.tolist() == m.table
        assert self.lens.tolist() == m.lens
        assert state[:m.P].tolist() == m.refs
        assert free_bits(state, m.P) == [r == 0 for r in m.refs]
        if moves:
            got = self.moves.tolist()
            assert got[:4] == m.head
            assert got[4:4 + 2 * m.head[0]] == [x for pair in m.pairs for x in pair]


@pytest.mark.parametrize("B,N,S,P", [(6, 100, 8, 60), (33, 4000, 16, 1500), (5, 64, 1, 200), (1500, 40, 8, 5000),
                                     (3, 30, 64, 4), (8, 300, 7, 257), (4096, 20, 8, 9000)])
def test_page_calls_follow_the_model(B, N, S, P):
    r = random.Random(B)
    c = Both(B, N, S, P)
    c.check()
    for step in range(30 if B < 100 else 8):
        what = r.choice(["reserve", "reserve", "one", "fork", "free", "compact"])
        if what == "reserve":
            c.reserve([r.choice([0, -3, 1, S, r.randrange(1, N + 5)]) for _ in range(B)])
        elif what == "one":
            c.reserve([1] * B)
        elif what == "fork":
            c.fork([r.choice([b, b, r.randrange(B), -1, B, 2 ** 31 - 1]) for b in range(B)])
        elif what == "free":
            c.free([r.randrange(-1, B + 1) for _ in range(r.randrange(1, B + 1))])
        else:
            c.compact()


def test_sharers_of_a_last_page_copy_it_in_order():
    c = Both(6, 100, 8, 40)
    c.reserve([12, 0, 0, 0, 0, 0])
    c.fork([0, 0, 0, 0, 0, -1])
    c.reserve([1, 0, 1, 1, 0, 5])   # two holders stay: all three copy
    assert c.m.head[0] == 3
    c.reserve([0, 1, 0, 0, 1, 0])   # the last two: one copies, the other writes in place
    assert c.m.head[0] == 1
    c.fork([1, 0, 3, 2, 5, 4])      # swapped rows only
    c.reserve([1] * 6)
    assert c.m.head[0] == 0


def test_too_few_pages_give_none():
    c = Both(4, 64, 8, 10)
    c.reserve([8, 16, 24, 8])
    c.reserve([64, 1, 0, 30])
    assert c.m.head[1] == 2 and c.m.grant == [0] * 4   # 64 would pass N; 1 + 4 of 3 free pages
    c.fork([0, 1, 1, 1])
    c.reserve([0, 1, 1, 40])       # exactly the 7 that are free
    assert c.m.grant == [0, 1, 1, 40] and c.m.head[3] == 0
    c.reserve([0, 0, 0, 0])


def test_compaction_of_full_and_empty_pools():
    for P in (32, 64, 33, 2):
        c = Both(2, P, 1, P)
        c.compact()
        c.reserve([P // 2, P - P // 2])
        c.compact()
        c.free([0])
        c.compact()
        c.free([0, 1])
        c.compact()
    c = Both(2, 40000, 1, 70000)   # more words than the scanning block has threads
    c.reserve([30000, 40000])
    c.free([0, 0, 0])
    c.reserve([123, 0])
    c.compact()
    assert c.m.head[0] > 9000


def test_a_broken_table_neither_faults_nor_frees_twice():
    c = Both(3, 64, 8, 12)
    c.reserve([20, 20, 20])
    c.table[0, 1] = 99              # outside the pool
    c.table[1, 0] = -7
    c.table[2, 2] = c.table[2, 1]   # one page twice
    pisa.pisa_pages_free(c.cfg, c.pages, torch.arange(3, dtype=torch.int32, device=DEV), c.state, c.table, c.lens)
    refs = c.state[:12].tolist()
    assert min(refs) == 0 and c.table.tolist() == [[-1] * 8] * 3 and c.lens.tolist() == [0] * 3
    assert free_bits(c.state.cpu().numpy(), 12) == [x == 0 for x in refs]
    # a partial last page that is missing: no room is given
    pisa.pisa_pages_init(c.cfg, c.pages, c.state, c.table, c.lens)
    add = torch.tensor([5, 5, 5], dtype=torch.int32, device=DEV)
    pisa.pisa_pages_reserve(c.cfg, c.pages, add, c.state, c.table, c.lens, c.grant, c.moves)
    c.table[1, 0] = -1
    pisa.pisa_pages_reserve(c.cfg, c.pages, add, c.state, c.table, c.lens, c.grant, c.moves)
    assert c.grant.tolist() == [5, 0, 5] and c.lens.tolist() == [10, 5, 10]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("Hkv,S,d", [(1, 1, 64), (8, 64, 128), (3, 7, 64), (2, 33, 128)])
def test_page_copies(Hkv, S, d, dtype):
    P = 50
    cfg = pisa.make_cfg(B=1, Hq=Hkv, Hkv=Hkv, N=64, d=d, C=16, K=4, dtype=dtype)
    pages = pisa.make_pages(S, P)
    g = torch.Generator().manual_seed(11)
    K, V = (torch.randn(P, Hkv, S, d, generator=g).to(dtype) for _ in range(2))
    perm = torch.randperm(P, generator=g)[:40].view(20, 2)
    pairs = torch.cat([perm, torch.tensor([[-1, 3], [P, 4], [5, P], [6, -8]])]).int()
    moves = torch.cat([torch.tensor([24, 0, 0, 0]), pairs.view(-1)]).int()
    Kd, Vd = K.to(DEV), V.to(DEV)
    pisa.pisa_pages_copy(cfg, pages, moves.to(DEV), Kd, Vd)
    for x, y in ((K, Kd), (V, Vd)):
        x[perm[:, 1]] = x[perm[:, 0]]
        assert torch.equal(x, y.cpu())
    # a count beyond the list reads no further than the list
    moves[0] = 10 ** 9
    pisa.pisa_pages_copy(cfg, pages, moves[:8].to(DEV), Kd, Vd)
    K[pairs[:2, 1].long()] = K[pairs[:2, 0].long()]
    assert torch.equal(K, Kd.cpu())
    moves[0] = 0
    pisa.pisa_pages_copy(cfg, pages, moves.to(DEV), Kd, Vd)
    assert torch.equal(K, Kd.cpu())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,S,d,Hkv", [(1, 64, 128, 8), (37, 16, 64, 3), (300, 7, 128, 2)])
def test_append_rows(T, S, d, Hkv, dtype):
    B, N, P = 7, 400, 500
    g = torch.Generator().manual_seed(12)
    lens = torch.tensor([T, T + 5, 0, 400, 300, 401, 350], dtype=torch.int32)
    count = torch.tensor([T, min(T, 2), 0, T, T + 1, 1, -1], dtype=torch.int32)   # the last three are refused
    table = torch.randperm(P, generator=g)[:B * (-(-N // S))].view(B, -1).int() if S > 6 else None
    table[3, (400 - 1) // S] = -1   # no page for the last rows
    K, V = (torch.randn(P, Hkv, S, d, generator=g).to(dtype) for _ in range(2))
    k, v = (torch.randn(B, Hkv, T, d, generator=g).to(dtype) for _ in range(2))
    cfg = pisa.make_cfg(B=B, Hq=Hkv, Hkv=Hkv, N=N, d=d, C=16, K=4, dtype=dtype)
    Kd, Vd = K.to(DEV), V.to(DEV)
    pisa.pisa_paged_append(cfg, pisa.make_pages(S, P), k.to(DEV), v.to(DEV), lens.to(DEV), count.to(DEV), table.to(DEV), Kd, Vd)
    for b in range(4):
        for i in range(int(count[b])):
            t = int(lens[b]) - int(count[b]) + i
            page = int(table[b, t // S])
            if page >= 0:
                K[page, :, t % S], V[page, :, t % S] = k[b, :, i], v[b, :, i]
    assert torch.equal(K, Kd.cpu()) and torch.equal(V, Vd.cpu())


# ---- the sparse step over pages --------------------------------------------------------------

def _selected64(q, K, V, idx, n, C, G):
    """Attention of one token over its leaves idx [Hkv, K] of K, V [Hkv, N, d], and what its tolerance needs; in 64 bits."""
    Hq, d = q.shape
    o, size = torch.zeros(Hq, d, dtype=torch.float64), torch.zeros(Hq, 2, dtype=torch.float64)
    for h in range(Hq):
        pos = torch.cat([torch.arange(int(i) * C, min(int(i) * C + C, n)) for i in idx[h // G] if i >= 0])
        k, v, x = K[h // G, pos].double(), V[h // G, pos].double(), q[h].double()
        o[h] = torch.softmax((k @ x) / math.sqrt(d), 0) @ v
        size[h, 0], size[h, 1] = ((k.abs() @ x.abs()) / math.sqrt(d)).max(), v.abs().max()
    return o, size


STEPS = [
    (1, 128, 64, 8, 64, torch.bfloat16, 4096, [1000, 2049, 3001, 1]),
    (2, 128, 64, 8, 128, torch.bfloat16, 4000, [1000, 2048, 3999, 64]),
    (1, 64, 16, 4, 48, torch.float32, 1024, [100, 512, 990, 17]),
    (4, 64, 32, 8, 32, torch.bfloat16, 2048, [333, 1024, 2000, 31]),
    (8, 128, 64, 16, 64, torch.bfloat16, 4096, [4000, 1600, 63, 1023]),
    (8, 128, 64, 16, 64, torch.float32, 4096, [4000, 1600, 63, 1023]),
    (16, 64, 24, 16, 24, torch.float32, 2048, [2040, 700, 23, 500]),
    (2, 64, 7, 5, 14, torch.bfloat16, 500, [490, 7, 8, 300]),        # leaves that end inside a tile
    (16, 128, 64, 16, 64, torch.bfloat16, 4096, [4000, 1600, 63, 1023]),
    (16, 128, 128, 4, 256, torch.bfloat16, 4096, [1500, 2600, 4050, 128]),
    (4, 128, 1024, 16, 1024, torch.float32, 20000, [19000, 16500, 5, 1025]),   # logits too many to keep
]


@pytest.mark.parametrize("G,d,C,K,S,dtype,N,lens,variant", [x + (0,) for x in STEPS] + [x + (v,) for x in STEPS[:4] for v in (1, 2)])
def test_sparse_step_chooses_and_attends_as_the_contiguous_cache(G, d, C, K, S, dtype, N, lens, variant):
    B, Hkv = len(lens), 2
    g = torch.Generator().manual_seed(13)
    cfg = pisa.make_cfg(B=B, Hq=Hkv * G, Hkv=Hkv, N=N, d=d, C=C, K=K, dtype=dtype, score_variant=variant)
    W = -(-N // S)
    P = B * W + 3
    table = torch.randperm(P, generator=g)[:B * W].view(B, W).int().to(DEV)
    Kc, Vc = (torch.randn(B, Hkv, N, d, generator=g).to(dtype).to(DEV) for _ in range(2))
    Kp, Vp = (torch.full((P, Hkv, S, d), math.nan, dtype=dtype, device=DEV) for _ in range(2))
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    pages = pisa.make_pages(S, P)
    pisa.pisa_paged_append(cfg, pages, Kc, Vc, n, n, table, Kp, Vp)
    R = pisa.pisa_pyramid_rows(cfg)
    pyr, pyp = (torch.zeros(B, Hkv, R, d, device=DEV) for _ in range(2))
    pisa.pisa_build_pyramid_prefix(cfg, Kc, n, pyr)
    pisa.pisa_paged_build_pyramid(cfg, pages, Kp, table, n, pyp)
    assert torch.equal(pyr, pyp)
    other = 0
    for _ in range(4):
        q = torch.randn(B, Hkv * G, d, generator=g).to(dtype).to(DEV)
        k, v = (torch.randn(B, Hkv, d, generator=g).to(dtype).to(DEV) for _ in range(2))
        idx, idp = (torch.full((B, Hkv, K), -7, dtype=torch.int32, device=DEV) for _ in range(2))
        o, op = torch.empty_like(q), torch.full_like(q, 9.0)
        pisa.pisa_decode_step(cfg, q, k, v, Kc, Vc, pyr, n, idx, o)
        n = n + 1
        pisa.pisa_paged_decode_step(cfg, pages, q, k, v, Kp, Vp, table, n, pyp, idp, op)
        torch.cuda.synchronize()
        # a summary is a mean of C rows in 32 bits, in an order of the kernel's
        assert float((pyr - pyp).abs().max()) <= 2 * C * 2.0 ** -24 * float(Kc.abs().max())
        other += int((idx != idp).any(-1).sum())   # a tie to 32 bits may fall either way
        host = [x.cpu() for x in (q, Kc, Vc, idp, op)]
        for b in range(B):
            if int(n[b]) > N:
                assert bool((idp[b] == -1).all()) and not op[b].any()
                continue
            ro, size = _selected64(host[0][b], host[1][b], host[2][b], host[3][b], int(n[b]), C, G)
            tol, _ = tolerances(ro[None], torch.zeros(1, G * Hkv), size[None], [K * C], d, dtype)
            assert bool(((host[4][b].double() - ro).abs() <= tol[0]).all())
    assert other <= 1
    # out of range, no page for the token: untouched, idx -1, o 0
    bad = torch.tensor([0, N + 1, -3, lens[3]], dtype=torch.int32, device=DEV)
    table[3, (lens[3] - 1) // S] = P
    before = [x.clone() for x in (Kp, Vp, pyp)]
    pisa.pisa_paged_decode_step(cfg, pages, q, k, v, Kp, Vp, table, bad, pyp, idp, op)
    assert bool((idp == -1).all()) and bool((op == 0).all())
    for x, y in zip(before, (Kp, Vp, pyp)):
        assert torch.equal(x.nan_to_num(5.0), y.nan_to_num(5.0))


@pytest.mark.parametrize("paged", [False, True], ids=["contiguous", "paged"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_groups_of_16_rank_every_candidate(d, dtype, paged):
    # 32 candidate leaves x 16 heads are more than a block has threads: against the oracle's selection
    from oracle import oracle
    from tests.parity import TIE_BAND
    B, Hkv, G, C, K, N, S = 3, 1, 16, 32, 16, 2048, 64
    cfg = pisa.make_cfg(B=B, Hq=G, Hkv=Hkv, N=N, d=d, C=C, K=K, dtype=dtype)
    lens = torch.tensor([2000, 1100, 700], dtype=torch.int32)
    checked = 0
    for seed in range(3):   # other data each time: what an earlier launch left behind does not fit
        g = torch.Generator().manual_seed(100 + seed)
        Kc, Vc = (torch.randn(B, Hkv, N, d, generator=g).to(dtype) for _ in range(2))
        q = torch.randn(B, G, d, generator=g).to(dtype)
        new = (lens - 1)[:, None, None, None].long().expand(B, Hkv, 1, d)
        k, v = (x.gather(2, new)[:, :, 0].contiguous().to(DEV) for x in (Kc, Vc))
        pyr = torch.zeros(B, Hkv, pisa.pisa_pyramid_rows(cfg), d, device=DEV)
        pisa.pisa_build_pyramid_prefix(cfg, Kc.to(DEV), (lens - 1).to(DEV), pyr)
        idx, o = torch.empty(B, Hkv, K, dtype=torch.int32, device=DEV), torch.empty(B, G, d, dtype=dtype, device=DEV)
        if paged:
            pool = [x.view(B, Hkv, N // S, S, d).transpose(1, 2).reshape(-1, Hkv, S, d).contiguous().to(DEV) for x in (Kc, Vc)]
            table = torch.arange(B * N // S, dtype=torch.int32, device=DEV).view(B, -1)
            pisa.pisa_paged_decode_step(cfg, pisa.make_pages(S, B * N // S), q.to(DEV), k, v, *pool, table, lens.to(DEV), pyr, idx, o)
        else:
            pisa.pisa_decode_step(cfg, q.to(DEV), k, v, Kc.to(DEV), Vc.to(DEV), pyr, (lens - 1).to(DEV), idx, o)
        for b in range(B):
            n = int(lens[b])
            Kh = oracle.to_f64(Kc[b, 0, :n])
            Ph = oracle.build_pyramid(Kh, C, N=n, N_layout=N)
            want, gap = oracle.select_rows(oracle.to_f64(q[b])[None], np.array([n - 1]), Kh, Ph, C=C, K=K, N=n, N_layout=N)
            if gap[0] >= TIE_BAND:
                checked += 1
                assert idx[b, 0].tolist() == want[0].tolist()
    assert checked >= 6


def test_sparse_step_without_some_leaves():
    # leaves whose page is missing count as empty: never read, and nothing of them in the output
    B, Hkv, G, d, C, K, S, N = 1, 2, 2, 128, 64, 16, 64, 2048
    g = torch.Generator().manual_seed(21)
    cfg = pisa.make_cfg(B=B, Hq=Hkv * G, Hkv=Hkv, N=N, d=d, C=C, K=K)
    P = 40
    table = torch.randperm(P, generator=g)[:32].view(1, 32).int()
    Kp, Vp = (torch.randn(P, Hkv, S, d, generator=g).bfloat16() for _ in range(2))
    n, gone = 1000, [3, 7, 14]
    dev = [x.to(DEV) for x in (Kp, Vp, table)]
    pyr = torch.zeros(B, Hkv, pisa.pisa_pyramid_rows(cfg), d, device=DEV)
    pages, lens = pisa.make_pages(S, P), torch.tensor([n], dtype=torch.int32, device=DEV)
    pisa.pisa_paged_build_pyramid(cfg, pages, dev[0], dev[2], lens, pyr)
    dev[2][0, gone] = torch.tensor([-1, P, 10 ** 9], dtype=torch.int32, device=DEV)
    q, k, v = (torch.randn(B, h, d, generator=g).bfloat16() for h in (Hkv * G, Hkv, Hkv))
    idx, o = torch.empty(B, Hkv, K, dtype=torch.int32, device=DEV), torch.empty(B, Hkv * G, d, dtype=torch.bfloat16, device=DEV)
    pisa.pisa_paged_decode_step(cfg, pages, q.to(DEV), k.to(DEV), v.to(DEV), *dev, lens, pyr, idx, o)
    rows = [x[table[0].long()].transpose(0, 1).reshape(Hkv, N, d).clone() for x in (Kp, Vp)]
    for x, y in zip(rows, (k, v)):
        x[:, n - 1] = y[0]
    here = [i for i in range(16) if i not in gone]
    want = torch.tensor(here).expand(Hkv, -1)
    ro, size = _selected64(q[0], rows[0], rows[1], want, n, C, G)
    tol, _ = tolerances(ro[None], torch.zeros(1, G * Hkv), size[None], [K * C], d, torch.bfloat16)
    assert bool(((o[0].cpu().double() - ro).abs() <= tol[0]).all())


def test_a_step_without_pages_writes_nothing():
    # the pool is full and both sequences share their last page: no grant, so no row may be written
    cfg = pisa.make_cfg(B=2, Hq=4, Hkv=2, N=64, d=64, C=8, K=4, dtype=torch.float32)
    c = pisa.PagedCache(cfg, pisa.make_pages(8, 3), device=DEV)
    g = torch.Generator().manual_seed(19)
    i32 = dict(dtype=torch.int32, device=DEV)
    c.reserve(torch.tensor([20, 0], **i32))
    k, v = (torch.randn(2, 2, 20, 64, generator=g).to(DEV) for _ in range(2))
    c.append(k, v)
    c.fork(torch.tensor([0, 0], **i32))
    before = [x.clone() for x in (c.K[0], c.V[0], c.pyr[0], c.table, c.lens)]
    assert c.reserve(torch.ones(2, **i32)).tolist() == [0, 0] and int(c.moves[1]) == 1
    q, k1, v1 = (torch.randn(2, h, 64, generator=g).to(DEV) for h in (4, 2, 2))
    o, lse, idx = torch.ones(2, 4, 64, device=DEV), torch.ones(2, 4, device=DEV), torch.zeros(2, 2, 4, **i32)
    c.attend(q, o, lse, k1, v1)
    assert not o.any() and bool((lse == -math.inf).all())
    c.step(q, k1, v1, idx, o)
    assert not o.any() and bool((idx == -1).all())
    for x, y in zip(before, (c.K[0], c.V[0], c.pyr[0], c.table, c.lens)):
        assert torch.equal(x, y)
    c.attend(q, o, lse)      # what is cached can still be attended to
    assert bool((lse > -math.inf).all())
    c.free(torch.tensor([1], **i32))
    assert c.reserve(torch.tensor([1, 0], **i32)).tolist() == [1, 0]
    c.attend(q, o, lse, k1, v1)
    assert c.lens.tolist() == [21, 0] and bool((lse[0] > -math.inf).all()) and not o[1].any()


# ---- as a serving program uses them ------------------------------------------------------------

@pytest.mark.parametrize("dtype,S,C", [(torch.bfloat16, 32, 16), (torch.float32, 16, 16)])
def test_a_service_run(dtype, S, C):
    """Prompts come, tokens are generated (dense and sparse layer), beams fork, sequences
    end, the pool is compacted; every sequence's history stays what was put in."""
    B, Hkv, G, d, N, P = 5, 2, 2, 64, 256, 100
    g, r = torch.Generator().manual_seed(14), random.Random(15)
    cfg = pisa.make_cfg(B=B, Hq=Hkv * G, Hkv=Hkv, N=N, d=d, C=C, K=4, dtype=dtype)
    c = pisa.PagedCache(cfg, pisa.make_pages(S, P), layers=2, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    hist = [[torch.zeros(Hkv, 0, d, dtype=dtype) for _ in range(4)] for _ in range(B)]   # K, V of two layers

    def rnd(*shape):
        return torch.randn(*shape, generator=g).to(dtype)

    def put(b, rows):
        hist[b] = [torch.cat([x, y], 1) for x, y in zip(hist[b], rows)]

    def verify():
        torch.cuda.synchronize()
        assert c.lens.tolist() == [hist[b][0].shape[1] for b in range(B)]
        table = c.table.cpu().long()
        for b in range(B):
            pos = torch.arange(hist[b][0].shape[1])
            for i, pool in enumerate((c.K[0], c.V[0], c.K[1], c.V[1])):
                assert torch.equal(pool.cpu()[table[b][pos // S], :, pos % S].transpose(0, 1), hist[b][i])

    for turn in range(25):
        # prompts for the empty slots
        T = 40
        add = [r.randrange(1, T) if hist[b][0].shape[1] == 0 else 0 for b in range(B)]
        rows = [rnd(B, Hkv, T, d) for _ in range(4)]
        grant = c.reserve(torch.tensor(add, **i32)).clone()
        for layer in range(2):
            c.append(rows[2 * layer].to(DEV), rows[2 * layer + 1].to(DEV), layer)
            c.build_pyramid(layer, c.lens * (grant > 0).int())
        for b, n in enumerate(grant.tolist()):
            put(b, [x[b, :, :n] for x in rows])
        verify()
        for _ in range(6):  # tokens
            grant = c.reserve(torch.ones(B, **i32)).tolist()
            if sum(grant) == 0:
                break
            q, rows = rnd(B, Hkv * G, d), [rnd(B, Hkv, d) for _ in range(4)]
            for b in range(B):
                if grant[b]:
                    put(b, [x[b][:, None] for x in rows])
            o, lse = torch.empty(B, Hkv * G, d, dtype=dtype, device=DEV), torch.empty(B, Hkv * G, device=DEV)
            c.attend(q.to(DEV), o, lse, rows[0].to(DEV), rows[1].to(DEV), 0)
            idx, o2 = torch.empty(B, Hkv, 4, **i32), torch.empty_like(o)
            c.step(q.to(DEV), rows[2].to(DEV), rows[3].to(DEV), idx, o2, 1)
        verify()
        _check(o.cpu(), lse.cpu(), q, c.K[0].cpu(), c.V[0].cpu(), c.table.cpu(), c.lens.cpu(), S, G)
        # the sparse layer against a contiguous cache with the same history
        Kc, Vc = (torch.zeros(B, Hkv, N, d, dtype=dtype) for _ in range(2))
        for b in range(B):
            n = hist[b][0].shape[1]
            Kc[b, :, :n], Vc[b, :, :n] = hist[b][2], hist[b][3]
        pyr = torch.zeros(B, Hkv, pisa.pisa_pyramid_rows(cfg), d, device=DEV)
        pisa.pisa_build_pyramid_prefix(cfg, Kc.to(DEV), c.lens, pyr)
        want, o3 = torch.empty_like(idx), torch.empty_like(o)
        pisa.pisa_decode(cfg, q.to(DEV), Kc.to(DEV), Vc.to(DEV), pyr, c.lens - 1, want, o3)
        same = (idx == want).all(-1)
        assert int((~same).sum()) <= 1   # a tie may fall either way: one pyramid grew, the other was built
        same = same.repeat_interleave(G, 1)
        assert float((o2 - o3)[same].abs().max()) <= 2.0 ** -7 * float(o3.abs().max())
        # beams, ends, defragmentation
        if turn % 3 == 1:
            parent = [r.choice([b, b, r.randrange(B), -1]) for b in range(B)]
            c.fork(torch.tensor(parent, **i32))
            hist = [list(hist[p]) if p >= 0 else [torch.zeros(Hkv, 0, d, dtype=dtype)] * 4 for p in parent]
        if turn % 4 == 2:
            gone = [r.randrange(B), r.randrange(B)]
            c.free(torch.tensor(gone, **i32))
            for b in gone:
                hist[b] = [torch.zeros(Hkv, 0, d, dtype=dtype) for _ in range(4)]
        if turn % 5 == 3:
            c.compact()
        verify()
        if max(h[0].shape[1] for h in hist) > N - 50:
            c.free(torch.arange(B, **i32))
            hist = [[torch.zeros(Hkv, 0, d, dtype=dtype) for _ in range(4)] for _ in range(B)]
