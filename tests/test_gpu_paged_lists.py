"""Attention over a paged cache where a unit has more tiles than a cluster takes: the list of
tiles in shares, its rows by TMA (pages of whole row groups) and by single copies (others).
Capacities of 8 K tokens for every head width and type: more than 32 tiles a unit."""
import math

import pytest
import torch

from hierarchical_block_sparse_b200 import pisa
from tests.paged_ref import attend64
from tests.test_gpu_paged import _attend, _cache, _check

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
N = 8192
TYPES = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
PAGES = pytest.mark.parametrize("S", [64, 20], ids=["tma", "copies"])   # 20: no multiple of a tile's 8, 16 or 32 rows


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("a CUDA device is required for the gpu-marked tests")
    pisa.load()


@TYPES
@PAGES
@pytest.mark.parametrize("Hkv,G,d,lens", [(2, 4, 128, [0, 1, 20, 64, 65, 21, 5000, 81, 700, 4097]), (1, 1, 64, [2600]), (2, 16, 64, [3000, 2, 33]),
                                          (4, 2, 64, [(i * 37) % 300 for i in range(90)]), (1, 8, 128, [4000, 0, 1])])
def test_the_token_appended_on_the_way(Hkv, G, d, lens, S, dtype):
    cfg, pages, q, K, V, table, n = _cache(lens, Hkv=Hkv, G=G, d=d, S=S, N=N, dtype=dtype, seed=61)
    lost = 7 if len(lens) > 7 else None
    if lost:
        table[lost, (lens[lost] - 1) // S] = -1   # no page for the token: not written, not counted
    g = torch.Generator().manual_seed(62)
    k_new, v_new = (torch.randn(len(lens), Hkv, d, generator=g).to(dtype) for _ in range(2))
    o, lse, K1, V1 = _attend(cfg, pages, q, K, V, table, n, k_new, v_new)
    Kw, Vw = K.clone(), V.clone()
    for b, x in enumerate(lens):
        if x and b != lost:
            at = int(table[b, (x - 1) // S]), slice(None), (x - 1) % S
            Kw[at], Vw[at] = k_new[b], v_new[b]
    for got, want in ((K1, Kw), (V1, Vw)):
        assert torch.equal(got.nan_to_num(5.0), want.nan_to_num(5.0))
    _check(o, lse, q, K1, V1, table, n, S, G)
    o2, lse2, _, _ = _attend(cfg, pages, q, K1, V1, table, n)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@TYPES
@PAGES
def test_a_length_past_the_capacity_appends_nothing(S, dtype):
    cfg, pages, q, K, V, table, _ = _cache([N, N, 0], Hkv=2, G=2, d=128, S=S, N=N, dtype=dtype, seed=63)
    k_new, v_new = torch.full((3, 2, 128), 9.0).to(dtype), torch.full((3, 2, 128), 9.0).to(dtype)
    lens = torch.tensor([N + 1, N, -1], dtype=torch.int32)
    o, lse, K1, V1 = _attend(cfg, pages, q, K, V, table, lens, k_new, v_new)
    page, row = table[:, (N - 1) // S].long(), (N - 1) % S
    for was, now in ((K, K1), (V, V1)):
        assert torch.equal(now[page[0], :, row], was[page[0], :, row]) and bool((now[page[1], :, row] == 9).all())
        assert int((now.nan_to_num(5.0) != was.nan_to_num(5.0)).any(-1).sum()) == 2   # two heads' rows
    _check(o, lse, q, K1, V1, table, lens.clamp(0, N), S, 2)


@TYPES
@PAGES
def test_absent_pages_and_clamped_lengths(S, dtype):
    cfg, pages, q, K, V, table, _ = _cache([6400, 6400, 200, 1000], Hkv=2, G=2, d=64, S=S, N=N, dtype=dtype, seed=64)
    table[0, 3], table[0, 7], table[0, 99] = -1, pages.P, -2000000000
    table[0, 40:45] = pages.P + 5
    table[3] = -1
    lens = torch.tensor([6400, 10 ** 9, -5, 1000], dtype=torch.int32)
    o, lse, _, _ = _attend(cfg, pages, q, K, V, table, lens)
    _check(o, lse, q, K, V, table, lens.clamp(0, N), S, 2)


@TYPES
@PAGES
def test_infinite_and_nan_keys_that_count(S, dtype):
    cfg, pages, q, K, V, table, lens = _cache([5000, 3000, 2000], Hkv=2, G=2, d=64, S=S, N=N, dtype=dtype, seed=65)
    K[int(table[0, 4000 // S]), 0, 4000 % S] = math.nan
    V[int(table[1, 100 // S]), 1, 100 % S, 9] = math.inf
    K[int(table[2, 5]), 0, 3] = math.inf     # logits of both signs of infinity, or of their sum
    o, lse, _, _ = _attend(cfg, pages, q, K, V, table, lens)
    assert torch.isnan(o[0, :2]).all() and torch.isnan(lse[0, :2]).all()
    assert bool((o[1, 2:, 9] == math.inf).all()) and bool(torch.isfinite(o[1, 2:, :9]).all())
    assert torch.isnan(o[2, :2]).all()
    whole = [(0, slice(2, 4)), (1, slice(0, 2)), (2, slice(2, 4))]
    ro, _, _ = attend64(q, K.nan_to_num(0.0, 0.0), V.nan_to_num(0.0, 0.0), table, lens, S, 2)
    for b, h in whole:
        assert float((o[b, h].double() - ro[b, h]).abs().max()) < 2e-2


@TYPES
@PAGES
def test_a_captured_call_follows_lengths_that_grow_and_shrink(S, dtype):
    # the shares, the cuts and the join change with the lengths alone
    lens = [4000, 2000, 1000, 0]
    cfg, pages, q, K, V, table, n = _cache([8000, 8000, 8000, 8000], Hkv=2, G=4, d=128, S=S, N=N, dtype=dtype, seed=66)
    dev = [x.to(DEV) for x in (q, K, V, table)]
    dl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    o, lse, ws = torch.empty_like(dev[0]), torch.empty(4, 8, device=DEV), pisa.alloc_paged_workspace(cfg, pages, DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pisa.pisa_paged_attn(cfg, pages, dev[0], None, None, *dev[1:], dl, o, lse, ws)
    for lens in ([4000, 2000, 1000, 0], [1, 0, 0, 0], [0, 0, 0, 0], [8000, 8000, 8000, 8000], [63, 64, 65, 7999], [0, 0, 5, 129]):
        dl.copy_(torch.tensor(lens, dtype=torch.int32))
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        _check(o.cpu(), lse.cpu(), q, K, V, table, torch.tensor(lens, dtype=torch.int32), S, 4)
