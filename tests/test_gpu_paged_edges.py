"""The paged decode cache at the edges of its number range: NaN and infinite keys and
summaries, values near the type's largest, probabilities that cancel."""
import math

import pytest
import torch

from hierarchical_block_sparse_b200 import pisa

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("a CUDA device is required for the gpu-marked tests")
    pisa.load()


def _step(cfg, S, q, Kc, Vc, lens, paged):
    """One step over keys Kc, Vc [B, Hkv, N, d], the token in hand being the last of lens[b]: idx and o."""
    B, Hkv, N, d = Kc.shape
    n = torch.tensor(lens, dtype=torch.int32)
    at = (n - 1)[:, None, None, None].long().expand(B, Hkv, 1, d)
    k, v = (x.gather(2, at)[:, :, 0].contiguous().to(DEV) for x in (Kc, Vc))
    pyr = torch.zeros(B, Hkv, pisa.pisa_pyramid_rows(cfg), d, device=DEV)
    pisa.pisa_build_pyramid_prefix(cfg, Kc.to(DEV), (n - 1).to(DEV), pyr)
    idx = torch.full((B, Hkv, cfg.K), -7, dtype=torch.int32, device=DEV)
    o = torch.full_like(q, 9.0, device=DEV)
    if paged:
        pool = [x.view(B, Hkv, N // S, S, d).transpose(1, 2).reshape(-1, Hkv, S, d).contiguous().to(DEV) for x in (Kc, Vc)]
        table = torch.arange(B * N // S, dtype=torch.int32, device=DEV).view(B, -1)
        pisa.pisa_paged_decode_step(cfg, pisa.make_pages(S, B * N // S), q.to(DEV), k, v, *pool, table, n.to(DEV), pyr, idx, o)
    else:
        pisa.pisa_decode_step(cfg, q.to(DEV), k, v, Kc.to(DEV), Vc.to(DEV), pyr, (n - 1).to(DEV), idx, o)
    torch.cuda.synchronize()
    return idx.cpu(), o.cpu()


STEP_FORMS = [(1, 128, 64, torch.bfloat16), (4, 128, 16, torch.bfloat16), (16, 64, 16, torch.bfloat16),
              (1, 64, 16, torch.float32), (8, 64, 32, torch.float32)]


@pytest.mark.parametrize("paged", [False, True], ids=["contiguous", "paged"])
@pytest.mark.parametrize("variant", [0, 1, 2])
@pytest.mark.parametrize("G,d,C,dtype", STEP_FORMS)
def test_nan_leaves_rank_behind_the_forced_ones_and_no_more_than_k_are_kept(G, d, C, dtype, variant, paged):
    # 40 leaves, K = 4: 0, 38 and 39 are forced, one place is left. A NaN leaf takes it, the lowest of several.
    B, Hkv, K, N = 4, 2, 4, 64 * C
    g = torch.Generator().manual_seed(31)
    cfg = pisa.make_cfg(B=B, Hq=Hkv * G, Hkv=Hkv, N=N, d=d, C=C, K=K, dtype=dtype, score_variant=variant)
    Kc, Vc = (torch.randn(B, Hkv, N, d, generator=g).to(dtype) for _ in range(2))
    q = torch.randn(B, Hkv * G, d, generator=g).to(dtype)
    n = 40 * C - 3
    Kc[0, :, 7 * C + 2] = math.nan
    for leaf in (20, 5, 31, 9):
        Kc[1, :, leaf * C + 1] = math.nan
    Kc[2, 0] = math.nan              # everything, of one head
    idx, o = _step(cfg, C, q, Kc, Vc, [n] * B, paged)
    assert idx[0].tolist() == [[0, 7, 38, 39]] * Hkv
    assert idx[1].tolist() == [[0, 5, 38, 39]] * Hkv
    assert idx[2, 0].tolist() == [0, 1, 38, 39]
    Kc[2, 0] = torch.randn(N, d, generator=g).to(dtype)
    Kc[:2] = torch.randn(2, Hkv, N, d, generator=g).to(dtype)
    again, o2 = _step(cfg, C, q, Kc, Vc, [n] * B, paged)   # the others do not notice
    assert torch.equal(again[3], idx[3]) and torch.equal(o2[3], o[3])
    assert torch.equal(again[2, 1], idx[2, 1]) and torch.equal(o2[2, G:], o[2, G:])
    assert bool(torch.isfinite(o2).all())
