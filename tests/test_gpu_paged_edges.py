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


def _dense(q, K, V, lens, N):
    """pisa_paged_attn over keys K, V [B, Hkv, N, d], a page a sequence of 32 rows each; o and lse."""
    B, Hkv, _, d = K.shape
    S = 32
    cfg = pisa.make_cfg(B=B, Hq=q.shape[1], Hkv=Hkv, N=N, d=d, C=16, K=4, dtype=q.dtype)
    pool = [x.view(B, Hkv, N // S, S, d).transpose(1, 2).reshape(-1, Hkv, S, d).contiguous().to(DEV) for x in (K, V)]
    pages = pisa.make_pages(S, B * N // S)
    table = torch.arange(B * N // S, dtype=torch.int32, device=DEV).view(B, -1)
    o, lse = torch.full_like(q, 9.0, device=DEV), torch.full(q.shape[:2], 9.0, device=DEV)
    pisa.pisa_paged_attn(cfg, pages, q.to(DEV), None, None, *pool, table, torch.tensor(lens, dtype=torch.int32, device=DEV), o, lse,
                         pisa.alloc_paged_workspace(cfg, pages, DEV))
    torch.cuda.synchronize()
    return o.cpu(), lse.cpu()


@pytest.mark.parametrize("form", ["attention", "step"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8, 16])
def test_probabilities_keep_their_32_bits(G, d, form):
    """Two keys with logits 0 and -x, values v0 = -p v1 to bf16: what is left of the sum shows an
    error of p. In the unit p |v1|: a logit is one exact product, scaled (2^-24 of the scale, 2^-24 of
    the result, 2^-24 of the difference from the maximum or the normaliser, which has 2^-22 itself),
    |z| <= 4 in log2 units: below 2^-20 with the exponential's 2^-22. The sums have three terms of a
    probability in parts, six additions of 2^-23: 2^-20.4. In all 2^-19 of (|v0| + p |v1|) <= 2.1 p |v1|, and half a
    step of the result."""
    B, N, C = 256, 64, 32
    q = torch.zeros(B, G, d).bfloat16()
    K, V = torch.zeros(B, 1, N, d).bfloat16(), torch.zeros(B, 1, N, d).bfloat16()
    x = torch.arange(1, B + 1).double() / 128                 # k entries: at most 8 bits, exact
    q[..., 0] = math.sqrt(d) if d == 64 else 11.0
    K[:, 0, 1, 0] = (-x).bfloat16()
    z = -x * float(q[0, 0, 0]) / math.sqrt(d)
    p = torch.exp(z)
    g = torch.Generator().manual_seed(41)
    v1 = (1 + torch.randint(0, 128, (B, d), generator=g) / 128).bfloat16()
    v0 = (-p[:, None] * v1.double()).bfloat16()
    V[:, 0, 0], V[:, 0, 1] = v0, v1
    if form == "attention":
        o, _ = _dense(q, K, V, [2] * B, N)
    else:
        cfg = pisa.make_cfg(B=B, Hq=G, Hkv=1, N=N, d=d, C=C, K=4)
        _, o = _step(cfg, C, q, K, V, [2] * B, True)
    want = ((v0.double() + p[:, None] * v1.double()) / (1 + p[:, None]))[:, None].expand(B, G, d)
    unit = (p[:, None] * v1.double() / (1 + p[:, None]))[:, None]
    tol = torch.finfo(torch.bfloat16).eps / 2 * want.abs() + 2.1 * 2.0 ** -19 * unit
    off = (o.double() - want).abs() / tol
    assert float(off.max()) <= 1, float(off.max())


@pytest.mark.parametrize("G,d", [(1, 128), (2, 64), (4, 128), (8, 128), (8, 64), (16, 128)])
def test_long_sums_are_rounded_not_cut(G, d):
    """The same odd weights with values v in one half of 256 K keys and -v in the other: the output is 0.
    600 units keep one unit's keys in one block of 4 warps. In the unit v = 255 / 128: a tile's product
    may be cut in each of at most 3 parts (3 * 2^-23), and a warp adds 4096 tiles, partial sums at most half
    of its weights: roundings of 2^-24 of that, independent, so of deviation 64 * 2^-25 / sqrt(3) = 1.1e-6;
    six of it are 6.6e-6 a warp, 3.3e-6 for the mean of four, and 0.4e-6 for the cuts. Cuts in every addition
    alike would be 4096 / 2 * 2^-24 / 4 = 3e-5."""
    B, N, Hkv, S = 300, 262144, 2, 64
    cfg = pisa.make_cfg(B=B, Hq=Hkv * G, Hkv=Hkv, N=N, d=d, C=64, K=16)
    pages = pisa.make_pages(S, N // S)
    g = torch.Generator().manual_seed(44)
    w = torch.randn(N // 2, generator=g)
    K, V = torch.zeros(N, d), torch.full((N, d), 255 / 128)
    K[:, 0] = torch.cat([w, w])
    V[N // 2:] *= -1
    pool = [x.bfloat16().view(N // S, 1, S, d).expand(-1, Hkv, -1, -1).contiguous().to(DEV) for x in (K, V)]
    table = torch.arange(N // S, dtype=torch.int32, device=DEV).expand(B, -1).contiguous()
    q = torch.zeros(B, Hkv * G, d, device=DEV).bfloat16()
    q[..., 0] = 5.0
    o = torch.empty_like(q)
    pisa.pisa_paged_attn(cfg, pages, q, None, None, *pool, table, torch.full((B,), N, dtype=torch.int32, device=DEV), o, None,
                         pisa.alloc_paged_workspace(cfg, pages, DEV))
    assert float(o.float().abs().max()) <= 3.7e-6 * 255 / 128, float(o.float().abs().max())


@pytest.mark.parametrize("form", ["attention", "step"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("G,d", [(1, 128), (2, 64), (4, 128), (8, 64), (16, 128)])
def test_infinite_values_that_count_stay_infinite(G, d, dtype, form):
    # whatever bits the probability has: 1 of a single key, equal ones of two, odd ones of more
    B, N, C = 5, 64, 16
    g = torch.Generator().manual_seed(43)
    q, K = torch.randn(B, G, d, generator=g).to(dtype), torch.randn(B, 1, N, d, generator=g).to(dtype)
    K[1] = 0.0
    V = torch.randn(B, 1, N, d, generator=g).to(dtype)
    V[:, :, 0, 5], V[:, :, 0, 6] = math.inf, -math.inf
    lens = [1, 2, 3, 17, 60]
    if form == "attention":
        o, _ = _dense(q, K, V, lens, N)
    else:
        _, o = _step(pisa.make_cfg(B=B, Hq=G, Hkv=1, N=N, d=d, C=C, K=4, dtype=dtype), C, q, K, V, lens, True)
    assert bool((o[..., 5] == math.inf).all()) and bool((o[..., 6] == -math.inf).all())
    assert bool(torch.isfinite(o[..., :5]).all()) and bool(torch.isfinite(o[..., 7:]).all())


@pytest.mark.parametrize("form", ["attention", "step"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("G,d", [(1, 128), (2, 64), (4, 128), (8, 64), (16, 128)])
def test_keys_without_weight_add_nothing(G, d, dtype, form):
    # keys 1, 3, 5, ...: logits 300 below the others', values near the largest of the type; e^-300 of them is nothing
    B, N, C, n = 3, 64, 16, 50
    g = torch.Generator().manual_seed(42)
    q = torch.zeros(B, G, d).to(dtype)
    q[..., 0] = math.sqrt(d) if d == 64 else 8.0
    K, V = torch.zeros(B, 1, N, d).to(dtype), torch.randn(B, 1, N, d, generator=g).to(dtype)
    K[:, :, 1::2, 0] = -300.0 * math.sqrt(d) / float(q[0, 0, 0])
    V[:, :, 1::2] = 3.0e38 * torch.sign(torch.randn(B, 1, N // 2, d, generator=g)).to(dtype)
    if form == "attention":
        o, _ = _dense(q, K, V, [n] * B, N)
    else:
        _, o = _step(pisa.make_cfg(B=B, Hq=G, Hkv=1, N=N, d=d, C=C, K=4, dtype=dtype), C, q, K, V, [n] * B, True)
    want = V[:, :, 0:n:2].double().mean(2).expand(B, G, d)
    # 25 equal weights: the division's and the sums' roundings of 32 bits, below 2^-18 of the largest value, and the output's
    tol = torch.finfo(dtype).eps / 2 * want.abs() + 2.0 ** -18 * V[:, :, 0:n:2].double().abs().max()
    assert bool(((o.double() - want).abs() <= tol).all()), float((o.double() - want).abs().max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("G,d", [(1, 128), (2, 64), (4, 128), (8, 64), (16, 128)])
def test_large_values_behind_growing_logits_stay_finite(G, d, dtype):
    # a weighted mean of values of 2^120 is one of them, whatever the order in which the logits come
    B, N = 2, 1024
    q = torch.zeros(B, G, d).to(dtype)
    q[..., 0] = 8.0
    K, V = torch.zeros(B, 1, N, d).to(dtype), torch.full((B, 1, N, d), 2.0 ** 120).to(dtype)
    K[0, :, 512:, 0] = 5.0 * math.sqrt(d) / 8.0       # 7.2 in log2 units, short of what moves the maximum at once
    V[..., 1::2] *= -1
    for lens in ([1024, 1024], [700, 3]):
        o, lse = _dense(q, K, V, lens, N)
        # the weights' sum and the weighted sum agree to the roundings of 1024 terms in 32 bits
        assert bool(((o.double() / V[:, :, 0].double() - 1).abs() <= 2.0 ** -13 + torch.finfo(dtype).eps / 2).all())
        z = (K[:, 0, :, 0].double() * 8.0 / math.sqrt(d))
        for b in range(B):
            assert float((lse[b].double() - torch.logsumexp(z[b, :lens[b]], 0)).abs().max()) <= 2.0 ** -13


@pytest.mark.parametrize("paged", [False, True], ids=["contiguous", "paged"])
@pytest.mark.parametrize("variant", [0, 1])
@pytest.mark.parametrize("G,d,C,dtype", STEP_FORMS)
def test_nan_in_a_kept_leaf_is_seen(G, d, C, dtype, variant, paged):
    B, Hkv, K, N = 3, 2, 4, 16 * C
    g = torch.Generator().manual_seed(32)
    cfg = pisa.make_cfg(B=B, Hq=Hkv * G, Hkv=Hkv, N=N, d=d, C=C, K=K, dtype=dtype, score_variant=variant)
    Kc, Vc = (torch.randn(B, Hkv, N, d, generator=g).to(dtype) for _ in range(2))
    q = torch.randn(B, Hkv * G, d, generator=g).to(dtype)
    n = 10 * C - 1
    Kc[0, 0, 3] = math.nan               # leaf 0 is always kept
    Vc[1, 1, n - 2, 5] = math.nan        # and so is the current one
    Vc[1, 1, n - 2, 6] = math.inf
    idx, o = _step(cfg, C, q, Kc, Vc, [n] * B, paged)
    assert bool(torch.isnan(o[0, :G]).all()) and bool(torch.isfinite(o[0, G:]).all())
    assert bool(torch.isnan(o[1, G:, 5]).all()) and bool((o[1, G:, 6] == math.inf).all())
    rest = torch.ones(d, dtype=torch.bool)
    rest[5:7] = False
    assert bool(torch.isfinite(o[1][:, rest]).all()) and bool(torch.isfinite(o[1, :G]).all()) and bool(torch.isfinite(o[2]).all())


@pytest.mark.parametrize("form", ["contiguous", "paged", "attention"])
@pytest.mark.parametrize("G,d,C,dtype", STEP_FORMS)
def test_nothing_but_keys_of_minus_infinity_gives_0(G, d, C, dtype, form):
    # as for a sequence without keys: no key has any weight
    B, N = 3, 16 * C
    g = torch.Generator().manual_seed(34)
    Kc, Vc = (torch.randn(B, 1, N, d, generator=g).to(dtype) for _ in range(2))
    q = torch.randn(B, G, d, generator=g).to(dtype)
    q[..., 0] = 1.0
    Kc[:2, :, :, 0] = -math.inf
    lens = [1, 9 * C + 2, 9 * C + 2]
    if form == "attention":
        o, lse = _dense(q, Kc, Vc, lens, N)
        assert bool((lse[:2] == -math.inf).all())
    else:
        _, o = _step(pisa.make_cfg(B=B, Hq=G, Hkv=1, N=N, d=d, C=C, K=4, dtype=dtype), C, q, Kc, Vc, lens, form == "paged")
    assert not bool(o[:2].any()) and bool(torch.isfinite(o[2]).all()) and bool(o[2].any())


@pytest.mark.parametrize("paged", [False, True], ids=["contiguous", "paged"])
@pytest.mark.parametrize("G,d,C,dtype", STEP_FORMS)
def test_keys_of_minus_infinity_have_no_weight(G, d, C, dtype, paged):
    # logits of -inf: a whole leaf of them, a new leaf's only key, every second key of another leaf
    B, Hkv, K, N = 3, 2, 4, 16 * C
    g = torch.Generator().manual_seed(33)
    cfg = pisa.make_cfg(B=B, Hq=Hkv * G, Hkv=Hkv, N=N, d=d, C=C, K=K, dtype=dtype)
    Kc, Vc = (torch.randn(B, Hkv, N, d, generator=g).to(dtype) for _ in range(2))
    q = torch.randn(B, Hkv * G, d, generator=g).to(dtype)
    q[..., 0] = 1.0
    lens = [4 * C, 3 * C + 1, 10 * C + 1]
    Kc[0, :, C:2 * C, 0] = -math.inf
    Kc[1, :, 3 * C, 0] = -math.inf
    Kc[:, :, 2 * C:3 * C:2, 0] = -math.inf
    Kc[2, :, 5 * C:6 * C, 0] = -math.inf      # ranks last: there are better ones
    idx, o = _step(cfg, C, q, Kc, Vc, lens, paged)
    assert idx[0].tolist() == [[0, 1, 2, 3]] * Hkv and idx[1].tolist() == [[0, 1, 2, 3]] * Hkv and not bool((idx[2] == 5).any())
    for b in range(B):
        for h in range(Hkv * G):
            pos = torch.cat([torch.arange(int(i) * C, min(int(i) * C + C, lens[b])) for i in idx[b, h // G]])
            pos = pos[Kc[b, h // G, pos, 0] > -math.inf]
            k, v, x = Kc[b, h // G, pos].double(), Vc[b, h // G, pos].double(), q[b, h].double()
            want = torch.softmax((k @ x) / math.sqrt(d), 0) @ v
            # logits: (d + 4) 2^-24 of sum |q||k|; sums of up to 4 C terms; both in numerator and denominator
            size = float(((k.abs() @ x.abs()) / math.sqrt(d)).max())
            tol = torch.finfo(dtype).eps / 2 * want.abs() + 2 * ((d + 4) * 2.0 ** -24 * size + 2.0 ** -17 + 4 * C * 2.0 ** -24) * v.abs().max()
            assert bool(((o[b, h].double() - want).abs() <= tol).all()), (b, h)
