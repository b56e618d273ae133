"""Host-side checks of the paged-cache calls: sizes, and refusals before anything
reaches a device."""
import ctypes

import pytest
import torch

from hierarchical_block_sparse_b200 import build as pisa_build
from hierarchical_block_sparse_b200 import pisa

A = [ctypes.c_void_p(1 << 16 | i << 12) for i in range(16)]   # distinct, aligned, never dereferenced
BAD4, BAD16 = ctypes.c_void_p((1 << 20) + 2), ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def lib():
    pisa_build.build()
    return pisa.load()


def _cfg(**kw):
    base = dict(B=2, Hq=4, Hkv=2, N=1000, d=128, C=16, K=4)
    base.update(kw)
    return pisa.make_cfg(**base)


# name -> (arguments after cfg and pages, positions of pointers that must be 16-byte aligned,
#          positions that may be null)
def _calls(cfg, pages):
    ws = max(int(pisa.load().pisa_paged_workspace_bytes(cfg, pages)), 0)
    big = 4 + 2 * max(cfg.B, pages.P)
    return {
        "pisa_pages_init": ([A[0], A[1], A[2]], [0], []),
        "pisa_pages_reserve": ([A[0], A[1], A[2], A[3], A[4], A[5], big], [1], []),
        "pisa_pages_fork": ([A[0], A[1], A[2], A[3], A[4], A[5]], [1], []),
        "pisa_pages_free": ([A[0], 2, A[1], A[2], A[3]], [2], []),
        "pisa_pages_compact": ([A[0], A[1], A[2], big], [0], []),
        "pisa_pages_copy": ([A[0], big, A[1], A[2]], [2, 3], []),
        "pisa_paged_append": ([A[0], A[1], 3, A[2], A[3], A[4], A[5], A[6]], [0, 1, 6, 7], []),
        "pisa_paged_attn": ([A[0], A[1], A[2], A[3], A[4], A[5], A[6], A[7], A[8], A[9], ws], [0, 1, 2, 3, 4, 7, 9], [1, 2, 8]),
        "pisa_paged_build_pyramid": ([A[0], A[1], A[2], A[3]], [0, 3], []),
        "pisa_paged_decode_step": ([A[i] for i in range(10)], [0, 1, 2, 3, 4, 7, 9], []),
    }


NAMES = ["pisa_pages_init", "pisa_pages_reserve", "pisa_pages_fork", "pisa_pages_free", "pisa_pages_compact",
         "pisa_pages_copy", "pisa_paged_append", "pisa_paged_attn", "pisa_paged_build_pyramid", "pisa_paged_decode_step"]


@pytest.mark.parametrize("name", NAMES)
def test_refused_before_launch(lib, name):
    pages = pisa.make_pages(64, 50)
    fn = getattr(lib, name)
    args, wide, optional = _calls(_cfg(), pages)[name]

    def call(cfg=None, pg=pages, a=args):
        return fn(cfg if cfg is not None else _cfg(), pg, *a, None)

    assert fn(None, pages, *args, None) == -1 and fn(_cfg(), None, *args, None) == -1
    for field, value, status in [("B", 0, -1), ("Hq", 3, -1), ("N", -1, -1), ("dtype", 9, -1), ("d", 96, -2), ("Hq", 6, -2),
                                 ("Hq", 64, -2), ("C", 2000, -2), ("N", 2 ** 30 + 1, -2)]:
        cfg = _cfg()
        setattr(cfg, field, value)
        assert call(cfg) == status, (field, value)
    for S, P, status in [(0, 50, -1), (64, 0, -1), (-4, 50, -1), (1025, 50, -2), (1024, 1 << 20, -2)]:
        assert call(pg=pisa.make_pages(S, P)) == status, (S, P)
    for i, x in enumerate(args):
        if not isinstance(x, ctypes.c_void_p):
            continue
        if i not in optional:
            assert call(a=args[:i] + [None] + args[i + 1:]) == -1, i
        bad = BAD16 if i in wide else BAD4
        assert call(a=args[:i] + [bad] + args[i + 1:]) == -4, i


def test_sizes(lib):
    assert pisa.pisa_pages_state_words(pisa.make_pages(64, 50)) == 2 * 52 + 3 * 4 + 16
    assert pisa.pisa_pages_state_words(pisa.make_pages(1, 1)) == 2 * 4 + 3 * 4 + 16
    assert lib.pisa_pages_state_words(pisa.make_pages(64, 0)) == -1
    for P in (1, 4, 5, 31, 32, 33, 127, 129, 100003):   # the binding's own count
        assert pisa.pisa_pages_state_words(pisa.make_pages(8, P)) == pisa._state_words(pisa.make_pages(8, P))
    pages = pisa.make_pages(64, 50)
    assert pisa.pages_width(_cfg(N=1000), pages) == 16
    one, sixteen = (pisa.pisa_paged_workspace_bytes(_cfg(Hq=2 * g), pages) for g in (1, 16))
    assert sixteen > 15 * one > 0
    assert lib.pisa_paged_workspace_bytes(_cfg(d=96), pages) == -2


def test_lists_too_short_and_aliases(lib):
    cfg, pages = _cfg(B=3), pisa.make_pages(64, 50)
    r, f = lib.pisa_pages_reserve, lib.pisa_pages_fork
    assert r(cfg, pages, *A[:6], 4 + 2 * 3 - 1, None) == -1
    assert r(_cfg(B=4097), pages, *A[:6], 1 << 20, None) == -2
    assert r(cfg, pages, A[0], A[1], A[2], A[3], A[0], A[5], 100, None) == -1     # grant over add
    assert r(cfg, pages, A[0], A[1], A[2], A[3], A[3], A[5], 100, None) == -1     # grant over len
    assert r(cfg, pages, A[3], A[1], A[2], A[3], A[4], A[5], 100, None) == -1     # add is len
    assert f(cfg, pages, A[0], A[1], A[2], A[3], A[2], A[5], None) == -1          # table in place
    assert f(cfg, pages, A[0], A[1], A[2], A[3], A[4], A[3], None) == -1          # lengths in place
    assert lib.pisa_pages_compact(cfg, pages, A[0], A[1], A[2], 4 + 50 - 1, None) == -1
    assert lib.pisa_pages_copy(cfg, pages, A[0], 3, A[1], A[2], None) == -1
    assert lib.pisa_pages_copy(cfg, pages, A[0], 10, A[1], A[1], None) == -1      # K and V one pool
    assert lib.pisa_pages_copy(cfg, pages, A[0], 5, A[1], A[2], None) == 0        # no room for a pair: nothing to do
    assert lib.pisa_pages_free(cfg, pages, A[0], -1, A[1], A[2], A[3], None) == -1
    assert lib.pisa_pages_free(cfg, pages, None, 0, A[1], A[2], A[3], None) == 0
    ap = lib.pisa_paged_append
    assert ap(cfg, pages, A[0], A[1], -1, *A[2:7], None) == -1
    assert ap(cfg, pages, A[0], A[1], 0, *A[2:7], None) == 0
    assert ap(cfg, pages, A[0], A[1], 1, A[2], A[3], A[4], A[5], A[5], None) == -1


def test_attention_refusals(lib):
    cfg, pages = _cfg(), pisa.make_pages(64, 50)
    n = pisa.pisa_paged_workspace_bytes(cfg, pages)
    fn = lib.pisa_paged_attn

    def call(c=cfg, k=A[1], v=A[2], ws=n):
        return fn(c, pages, A[0], k, v, *A[3:10], ws, None)

    assert call(k=None) == -1 and call(v=None) == -1        # one of the new rows only
    assert call(ws=n - 1) == -1
    assert call(_cfg(causal=False, forced_mask=4)) == -1
    assert call(_cfg(N=0)) == 0
    assert call(_cfg(B=64, N=2 ** 30), ws=1 << 30) == -2     # more tiles than 32 bits count


def test_sparse_calls_need_whole_leaves_in_a_page(lib):
    pages = pisa.make_pages(40, 50)
    args = _calls(_cfg(), pages)
    for name in ("pisa_paged_build_pyramid", "pisa_paged_decode_step"):
        assert getattr(lib, name)(_cfg(), pages, *args[name][0], None) == -2
    step = lib.pisa_paged_decode_step
    assert step(_cfg(causal=False, forced_mask=4), pisa.make_pages(64, 50), *args["pisa_paged_decode_step"][0], None) == -1


def test_binding_checks_its_tensors(lib):
    cfg, pages = _cfg(), pisa.make_pages(64, 50)
    i32 = torch.zeros(200, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pisa.pisa_pages_init(cfg, pages, i32, i32, i32)

    class Fake:   # a CUDA tensor as far as the checks see
        def __init__(self, dtype, n, contiguous=True, at=0):
            self.dtype, self.n, self.contiguous, self.at = dtype, n, contiguous, at
            self.is_cuda = at >= 0

        def get_device(self):
            return self.at

        def numel(self):
            return self.n

        def is_contiguous(self):
            return self.contiguous

        def data_ptr(self):
            return 1 << 16

    good = [Fake(torch.int32, 1000) for _ in range(3)]
    for i in range(3):
        for bad, text in ((Fake(torch.int64, 1000), "elements"), (Fake(torch.int32, 1), "elements"),
                          (Fake(torch.int32, 1000, contiguous=False), "contiguous"),
                          (Fake(torch.int32, 1000, at=1), "different devices"), (Fake(torch.int32, 1000, at=-1), "CUDA")):
            with pytest.raises(ValueError, match=text):
                pisa.pisa_pages_init(cfg, pages, *[bad if j == i else x for j, x in enumerate(good)])
