"""Refusals of pisa_paged_pyramid_append before anything reaches a device."""
import ctypes

import pytest

from hierarchical_block_sparse_b200 import build as pisa_build
from hierarchical_block_sparse_b200 import pisa

A = [ctypes.c_void_p(1 << 16 | i << 12) for i in range(7)]   # distinct, aligned, never dereferenced
BAD4, BAD16 = ctypes.c_void_p((1 << 20) + 2), ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def fn():
    pisa_build.build()
    return pisa.load().pisa_paged_pyramid_append


def _cfg(**kw):
    return pisa.make_cfg(**{**dict(B=2, Hq=4, Hkv=2, N=1000, d=128, C=16, K=4), **kw})


def test_refused_before_launch(fn):
    pages = pisa.make_pages(64, 50)
    assert fn(None, pages, *A, None) == -1 and fn(_cfg(), None, *A, None) == -1
    for kw, status in [(dict(B=0), -1), (dict(N=-1), -1), (dict(d=96), -2), (dict(C=2000), -2), (dict(N=2 ** 30 + 1), -2), (dict(N=0), 0)]:
        assert fn(_cfg(**kw), pages, *A, None) == status, kw
    assert fn(_cfg(), pisa.make_pages(40, 50), *A, None) == -2       # pages that split leaves
    assert fn(_cfg(), pisa.make_pages(1025, 50), *A, None) == -2
    assert fn(_cfg(), pages, A[0], A[1], A[2], A[2], *A[4:], None) == -1   # K and V one pool
    for i in range(7):   # k_new, v_new, K, V, table, len, pyr
        assert fn(_cfg(), pages, *A[:i], None, *A[i + 1:], None) == -1, i
        bad = BAD4 if i in (4, 5) else BAD16
        assert fn(_cfg(), pages, *A[:i], bad, *A[i + 1:], None) == -4, i
