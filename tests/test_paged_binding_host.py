"""Checks that the paged calls' binding makes on its tensors' shapes."""
import pytest
import torch

from hierarchical_block_sparse_b200 import pisa


class Fake:
    """A CUDA tensor of bf16 as far as the checks see."""
    is_cuda = True
    dtype = torch.bfloat16

    def __init__(self, *shape):
        self.shape = shape

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for x in self.shape:
            n *= x
        return n

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 16


class Ints(Fake):
    dtype = torch.int32


def test_appended_keys_and_values_have_as_many_rows():
    # with other rows a head's values would be read at the keys' stride
    cfg, pages = pisa.make_cfg(B=2, Hq=4, Hkv=2, N=100, d=64, C=16, K=4), pisa.make_pages(16, 20)
    pool = Fake(20, 2, 16, 64)
    for k, v in ((Fake(2, 2, 3, 64), Fake(2, 2, 5, 64)), (Fake(2, 2, 64), Fake(2, 2, 5, 64)), (Fake(2, 2, 5, 64), Fake(2, 2, 3, 64)),
                 (Fake(2, 2, 5, 64), Fake(2, 2, 64))):
        with pytest.raises(ValueError, match="rows|elements"):
            pisa.pisa_paged_append(cfg, pages, k, v, Ints(2), Ints(2), Ints(2, 7), pool, pool)


def test_calls_of_one_token_refuse_rows_of_several():
    # [B, Hkv, T, d] holds enough elements, but its rows are not where [B, Hkv, d] has them
    cfg, pages = pisa.make_cfg(B=2, Hq=4, Hkv=2, N=100, d=64, C=16, K=4), pisa.make_pages(16, 20)
    q, one, many, pool, table, lens, ws = Fake(2, 4, 64), Fake(2, 2, 64), Fake(2, 2, 3, 64), Fake(20, 2, 16, 64), Ints(2, 7), Ints(2), Fake(1)
    for k, v in ((many, many), (one, many), (many, one)):
        for call in (lambda: pisa.pisa_paged_attn(cfg, pages, q, k, v, pool, pool, table, lens, q, None, ws),
                     lambda: pisa.pisa_paged_pyramid_append(cfg, pages, k, v, pool, pool, table, lens, ws),
                     lambda: pisa.pisa_paged_decode_step(cfg, pages, q, k, v, pool, pool, table, lens, ws, lens, q)):
            with pytest.raises(ValueError, match="one row"):
                call()
