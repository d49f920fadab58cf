"""GPU tests of the block-scaled write at the ends of its ranges: block ids, positions and lengths near 2^31.

Exact: codes are roundings of exact values, counts are whole numbers."""
import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_slot_gb300 import bkv

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def test_a_cache_of_2_to_the_31_blocks():
    """A block past the table's columns is an error and none of the cache, whose last block's id is INT32_MAX, too."""
    total = 1 << 31
    k, v = (torch.zeros((total, 1, 1, 1), dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.ones((total, 1), device=DEV) for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    x = torch.tensor([3.0, 5.0], device=DEV).view(2, 1, 1)
    bkv.bkv_cache_write_fp8_blocks(x, x, _i32(0, 2), _i32(2), _i32(7).view(1, 1), k, v, ks, vs, err_count=err)
    assert int(err) == 1
    assert int(k[-1]) == 0 and int(v[-1]) == 0 and float(ks[-1]) == 1 and float(vs[-1]) == 1
    want = oracle.e4m3_encode(np.array([384.0], np.float32))[0]      # 3 / 2^-7, the smallest power with 3 <= 448 s
    assert int(k[7]) == want and int(v[7]) == want and float(ks[7]) == 2.0 ** -7
    # the last block, by its id
    bkv.bkv_cache_write_fp8_blocks(x, x, _i32(0, 1), _i32(1), _i32(2 ** 31 - 1).view(1, 1), k, v, ks, vs, err_count=err)
    assert int(err) == 1
    assert float(ks[-1]) == float(ks[7]) and int(k[-1]) == int(k[7]) != 0
    assert int((k.view(-1) != 0).sum()) == 2


def test_lengths_near_2_to_the_31():
    """A request that ends at position 2^31 - 2, with rows of the step behind its last token: its one block is past the
    table's columns, and the rows behind belong to nobody."""
    k, v = (torch.zeros((5, 1, 1, 8), dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.ones((5, 1), device=DEV) for _ in range(2))
    x = torch.ones((6, 1, 8), device=DEV)
    for lens, qsl in (([2 ** 31 - 1], [0, 1]), ([1, 2 ** 31 - 1], [0, 1, 2]), ([2 ** 31 - 1, 1], [0, 1, 2])):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        k.zero_(), v.zero_()
        table = torch.full((len(lens), 3), 2, dtype=torch.int32, device=DEV)
        bkv.bkv_cache_write_fp8_blocks(x, x, _i32(*qsl), _i32(*lens), table, k, v, ks, vs, err_count=err)
        assert int(err) == 1
        assert bool((k[[0, 1, 3, 4]] == 0).all()) and bool((v[[0, 1, 3, 4]] == 0).all())
        assert bool((k[2] != 0).all()) == (len(lens) == 2)
