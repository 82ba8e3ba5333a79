"""Cached numbers as E5M2, at the low end of its range: what the header says it holds comes back as it is, the rest
as the nearest, ties to the even code."""
import os
import re

import numpy as np
import pytest
import torch

import mx4_reference as M

D = 256
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "dflash_mx4_cache.h")


def nearest(x):
    """FP64 numbers as E5M2 ones: steps of 2^-16 below 2^-14, two bits behind the leading one above."""
    e = np.maximum(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -40))), -14)
    step = 2.0 ** (e - 2)
    return np.clip(np.round(x / step) * step, -57344, 57344)  # (numpy rounds halves to even)


def test_the_range_that_the_header_states():
    with open(HEADER) as f:
        low, high, also = re.search(r"E5M2 2 /\* holds every number of the format from 2\^(-\d+) to (\d+), and 2\^(-\d+)",
                                    f.read()).groups()
    every = np.unique(np.concatenate([M.GRID[1:] * 2.0 ** e for e in range(-30, 20)]))
    held = every[nearest(every) == every]
    inside = (every >= 2.0 ** int(low)) & (every <= float(high))
    assert set(every[inside]) | {2.0 ** int(also)} == set(held)
    assert nearest(np.array([1.5 * 2.0 ** -16]))[0] == 2.0 ** -15


@pytest.mark.gpu
def test_read_at_the_low_end():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_verify_paged_e4m3_gb300 import binding as B, build
    build.build()
    codes = np.tile(np.arange(16, dtype=np.uint8), (16, 2, 16))
    scales = np.broadcast_to(127 - np.arange(12, 28, dtype=np.uint8)[:, None, None], (16, 2, 8))
    want = nearest(M.numbers(codes, scales))
    cache = B.Mx4Cache(2, D, 16, 1)
    pools = []
    for of_v in (False, True):
        pool = M.empty_pool(1, 16, 2)
        M.put(pool, np.arange(16), codes, scales, of_v)
        pools.append(torch.from_numpy(pool).cuda())
    got = cache.read(*pools, torch.arange(16, device="cuda"), dtype=torch.float8_e5m2)
    for x in got:
        assert np.array_equal(x.double().cpu().numpy(), want)
    assert (want == 1.5 * 2.0 ** -16).sum() == 0 and (want == 2.0 ** -15).any()
