"""Edges of the paged-cache operators on the GPU: orders between units, weights near the types' ends, sizes near
32 bits.  Bounds and helpers are those of test_gpu_paged.
"""
import pytest
import torch

import test_gpu_paged as base
from test_gpu_paged import sdpa  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


# ------------------------------------------------------------------ one unit after the other
@pytest.mark.parametrize("fp8", [False, True], ids=["16_bits", "e4m3"])
def test_units_of_one_tile_behind_units_of_more(sdpa, fp8):  # noqa: F811
    """65 to 128 rows a key/value head: the chains take a unit's key tiles in turn and their sums meet in shared
    memory.  Behind a unit of two or three tiles comes one of a single tile, whose second chain has nothing to wait
    for: it must leave the sums before it alone until they are read.  About eight units a CTA, many times over."""
    b = 600
    lens = [(300, 100, 384, 60, 129, 128)[i % 6] for i in range(b)]
    news = [17 + i % 16 for i in range(b)]
    c = base._attend_case(41 + fp8, lens, news, 8, 2, 128, 16, BF, fp8)
    o, lse = base._call(sdpa, c)
    sdpa.sdpa_check_device_error()
    base._check(c, o, lse)
    for _ in range(60):
        x, y = base._call(sdpa, c)
        assert torch.equal(x, o) and torch.equal(y, lse)
