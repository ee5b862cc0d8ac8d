"""Commits of prompts into the 8-bit cache, whose pages' entries several groups of lanes share, bit-exact against the oracle."""
import math

import pytest
import torch

from test_gpu_kv8 import Commit

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,dtype", [("e4m3", "fp16"), ("e5m2", "bf16")])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page,S", [(9, 33), (16, 131), (24, 300), (100, 257), (600, 601)])
def test_prompts(fmt, dtype, D, page, S):
    """Twice, so that the second run's first page has a scale that may rise."""
    cols = -(-(2 * S + 8) // page) + 1
    c = Commit(3, S, 2, 2, D, page, 3 * cols, cols, fmt, dtype, seed=S + D)
    L = c.run([S - 1, S // 2, 0], [0, 3, 8])
    c.run([S // 3, S - 1, S - 1], L)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
def test_prompts_with_special_values(fmt, dtype, D):
    c = Commit(2, 40, 1, 2, D, 16, 12, 6, fmt, dtype, seed=D)
    x = c.staged.view(1, 2, 40, 2, 2, D)
    x[0, 0, 3, 0, 1, 5], x[0, 0, 14, 1, 0, D - 1], x[0, 0, 15, 0, 0, 0] = math.inf, -math.inf, math.nan
    x[0, 0, 20, 1, 1] = math.nan                              # an entry without a number
    x[0, 0, 32:, 0, 0] = -math.inf                            # a page without one
    x[0, 1, :17] = 0.0
    x[0, 1, 16, 1] = torch.finfo(x.dtype).smallest_normal / 8
    x[0, 1, 39] = torch.finfo(x.dtype).max
    L = c.run([39, 39], [1, 0])
    c.staged.mul_(4)
    c.run([9, 20], L)                                         # codes that are not finite, rounded again
    assert (c.scales > 0).all()


@pytest.mark.parametrize("page,S", [(1, 300), (2, 700)])
def test_ranges_of_more_pages_than_are_kept_at_hand(page, S):
    """More than 256 pages: the rest is looked up again."""
    cols = -(-(S + 8) // page) + 1
    c = Commit(2, S, 1, 1, 64, page, 2 * cols, cols, "e4m3", "bf16", seed=S)
    c.run([S - 1, S - 20], [0, 5])
