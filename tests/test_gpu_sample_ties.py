"""Nuclei whose border lies among equal logits, every row against oracle/sample.py."""
import pytest
import torch

from test_gpu_sample import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [700, 20000, 128256])
def test_no_row_is_near_a_border(V):
    """The shares asked for are nowhere a whole number of equals, and no uniform is (with these inputs): none is exempt."""
    g = torch.Generator().manual_seed(V)
    equal = torch.full((4, V), -3.25)
    few = torch.randint(0, 3, (4, V), generator=g).float() * 0.5
    zeros = torch.where(torch.rand((4, V), generator=g) < 0.5, 0.0, -0.0)
    u = torch.rand(4, generator=g).cuda()
    for z in (equal, few, zeros):
        for kw in (dict(top_p=0.37113), dict(top_p=0.91927), dict(top_k=600, top_p=0.41713),
                   dict(top_k=V // 2, top_p=0.71234, min_p=0.3)):
            check(z.cuda(), u, most_near=0, **kw)
