"""Attention over the 8-bit cache at the ends of its numbers: queries up to the
largest finite one.  Tolerances as in test_fp8_attention.py.
"""
import pytest
import torch

from test_fp8_attention import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("new,group", [([1, 3], 4), ([9], 16)])
def test_the_largest_finite_queries(dtype, new, group):
    # coordinates in [2^127, 2^128) beside small ones, with a scale that brings the scores to ordinary size
    c = Case(new, [400, 300][:len(new)], group=group, dtype=dtype, scale=2.0 ** -126, seed=30)
    huge = torch.finfo(dtype).max
    q = torch.rand(c.q.shape, generator=c.g, device="cuda").sub_(0.5).mul_(2.0 ** 125)
    q[..., ::16] = 1.7e38 * 1.1 * torch.sign(q[..., ::16])
    q[..., 5] = -huge
    c.q.copy_(q.to(dtype))
    c.run()
    c.check()
