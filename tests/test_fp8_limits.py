"""Attention over the 8-bit cache at the ends of its numbers: queries up to the
largest finite one, and weights far below a row's largest.  Tolerances as in
test_fp8_attention.py.
"""
import math

import numpy as np
import pytest
import torch

import test_fp8_run
from test_fp8_attention import Case, reference
from test_fp8_cache import Model

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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("depth", [4, 12, 15, 18, 21, 24])
def test_a_long_tail_beside_a_token_with_small_values(depth, dtype):
    # The first token's weight is 2^depth times that of each other and its values are small: the output is what the others
    # give.  A weight is held to 2^-11 of itself or 2^-26 of the row's largest (all blocks have one value scale), a score to D
    # (test_fp8_attention.py), the output rounded to bf16.
    ctx = 20000
    c = Case([2], [ctx], n_kv=1, group=4, dtype=dtype, seed=31)
    kv = torch.zeros((ctx, 2, 1, 128), device="cuda")
    kv[:, 1] = torch.rand((ctx, 1, 128), generator=c.g, device="cuda") + 0.5
    kv[0, 1] = 2.0 ** -9
    kv[0, 0] = 1.0
    c.write(kv, [ctx], [ctx])
    c.q.fill_(depth * math.log(2.0) / math.sqrt(128))     # (a key of ones: the first score is depth, base 2)
    c.run()
    c.check()
    k, v = (Model(c.cache).values(x, c.table[0], 0, ctx, 0) for x in "kv")
    q = c.q[-1, 0].double().cpu().numpy()
    s = k @ q / math.sqrt(128)
    p = np.exp(s - s[0]) / np.exp(s - s[0]).sum()
    d = np.linalg.norm(q)                                  # |q| |k| / sqrt(128), |k| at most sqrt(128)
    held = max(2.0 ** -11, 2.0 ** -26 * p[0] / p[1]) + np.expm1(2.0 ** -14 * d)
    bound = p[1:] @ v[1:] * held + p[0] * v[0] * held + 1.01 * 2.0 ** -8 * (p @ v)
    assert (np.abs(c.out[-1].double().cpu().numpy() - p @ v) <= bound).all()


def test_the_serving_loop_within_the_bound_of_few_rows(monkeypatch):
    # (the loop's calls are too small for the form with the wider one)
    monkeypatch.setattr(test_fp8_run, "reference", lambda q, k, v, n, scale, wide: reference(q, k, v, n, scale, False))
    loop = test_fp8_run.Loop()
    assert loop.nbytes < 16 << 20
    model, past = Model(loop.cache), [0, 0, 0]
    for new in ([70, 33, 0], [1, 40, 90], [1, 1, 1], [4, 0, 2], [1, 1, 1], [8, 8, 8]):
        loop.fill(new)
        loop.step()
        past = loop.check(model, new, past)
