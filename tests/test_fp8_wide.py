"""Attention over the 8-bit cache by the form for many rows of a sequence (key
tiles expanded once, then read by row tiles of 256): every case here is large
enough for it, which its workspace shows, and the wide bound of
test_fp8_attention.py is used only for sequences that take it.
"""
import math

import numpy as np
import pytest
import torch

from online_kv_cache_tq_gb300 import binding as B

import test_fp8_attention as few
from test_fp8_cache import Model, ints

pytestmark = pytest.mark.gpu
WIDE_FROM = 144               # rows from which a sequence takes the form
WIDE_BYTES = 16 << 20         # more workspace than the other form has for any call


class Case(few.Case):
    def __init__(self, new, ctx, group=16, n_kv=1, **kw):
        super().__init__(new, ctx, group=group, n_kv=n_kv, **kw)
        assert self.nbytes > WIDE_BYTES, "the call is too small for the wide form"

    def check(self, sequences=None, tokens=40, blocked=(), code=0):
        torch.cuda.synchronize()
        assert B.tq_get_last_device_error(self.book) == code
        for b in range(self.batch) if sequences is None else sequences:
            super().check([b], tokens, blocked, wide=self.new[b] * self.group >= WIDE_FROM)


@pytest.mark.parametrize("near", [False, True])
def test_scores_far_below_zero_beside_blocks_of_tiny_scale(near):
    # Every score is -87, but the first of each 128 tokens', -79 (base 2; near: -43 and -47), and only two blocks hold values:
    # the others' scale is 2^-40, and their tokens are most of a row's sum.  Queries and keys are exact in fp16 and e4m3.
    ctx = 1984
    c = Case([300], [ctx], seed=1)
    kv = torch.zeros((ctx, 2, 1, 128), device="cuda")
    kv[:, 0] = -1.375
    kv[::128, 0] = -1.25
    kv[640:704, 1] = torch.randn((64, 1, 128), generator=c.g, device="cuda")
    kv[1280:1344, 1] = torch.randn((64, 1, 128), generator=c.g, device="cuda")
    c.write(kv, [ctx], [ctx])
    c.q.fill_(2.125 if near else 3.875)
    c.run()
    c.check(tokens=300)


def test_one_chunk_among_many_empty_sequences():
    # a sequence has all tokens of the call, which has as many tokens as sequences: before, behind and among empty ones
    ctx = 16384
    for at in (0, 100, 255):
        new, lengths = [0] * 256, [1] * 256
        new[at], lengths[at] = 256, ctx
        c = Case(new, lengths, group=64, seed=2)
        c.run()
        c.check([at], tokens=3)


def test_decode_steps_have_no_workspace_for_it():
    book = B.Codebook(block_size=64)
    for batch, n_q, n_kv, ctx in ((64, 64, 8, 32768), (256, 64, 8, 8192), (1, 64, 8, 1 << 20), (128, 64, 8, 700)):
        assert B.tq_fp8_workspace_bytes(book, batch, batch, n_q, n_kv, ctx) < WIDE_BYTES
