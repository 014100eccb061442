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
from online_kv_cache_tq_gb300 import cache as C

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
        for wide in (False, True):
            those = [b for b in (range(self.batch) if sequences is None else sequences)
                     if (self.new[b] * self.group >= WIDE_FROM) == wide]
            super().check(those, tokens, blocked, wide=wide)


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
    ctx = 8192
    for at in (0, 200, 511):
        new, lengths = [0] * 512, [1] * 512
        new[at], lengths[at] = 512, ctx
        c = Case(new, lengths, group=64, seed=2)
        c.run()
        c.check([at], tokens=3)


def test_decode_steps_have_no_workspace_for_it():
    book = B.Codebook(block_size=64)
    for batch, n_q, n_kv, ctx in ((64, 64, 8, 32768), (256, 64, 8, 1 << 20), (1, 64, 8, 1 << 20), (2048, 64, 8, 700)):
        assert B.tq_fp8_workspace_bytes(book, batch, batch, n_q, n_kv, ctx) < WIDE_BYTES


@pytest.mark.parametrize("bs", [32, 64, 96, 128, 256, 160])
@pytest.mark.parametrize("new,ctx,n_kv,group", [([200], [700], 2, 16), ([129, 250], [1000, 2051], 2, 4), ([37, 16, 300], [2000, 16, 555], 1, 16),
                                                ([300, 1, 128], [299, 2000, 600], 2, 8), ([513], [513], 4, 8), ([145], [9000], 5, 1)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prompt_chunks(bs, new, ctx, n_kv, group, dtype):
    c = Case(new, ctx, bs=bs, n_kv=n_kv, group=group, dtype=dtype, seed=bs, pad=2)
    c.run()
    c.check()


@pytest.mark.parametrize("rows", [143, 144, 145, 256, 257])
def test_the_rows_from_which_a_sequence_takes_it(rows):
    # (three such sequences and one of 600 rows; below the limit the narrower bound holds)
    c = Case([rows, rows, 600, rows], [rows, 2500, 3000, 700], group=1, n_kv=3, seed=rows)
    c.run()
    c.check(tokens=60)


@pytest.mark.parametrize("q_scale,scale", [(0.0, 0.0), (1e-30, 0.0), (300.0, 1 / 300.0), (3e4, 1 / 3e4), (1e30, 1e-30), (3e37, 3e-38)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_query_magnitudes(q_scale, scale, dtype):
    c = Case([150, 40], [2300, 300], q_scale=q_scale, scale=scale, dtype=dtype, seed=3)
    c.run()
    c.check()


@pytest.mark.parametrize("q_scale", [4e33, 4e20, 1e5])
def test_scores_of_huge_magnitude(q_scale):
    # one key wins by far: the output is its value
    c = Case([300], [1000], q_scale=q_scale, dtype=torch.float32, seed=4)
    c.run()
    torch.cuda.synchronize()
    assert B.tq_get_last_device_error(c.book) == 0
    model = Model(c.cache)
    for back in (1, 100, 300):
        k, v = (model.values(x, c.table[0], 0, 1001 - back, 0) for x in "kv")
        s = c.q[-back].double().cpu().numpy() @ k.T
        order = np.sort(s, axis=1)
        sure = (order[:, -1] - order[:, -2]) > 2.0 ** -9 * np.abs(order[:, -1])
        assert sure.any()
        got = c.out[-back].double().cpu().numpy()[sure]
        assert (np.abs(got - v[s.argmax(1)[sure]]) <= few.V * np.abs(got) * 1.01 + 1e-30).all()


@pytest.mark.parametrize("lo,hi", [(-45, 13), (-40, -30), (5, 14)])
def test_scales_over_their_whole_range(lo, hi):
    # blocks whose values lie decades apart, and zero vectors; every row sees several of them
    c = Case([300], [1280], seed=5)
    block = torch.arange(1280, device="cuda") // 64
    kv = torch.randn((1280, 2, 1, 128), generator=c.g, device="cuda")
    kv[:, 1] *= torch.exp2(torch.linspace(lo, hi, 20, device="cuda").round())[block][:, None, None]
    kv[100:140] = 0.0
    c.write(kv, [1280], [1280])
    c.run()
    c.check()
    # weight only on the tokens of a block with small values: their own rounding decides
    kv = torch.randn((1280, 2, 1, 128), generator=c.g, device="cuda")
    kv[:, 1, 0] *= torch.exp2(torch.where(block == 3, -20.0, 8.0))[:, None]
    kv[192:256, 0] = 6.0 + 0.1 * kv[192:256, 0]
    c.write(kv, [1280], [1280])
    c.q.fill_(3.0)
    c.run()
    torch.cuda.synchronize()
    model = Model(c.cache)
    k, v = (model.values(x, c.table[0], 0, 1280, 0) for x in "kv")
    s = c.q[-1].double().cpu().numpy() @ k.T / math.sqrt(128)
    p = np.exp(s - s.max(1, keepdims=True))
    expect = p @ v / p.sum(1, keepdims=True)
    got = c.out[-1].double().cpu().numpy()
    assert np.linalg.norm(got - expect) <= 0.005 * np.linalg.norm(expect)


@pytest.mark.parametrize("ctx", [1083, 1152])
@pytest.mark.parametrize("group", [16, 64])
def test_what_a_row_does_not_see_has_no_influence(ctx, group):
    new = 300
    c = Case([new, 1], [ctx, 50], group=group, seed=6)
    c.run()
    c.check()
    first = c.out.clone()
    # stale slots behind both contexts: every bit pattern, NaN among them
    for b, length in enumerate(c.ctx):
        blk, off = int(c.table[b, (length - 1) // 64]), (length - 1) % 64 + 1
        k, v = c.cache["k_codes"][blk].permute(0, 1, 3, 2, 4), c.cache["v_codes"][blk].permute(0, 1, 3, 2)
        for t in range(off, 64):
            k[:, t // 8, t % 8] = 127 if t % 2 else 255
            v[:, t // 16, t % 16] = 255 if t % 3 else 127
    spare = int(np.setdiff1d(np.arange(c.num_blocks), c.table[c.table >= 0])[0])
    c.cache["k_scale"][spare] = c.cache["v_scale"][spare] = float("nan")
    c.out.fill_(5.0)
    c.run()
    torch.cuda.synchronize()
    assert torch.equal(first, c.out)
    # a NaN in the key or value of one of the new tokens: the rows behind it see it, those before do not
    for which in (0, 1):
        for back in (1, 70, 260):
            d = Case([new, 1], [ctx, 50], group=group, seed=6)
            blk, off = int(d.table[0, (ctx - back) // 64]), (ctx - back) % 64
            if which == 0:
                d.cache["k_codes"][blk, 0, off // 8, :, off % 8] = 127
            else:
                d.cache["v_codes"][blk, 0, off // 16, :, off % 16] = 255
            d.run()
            torch.cuda.synchronize()
            assert bool(torch.isnan(d.out[new - back:new]).all())
            assert torch.equal(first[:new - back], d.out[:new - back]) and torch.equal(first[new:], d.out[new:])


@pytest.mark.parametrize("bs,where", [(64, range(128, 192)), (32, range(64, 96)), (256, range(512, 768))])
def test_bad_blocks_are_skipped_and_recorded(bs, where):
    c = Case([300, 200], [1500, 900], bs=bs, n_kv=2, group=8, seed=7)
    for bad in (-1, c.num_blocks, (1 << 31) - 1):
        c.table_t[0, where[0] // bs] = bad
        c.run()
        c.check([0], 60, where, code=2)
        c.run()
        c.check([1], code=2)


def test_bad_lengths_are_recorded():
    c = Case([200, 300, 1], [1000, 2000, 300], seed=8)
    for bad in (-1, 2001, 1 << 30, -(1 << 31)):
        c.out.fill_(5.0)
        c.ctx_t[1] = bad
        c.run()
        c.check([0, 2], code=3)
        assert bool((c.out[200:500] == 0.0).all())
    c.ctx_t[1] = 2000
    for start in ([0, 200, 600, 501], [0, -2, 500, 501], [0, 200, 100, 501], [0, 200, 500, 9999]):
        c.start.copy_(ints(start))
        c.run()
        torch.cuda.synchronize()
        assert B.tq_get_last_device_error(c.book) == 3


def test_accuracy_of_ordinary_scores():
    # the output's own rounding is 2^-8 / sqrt(3) times the mean place of a number in its binade: 0.00165; the weights' adds half
    c = Case([100] * 8, [3000] * 8, n_kv=2, group=8, seed=9)
    c.run()
    torch.cuda.synchronize()
    assert few.Case.check(c, tokens=30, wide=True) <= 0.0027


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_query_that_is_not_finite_spoils_its_own_row_only(bad):
    c = Case([300, 1], [1300, 90], seed=10)
    at = 260
    c.q[at, 2, 17] = bad
    c.run()
    torch.cuda.synchronize()
    spoilt = c.out[at, 2].clone()
    c.q[at, 2, 17] = 0.0
    once = c.out.clone()
    c.run()
    once[at, 2] = c.out[at, 2]                            # (the others: within the bound, beside the row and far from it)
    c.out.copy_(once)
    c.check(tokens=60)
    if bad != bad:
        assert bool(torch.isnan(spoilt).all())


@pytest.mark.parametrize("new,ctx", [([300, 1], [0, 1000]), ([300, 1], [3, 1000]), ([300, 300], [299, 1000]), ([200, 0, 200], [200, 0, 1000])])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_empty_and_short_contexts(new, ctx, dtype):
    c = Case(new, ctx, dtype=dtype, seed=11)
    c.run()
    c.check()


@pytest.mark.parametrize("kw", [dict(k_bits=2, v_bits=2, qjl_m=0), dict(norm_bits=16), dict(k_bits=0, v_bits=0, qjl_m=0, codec=1)])
def test_any_device_handle_serves(kw):
    c = Case([1, 2, 300], [100, 40, 1300], seed=12)
    c.run()
    torch.cuda.synchronize()
    first = c.out.clone()
    c.book = B.Codebook(block_size=64, **kw)
    c.out.fill_(5.0)
    c.run()
    torch.cuda.synchronize()
    assert torch.equal(first, c.out)


def test_blocks_beyond_four_gigabytes():
    # the same tokens in a small cache and at the end of one of 4.6 GB of keys and as much of values
    c = Case([300, 2], [1000, 90], n_kv=8, group=2, seed=13)
    c.run()
    torch.cuda.synchronize()
    first = c.out.clone()
    num_blocks, used = 70000, np.unique(c.table[c.table >= 0])
    big = {name: torch.empty((num_blocks,) + tuple(t.shape[1:]), dtype=t.dtype, device="cuda") for name, t in c.cache.items()}
    far = {int(b): num_blocks - 1 - i for i, b in enumerate(used)}
    for name in big:
        big[name][torch.tensor([far[int(b)] for b in used], device="cuda")] = c.cache[name][ints(used).long()]
    c.table_t = ints(np.vectorize(lambda b: far.get(int(b), -1))(c.table))
    c.view = C.fp8_view(c.book, big)
    c.out.fill_(5.0)
    c.run()
    torch.cuda.synchronize()
    assert B.tq_get_last_device_error(c.book) == 0
    assert torch.equal(first, c.out)


@pytest.mark.parametrize("batch,group", [(300, 16), (700, 9)])
def test_many_sequences_of_many_and_few_rows(batch, group):
    rng = np.random.default_rng(batch)
    new = [int(n) for n in rng.choice([0, 1, 1, 2, 9, 10, 20, 40], batch)]
    ctx = [n + int(x) for n, x in zip(new, rng.integers(0, 400, batch))]
    ctx[batch // 2] += 1000
    c = Case(new, ctx, group=group, bs=32, seed=14)
    c.run()
    c.check()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("new,ctx", [([300, 200], [2000, 900]), ([600, 1, 1], [1300, 700, 900])])
def test_same_call_same_bits_on_streams_and_in_graphs(new, ctx, dtype):
    c = Case(new, ctx, n_kv=2, group=8, dtype=dtype, seed=15)
    c.run()
    torch.cuda.synchronize()
    first = c.out.clone()
    outs, spaces = [torch.zeros_like(c.out) for _ in range(2)], [torch.full_like(c.ws, 255) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.run(out=outs[0], ws=spaces[0])
    c.run(out=outs[1], ws=spaces[1], stream=side)         # both at once, a workspace each
    torch.cuda.synchronize()
    assert torch.equal(first, outs[0]) and torch.equal(first, outs[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(out=outs[0], ws=spaces[0])
        c.run(out=outs[1], ws=spaces[0])                  # one after another in one workspace
    for out in outs:
        out.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, outs[0]) and torch.equal(first, outs[1])
    # shorter contexts, fewer rows and other queries in the captured shape
    c.new = [n // 2 if n > 1 else n for n in c.new]
    c.ctx = [n - 50 for n in c.ctx]
    c.start.copy_(ints(np.concatenate([[0], np.cumsum(c.new)])))
    c.ctx_t.copy_(ints(c.ctx))
    c.q.mul_(0.5)
    outs[0].fill_(5.0)
    graph.replay()
    torch.cuda.synchronize()
    c.out.copy_(outs[0])
    c.check()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("new,ctx", [([300, 200], [2000, 900]), ([600, 1, 1], [1300, 700, 900])])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_correct(new, ctx, dtype):
    # the test aid withholds one product's completion in a CTA of each form: its waits run out after a second, what it has in
    # flight is drained, the call ends with device error 4 and the handle works on
    c = Case(new, ctx, n_kv=2, group=8, dtype=dtype, seed=16)
    B.tq_debug_withhold_commit(c.book, True)
    c.run()
    torch.cuda.synchronize()
    assert B.tq_get_last_device_error(c.book) == 4
    B.tq_debug_withhold_commit(c.book, False)
    c.run()
    c.check()


@pytest.mark.parametrize("max_context", [1 << 15, 1 << 20])
@pytest.mark.parametrize("past", [0, 5])
def test_a_decode_step_large_enough_for_its_launches(max_context, past):
    # no sequence takes the form: the others run before its launches, or behind them (where its tiles may have no room)
    rng = np.random.default_rng(max_context)
    ctx = [int(x) for x in rng.integers(1, 400, 600)]
    c = few.Case([1] * 600, ctx, n_kv=2, group=8, seed=17, pad=past)
    ws, nbytes = C.allocate_fp8_workspace(c.book, c.total, c.batch, c.n_q, c.n_kv, max_context)
    assert nbytes > WIDE_BYTES
    B.tq_fp8_attention(c.book, c.q, B.TQ_BF16, c.total, c.batch, c.n_q, c.n_kv, c.view, c.table_t, c.max_blocks, c.start,
                       c.ctx_t, max_context, 0.0, c.out, ws, nbytes)
    c.check(wide=False)
