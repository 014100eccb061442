"""Attention over the 8-bit cache, against the formula in 64 bits on the values
that the cache holds.

Tolerance of an output coordinate j, with a_j = sum_t p_t |v_tj| (p the softmax
weights) and V = 2^-8 (half a step of bf16, relative).
Few rows: a query coordinate is held to 2^-16 of itself, keys exactly, and a
score is summed and shifted in float32, so |delta s_t| <= D = 2^-15 scale |q| |k_t|
(Cauchy-Schwarz), which changes p-weighted means by at most (e^{2 D} - 1) a_j.
Weights are held to 2^-11 of themselves (an fp16 rounding, then three e4m3
pieces of it) and 2^-26 of the largest weight times
the largest scale.  The output is rounded to bf16 once: V |o_j|.
Many rows (from WIDE rows of a sequence and KV head): queries are fp16 numbers
(u = 2^-11), D = 1.5 u scale |q| |k|; weights bf16 (V); the output passes once
through fp16 (u of its largest coordinate).
"""
import math

import numpy as np
import pytest
import torch

from online_kv_cache_tq_gb300 import binding as B
from online_kv_cache_tq_gb300 import cache as C

from test_fp8_cache import Model, generator, ints, random_cache

pytestmark = pytest.mark.gpu
U, V = 2.0 ** -11, 2.0 ** -8
WIDE = 128                    # rows from which the wider bound is allowed


def reference(q, k, v, n_new, scale, wide, blocked=()):
    """q [n][G][128], k, v [ctx][128] float64 -> outputs and bounds [n][G][128]."""
    n, g, length = q.shape[0], q.shape[1], k.shape[0]
    out, bound = np.zeros((n, g, 128)), np.zeros((n, g, 128))
    for i in range(n):
        seen = np.arange(length) <= length - n_new + (n_new - n) + i
        seen[list(blocked)] = False
        if not seen.any():
            continue
        ks, vs = k[seen], v[seen]
        s = q[i] @ ks.T * scale
        p = np.exp(s - s.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        out[i] = p @ vs
        a = p @ np.abs(vs)
        d = (np.linalg.norm(q[i], axis=1)[:, None] * np.linalg.norm(ks, axis=1)[None, :]).max(1, keepdims=True) * scale
        top = np.abs(vs).max()
        if wide:
            with np.errstate(over="ignore"):
                bound[i] = a * (np.expm1(3 * U * d) + 1.05 * V) + U * np.abs(out[i]).max(1, keepdims=True)
        else:
            with np.errstate(over="ignore"):
                bound[i] = a * (np.expm1(2.0 ** -14 * d) + 2.0 ** -11) + 2.0 ** -25 * seen.sum() * p.max(1, keepdims=True) * top
        bound[i] += 1.01 * V * np.abs(out[i])
    return out, bound


class Case:
    def __init__(self, new, ctx, bs=64, n_kv=2, group=4, seed=0, dtype=torch.bfloat16, q_scale=1.0, k_scale=1.0,
                 v_scale=1.0, pad=0, scale=0.0, identity=False):
        self.new, self.ctx, self.n_kv, self.group, self.n_q, self.scale = list(new), list(ctx), n_kv, group, n_kv * group, scale
        self.batch, self.total, self.bs = len(new), sum(new) + pad, bs
        self.book = B.Codebook(block_size=bs)
        need = [-(-max(c, 1) // bs) for c in ctx]
        self.max_blocks = max(need)
        self.num_blocks = sum(need) + 1 if not identity else self.batch * self.max_blocks
        ids = np.random.default_rng(seed).permutation(self.num_blocks)
        self.table = np.full((self.batch, self.max_blocks), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        if identity:
            self.table = np.arange(self.num_blocks, dtype=np.int32).reshape(self.batch, self.max_blocks)
        self.table_t = None if identity else ints(self.table)
        self.g = g = generator(seed)
        self.cache = random_cache(self.book, self.num_blocks, n_kv, g)
        self.view = C.fp8_view(self.book, self.cache)
        # every position of every sequence, with a profile of channels and tokens
        rows = sum(ctx)
        prof = torch.exp(0.5 * torch.randn((2, n_kv, 128), generator=g, device="cuda"))
        kv = torch.randn((rows, 2, n_kv, 128), generator=g, device="cuda") * prof
        kv *= torch.tensor([k_scale, v_scale], device="cuda")[:, None, None]
        self.write(kv, ctx, ctx)
        self.q = (torch.randn((self.total, self.n_q, 128), generator=g, device="cuda") * q_scale).to(dtype)
        self.start = ints(np.concatenate([[0], np.cumsum(new)]))
        self.ctx_t = ints(ctx)
        self.ws, self.nbytes = C.allocate_fp8_workspace(self.book, max(1, self.total), self.batch, self.n_q, n_kv,
                                                        int(max(ctx)))
        self.ws.fill_(255)
        self.out = torch.full((self.total, self.n_q, 128), 5.0, dtype=torch.bfloat16, device="cuda")

    def write(self, kv, new, ctx):
        if kv.shape[0] == 0:
            return
        row = 2 * self.n_kv * 128
        start = ints(np.concatenate([[0], np.cumsum(new)]))
        B.tq_fp8_append(self.book, kv[:, 0], kv[:, 1], B.TQ_FP32, kv.shape[0], self.batch, self.n_kv, row, row, self.view,
                        self.table_t, self.max_blocks, start, ints(ctx))
        assert B.tq_get_last_device_error(self.book) == 0

    def run(self, out=None, ws=None, stream=None):
        B.tq_fp8_attention(self.book, self.q, B.TQ_BF16 if self.q.dtype == torch.bfloat16 else B.TQ_FP32, self.total,
                           self.batch, self.n_q, self.n_kv, self.view, self.table_t, self.max_blocks, self.start,
                           self.ctx_t, int(max(self.ctx)), self.scale, self.out if out is None else out,
                           self.ws if ws is None else ws, self.nbytes, stream)

    def check(self, sequences=None, tokens=None, blocked=(), code=0, wide=None):
        torch.cuda.synchronize()
        assert B.tq_get_last_device_error(self.book) == code
        model = Model(self.cache)
        got, qn = self.out.double().cpu().numpy(), self.q.double().cpu().numpy()
        scale = self.scale or 1.0 / math.sqrt(128)
        starts = np.concatenate([[0], np.cumsum(self.new)])
        err2 = ref2 = 0.0
        for b in range(self.batch) if sequences is None else sequences:
            n, length = self.new[b], self.ctx[b]
            none = max(0, n - length)
            assert (got[starts[b]:starts[b] + none] == 0.0).all()
            take = n - none if tokens is None else min(tokens, n - none)
            if take == 0:
                continue
            many = n * self.group >= WIDE if wide is None else wide
            for h in range(self.n_kv):
                hs, rs = slice(h * self.group, (h + 1) * self.group), slice(starts[b + 1] - take, starts[b + 1])
                k, v = (model.values(x, self.table[b], 0, length, h) for x in "kv")
                expect, bound = reference(qn[rs, hs], k, v, n, scale, many, blocked)
                err = np.abs(got[rs, hs] - expect)
                assert np.isfinite(got[rs, hs]).all()
                assert (err <= bound + 1e-30).all(), "seq %d KV head %d: worst %.3g of the bound" % (
                    b, h, (err / np.maximum(bound, 1e-30)).max())
                err2 += (err ** 2).sum()
                ref2 += (expect ** 2).sum()
        assert (got[starts[-1]:] == 5.0).all()           # rows behind the last sequence
        return math.sqrt(err2 / ref2) if ref2 else 0.0


@pytest.mark.parametrize("bs", [32, 64, 96, 128, 256, 160])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode_of_ragged_contexts(bs, dtype):
    # one token each, contexts around the ends of blocks, of 32, of 128 tokens
    ctx = [1, 2, 31, 32, 33, 95, 96, 97, 127, 128, 129, 255, 256, 257, 500, 1000]
    c = Case([1] * len(ctx), ctx, bs=bs, dtype=dtype, seed=bs, pad=3)
    c.run()
    assert c.check() <= 0.0019


@pytest.mark.parametrize("group,n_kv", [(1, 1), (1, 5), (2, 2), (3, 2), (5, 1), (8, 1), (7, 1), (12, 1), (16, 1), (40, 2), (64, 1)])
def test_groups_and_ragged_batches(group, n_kv):
    new = [1, 0, 3, 7, 2, 1, 0, 9, 5]
    c = Case(new, [5, 700, 129, 7, 1, 300, 0, 64, 3], n_kv=n_kv, group=group, seed=group, pad=4)
    c.run()
    c.check()


@pytest.mark.parametrize("n_kv,group,new,ctx", [(33000, 1, [2], [3]), (700, 3, [1, 4], [130, 5]), (300, 1, [200, 2], [260, 40])])
def test_many_kv_heads(n_kv, group, new, ctx):
    c = Case(new, ctx, bs=32, n_kv=n_kv, group=group, seed=n_kv)
    c.run()
    c.check(tokens=2)


@pytest.mark.parametrize("group,bs", [(8, 64), (16, 32), (4, 96)])
@pytest.mark.parametrize("seed", range(3))
def test_many_short_sequences_of_changing_row_counts(group, bs, seed):
    # a CTA works on several sequences, one after another, with fewer and more rows and key tiles than the one before
    rng = np.random.default_rng(seed)
    batch = 260
    new = [int(n) for n in rng.choice([0, 1, 1, 2, 3, 4, 6, 9], batch)]
    ctx = [n + int(c) for n, c in zip(new, rng.integers(0, 500, batch))]
    c = Case(new, ctx, n_kv=2, group=group, bs=bs, seed=seed)
    c.run()
    c.check()


@pytest.mark.parametrize("new,ctx", [([1], [20000]), ([2, 5, 1], [9000, 30, 12345]), ([4], [4]), ([33], [5000])])
def test_few_tokens_on_long_contexts(new, ctx):
    c = Case(new, ctx, n_kv=1, group=8, seed=1)
    c.run()
    c.check()


@pytest.mark.parametrize("bs", [32, 64, 96, 128])
@pytest.mark.parametrize("new,ctx", [([200], [200]), ([129, 250], [1000, 251]), ([33, 16, 300], [2000, 16, 555]),
                                     ([300, 1, 128], [299, 1000, 600])])
def test_prompt_chunks(bs, new, ctx):
    c = Case(new, ctx, bs=bs, n_kv=2, group=4, seed=2, pad=2)
    c.run()
    c.check()


@pytest.mark.parametrize("group", [1, 4, 8])
def test_many_and_few_rows_in_one_call(group):
    c = Case([600, 1, 3, 520, 0, 40], [900, 3000, 700, 520, 5, 41], n_kv=1, group=group, seed=3, dtype=torch.float32)
    c.run()
    c.check(tokens=70)


def test_accuracy_of_ordinary_scores():
    # the output's own rounding is 2^-8 / sqrt(3) times the mean place of a number in its binade: 0.00165
    c = Case([1] * 8, [3000] * 8, group=8, seed=4)
    c.run()
    assert c.check() <= 0.0019
    c = Case([100], [3000], group=8, n_kv=1, seed=4)
    c.run()
    assert c.check(tokens=30) <= 0.0027


def test_scale_identity_table_and_float_queries():
    c = Case([2, 1, 150], [300, 70, 200], scale=0.3, identity=True, dtype=torch.float32, seed=5)
    c.run()
    c.check()


@pytest.mark.parametrize("new", [[1, 3], [150, 40]])
@pytest.mark.parametrize("q_scale", [0.0, 1e-30, 300.0, 3e4])
def test_query_magnitudes(new, q_scale):
    c = Case(new, [400, 300], group=4, q_scale=q_scale, scale=0.0 if q_scale < 1 else 1.0 / q_scale, seed=6,
             dtype=torch.float32)
    c.run()
    c.check()


@pytest.mark.parametrize("new", [1, 300])
@pytest.mark.parametrize("q_scale", [4e33, 4e20, 1e5])
def test_scores_of_huge_magnitude(new, q_scale):
    # one key wins by far: the output is its value
    c = Case([new], [400], n_kv=1, group=4, q_scale=q_scale, seed=7, dtype=torch.float32)
    c.run()
    torch.cuda.synchronize()
    assert B.tq_get_last_device_error(c.book) == 0
    model = Model(c.cache)
    k, v = (model.values(x, c.table[0], 0, 400, 0) for x in "kv")
    s = c.q[-1].double().cpu().numpy() @ k.T
    order = np.sort(s, axis=1)
    sure = (order[:, -1] - order[:, -2]) > 2.0 ** -9 * np.abs(order[:, -1])
    assert sure.any()
    got = c.out[-1].double().cpu().numpy()[sure]
    assert (np.abs(got - v[s.argmax(1)[sure]]) <= V * np.abs(got) * 1.01 + 1e-30).all()


@pytest.mark.parametrize("new", [1, 4, 300])
def test_scales_over_their_whole_range(new):
    # blocks whose values lie decades apart, and zero vectors; every row sees several of them
    c = Case([new], [640], n_kv=1, group=4, seed=8)
    e = torch.linspace(-45, 13, 10, device="cuda").round()
    kv = torch.randn((640, 2, 1, 128), generator=c.g, device="cuda")
    kv[:, 1] *= torch.exp2(e)[torch.arange(640, device="cuda") // 64][:, None, None]
    kv[100:140] = 0.0
    c.write(kv, [640], [640])
    c.run()
    c.check()
    # weight only on the tokens of a block with small values: their own rounding decides
    kv = torch.randn((640, 2, 1, 128), generator=c.g, device="cuda")
    kv[:, 1, 0] *= torch.exp2(torch.where(torch.arange(640, device="cuda") // 64 == 3, -20.0, 8.0))[:, None]
    kv[192:256, 0] = 6.0 + 0.1 * kv[192:256, 0]
    c.write(kv, [640], [640])
    c.q.fill_(3.0)
    c.run()
    torch.cuda.synchronize()
    model = Model(c.cache)
    k, v = (model.values(x, c.table[0], 0, 640, 0) for x in "kv")
    s = c.q[-1].double().cpu().numpy() @ k.T / math.sqrt(128)
    p = np.exp(s - s.max(1, keepdims=True))
    expect = p @ v / p.sum(1, keepdims=True)
    got = c.out[-1].double().cpu().numpy()
    assert np.linalg.norm(got - expect) <= 0.005 * np.linalg.norm(expect)


@pytest.mark.parametrize("new", [1, 3, 40, 300])
def test_what_a_row_does_not_see_has_no_influence(new):
    ctx = new + 83
    c = Case([new, 1], [ctx, 50], n_kv=1, group=4, seed=9)
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
    # the last token's key or value is NaN: only the last row sees it
    for which in (0, 1):
        d = Case([new, 1], [ctx, 50], n_kv=1, group=4, seed=9)
        kv = torch.zeros((2, 2, 1, 128), device="cuda")
        last, row = d.read_last()
        kv[:] = last
        kv[0, which, 0, 77] = float("nan")
        d.write(kv, [1, 1], d.ctx)
        d.run()
        torch.cuda.synchronize()
        assert bool(torch.isnan(d.out[new - 1]).all())
        assert torch.equal(first[:new - 1], d.out[:new - 1]) and torch.equal(first[new:], d.out[new:])


def _read_last(self):
    out = torch.zeros((2, 2, self.n_kv, 128), device="cuda")
    row = self.n_kv * 128
    B.tq_fp8_read(self.book, self.view, self.table_t, self.max_blocks, 2, 2, self.n_kv, ints([0, 1, 2]), self.ctx_t,
                  B.TQ_FP32, out[0], out[1], row, row)
    return out.transpose(0, 1).contiguous(), row


Case.read_last = _read_last


@pytest.mark.parametrize("new", [2, 200])
def test_bad_blocks_are_skipped_and_recorded(new):
    c = Case([new, 3], [700, 500], n_kv=2, group=4, seed=10)
    for bad in (-1, c.num_blocks, (1 << 31) - 1):
        c.table_t[0, 2] = bad                            # positions 128 .. 191
        c.run()
        c.check(sequences=[0], code=2, blocked=range(128, 192), tokens=60)
        c.run()
        c.check(sequences=[1], code=2)


def test_bad_lengths_are_recorded():
    c = Case([2, 3, 1], [100, 200, 300], seed=11)
    for bad in (-1, 301, 1 << 30, -(1 << 31)):
        c.out.fill_(5.0)
        c.ctx_t[1] = bad
        c.run()
        c.check(sequences=[0, 2], code=3)
        assert bool((c.out[2:5] == 0.0).all())
    c.ctx_t[1] = 200
    for start in ([0, 2, 9, 6], [0, -2, 5, 6], [0, 2, 1, 6], [0, 2, 5, 99]):
        c.out.fill_(5.0)
        c.start.copy_(ints(start))
        c.run()
        torch.cuda.synchronize()
        assert B.tq_get_last_device_error(c.book) == 3


def test_more_expanded_tiles_than_the_workspace_holds():
    # forty sequences of many rows whose contexts share blocks: what has no room takes the other form
    c = Case([70] * 3, [400] * 3, n_kv=1, group=8, seed=12)
    batch, ctx, max_blocks = 40, 110000, 1720
    table = c.table_t[:1, :6].repeat(batch, 287)[:, :max_blocks].contiguous()
    new, group = 64, 8
    q = torch.randn((batch * new, group, 128), generator=c.g, device="cuda").to(torch.bfloat16)
    q[new:] = q[:new].repeat(batch - 1, 1, 1)
    start, ctx_t = ints(np.arange(batch + 1) * new), ints([ctx] * batch)
    ws, nbytes = C.allocate_fp8_workspace(c.book, batch * new, batch, group, 1, ctx)
    assert nbytes < 2.4e9
    out = torch.zeros((batch * new, group, 128), dtype=torch.bfloat16, device="cuda")
    B.tq_fp8_attention(c.book, q, B.TQ_BF16, batch * new, batch, group, 1, c.view, table, max_blocks, start, ctx_t, ctx,
                       0.0, out, ws, nbytes)
    torch.cuda.synchronize()
    assert B.tq_get_last_device_error(c.book) == 0
    o = out.float().reshape(batch, -1)
    assert bool(((o - o[:1]).norm(dim=1) <= 0.005 * o[0].norm()).all())


@pytest.mark.parametrize("new,ctx", [([1, 1, 1], [3000, 700, 9]), ([4, 3], [3000, 700]), ([400, 20], [900, 4000])])
def test_same_call_same_bits_on_streams_and_in_graphs(new, ctx):
    c = Case(new, ctx, group=8, n_kv=2, seed=13)
    c.run()
    torch.cuda.synchronize()
    first = c.out.clone()
    outs = [torch.zeros_like(c.out) for _ in range(3)]
    ws = [torch.full_like(c.ws, 255) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.run(out=outs[0])
    c.run(out=outs[1], ws=ws[0], stream=side)            # both at once, a workspace each
    torch.cuda.synchronize()
    assert torch.equal(first, outs[0]) and torch.equal(first, outs[1])
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph, out, w in zip(graphs, outs[1:], ws):
        out.zero_()
        with torch.cuda.graph(graph):
            c.run(out=out, ws=w)
    for graph in graphs + graphs:
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, outs[1]) and torch.equal(first, outs[2])
    # shorter contexts and other queries in the captured shape
    c.ctx = [x - 5 for x in c.ctx]
    c.ctx_t.copy_(ints(c.ctx))
    c.q.mul_(0.5)
    graphs[0].replay()
    torch.cuda.synchronize()
    c.out.copy_(outs[1])
    c.check(tokens=30)
    assert B.tq_get_last_device_error(c.book) == 0


def test_refusals():
    c = Case([3], [100])
    base = [c.q, B.TQ_BF16, 3, 1, c.n_q, c.n_kv, c.view, c.table_t, c.max_blocks, c.start, c.ctx_t, 100, 0.0, c.out, c.ws,
            c.nbytes]
    ptr = lambda t, n: t.data_ptr() + n
    for i, value, status in ((0, None, 1), (0, ptr(c.q, 8), 1), (1, 2, 1), (2, -1, 1), (3, -1, 1), (4, 0, 1), (4, 7, 1),
                             (5, 0, 1), (5, 1, 1), (7, ptr(c.table_t, 2), 1), (8, 0, 1), (9, None, 1), (10, None, 1),
                             (9, ptr(c.start, 1), 1), (10, ptr(c.ctx_t, 2), 1), (11, -1, 1), (11, (1 << 30) + 1, 2),
                             (12, -1.0, 1), (12, float("nan"), 1), (12, float("inf"), 1), (13, None, 1),
                             (13, ptr(c.out, 8), 1), (14, None, 5), (14, ptr(c.ws, 16), 5), (15, c.nbytes - 1, 5),
                             (2, 1 << 30, 1)):
        args = list(base)
        args[i] = value
        with pytest.raises(B.TQError) as err:
            B.tq_fp8_attention(c.book, *args)
        assert err.value.status == status, (i, value)
    args = list(base)
    args[7], args[8] = None, c.num_blocks + 1            # an identity table beyond the cache
    with pytest.raises(B.TQError):
        B.tq_fp8_attention(c.book, *args)
    for i in (2, 3):
        args = list(base)
        args[i] = 0
        B.tq_fp8_attention(c.book, *args)                # nothing to do
    for args in ((0, 1, 8, 2, 100), (1, 0, 8, 2, 100), (1, 1, 7, 2, 100), (1, 1, 8, 0, 100), (1, 1, 8, 2, -1)):
        assert B.tq_fp8_workspace_bytes(c.book, *args) == 0
    torch.cuda.synchronize()
    assert bool((c.out == 5.0).all())


@pytest.mark.parametrize("kw", [dict(k_bits=2, v_bits=2, qjl_m=0), dict(norm_bits=16), dict(k_bits=0, v_bits=0, qjl_m=0, codec=1)])
def test_any_device_handle_serves(kw):
    c = Case([1, 2, 200], [100, 40, 300], seed=14)
    c.run()
    first = c.out.clone()
    c.book = B.Codebook(block_size=64, **kw)
    c.out.fill_(5.0)
    c.run()
    torch.cuda.synchronize()
    assert torch.equal(first, c.out)


@pytest.mark.parametrize("new", [[1, 1], [2, 5], [300, 200]])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_correct(new, dtype):
    # the test aid withholds one product's completion in the first CTA of each launch: its waits run out after a second,
    # what it has in flight is drained, the call ends with device error 4 and the handle works on
    c = Case(new, [n + 700 for n in new], n_kv=2, group=4, seed=24, dtype=dtype)
    B.tq_debug_withhold_commit(c.book, True)
    c.run()
    torch.cuda.synchronize()
    assert B.tq_get_last_device_error(c.book) == 4
    B.tq_debug_withhold_commit(c.book, False)
    c.run()
    c.check(tokens=40)


@pytest.mark.parametrize("group,new", [(4, [1]), (4, [4, 3, 0, 5]), (2, [1, 0, 90])])
def test_more_sequences_than_threads(group, new):
    rng = np.random.default_rng(group + len(new))
    batch = 900
    new = [new[i % len(new)] for i in range(batch)]
    ctx = [max(n, 1) + int(c) for n, c in zip(new, rng.integers(0, 140, batch))]
    c = Case(new, ctx, n_kv=1, group=group, bs=32, seed=20)
    c.run()
    c.check()


@pytest.mark.parametrize("new,ctx", [([1, 1], [0, 40]), ([5, 2], [0, 1]), ([200, 1], [0, 30]), ([300], [3])])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_empty_contexts(new, ctx, dtype):
    c = Case(new, ctx, group=4, dtype=dtype, seed=21)
    c.run()
    c.check()


@pytest.mark.parametrize("new", [2, 6, 200])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_query_that_is_not_finite_spoils_its_own_row_only(new, bad):
    c = Case([new, 1], [300, 90], n_kv=1, group=4, seed=22)
    c.run()
    torch.cuda.synchronize()
    first = c.out.clone()
    c.q[1, 2, 17] = bad
    c.run()
    torch.cuda.synchronize()
    keep = torch.ones_like(first[..., 0], dtype=torch.bool)
    keep[1, 2] = False
    assert torch.equal(first[keep], c.out[keep])
    if bad != bad:
        assert bool(torch.isnan(c.out[1, 2]).all())


@pytest.mark.parametrize("new", [1, 4, 200])
def test_blocks_beyond_four_gigabytes(new):
    # the same tokens in a small cache and at the end of one of 4.6 GB of keys and as much of values
    c = Case([new, 2], [300, 90], n_kv=8, group=1, seed=23)
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
