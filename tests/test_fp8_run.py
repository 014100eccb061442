"""The 8-bit cache in a serving loop, as it would be used: token map, head norms
with rotation, append and attention of a prompt step, a mixed step and decode
steps on a padded batch, one step captured and replayed; then a sequence read
back and its tokens appended to the packed cache.  Each stage is checked from
the GPU's own inputs to it."""
import numpy as np
import pytest
import torch

from online_kv_cache_tq_gb300 import binding as B
from online_kv_cache_tq_gb300 import cache as C

from parity_helpers import books, check_append
from test_fp8_attention import reference
from test_fp8_cache import Model, generator, ints

pytestmark = pytest.mark.gpu


class Loop:
    def __init__(self, bs=32, n_kv=2, group=4, batch=3, rows=200):
        self.bs, self.n_kv, self.group, self.batch, self.rows, self.n_q = bs, n_kv, group, batch, rows, n_kv * group
        self.num_blocks, self.max_blocks = 64, 12
        self.book, self.ref = books(3, 3, 128, seed=1, block_size=bs)
        self.g = generator(0)
        self.cache = C.allocate_fp8_cache(self.book, self.num_blocks, n_kv)
        self.view = C.fp8_view(self.book, self.cache)
        self.free = ints(np.random.default_rng(0).permutation(self.num_blocks))
        dev = lambda n, dt=torch.int32: torch.zeros(n, dtype=dt, device="cuda")
        self.table = torch.full((batch, self.max_blocks), -1, dtype=torch.int32, device="cuda")
        self.past, self.new, self.ctx, self.start, self.taken = dev(batch), dev(batch), dev(batch), dev(batch + 1), dev(1)
        self.pos, self.slots = dev(rows), dev(rows, torch.int64)
        self.w = [(1 + 0.2 * torch.randn(128, generator=self.g, device="cuda")).to(torch.bfloat16) for _ in range(2)]
        self.inv = 10000.0 ** (-torch.arange(64, dtype=torch.float64, device="cuda") / 64)
        self.qkv = torch.zeros((rows, self.n_q + 2 * n_kv, 128), dtype=torch.bfloat16, device="cuda")
        self.out = torch.zeros((rows, self.n_q, 128), dtype=torch.bfloat16, device="cuda")
        self.ws, self.nbytes = C.allocate_fp8_workspace(self.book, rows, batch, self.n_q, n_kv, self.max_blocks * bs)

    def step(self):
        nq, nkv, rows, batch = self.n_q, self.n_kv, self.rows, self.batch
        stride = (nq + 2 * nkv) * 128
        q, k, v = self.qkv[:, :nq], self.qkv[:, nq:nq + nkv], self.qkv[:, nq + nkv:]
        B.tq_map_tokens(self.book, batch, self.past, self.new, self.table, self.max_blocks, self.num_blocks, self.free,
                        self.free.numel(), rows, self.ctx, self.start, self.pos, self.slots, self.taken)
        B.tq_norm_rope(self.book, q, k, B.TQ_BF16, rows, nq, nkv, stride, stride, self.w[0], self.w[1], 1e-6, self.pos,
                       self.inv, 128, False, q, k, stride, stride)
        B.tq_fp8_append(self.book, k, v, B.TQ_BF16, rows, batch, nkv, stride, stride, self.view, self.table,
                        self.max_blocks, self.start, self.ctx)
        self.q = q.contiguous()
        B.tq_fp8_attention(self.book, self.q, B.TQ_BF16, rows, batch, nq, nkv, self.view, self.table, self.max_blocks,
                           self.start, self.ctx, self.max_blocks * self.bs, 0.0, self.out, self.ws, self.nbytes)

    def fill(self, new):
        self.new.copy_(ints(new))
        self.qkv.copy_(torch.randn(self.qkv.shape, generator=self.g, device="cuda").to(torch.bfloat16))
        self.out.fill_(5.0)

    def check(self, model, new, past):
        torch.cuda.synchronize()
        assert B.tq_get_last_device_error(self.book) == 0
        ctx, total = [p + n for p, n in zip(past, new)], sum(new)
        table = self.table.cpu().numpy()
        assert self.ctx.tolist() == ctx
        kv = self.qkv[:total, self.n_q:].double().cpu().numpy().reshape(total, 2, self.n_kv, 128)
        for i, name in enumerate("kv"):
            model.append(name, kv[:, i], table, new, ctx)
        model.check(self.cache)
        got, q = self.out.double().cpu().numpy(), self.q.double().cpu().numpy()
        row = 0
        for b, n in enumerate(new):
            for h in range(self.n_kv):
                hs = slice(h * self.group, (h + 1) * self.group)
                if n:
                    k, v = (model.values(x, table[b], 0, ctx[b], h) for x in "kv")
                    expect, bound = reference(q[row:row + n, hs], k, v, n, 128 ** -0.5, True)
                    assert (np.abs(got[row:row + n, hs] - expect) <= bound).all()
            row += n
        assert (got[total:] == 5.0).all()
        # the loop moves on
        self.past.copy_(self.ctx)
        self.free = self.free[int(self.taken):].contiguous()
        return ctx


def test_a_serving_loop_and_the_way_to_the_packed_cache():
    loop = Loop()
    model, past = Model(loop.cache), [0, 0, 0]
    for new in ([70, 33, 0], [1, 40, 90], [1, 1, 1], [4, 0, 2]):
        loop.fill(new)
        loop.step()
        past = loop.check(model, new, past)
    # a decode step captured, replayed with other tokens (its blocks are there already)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    loop.fill([1, 1, 1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        loop.step()
    loop.fill([1, 1, 1])
    graph.replay()
    past = loop.check(model, [1, 1, 1], past)

    # sequence 2 as vectors, and to fewer bits
    n = past[2]
    k, v = torch.empty((2, n, loop.n_kv, 128), dtype=torch.bfloat16, device="cuda")
    start, ctx = ints([0, 0, 0, n]), ints([0, 0, n])
    row = loop.n_kv * 128
    B.tq_fp8_read(loop.book, loop.view, loop.table, loop.max_blocks, n, loop.batch, loop.n_kv, start, ctx, B.TQ_BF16, k, v,
                  row, row)
    assert B.tq_get_last_device_error(loop.book) == 0
    table = loop.table.cpu().numpy()
    for i, (x, name) in enumerate(zip((k, v), "kv")):
        for h in range(loop.n_kv):
            assert np.array_equal(x[:, h].double().cpu().numpy(), model.values(name, table[2], 0, n, h))
    packed = C.allocate_cache(loop.book, loop.num_blocks, loop.n_kv)
    pos = np.arange(n)
    slots = table[2][pos // loop.bs].astype(np.int64) * loop.bs + pos % loop.bs
    B.tq_quantize_append(loop.book, k, v, B.TQ_BF16, n, loop.n_kv, torch.as_tensor(slots, device="cuda"),
                         C.cache_view(loop.book, packed))
    torch.cuda.synchronize()
    assert B.tq_get_last_device_error(loop.book) == 0
    check_append(loop.book, loop.ref, packed, k, v, slots)
