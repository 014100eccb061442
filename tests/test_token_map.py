"""Token map of a step (context lengths, query starts, positions, slots, fresh
block table entries) against a loop over the batch; whole numbers are equal."""
import ctypes

import numpy as np
import pytest
import torch

from online_kv_cache_tq_gb300 import binding as B
from online_kv_cache_tq_gb300 import build as libbuild


def reference(past, new, table, free, n_tokens, bs, num_blocks):
    """Plain loop; table is modified in place."""
    batch, max_blocks = table.shape
    ctx, start = [], [0]
    positions, slots = np.full(n_tokens, -1, np.int32), np.full(n_tokens, -1, np.int64)
    used = t = 0
    for b in range(batch):
        p, n = int(past[b]), int(new[b])
        if p < 0 or n < 0 or p + n > max_blocks * bs:
            p = n = 0
        ctx.append(p + n)
        start.append(start[-1] + n)
        for col in range(-(-p // bs), -(-(p + n) // bs)):
            ok = used < len(free) and 0 <= free[used] < num_blocks
            table[b, col] = free[used] if ok else -1
            used += 1
        for pos in range(p, p + n):
            if t < n_tokens:
                blk = int(table[b, pos // bs])
                positions[t] = pos
                slots[t] = blk * bs + pos % bs if 0 <= blk < num_blocks else -1
            t += 1
    return np.array(ctx, np.int32), np.array(start, np.int32), positions, slots, used


def make(batch, bs, seed, past_hi, new_hi, zero_new=0.3):
    rng = np.random.default_rng(seed)
    past = rng.integers(0, past_hi + 1, batch).astype(np.int32)
    new = rng.integers(0, new_hi + 1, batch).astype(np.int32)
    new[rng.random(batch) < zero_new] = 0
    before, after = -(-past // bs), -(-(past + new) // bs)
    max_blocks = max(1, int(after.max()) + 1)
    num_blocks = int(after.sum()) + 5
    ids = rng.permutation(num_blocks).astype(np.int32)
    table = np.full((batch, max_blocks), -7, np.int32)
    pos = 0
    for b in range(batch):
        table[b, :before[b]] = ids[pos:pos + before[b]]
        pos += before[b]
    return past, new, table, ids[pos:].copy(), num_blocks


class Call:
    """Device buffers of one call, outputs pre-filled with a sentinel."""

    def __init__(self, past, new, table, free, num_blocks, n_tokens):
        dev = lambda x: torch.as_tensor(x, device="cuda")
        self.batch, self.num_blocks, self.n_tokens = len(past), num_blocks, n_tokens
        self.past, self.new, self.table, self.free = dev(past), dev(new), dev(table.copy()), dev(free)
        self.ctx = torch.full((max(1, self.batch),), -9, dtype=torch.int32, device="cuda")
        self.start = torch.full((self.batch + 1,), -9, dtype=torch.int32, device="cuda")
        self.positions = torch.full((n_tokens + 3,), -9, dtype=torch.int32, device="cuda")
        self.slots = torch.full((n_tokens + 3,), -9, dtype=torch.int64, device="cuda")
        self.taken = torch.full((1,), -9, dtype=torch.int32, device="cuda")

    def run(self, book, stream=None):
        B.tq_map_tokens(book, self.batch, self.past, self.new, self.table, self.table.shape[1], self.num_blocks,
                        self.free, self.free.numel(), self.n_tokens, self.ctx, self.start, self.positions, self.slots,
                        self.taken, stream)

    def check(self, table, free, past, new, bs):
        expect_table = table.copy()
        ctx, start, positions, slots, used = reference(past, new, expect_table, free, self.n_tokens, bs,
                                                       self.num_blocks)
        torch.cuda.synchronize()
        n = self.n_tokens
        assert np.array_equal(self.ctx.cpu().numpy()[:self.batch], ctx)
        assert np.array_equal(self.start.cpu().numpy(), start)
        assert np.array_equal(self.positions.cpu().numpy()[:n], positions)
        assert np.array_equal(self.slots.cpu().numpy()[:n], slots)
        assert np.array_equal(self.table.cpu().numpy(), expect_table)
        assert int(self.taken) == used
        # nothing behind the rows is written
        assert bool((self.positions[n:] == -9).all()) and bool((self.slots[n:] == -9).all())


def test_host_only_handle_is_refused():
    libbuild.build()
    book = B.Codebook(device=-1)
    one = ctypes.c_int(0)
    p = ctypes.addressof(one)
    with pytest.raises(B.TQError) as err:
        B.tq_map_tokens(book, 1, p, p, p, 1, 1, p, 1, 1, p, p, p, p, p, stream=0)
    assert err.value.status == 1
    book.close()


@pytest.mark.gpu
@pytest.mark.parametrize("batch,bs,past_hi,new_hi,pad", [
    (1, 64, 0, 1, 0), (1, 32, 0, 5000, 0), (1, 64, 200000, 3, 1), (7, 96, 500, 40, 5), (64, 64, 32768, 1, 0),
    (255, 32, 300, 300, 17), (256, 64, 0, 70, 0), (257, 128, 1000, 33, 1), (1000, 32, 40, 9, 2000),
    (8192, 32, 100, 2, 3)])
def test_against_the_loop(batch, bs, past_hi, new_hi, pad):
    book = B.Codebook(block_size=bs)
    past, new, table, free, num_blocks = make(batch, bs, batch + bs, past_hi, new_hi, 0.0 if batch == 1 else 0.3)
    call = Call(past, new, table, free, num_blocks, int(new.sum()) + pad)
    call.run(book)
    call.check(table, free, past, new, bs)
    call.run(book)                                 # the same inputs: the same outputs
    call.check(table, free, past, new, bs)
    assert B.tq_get_last_device_error(book) == 0


@pytest.mark.gpu
def test_no_tokens_and_no_sequences():
    book = B.Codebook()
    table = np.full((3, 2), -1, np.int32)
    past, new = np.array([0, 64, 5], np.int32), np.zeros(3, np.int32)
    call = Call(past, new, table, np.zeros(0, np.int32), 4, 0)
    call.run(book)
    call.check(table, [], past, new, 64)
    empty = Call(np.zeros(0, np.int32), np.zeros(0, np.int32), np.zeros((0, 2), np.int32), np.zeros(0, np.int32), 4, 6)
    B.tq_map_tokens(book, 0, None, None, None, 2, 4, None, 0, 6, None, empty.start, empty.positions, empty.slots,
                    empty.taken)
    torch.cuda.synchronize()
    assert empty.start.tolist() == [0] and int(empty.taken) == 0
    assert empty.positions.tolist() == [-1] * 6 + [-9] * 3 and empty.slots.tolist() == [-1] * 6 + [-9] * 3
    assert B.tq_get_last_device_error(book) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("what,code", [("short_list", 6), ("bad_free", 2), ("bad_entry", 2), ("negative", 3),
                                       ("too_long", 3), ("few_rows", 7)])
def test_recorded_errors(what, code):
    book = B.Codebook()
    past = np.array([10, 64, 0, 100], np.int32)
    new = np.array([3, 130, 65, 1], np.int32)
    table = np.full((4, 5), -1, np.int32)
    table[0, 0], table[1, 0], table[3, :2] = 0, 1, (2, 3)
    free, n_tokens = np.arange(4, 20, dtype=np.int32), int(new.sum())
    if what == "short_list":
        free = free[:2]
    elif what == "bad_free":
        free[1] = 1000
    elif what == "bad_entry":
        table[0, 0] = 20
    elif what == "negative":
        past[1] = -1
    elif what == "too_long":
        new[2] = 5 * 64 + 1
    elif what == "few_rows":
        n_tokens -= 50
    call = Call(past, new, table, free, 20, n_tokens)
    call.run(book)
    call.check(table, free, past, new, 64)
    assert B.tq_get_last_device_error(book) == code
    assert B.tq_get_last_device_error(book) == 0


@pytest.mark.gpu
def test_refusals():
    book = B.Codebook()
    past, new, table, free, num_blocks = make(4, 64, 0, 100, 10)
    ok = Call(past, new, table, free, num_blocks, int(new.sum()))
    base = [4, ok.past, ok.new, ok.table, table.shape[1], num_blocks, ok.free, ok.free.numel(), ok.n_tokens, ok.ctx,
            ok.start, ok.positions, ok.slots, ok.taken]
    for i, value, status in ((0, -1, 1), (0, 8193, 2), (1, None, 1), (2, None, 1), (3, None, 1), (4, 0, 1),
                             (4, 1 << 30, 1), (5, 0, 1), (6, None, 1), (7, -1, 1), (8, -1, 1), (9, None, 1),
                             (9, ok.past, 1), (9, ok.new, 1), (10, None, 1), (11, None, 1), (12, None, 1),
                             (12, ok.slots.data_ptr() + 4, 1), (13, None, 1)):
        args = list(base)
        args[i] = value
        with pytest.raises(B.TQError) as err:
            B.tq_map_tokens(book, *args)
        assert err.value.status == status, i
    torch.cuda.synchronize()
    assert bool((ok.slots == -9).all()) and bool((ok.start == -9).all())   # a rejected call leaves its buffers


@pytest.mark.gpu
def test_captured_and_replayed_with_other_lengths():
    book = B.Codebook()
    past, new, table, free, num_blocks = make(30, 64, 3, 2000, 50)
    call = Call(past, new, table, free, num_blocks, int(new.sum()) + 40)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call.run(book)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call.run(book)
    graph.replay()
    call.check(table, free, past, new, 64)
    fewer = np.maximum(new - 3, 0).astype(np.int32)
    call.new.copy_(torch.as_tensor(fewer))
    call.table.copy_(torch.as_tensor(table))
    graph.replay()
    call.check(table, free, past, fewer, 64)
    assert B.tq_get_last_device_error(book) == 0


@pytest.mark.gpu
def test_large_and_middling_batches_from_several_threads():
    # the starts of a batch take shared memory beyond the default limit, which is raised for the whole process
    import threading
    book = B.Codebook(block_size=32)
    calls, failed = [], []
    for batch in (8192, 5200, 8192, 5300):
        past, new, table, free, num_blocks = make(batch, 32, batch, 100, 2)
        call = Call(past, new, table, free, num_blocks, int(new.sum()) + 3)
        calls.append((call, (table, free, past, new, 32)))
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    entry, ptr = B.load().tq_map_tokens, lambda t: ctypes.c_void_p(t.data_ptr())

    def work(c, stream):
        # (arguments made once, so that the threads spend their time in the library)
        args = [book.handle, c.batch, ptr(c.past), ptr(c.new), ptr(c.table), c.table.shape[1], c.num_blocks,
                ptr(c.free), c.free.numel(), c.n_tokens, ptr(c.ctx), ptr(c.start), ptr(c.positions), ptr(c.slots),
                ptr(c.taken), ctypes.c_void_p(stream.cuda_stream)]
        for _ in range(20000):
            status = entry(*args)
            if status:
                failed.append(status)
                return

    threads = [threading.Thread(target=work, args=(c, s)) for (c, _), s in zip(calls, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for call, args in calls:
        call.check(*args)
    assert B.tq_get_last_device_error(book) == 0


@pytest.mark.gpu
def test_misaligned_lengths_and_outputs_are_refused():
    book = B.Codebook()
    past, new, table, free, num_blocks = make(4, 64, 0, 100, 10)
    ok = Call(past, new, table, free, num_blocks, int(new.sum()))
    base = [4, ok.past, ok.new, ok.table, table.shape[1], num_blocks, ok.free, ok.free.numel(), ok.n_tokens, ok.ctx,
            ok.start, ok.positions, ok.slots, ok.taken]
    for i in (1, 2, 3, 6, 9, 10, 11, 13):
        args = list(base)
        args[i] = base[i].data_ptr() + 2
        with pytest.raises(B.TQError) as err:
            B.tq_map_tokens(book, *args)
        assert err.value.status == 1, i
    torch.cuda.synchronize()
    assert bool((ok.slots == -9).all()) and bool((ok.start == -9).all())


@pytest.mark.gpu
def test_a_captured_step_moves_on_in_its_free_list():
    # the list in a buffer of fixed capacity, -1 behind its end: lengths and list move on on the device, so that a replay is
    # the next step; the last steps find the list used up
    bs, batch, num_blocks, cap = 32, 5, 40, 64
    book = B.Codebook(block_size=bs)
    rng = np.random.default_rng(11)
    free = np.full(cap, -1, np.int32)
    free[:num_blocks] = rng.permutation(num_blocks)
    past, new = np.zeros(batch, np.int32), np.array([33, 0, 70, 1, 64], np.int32)
    table = np.full((batch, 30), -1, np.int32)
    call = Call(past, new, table, free, num_blocks, 220)
    index = torch.arange(cap, device="cuda")
    padded = torch.full((2 * cap,), -1, dtype=torch.int32, device="cuda")

    def step():
        call.run(book)
        call.past.copy_(call.ctx)
        padded[:cap].copy_(call.free)
        call.free.copy_(padded[index + call.taken])

    side = torch.cuda.Stream()                     # (a step outside the graph first, as PyTorch asks, then the start again)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    call.past.copy_(torch.as_tensor(past))
    call.table.copy_(torch.as_tensor(table))
    call.free.copy_(torch.as_tensor(free))
    assert B.tq_get_last_device_error(book) == 0
    codes = []
    for _ in range(9):
        graph.replay()
        ctx, start, positions, slots, used = reference(past, new, table, free, 220, bs, num_blocks)
        torch.cuda.synchronize()
        assert np.array_equal(call.ctx.cpu().numpy(), ctx) and int(call.taken) == used
        assert np.array_equal(call.positions.cpu().numpy()[:220], positions)
        assert np.array_equal(call.slots.cpu().numpy()[:220], slots)
        assert np.array_equal(call.table.cpu().numpy(), table)
        past, free = ctx, np.concatenate([free[used:], np.full(min(used, cap), -1, np.int32)])[:cap]
        assert np.array_equal(call.free.cpu().numpy(), free)
        codes.append(B.tq_get_last_device_error(book))
    assert codes[0] == 0 and codes[-1] == 2
