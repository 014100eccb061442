"""The 8-bit cache written and read back, against a plain model in 64 bits that
holds every byte of it: codes, scales and what the calls leave alone have to be
the same, bit for bit (the read's values are exact in either type)."""
import numpy as np
import pytest
import torch

from online_kv_cache_tq_gb300 import binding as B
from online_kv_cache_tq_gb300 import build as libbuild
from online_kv_cache_tq_gb300 import cache as C

LEAST, MOST = -40, 14
CODE_VALUES = np.array([(-1.0 if b & 128 else 1.0) * (np.nan if b & 127 == 127 else
                        ((b & 7) / 8.0 * 2.0 ** -6 if b & 120 == 0 else (1 + (b & 7) / 8.0) * 2.0 ** ((b >> 3 & 15) - 7)))
                        for b in range(256)])


def to_codes(x):
    """float64 -> e4m3 codes, to nearest even, saturating, NaN 0x7f."""
    x = np.asarray(x, np.float64)
    nan, sign = np.isnan(x), np.where(np.signbit(x), 128, 0)
    a = np.minimum(np.abs(np.where(nan, 0.0, x)), 448.0)
    e = np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -6.0)
    step = 2.0 ** (e - 3)
    a = np.rint(a / step) * step                     # (np.rint: half to even)
    a = np.minimum(a, 448.0)
    low = np.rint(a * 2.0 ** 9).astype(np.int64)     # subnormals and 2^-6: multiples of 2^-9
    e = np.floor(np.log2(np.where(a > 0, a, 1.0)))
    high = ((e + 7) * 8 + np.rint((a / 2.0 ** e - 1) * 8)).astype(np.int64)
    code = np.where(a < 2.0 ** -6, low, high)
    return np.where(nan, 127, code | sign).astype(np.uint8)


def scale_exponent(amax):
    if not amax > 0:
        return LEAST
    m, e = np.frexp(min(float(amax), 3e38))
    return int(min(MOST, max(LEAST, (e + 1 if m > 0.875 else e) - 9)))


class Model:
    """The cache as token-major codes [blocks][heads][offset][128] and scale exponents, for "k" and "v"."""

    def __init__(self, cache):
        k, v = cache["k_codes"].cpu().numpy(), cache["v_codes"].cpu().numpy()
        n, h = k.shape[:2]
        self.codes = dict(k=k.transpose(0, 1, 2, 4, 3, 5).reshape(n, h, -1, 128).copy(),
                          v=v.transpose(0, 1, 2, 4, 3).reshape(n, h, -1, 128).copy())
        self.scale = dict(k=cache["k_scale"].cpu().numpy().copy(), v=cache["v_scale"].cpu().numpy().copy())
        self.block_size = self.codes["k"].shape[2]

    def append(self, name, rows, table, new, ctx):
        """rows [tokens][heads][128] float64; sequences that the call leaves out have new 0 here."""
        bs, row = self.block_size, 0
        for b, (n, length) in enumerate(zip(new, ctx)):
            pos = length - n
            while pos < length:
                block, off = int(table[b][pos // bs]), pos % bs
                count = min(bs - off, length - pos)
                if block >= 0:
                    self.run(name, block, off, rows[row:row + count])
                pos, row = pos + count, row + count

    def run(self, name, block, off, x):
        codes, scale = self.codes[name][block], self.scale[name][block]
        for h in range(x.shape[1]):
            amax = np.nanmax(np.abs(np.where(np.isnan(x[:, h]), 0.0, x[:, h])))
            e = scale_exponent(amax)
            old = int(np.round(np.log2(scale[h]))) if off else e
            if off and e > old:
                codes[h, :off] = to_codes(CODE_VALUES[codes[h, :off]] * 2.0 ** (old - e))
            e = max(e, old)
            new = to_codes(x[:, h] / 2.0 ** e)
            new[np.isnan(x[:, h]).any(-1)] = 127
            codes[h, off:off + len(x)] = new
            scale[h] = 2.0 ** e

    def values(self, name, table_row, first, last, head):
        """[last - first][128] float64."""
        pos = np.arange(first, last)
        blk = np.asarray(table_row)[pos // self.block_size]
        return CODE_VALUES[self.codes[name][blk, head, pos % self.block_size]] * \
            self.scale[name][blk, head].astype(np.float64)[:, None]

    def check(self, cache):
        other = Model(cache)
        for name in ("k", "v"):
            assert np.array_equal(self.scale[name], other.scale[name]), name
            bad = self.codes[name] != other.codes[name]
            assert not bad.any(), "%s: %d codes differ, first at %s" % (name, bad.sum(), np.argwhere(bad)[0])


def random_cache(book, num_blocks, n_kv, g):
    """A cache whose blocks hold what earlier use left: any codes (no NaN), ordinary scales."""
    cache = C.allocate_fp8_cache(book, num_blocks, n_kv)
    for name in ("k_codes", "v_codes"):
        c = torch.randint(0, 255, cache[name].shape, generator=g, device="cuda", dtype=torch.uint8)
        cache[name].copy_(torch.where((c & 127) == 127, 3, c))
    for name in ("k_scale", "v_scale"):
        cache[name].copy_(torch.exp2(torch.randint(-9, -5, cache[name].shape, generator=g, device="cuda").float()))
    return cache


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def ints(x):
    return torch.as_tensor(np.asarray(x, np.int32), device="cuda")


class Case:
    def __init__(self, new, past, bs=64, n_kv=2, dtype=torch.bfloat16, seed=0, pad=0, identity=False, spare=2):
        self.new, self.ctx, self.n_kv, self.bs, self.dtype = list(new), [p + n for p, n in zip(past, new)], n_kv, bs, dtype
        self.batch, self.total = len(new), sum(new) + pad
        self.book = B.Codebook(block_size=bs)
        need = [-(-max(c, 1) // bs) for c in self.ctx]
        self.max_blocks = max(need)
        rng = np.random.default_rng(seed)
        self.num_blocks = self.batch * self.max_blocks + spare
        ids = np.arange(self.num_blocks) if identity else rng.permutation(self.num_blocks)
        self.table = ids[:self.batch * self.max_blocks].reshape(self.batch, self.max_blocks).astype(np.int32)
        self.table_t = None if identity else ints(self.table)
        self.g = generator(seed)
        self.cache = random_cache(self.book, self.num_blocks, n_kv, self.g)
        self.view = C.fp8_view(self.book, self.cache)
        self.start, self.ctx_t = ints(np.concatenate([[0], np.cumsum(new)])), ints(self.ctx)
        self.kv = (torch.randn((self.total, 2, n_kv, 128), generator=self.g, device="cuda") *
                   torch.exp(torch.randn((self.total, 1, 1, 1), generator=self.g, device="cuda"))).to(dtype)

    @property
    def code(self):
        return B.TQ_BF16 if self.dtype == torch.bfloat16 else B.TQ_FP32

    def append(self, k=True, v=True, stream=None):
        row = 2 * self.n_kv * 128
        B.tq_fp8_append(self.book, self.kv[:, 0] if k else None, self.kv[:, 1] if v else None, self.code, self.total,
                        self.batch, self.n_kv, row, row, self.view, self.table_t, self.max_blocks, self.start,
                        self.ctx_t, stream)

    def read(self, k=True, v=True, dtype=None, start=None, ctx=None, total=None, stream=None):
        dtype, total = dtype or self.dtype, self.total if total is None else total
        out = torch.full((2, total, self.n_kv + 1, 128), 7.0, dtype=dtype, device="cuda")
        row = (self.n_kv + 1) * 128
        B.tq_fp8_read(self.book, self.view, self.table_t, self.max_blocks, total, self.batch, self.n_kv,
                      self.start if start is None else start, self.ctx_t if ctx is None else ctx,
                      B.TQ_BF16 if dtype == torch.bfloat16 else B.TQ_FP32, out[0] if k else None,
                      out[1] if v else None, row, row, stream)
        return out

    def check_append(self, k=True, v=True, code=0, new=None):
        model = Model(self.cache)
        self.append(k, v)
        assert B.tq_get_last_device_error(self.book) == code
        x = self.kv.double().cpu().numpy()
        for i, name in enumerate("kv"):
            if (k, v)[i]:
                model.append(name, x[:, i], self.table, self.new if new is None else new, self.ctx)
        model.check(self.cache)
        return model

    def check_read(self, model, dtype=None, new=None, ctx=None, k=True, v=True):
        new, ctx = new or self.new, ctx or self.ctx
        start = np.concatenate([[0], np.cumsum(new)])
        total = int(start[-1]) + 3
        out = self.read(k, v, dtype, ints(start), ints(ctx), total)
        assert B.tq_get_last_device_error(self.book) == 0
        got = out.double().cpu().numpy()
        for i, name in enumerate("kv"):
            if not (k, v)[i]:
                assert (got[i] == 7.0).all()
                continue
            for b in range(self.batch):
                for h in range(self.n_kv):
                    expect = model.values(name, self.table[b], ctx[b] - new[b], ctx[b], h)
                    assert np.array_equal(got[i, start[b]:start[b + 1], h], expect, equal_nan=True)
            assert (got[i, start[-1]:] == 7.0).all() and (got[i, :, self.n_kv] == 7.0).all()


def test_codes_of_the_model():
    # every code stands for itself, midpoints go to the even code, what is beyond saturates
    finite = CODE_VALUES[np.isfinite(CODE_VALUES)]
    assert np.array_equal(CODE_VALUES[to_codes(finite)], finite)
    up = np.sort(finite[finite >= 0])[1:]
    mid = 0.5 * (up[:-1] + up[1:])
    assert (to_codes(mid) % 2 == 0).all()
    assert (to_codes([500.0, -1e30, np.inf]) == [126, 254, 126]).all() and to_codes(np.nan) == 127
    assert scale_exponent(448.0) == 0 and scale_exponent(448.0001) == 1 and scale_exponent(0.0) == LEAST
    assert scale_exponent(224.0) == -1 and scale_exponent(1e30) == MOST and scale_exponent(1e-30) == LEAST


def test_host_only_handle_is_refused():
    libbuild.build()
    book = B.Codebook(device=-1)
    view = B.make_fp8_view(16, 16, 16, 16, 4, 1, 64)
    calls = [lambda: B.tq_fp8_append(book, 16, 16, 0, 4, 1, 1, 128, 128, view, None, 4, 16, 16, 0),
             lambda: B.tq_fp8_read(book, view, None, 4, 4, 1, 1, 16, 16, 0, 16, 16, 128, 128, 0),
             lambda: B.tq_fp8_attention(book, 16, 0, 4, 1, 1, 1, view, None, 4, 16, 16, 64, 0.0, 16, 256, 1 << 30, 0)]
    for call in calls:
        with pytest.raises(B.TQError) as err:
            call()
        assert err.value.status == 1
    assert B.tq_fp8_workspace_bytes(book, 4, 1, 1, 1, 64) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("bs", [32, 64, 96, 128, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ragged_appends_and_reads(bs, dtype):
    # empty, single and long runs; fresh blocks, blocks with earlier tokens, runs that end inside sixteen tokens
    c = Case([1, 0, 3, 9, 70, 300, 1, 17, 8, 33], [0, 5, 30, 31, 100, 0, 63, 15, 511, 95], bs=bs, n_kv=3, dtype=dtype,
             seed=bs, pad=5)
    model = c.check_append()
    c.check_read(model)
    # a second step behind the first: blocks go on, scales grow
    c.ctx = [x + n for x, n in zip(c.ctx, [0] * 10)]
    c.check_read(model, dtype=torch.float32, new=c.ctx, ctx=c.ctx)
    c.check_read(model, dtype=torch.bfloat16, new=[min(x, 21) for x in c.ctx], ctx=c.ctx)


@pytest.mark.gpu
@pytest.mark.parametrize("bs,dtype", [(64, torch.bfloat16), (96, torch.float32), (32, torch.bfloat16)])
def test_a_sequence_token_by_token(bs, dtype):
    # 150 steps of one token (two sequences, one beginning inside a block), magnitudes that grow and shrink
    c = Case([1, 1], [0, 40], bs=bs, dtype=dtype, seed=3)
    c.max_blocks, c.num_blocks = 8, 18
    c.cache = random_cache(c.book, 18, c.n_kv, c.g)
    c.view = C.fp8_view(c.book, c.cache)
    c.table = np.random.default_rng(1).permutation(18)[:16].reshape(2, 8).astype(np.int32)
    c.table_t = ints(c.table)
    model = Model(c.cache)
    rng = np.random.default_rng(2)
    for step in range(150):
        c.kv.copy_((torch.randn(c.kv.shape, generator=c.g, device="cuda") * float(np.exp(rng.normal() * 2))).to(dtype))
        c.append()
        x = c.kv.double().cpu().numpy()
        for i, name in enumerate("kv"):
            model.append(name, x[:, i], c.table, [1, 1], c.ctx)
        c.ctx = [v + 1 for v in c.ctx]
        c.ctx_t += 1
    torch.cuda.synchronize()
    assert B.tq_get_last_device_error(c.book) == 0
    model.check(c.cache)


@pytest.mark.gpu
@pytest.mark.parametrize("new,past", [([40], [10]), ([3], [50]), ([200, 5], [33, 129])])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_unusual_values(new, past, dtype):
    c = Case(new, past, dtype=dtype, seed=4)
    t = min(new)
    c.kv[0, :, 0] = 0.0
    c.kv[t // 2, 0, 0, 5] = float("nan")                 # one coordinate of a key
    c.kv[t - 1, 1, 1, 127] = float("-nan")
    c.kv[t // 2, 1, 0, 64] = float("inf")
    c.kv[0, 1, 1, 3] = -3e38
    c.check_append()
    for factor in (0.0, 1e-30, 1e-12, 2.0 ** -40, 1e9):
        d = Case(new, past, dtype=dtype, seed=5)
        d.kv *= factor
        d.check_read(d.check_append())


@pytest.mark.gpu
def test_magnitudes_at_the_borders_of_a_scale():
    for top in (447.0, 448.0, 449.0, 464.0, 480.0, 512.0, 0.875, 0.8751):
        c = Case([20], [0], dtype=torch.float32, seed=6)
        c.kv.clamp_(-1, 1).mul_(top)
        c.kv[3, :, :, 9] = top
        c.check_append()


@pytest.mark.gpu
def test_keys_or_values_alone_and_the_identity_table():
    c = Case([50, 1, 9], [3, 64, 20], identity=True, seed=7)
    model = c.check_append(k=True, v=False)
    c.check_read(model, k=False)
    model = c.check_append(k=False, v=True)
    c.check_read(model, v=False)
    c.check_read(model)


@pytest.mark.gpu
@pytest.mark.parametrize("batch", [300, 700])
def test_many_sequences(batch):
    rng = np.random.default_rng(batch)
    new = rng.choice([0, 1, 1, 1, 2, 40], batch)
    c = Case([int(n) for n in new], [int(p) for p in rng.integers(0, 90, batch)], bs=32, n_kv=1, seed=8, pad=3)
    c.check_read(c.check_append())


@pytest.mark.gpu
def test_long_prompt():
    c = Case([5000, 1, 3333], [77, 300, 0], bs=64, n_kv=2, seed=9)
    c.check_read(c.check_append())


@pytest.mark.gpu
def test_bad_lengths_and_blocks_are_recorded_and_left_out():
    base = dict(new=[5, 40, 7, 1], past=[10, 100, 0, 200])
    c = Case(seed=10, **base)
    c.ctx_t[1] = 39                                       # fewer than its rows
    c.ctx[1] = 39
    model = Model(c.cache)
    c.append()
    assert B.tq_get_last_device_error(c.book) == 3
    x = c.kv.double().cpu().numpy()
    rows = np.concatenate([x[:5], x[45:]])
    for i, name in enumerate("kv"):
        model.append(name, rows[:, i], c.table[[0, 2, 3]], [5, 7, 1], [15, 7, 201])
    model.check(c.cache)
    for bad in (-1, 1 << 30, -(1 << 31)):
        c = Case(seed=11, **base)
        c.table[1, 1] = -1
        c.table_t[1, 1] = bad
        c.check_append(code=2)
        out = c.read()
        assert B.tq_get_last_device_error(c.book) == 2
        # the block's tokens are positions 100 .. 127 of sequence 1
        assert bool((out[:, 5:33] == 7.0).all()) and bool((out[:, :5, :2] != 7.0).any())
    for start in ([0, 5, 3, 52, 53], [0, 5, 45, 52, 99], [0, -5, 45, 52, 53], [7, 5, 45, 52, 53]):
        c = Case(seed=12, **base)
        c.start.copy_(ints(start))
        c.append()
        c.read()
        assert B.tq_get_last_device_error(c.book) in (0, 3)
    for ctx in (-1, -(1 << 31), (1 << 31) - 1, 10 ** 6):
        c = Case(seed=13, **base)
        c.ctx_t[3] = ctx
        c.append()
        assert B.tq_get_last_device_error(c.book) == 3
        out = c.read()
        assert B.tq_get_last_device_error(c.book) == 3 and bool((out[:, 52:] == 7.0).all())


@pytest.mark.gpu
def test_refusals():
    c = Case([4], [60])
    row = 2 * c.n_kv * 128
    before = {k: v.clone() for k, v in c.cache.items()}
    out = torch.full((4, c.n_kv, 128), 7.0, dtype=c.dtype, device="cuda")
    append = [c.kv[:, 0], c.kv[:, 1], B.TQ_BF16, 4, 1, c.n_kv, row, row, c.view, c.table_t, c.max_blocks, c.start, c.ctx_t]
    read = [c.view, c.table_t, c.max_blocks, 4, 1, c.n_kv, c.start, c.ctx_t, B.TQ_BF16, out, out, 256, 256]
    view = lambda **kw: B.make_fp8_view(*[{**dict(k=c.cache["k_codes"], v=c.cache["v_codes"], ks=c.cache["k_scale"],
                                                  vs=c.cache["v_scale"], n=c.num_blocks, h=c.n_kv, bs=64), **kw}[x]
                                          for x in ("k", "v", "ks", "vs", "n", "h", "bs")])
    views = [view(k=None), view(v=None), view(ks=None), view(vs=None), view(n=0), view(h=1), view(bs=32),
             view(k=c.cache["k_codes"].data_ptr() + 8), view(vs=c.cache["v_scale"].data_ptr() + 4)]
    for fn, base, changes in (
            (B.tq_fp8_append, append,
             [(2, 2), (3, -1), (4, -1), (5, 0), (6, 255), (6, row + 4), (7, row - 256 * 2 - 8), (10, 0), (11, None), (12, None),
              (0, c.kv.data_ptr() + 2), (11, c.start.data_ptr() + 2), (12, c.ctx_t.data_ptr() + 1),
              (9, c.table_t.data_ptr() + 2)] + [(8, v) for v in views]),
            (B.tq_fp8_read, read,
             [(8, 3), (3, -1), (4, -1), (5, 0), (11, 128), (12, 258), (2, 0), (6, None), (7, None),
              (9, out.data_ptr() + 2), (6, c.start.data_ptr() + 2)] + [(0, v) for v in views])):
        for i, value in changes:
            args = list(base)
            args[i] = value
            with pytest.raises(B.TQError) as err:
                fn(c.book, *args)
            assert err.value.status == 1, (fn.__name__, i, value)
        both = list(base)
        for i in (0, 1) if fn is B.tq_fp8_append else (9, 10):
            both[i] = None
        with pytest.raises(B.TQError):
            fn(c.book, *both)
        # a table of its own: more blocks than there are
        args = list(base)
        at = 9 if fn is B.tq_fp8_append else 1
        args[at], args[at + 1] = None, c.num_blocks + 1
        with pytest.raises(B.TQError):
            fn(c.book, *args)
        # nothing to do
        args = list(base)
        for i in ((3, 4) if fn is B.tq_fp8_append else (3, 4)):
            args[i] = 0
            fn(c.book, *args)
    torch.cuda.synchronize()
    assert bool((out == 7.0).all())
    assert all(torch.equal(before[k], c.cache[k]) for k in before)


@pytest.mark.gpu
def test_streams_and_graphs():
    c = Case([70, 1, 9], [0, 40, 100], seed=14)
    start = {k: v.clone() for k, v in c.cache.items()}
    c.append()
    out = c.read()
    first = {k: v.clone() for k, v in c.cache.items()}
    restore = lambda: [c.cache[k].copy_(v) for k, v in start.items()]
    restore()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.append(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(first[k], c.cache[k]) for k in first)
    restore()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.append()
        again = c.read()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(first[k], c.cache[k]) for k in first)
    assert torch.equal(out, again)
    # other tokens and lengths in the captured shape
    restore()
    c.kv.mul_(3.0)
    c.start.copy_(ints([0, 30, 31, 35]))
    c.new, c.ctx = [30, 1, 4], [35, 42, 104]
    c.ctx_t.copy_(ints(c.ctx))
    model = Model(c.cache)
    graph.replay()
    torch.cuda.synchronize()
    x = c.kv.double().cpu().numpy()
    for i, name in enumerate("kv"):
        model.append(name, x[:, i], c.table, c.new, c.ctx)
    model.check(c.cache)


@pytest.mark.gpu
@pytest.mark.parametrize("batch,dtype", [(300, torch.float32), (1500, torch.bfloat16), (900, torch.float32)])
def test_more_sequences_than_threads(batch, dtype):
    # single tokens, and a few long runs among them
    rng = np.random.default_rng(batch)
    new = rng.choice([0, 1, 1, 1, 1, 1, 3], batch)
    new[[5, batch // 2, batch - 1]] = [130, 70, 40]
    c = Case([int(n) for n in new], [int(p) for p in rng.integers(0, 60, batch)], bs=32, n_kv=2, dtype=dtype, seed=15)
    c.check_read(c.check_append())


@pytest.mark.gpu
def test_rows_that_overlap_are_recorded():
    # query_start goes down: every other sequence would have all rows
    c = Case([40] * 6, [100] * 6, seed=16)
    before = {k: v.clone() for k, v in c.cache.items()}
    c.start.copy_(ints([0, 240, 0, 240, 0, 240, 240]))
    c.ctx_t.fill_(240)
    c.append()
    assert B.tq_get_last_device_error(c.book) == 3
    assert all(torch.equal(before[k], c.cache[k]) for k in before)


@pytest.mark.gpu
def test_blocks_beyond_four_gigabytes():
    # the same tokens in a small cache and at the end of one of 4.6 GB of keys and as much of values
    bs, n_kv, num_blocks = 64, 8, 70000
    small = Case([150, 1, 9], [0, 70, 120], bs=bs, n_kv=n_kv, identity=False, seed=17)
    ids = np.unique(small.table)
    far = {int(b): num_blocks - 1 - i for i, b in enumerate(ids)}
    keys = torch.empty((num_blocks, n_kv, bs // 8, 8, 8, 16), dtype=torch.uint8, device="cuda")
    values = torch.empty((num_blocks, n_kv, bs // 16, 128, 16), dtype=torch.uint8, device="cuda")
    scales = torch.ones((2, num_blocks, n_kv), device="cuda")
    big = dict(k_codes=keys, v_codes=values, k_scale=scales[0], v_scale=scales[1])
    near_t, far_t = ints(ids).long(), torch.tensor([far[int(b)] for b in ids], device="cuda")
    for name in big:
        big[name][far_t] = small.cache[name][near_t]
    small.append()
    out = small.read()
    small.table_t = ints(np.vectorize(far.get)(small.table))
    small.view = C.fp8_view(small.book, big)
    small.append()
    assert B.tq_get_last_device_error(small.book) == 0
    for name in big:
        assert torch.equal(big[name][far_t], small.cache[name][near_t]), name
    assert torch.equal(out, small.read())


@pytest.mark.gpu
@pytest.mark.parametrize("bs,new,past", [(64, [3], [50]), (64, [40], [10]), (64, [60], [0]), (96, [90], [3]), (128, [100], [28]),
                                         (256, [200], [40]), (256, [256], [0])])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_vector_with_a_nan_leaves_its_block_alone(bs, new, past, dtype):
    # its other coordinates, however large, do not count for the scale: the other tokens, earlier ones among them, are stored
    # as if it were a vector of zeros
    spoilt = [(1, 0, 5, 1e4), (new[0] - 1, 1, 127, float("inf")), (new[0] // 2, 0, 64, -1e4)]
    first = Case(new, past, bs=bs, dtype=dtype, seed=20)
    for t, head, at, _ in spoilt:
        first.kv[t, :, head] = 0.0
    model = first.check_append()
    for values in (1, 8, 128):                            # huge coordinates: beside the NaN, in its eighth, all
        c = Case(new, past, bs=bs, dtype=dtype, seed=20)
        for t, head, at, huge in spoilt:
            lo = at // values * values
            c.kv[t, :, head, lo:lo + values] = huge
            c.kv[t, 0, head, (at + 1) % 128] = c.kv[t, 1, head, at] = float("nan")
            c.kv[t, 0, head, at] = huge
        c.append()
        assert B.tq_get_last_device_error(c.book) == 0
        for t, head, _, _ in spoilt:
            pos = past[0] + t
            for name in "kv":
                model.codes[name][c.table[0, pos // bs], head, pos % bs] = 127
        model.check(c.cache)


@pytest.mark.gpu
@pytest.mark.parametrize("start", [[0, 20, 10, 30], [0, 20, 20, 19], [5, 3, 20, 30], [0, 60, 59, 59], [0, 10, -1, 30]])
@pytest.mark.parametrize("batch", [3, 400])
def test_an_append_whose_query_start_goes_down_writes_nothing(start, batch):
    # rows to spare: the sum of the sequences' rows is no more than there are
    c = Case([20, 0, 20] + [0] * (batch - 3), [100] * batch, seed=21, pad=24)
    before = {k: v.clone() for k, v in c.cache.items()}
    c.start.copy_(ints(start + [start[-1]] * (batch - 3)))
    c.append()
    assert B.tq_get_last_device_error(c.book) == 3
    assert all(torch.equal(before[k], c.cache[k]) for k in before)


@pytest.mark.gpu
@pytest.mark.parametrize("start", [[0, 20, 10, 30], [0, 20, 20, 19], [5, 3, 20, 30], [0, 60, 59, 59], [0, 10, -1, 30]])
@pytest.mark.parametrize("batch", [3, 400])
def test_a_read_whose_query_start_goes_down_writes_nothing(start, batch):
    c = Case([20, 0, 20] + [0] * (batch - 3), [100] * batch, seed=22, pad=24)
    out = c.read(start=ints(start + [start[-1]] * (batch - 3)))
    assert B.tq_get_last_device_error(c.book) == 3
    assert bool((out == 7.0).all())
