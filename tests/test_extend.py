"""Attention of several new tokens per sequence over the packed cache, against
the oracle's reconstruction of the GPU's own cache in 64 bits.

Tolerance of an output row, with u = 2^-11 (half a step of fp16, relative) and
v = 2^-8 (of bf16).  A score is a product of two rounded vectors: the rotated
query (constants and result rounded, 2 u, plus u for the query itself scaled
to fp16) and the key's levels (u; signs are exact but their factor is rounded,
u), so |delta s_t| <= 4 u scale (|R q| n_t |c_t| + |S q| gamma_t coef sqrt(m))
by Cauchy-Schwarz, plus a few fp32 roundings (the factor 5 below).  A change
of every score by at most D changes softmax-weighted means by at most
(e^{2 D} - 1) max |v^|.  Weights and value levels are rounded to bf16 (2 v
relative to sum p |v^| <= max |v^|), the back-rotation's operands to fp16
(2 u), the output to bf16 (v relative to itself).
"""
import math

import numpy as np
import pytest
import torch

from online_kv_cache_tq_gb300 import binding as B
from online_kv_cache_tq_gb300 import build as libbuild
from online_kv_cache_tq_gb300 import cache as C
from online_kv_cache_tq_gb300 import workloads as W
from oracle import attention, packing, quantize

from parity_helpers import books, dtype_code, fill_cache, generator, host_cache

U, V = 2.0 ** -11, 2.0 ** -8


def reference(q, hc, row, length, n_new, kvh, ref, scale, blocked=()):
    """Outputs [n_new][G][128] of one sequence and KV head in float64, and the
    bound on each row's error.  Positions in ``blocked`` are skipped."""
    bs = hc["k_norm"].shape[2]
    rows = attention.read_sequence(hc, row, length, kvh, bs)
    codes = packing.unpack_planes(rows["k_codes"], ref["k_bits"], 128)
    kn, vn = rows["k_norm"].reshape(-1).astype(np.float64), rows["v_norm"].reshape(-1).astype(np.float64)
    khat = quantize.reconstruct_mse(rows["k_norm"].reshape(-1), codes, ref["rot"], ref["k_levels"])
    vhat = quantize.reconstruct_mse(rows["v_norm"].reshape(-1), rows["v_code_values"], ref["rot"], ref["v_levels"])
    level_norm = np.linalg.norm(ref["k_levels"][codes], axis=1)
    g = q.shape[1]
    qf = q.reshape(n_new * g, 128)
    s = qf @ khat.T
    reach = np.linalg.norm(qf, axis=1)[:, None] * (kn * level_norm)[None, :]
    if ref["proj"].shape[0]:
        sq = qf @ ref["proj"].T
        signs = 2.0 * packing.unpack_signs(rows["k_qjl"], 128) - 1.0
        coef = rows["k_rnorm"].reshape(-1).astype(np.float64) * math.sqrt(math.pi / 2) / 128
        s = s + (sq @ signs.T) * coef
        reach = reach + np.linalg.norm(sq, axis=1)[:, None] * (coef * math.sqrt(128))[None, :]
    s = (s * scale).reshape(n_new, g, length)
    reach = (reach * scale * 5 * U).reshape(n_new, g, length)
    seen = np.arange(length)[None, :] <= (length - n_new + np.arange(n_new))[:, None]
    seen[:, list(blocked)] = False
    out, bound = np.zeros((n_new, g, 128)), np.zeros((n_new, g, 1))
    for i in range(n_new):
        if not seen[i].any():
            continue
        z = s[i][:, seen[i]]
        p = np.exp(z - z.max(1, keepdims=True))
        out[i] = p @ vhat[seen[i]] / p.sum(1, keepdims=True)
        vmax = np.linalg.norm(vhat[seen[i]], axis=1).max()
        d = reach[i][:, seen[i]].max(1, keepdims=True)
        bound[i] = vmax * (np.expm1(2 * d) + 2.1 * V + 4 * U)
    return out, bound + V * np.abs(out)


class Case:
    def __init__(self, new, ctx, k_bits=3, v_bits=3, qjl=128, norm_bits=32, bs=64, n_kv=2, group=4, seed=0,
                 dtype=torch.bfloat16, q_scale=1.0, profile=None, pad=0, scale=0.0, identity=False):
        self.new, self.ctx, self.n_kv, self.group, self.n_q, self.scale = new, ctx, n_kv, group, n_kv * group, scale
        cfg = dict(n_kv=n_kv, block_size=bs, dtype="bf16", seed=seed, log_uniform=(0.3, 3.0), outliers=1,
                   outlier_scale=5.0)
        cfg.update(profile or {})
        self.book, self.ref = books(k_bits, v_bits, qjl, seed=1, block_size=bs, norm_bits=norm_bits)
        self.table, _ = W.block_layout(np.maximum(ctx, 1), bs, True, seed=seed)
        if identity:
            self.table = np.arange(self.table.size, dtype=np.int32).reshape(self.table.shape)
        g = generator(seed)
        self.cache = fill_cache(self.book, cfg, ctx, self.table, g)
        self.total = int(sum(new)) + pad
        self.q = (torch.randn((self.total, self.n_q, 128), generator=g, device="cuda") * q_scale).to(dtype)
        self.start = torch.as_tensor(np.concatenate([[0], np.cumsum(new)]).astype(np.int32), device="cuda")
        self.ctx_t = torch.as_tensor(np.asarray(ctx, np.int32), device="cuda")
        self.table_t = None if identity else torch.as_tensor(self.table, device="cuda")
        self.ws, self.nbytes = C.allocate_extend_workspace(self.book, max(1, self.total), len(new), self.n_q, n_kv,
                                                           int(max(ctx)))
        self.out = torch.full((self.total, self.n_q, 128), 5.0, dtype=torch.bfloat16, device="cuda")

    def run(self, stream=None, out=None, ws=None):
        B.tq_extend_attention(self.book, self.q, dtype_code(self.q), self.total, len(self.new), self.n_q, self.n_kv,
                              C.cache_view(self.book, self.cache), self.table_t, self.table.shape[1], self.start,
                              self.ctx_t, int(max(self.ctx)), self.scale, self.out if out is None else out,
                              self.ws if ws is None else ws, self.nbytes, stream)

    def check(self, sequences=None, tokens=None, blocked=(), code=0):
        """Compare sequences (all by default); tokens: at most that many new
        tokens of each, the last ones."""
        torch.cuda.synchronize()
        assert B.tq_get_last_device_error(self.book) == code
        got = self.out.double().cpu().numpy()
        hc = host_cache(self.cache)
        qn = self.q.double().cpu().numpy()
        scale = self.scale or 1.0 / math.sqrt(128)
        starts = np.concatenate([[0], np.cumsum(self.new)])
        err2 = ref2 = 0.0
        for b in range(len(self.new)) if sequences is None else sequences:
            n, length = int(self.new[b]), int(self.ctx[b])
            if n == 0:
                continue
            seen_none = max(0, n - length)
            assert (got[starts[b]:starts[b] + seen_none] == 0.0).all()
            take = n - seen_none if tokens is None else min(tokens, n - seen_none)
            for h in range(self.n_kv):
                if take == 0 or length == 0:
                    continue
                hs = slice(h * self.group, (h + 1) * self.group)
                rs = slice(starts[b] + n - take, starts[b] + n)
                expect, bound = reference(qn[rs, hs], hc, self.table[b], length, take, h, self.ref, scale, blocked)
                err = np.abs(got[rs, hs] - expect)
                assert np.isfinite(got[rs, hs]).all()
                assert (err <= bound + 1e-30).all(), "seq %d KV head %d: worst %.3g of the bound" % (
                    b, h, (err / np.maximum(bound, 1e-30)).max())
                err2 += (err ** 2).sum()
                ref2 += (expect ** 2).sum()
        assert (got[starts[-1]:] == 5.0).all()     # rows behind the last sequence
        # the roundings are independent: far below the worst case together
        assert ref2 == 0.0 or math.sqrt(err2 / ref2) <= 2.0 * V, math.sqrt(err2 / ref2)
        return math.sqrt(err2 / ref2) if ref2 else 0.0


def test_host_only_handle_is_refused():
    libbuild.build()
    book = B.Codebook(device=-1)
    view = B.tq_cache_view(16, 16, 16, 16, 16, 16, 1, 1, 64)
    assert B.tq_extend_workspace_bytes(book, 4, 1, 1, 1, 64) == 0
    with pytest.raises(B.TQError) as err:
        B.tq_extend_attention(book, 16, 0, 1, 1, 1, 1, view, None, 1, 16, 16, 64, 0.0, 16, 256, 1 << 20, stream=0)
    assert err.value.status == 1
    book.close()


@pytest.mark.gpu
@pytest.mark.parametrize("k_bits,v_bits,qjl,norm_bits,bs", [
    (3, 3, 128, 32, 64), (2, 1, 128, 32, 32), (5, 4, 128, 16, 96), (4, 2, 128, 32, 128), (1, 3, 0, 32, 64),
    (2, 2, 0, 16, 32), (3, 4, 0, 32, 256), (4, 1, 0, 32, 64)])
def test_bit_widths_and_block_sizes(k_bits, v_bits, qjl, norm_bits, bs):
    c = Case([5, 1, 3], [300, 1, 129], k_bits, v_bits, qjl, norm_bits, bs, seed=k_bits)
    c.run()
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("group,n_kv", [(1, 1), (1, 5), (2, 2), (3, 2), (8, 1), (7, 1), (16, 1), (40, 2)])
def test_ragged_batches(group, n_kv):
    # no new tokens, all of the context new, one token, more new tokens than context, contexts of 0 and 1
    c = Case([0, 64, 1, 37, 3, 1, 2], [40, 64, 700, 20, 128, 1, 0], n_kv=n_kv, group=group, seed=group, pad=3)
    c.run()
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("k_bits,v_bits,qjl", [(3, 3, 128), (4, 4, 0)])
@pytest.mark.parametrize("new,ctx", [([200], [200]), ([129, 250], [1000, 251]), ([33, 16, 300], [2000, 16, 555])])
def test_prompt_chunks(k_bits, v_bits, qjl, new, ctx):
    c = Case(new, ctx, k_bits, v_bits, qjl, n_kv=2, group=8, seed=3)
    c.run()
    print("relative rms error %.3g" % c.check())


@pytest.mark.gpu
@pytest.mark.parametrize("bs", [32, 64, 128])
def test_long_prompt(bs):
    c = Case([1500], [2011], n_kv=1, group=4, bs=bs, seed=5)
    c.run()
    c.check(tokens=40)
    c.check(tokens=1500) if bs == 64 else None


@pytest.mark.gpu
@pytest.mark.parametrize("new,ctx", [([4], [20000]), ([2, 5, 1], [9000, 30, 12345])])
def test_few_tokens_on_long_contexts(new, ctx):
    c = Case(new, ctx, n_kv=2, group=4, seed=6)
    c.run()
    c.check()


@pytest.mark.gpu
def test_float_queries_scale_and_identity_table():
    c = Case([9, 40], [130, 500], dtype=torch.float32, scale=0.05, identity=True, seed=7)
    c.run()
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("q_scale", [0.0, 1e-30, 3e4])
def test_query_magnitudes(q_scale):
    # zero queries (every key weighs the same), tiny ones, and a softmax that is one token (its bound in this file
    # is loose, the outputs are finite and the token the same)
    c = Case([6, 20], [200, 90], q_scale=q_scale, seed=8)
    c.run()
    torch.cuda.synchronize()
    if q_scale < 1.0:
        c.check()
    else:
        assert bool(torch.isfinite(c.out.float()).all()) and B.tq_get_last_device_error(c.book) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("new", [3, 300])
@pytest.mark.parametrize("q_scale,k_scale", [(4e33, 1.0), (1 / 30, 1e9), (4e8, 1e4)])
def test_scores_of_huge_magnitude(new, dtype, q_scale, k_scale):
    # every query points along one long key (30 times the others), with coordinates up to 2^118 or keys of 1e11: the
    # scores are finite numbers in 32 bits (6e37, 5e11, 6e16), and the weights are those of that token alone
    c = Case([new], [400], n_kv=1, group=4, seed=20, dtype=dtype)
    g = generator(5)
    k = torch.randn((400, 1, 128), generator=g, device="cuda")
    k[5] *= 30.0
    direction = k[5] * q_scale
    k *= k_scale
    v = torch.randn((400, 1, 128), generator=g, device="cuda")
    slots = torch.as_tensor(W.slots_for(c.table[0], np.arange(400), 64), device="cuda")
    B.tq_quantize_append(c.book, k, v, B.TQ_FP32, 400, 1, slots, C.cache_view(c.book, c.cache))
    c.q.copy_(direction.expand_as(c.q))
    c.run()
    torch.cuda.synchronize()
    assert B.tq_get_last_device_error(c.book) == 0
    expect, _ = reference(c.q.double().cpu().numpy(), host_cache(c.cache), c.table[0], 400, new, 0, c.ref,
                          1.0 / math.sqrt(128))
    got = c.out.double().cpu().numpy()
    assert np.isfinite(got).all()
    # one weight, so only the weight's and the value levels' roundings, R^T's and the output's are left
    size = np.linalg.norm(expect, axis=2, keepdims=True)
    assert (np.abs(got - expect) <= size * (2.1 * V + 4 * U) + V * np.abs(expect)).all()


@pytest.mark.gpu
def test_tokens_over_decades_of_magnitude_and_zero_vectors():
    c = Case([30], [400], seed=9, n_kv=1, group=8)
    g = generator(3)
    mags = 10.0 ** torch.empty(400, device="cuda").uniform_(-4, 1, generator=g)
    mags[::17] = 0.0
    k = torch.randn((400, 1, 128), generator=g, device="cuda") * mags[:, None, None]
    v = torch.randn((400, 1, 128), generator=g, device="cuda") * mags.flip(0)[:, None, None]
    slots = torch.as_tensor(W.slots_for(c.table[0], np.arange(400), 64), device="cuda")
    B.tq_quantize_append(c.book, k.contiguous(), v.contiguous(), B.TQ_FP32, 400, 1, slots, C.cache_view(c.book, c.cache))
    c.run()
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_stale_slots_behind_the_context_do_not_matter(bad):
    c = Case([3, 70], [65, 90], seed=10)
    for b, length in enumerate(c.ctx):
        blk, off = int(c.table[b, (length - 1) // 64]), length % 64
        for f in ("k_norm", "k_rnorm", "v_norm"):
            c.cache[f][blk, :, off:] = bad
    # ... nor does the value of a position that a token does not see yet
    last = (int(c.table[1, 89 // 64]), slice(None), 89 % 64)
    keep = c.out.clone()
    c.run()
    torch.cuda.synchronize()
    first = c.out.clone()
    for f in ("k_norm", "k_rnorm", "v_norm"):
        c.cache[f][last] = bad
    c.out.copy_(keep)
    c.run()
    torch.cuda.synchronize()
    assert torch.equal(first[:72], c.out[:72]) and bool(torch.isfinite(first.float()).all())
    assert bool(torch.isnan(c.out[72].float()).any()) or not math.isnan(bad)


@pytest.mark.gpu
def test_bad_blocks_are_skipped_and_recorded():
    c = Case([4, 2], [300, 100], seed=11)
    c.table_t[0, 1] = -1
    c.table_t[0, 3] = 1 << 20
    c.run()
    c.check(sequences=[0], blocked=list(range(64, 128)) + list(range(192, 256)), code=2)
    c.table_t[0] = -1                              # nothing left: zero rows
    c.run()
    torch.cuda.synchronize()
    assert bool((c.out[:4] == 0).all()) and B.tq_get_last_device_error(c.book) == 2


@pytest.mark.gpu
def test_bad_lengths_are_recorded():
    for ctx in (-1, 10 ** 6):
        c = Case([3, 2], [100, 100], seed=12)
        c.ctx_t[0] = ctx
        c.run()
        torch.cuda.synchronize()
        assert bool((c.out[:3] == 0).all()) and B.tq_get_last_device_error(c.book) == 3
        c.new, c.out[:3] = [3, 2], 0.0
        c.check(sequences=[1])
    for start in ([0, 9, 5], [-2, 3, 5], [0, 3, 50]):
        c = Case([3, 2], [100, 100], seed=13)
        c.start.copy_(torch.as_tensor(start, dtype=torch.int32))
        c.run()
        torch.cuda.synchronize()
        assert B.tq_get_last_device_error(c.book) == 3
        assert bool(torch.isfinite(c.out.float()).all())


@pytest.mark.gpu
def test_more_expanded_tiles_than_the_workspace_holds():
    # five sequences of 512 rows over 64 KV heads: 8256 expanded tiles each, of
    # which the workspace holds 32768, so the last one is read from its packed cache
    c = Case([512] * 5, [16500, 16400, 16512, 16385, 16450], n_kv=64, group=1, seed=17, bs=128)
    assert c.nbytes < 3 << 30
    c.run()
    torch.cuda.synchronize()
    hc, got, qn = host_cache(c.cache), c.out.double().cpu().numpy(), c.q.double().cpu().numpy()
    assert B.tq_get_last_device_error(c.book) == 0
    for b in range(5):
        last = slice(512 * b + 509, 512 * b + 512)
        for h in (0, 41, 63):
            expect, bound = reference(qn[last, h:h + 1], hc, c.table[b], int(c.ctx[b]), 3, h, c.ref,
                                      1.0 / math.sqrt(128))
            err = np.abs(got[last, h:h + 1] - expect)
            assert (err <= bound).all()
            assert math.sqrt((err ** 2).sum() / (expect ** 2).sum()) <= 2.0 * V


@pytest.mark.gpu
@pytest.mark.parametrize("group", [1, 4, 8])
def test_both_forms_in_one_call(group):
    # sequences on either side of 512 rows, some with rows that see nothing, row tiles cut at every place
    n = 512 // group
    c = Case([n - 1, n, n + 1, 2, 3 * n, n + 5], [n + 70, n, 4000, 5000, 3 * n + 1, n - 9], n_kv=2, group=group, seed=18)
    c.run()
    c.check(tokens=40)
    c.run()
    c.check(sequences=[0, 2, 4], tokens=n - 1)


@pytest.mark.gpu
@pytest.mark.parametrize("new", [3, 300])
def test_a_later_tile_passes_the_reference(new):
    # keys that grow along the context raise the reference again and again; a huge value behind a row's limit
    # leaves the rows before it as they are
    c = Case([new], [900], n_kv=1, group=4, seed=19)
    g = generator(4)
    k = torch.randn((900, 1, 128), generator=g, device="cuda") * torch.linspace(1, 60, 900, device="cuda")[:, None, None]
    v = torch.randn((900, 1, 128), generator=g, device="cuda")
    v[899] *= 1e6
    slots = torch.as_tensor(W.slots_for(c.table[0], np.arange(900), 64), device="cuda")
    B.tq_quantize_append(c.book, k.contiguous(), v.contiguous(), B.TQ_FP32, 900, 1, slots, C.cache_view(c.book, c.cache))
    c.run()
    torch.cuda.synchronize()
    hc, got, qn = host_cache(c.cache), c.out.double().cpu().numpy(), c.q.double().cpu().numpy()
    expect, bound = reference(qn, hc, c.table[0], 900, new, 0, c.ref, 1.0 / math.sqrt(128))
    assert np.isfinite(got).all() and (np.abs(got - expect) <= bound).all()
    before = np.abs(got - expect)[:-1], expect[:-1]
    # A score is a sum of 128 products with |q| n scale up to 680, of rms 60; the fp16 roundings of the query, its
    # rotation and the keys (2^-11 each at most, 2e-4 in the rms) move it by 0.03 in the rms.  An output of a few
    # weights moves by twice that at most, 6 %, relative to itself: half of 32 2^-8.
    assert math.sqrt((before[0] ** 2).sum() / (before[1] ** 2).sum()) <= 32.0 * V


@pytest.mark.gpu
def test_one_token_agrees_with_decode():
    c = Case([1, 1, 1], [77, 512, 1300], seed=14)
    c.run()
    ws, nbytes = C.allocate_workspace(c.book, 3, c.n_q, 1300)
    out = torch.zeros((3, c.n_q, 128), device="cuda")
    B.tq_decode_attention(c.book, c.q, B.TQ_BF16, 3, c.n_q, c.n_kv, C.cache_view(c.book, c.cache), c.table_t,
                          c.table.shape[1], c.ctx_t, 1300, 0.0, out, ws, nbytes)
    c.check()
    err = (c.out.float() - out).norm() / out.norm()
    assert float(err) <= 2.0 * V


@pytest.mark.gpu
@pytest.mark.parametrize("new,ctx", [([4, 3], [3000, 700]), ([400, 20], [900, 4000])])
def test_same_call_same_bits_on_streams_and_in_graphs(new, ctx):
    c = Case(new, ctx, n_kv=2, group=4, seed=15)
    c.run()
    torch.cuda.synchronize()
    first = c.out.clone()
    # two calls at once, each with its own workspace
    side = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(c.out) for _ in range(2)]
    spaces = [torch.full_like(c.ws, 255) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, o, w in zip(side, outs, spaces):
            c.run(stream=s, out=o, ws=w)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], first) and torch.equal(outs[1], first)
    # two captured graphs that share a workspace, replayed one after the other
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for gph, o in zip(graphs, outs):
        o.zero_()
        with torch.cuda.graph(gph):
            c.run(out=o)
    for gph in graphs + graphs[::-1]:
        gph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], first) and torch.equal(outs[1], first)
    c.q.mul_(0.5)
    graphs[0].replay()
    c.run()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], c.out) and not torch.equal(outs[0], first)


@pytest.mark.gpu
def test_shorter_sequences_in_a_captured_shape():
    # a graph captured for the largest step, replayed with fewer tokens and shorter contexts
    c = Case([40, 30], [1000, 600], seed=16)
    c.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    c.new, c.ctx = [7, 0], [555, 600]
    c.start.copy_(torch.as_tensor([0, 7, 7], dtype=torch.int32))
    c.ctx_t.copy_(torch.as_tensor([555, 600], dtype=torch.int32))
    c.out.fill_(5.0)
    graph.replay()
    c.check()


@pytest.mark.gpu
def test_refusals():
    c = Case([3], [100])
    view = C.cache_view(c.book, c.cache)
    base = [c.q, B.TQ_BF16, 3, 1, c.n_q, c.n_kv, view, c.table_t, c.table.shape[1], c.start, c.ctx_t, 100, 0.0, c.out,
            c.ws, c.nbytes]
    other = B.tq_cache_view(*[getattr(view, n) for n, _ in view._fields_])
    other.n_kv_heads = 1
    odd = B.tq_cache_view(*[getattr(view, n) for n, _ in view._fields_])
    odd.k_codes = view.k_codes + 4
    for i, value, status in ((0, None, 1), (0, c.q.data_ptr() + 2, 1), (1, 7, 1), (2, -1, 1), (3, -1, 1), (4, 0, 1),
                             (4, 7, 1), (5, 0, 1), (6, other, 1), (6, odd, 1), (8, 0, 1), (9, None, 1),
                             (10, None, 1), (11, -1, 1), (12, -1.0, 1), (12, float("nan"), 1), (13, None, 1),
                             (13, c.out.data_ptr() + 2, 1), (14, None, 5), (14, c.ws.data_ptr() + 16, 5),
                             (15, c.nbytes - 1, 5)):
        args = list(base)
        args[i] = value
        with pytest.raises(B.TQError) as err:
            B.tq_extend_attention(c.book, *args)
        assert err.value.status == status, i
    polar = B.Codebook(k_bits=0, v_bits=0, qjl_m=0, codec=1)
    pc = C.allocate_cache(polar, 2, 1)
    with pytest.raises(B.TQError) as err:
        B.tq_extend_attention(polar, c.q, B.TQ_BF16, 3, 1, 4, 1, C.cache_view(polar, pc), None, 2, c.start, c.ctx_t, 100,
                              0.0, c.out, c.ws, c.nbytes)
    assert err.value.status == 2
    torch.cuda.synchronize()
    assert bool((c.out == 5.0).all())
    args = list(base)
    args[2] = 0
    B.tq_extend_attention(c.book, *args)           # no tokens: nothing to do
    assert B.tq_get_last_device_error(c.book) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("new", [3, 300])
def test_zero_values_under_small_weights(new):
    # every score is near -15 (as a power of two), so the weights sum to 2^-6 or less; the values a row sees first are
    # zero vectors: zero rows, not 0 * infinity
    c = Case([new], [new], n_kv=1, group=4, seed=25)
    g = generator(8)
    base = torch.randn((1, 1, 128), generator=g, device="cuda")
    k = base + 0.05 * torch.randn((new, 1, 128), generator=g, device="cuda")
    v = torch.randn((new, 1, 128), generator=g, device="cuda")
    v[:max(2, new // 2)] = 0.0
    slots = torch.as_tensor(W.slots_for(c.table[0], np.arange(new), 64), device="cuda")
    B.tq_quantize_append(c.book, k, v, B.TQ_FP32, new, 1, slots, C.cache_view(c.book, c.cache))
    c.q.copy_((base[0, 0] * (-10.0 * math.sqrt(128.0) / float(base.norm()) ** 2)).expand_as(c.q))
    c.run()
    c.check()
    assert bool((c.out[:max(2, new // 2)] == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("new", [3, 300])
@pytest.mark.parametrize("size", [300.0, 500.0, 800.0, 1000.0])
def test_queries_along_rows_of_the_sketch(new, size):
    # the signs of a row of S make S q as large as it can be: `size` times the row's sum of magnitudes, 118000 for 1000
    c = Case([new], [400], n_kv=1, group=4, scale=1e-4, seed=21)
    rows = np.sign(c.ref["proj"][np.arange(c.total * 4) % 128]).reshape(c.total, 4, 128)
    c.q.copy_(torch.as_tensor(size * rows))
    c.run()
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("new", [6, 140])
def test_nan_of_a_hidden_key_next_to_large_scores(new):
    # the last token's key is NaN and lies in the same group of 32 tokens as a key whose score is 2^140 above the
    # others'; only the last token sees it
    ctx = max(30, new)
    c = Case([new], [ctx], n_kv=1, group=4, seed=22)
    g = generator(6)
    k = torch.randn((ctx, 1, 128), generator=g, device="cuda")
    long = ctx - new                               # (every row sees it)
    k[long] *= 30.0
    v = torch.randn((ctx, 1, 128), generator=g, device="cuda")
    slots = torch.as_tensor(W.slots_for(c.table[0], np.arange(ctx), 64), device="cuda")
    B.tq_quantize_append(c.book, k, v, B.TQ_FP32, ctx, 1, slots, C.cache_view(c.book, c.cache))
    direction = k[long, 0].cpu().numpy() * (100.0 * math.sqrt(128.0) / float(k[long].norm()) ** 2)
    c.q.copy_(torch.as_tensor(direction).expand_as(c.q))
    c.run()
    c.check(sequences=[])
    first = c.out.clone()
    assert bool(torch.isfinite(first.float()).all())
    for hidden in (ctx - 1, (long // 32) * 32 + 31):
        if hidden <= long or hidden >= ctx:
            continue
        last = (int(c.table[0, hidden // 64]), slice(None), hidden % 64)
        kept = c.cache["k_norm"][last].clone()
        c.cache["k_norm"][last] = float("nan")
        c.run()
        torch.cuda.synchronize()
        rows = new - (ctx - hidden)                # rows before the hidden token
        assert torch.equal(first[:rows], c.out[:rows])
        assert bool(torch.isnan(c.out[rows:].float()).any())
        c.cache["k_norm"][last] = kept


@pytest.mark.gpu
@pytest.mark.parametrize("new", [3, 300])
@pytest.mark.parametrize("score,value_scale", [(52.0, 2.0 ** 23), (-52.0, 2.0 ** -43)])
def test_values_at_the_ends_of_their_range_with_scores_far_from_zero(new, score, value_scale):
    # every score is near +-75 (as a power of two), just inside the bound below which no maximum is searched, and the
    # values have the largest and smallest lengths that the interface allows
    c = Case([new], [400], n_kv=1, group=4, seed=23)
    g = generator(7)
    base = torch.randn((1, 1, 128), generator=g, device="cuda")
    k = base + 0.05 * torch.randn((400, 1, 128), generator=g, device="cuda")
    v = torch.randn((400, 1, 128), generator=g, device="cuda") * value_scale
    slots = torch.as_tensor(W.slots_for(c.table[0], np.arange(400), 64), device="cuda")
    B.tq_quantize_append(c.book, k, v, B.TQ_FP32, 400, 1, slots, C.cache_view(c.book, c.cache))
    q = base[0, 0] * (score * math.sqrt(128.0) / float(base.norm()) ** 2)
    c.q.copy_(q.expand_as(c.q))
    c.run()
    c.check()


@pytest.mark.gpu
def test_misaligned_lengths_and_tables_are_refused():
    c = Case([3], [100])
    base = [c.q, B.TQ_BF16, 3, 1, c.n_q, c.n_kv, C.cache_view(c.book, c.cache), c.table_t, c.table.shape[1], c.start,
            c.ctx_t, 100, 0.0, c.out, c.ws, c.nbytes]
    for i in (7, 9, 10):
        args = list(base)
        args[i] = base[i].data_ptr() + 2
        with pytest.raises(B.TQError) as err:
            B.tq_extend_attention(c.book, *args)
        assert err.value.status == 1, i
    torch.cuda.synchronize()
    assert bool((c.out == 5.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("new,n_kv", [([2, 5], 1), ([300, 200], 2), ([3, 400], 2)])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_correct(new, n_kv):
    # the test aid withholds one product's completion in the first CTA of each launch: its waits run out after a second,
    # what it has in flight is drained, the call ends with device error 4 and the handle works on
    c = Case(new, [n + 700 for n in new], n_kv=n_kv, group=4, seed=24)
    B.tq_debug_withhold_commit(c.book, True)
    c.run()
    torch.cuda.synchronize()
    assert B.tq_get_last_device_error(c.book) == 4
    B.tq_debug_withhold_commit(c.book, False)
    c.run()
    c.check(tokens=40)
