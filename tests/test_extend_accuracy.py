"""How far the multi-token attention is from 64 bits, on the value profiles of the library's own workloads.

The roundings are independent of one another and each is known, so the expected square of an output row's error follows
from the oracle's own numbers; the test compares the measured root-mean-square with it.  A rounding to s bits of a
number with an even spread of mantissas is off by 2^-s sqrt(1/3) sqrt(3 / (8 ln 2)) of it in the rms (s = 8 for bf16, 11
for fp16; half a step, its mean square, and the mean of 1 / mantissa^2).  Per row, with weights p_t (sum 1), values v_t
and output o = sum p_t v_t:
  output     b |o|, b for bf16 (and fp16 for the back-rotation's two operands, value levels within 2^-10.4)
  weights    b p_t |v_t| for each token whose weight has no remainder (three in four, by place in the cache)
  scores     d_t p_t |v_t - o|, d_t the rms error of score t (times scale):
             narrow form: R q and S q rounded (f for fp16) and their constants rounded; the sketch's factor as the two
             fp16 numbers around it, a step 2^-10 apart, sqrt(1/6) of it in the rms, with a mean within 2^-14.5,
             wide form: the key in the original space rounded and its constants rounded;
             fp32 queries: the query rounded.  Key levels are within 2^-12.9 (one rounding in 2^-13 each, rms).
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

from test_extend import Case
from parity_helpers import generator, host_cache

MANTISSA = math.sqrt(1.0 / 3.0) * math.sqrt(3.0 / (8.0 * math.log(2.0)))
BF16, FP16 = 2.0 ** -8 * MANTISSA, 2.0 ** -11 * MANTISSA
AROUND = 2.0 ** -10 * math.sqrt(1.0 / 6.0) * math.sqrt(3.0 / (8.0 * math.log(2.0)))


def has_remainder(tokens):
    """Tokens whose weights have a remainder: those of the last sixteen of 64 columns, in expansion order."""
    return (tokens % 64 >= 32) & (tokens % 4 >= 2)


def expected(q, hc, row, length, n_new, kvh, ref, scale, wide, round_q):
    """(outputs [n_new][G][128], expected square of each row's error) in float64; q: the sequence's last n_new tokens."""
    rows = attention.read_sequence(hc, row, length, kvh, hc["k_norm"].shape[2])
    codes = packing.unpack_planes(rows["k_codes"], ref["k_bits"], 128)
    kn, vn = rows["k_norm"].reshape(-1).astype(np.float64), rows["v_norm"].reshape(-1).astype(np.float64)
    c = ref["k_levels"][codes] * kn[:, None]
    vhat = quantize.reconstruct_mse(rows["v_norm"].reshape(-1), rows["v_code_values"], ref["rot"], ref["v_levels"])
    g = q.shape[1]
    qf = q.reshape(n_new * g, 128)
    q2, rq = qf ** 2, qf @ ref["rot"].T
    khat = c @ ref["rot"]
    s, d2 = rq @ c.T, (q2 @ (ref["rot"] ** 2).T) @ (c ** 2).T       # (R's constants)
    d2 += (rq ** 2) @ (c ** 2).T * (2.0 ** -13 / FP16) ** 2         # (key levels)
    if not wide:
        d2 += (rq ** 2) @ (c ** 2).T
    if ref["proj"].shape[0]:
        sq = qf @ ref["proj"].T
        signs = 2.0 * packing.unpack_signs(rows["k_qjl"], 128) - 1.0
        coef = rows["k_rnorm"].reshape(-1).astype(np.float64) * math.sqrt(math.pi / 2) / 128
        sketch = (sq @ signs.T) * coef
        khat = khat + coef[:, None] * (signs @ ref["proj"])
        s = s + sketch
        d2 += (q2 @ (ref["proj"] ** 2).T).sum(1)[:, None] * coef ** 2
        if not wide:
            d2 += (sq ** 2).sum(1)[:, None] * coef ** 2 * (1.0 + (AROUND / FP16) ** 2)
            d2 += (sketch * 2.0 ** -14.5 / FP16) ** 2
    d2 += (int(wide) + int(round_q)) * (q2 @ (khat ** 2).T)
    s, d2 = [x.reshape(n_new, g, length) for x in (s * scale, d2 * (FP16 * scale) ** 2)]
    seen = np.arange(length)[None, :] <= (length - n_new + np.arange(n_new))[:, None]
    v2, plain = (vhat ** 2).sum(1), (~has_remainder(np.arange(length))).astype(np.float64)
    out, err2 = np.zeros((n_new, g, 128)), np.zeros((n_new, g))
    for i in range(n_new):
        z = s[i][:, seen[i]]
        p = np.exp(z - z.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        v, d = vhat[seen[i]], d2[i][:, seen[i]]
        out[i] = o = p @ v
        o2 = (o ** 2).sum(1)
        apart = v2[seen[i]][None, :] - 2.0 * (o @ v.T) + o2[:, None]
        err2[i] = o2 * (BF16 ** 2 + 2 * FP16 ** 2 + 2.0 ** -22.8) + BF16 ** 2 * (p ** 2) @ (v2 * plain)[seen[i]] + \
            (p ** 2 * d * apart).sum(1)
    return out, err2


def measure(c, tokens, wide):
    """(measured rms, expected rms, rms of rounding the exact output alone, worst normalised error) of all sequences."""
    c.run()
    torch.cuda.synchronize()
    assert B.tq_get_last_device_error(c.book) == 0
    got, qn, hc = c.out.double().cpu().numpy(), c.q.double().cpu().numpy(), host_cache(c.cache)
    starts = np.concatenate([[0], np.cumsum(c.new)])
    sums, worst = np.zeros(4), 0.0
    for b, n in enumerate(c.new):
        take = min(tokens, n)
        rs = slice(starts[b] + n - take, starts[b] + n)
        for h in range(c.n_kv):
            hs = slice(h * c.group, (h + 1) * c.group)
            out, err2 = expected(qn[rs, hs], hc, c.table[b], int(c.ctx[b]), take, h, c.ref, 1.0 / math.sqrt(128.0), wide,
                                 c.q.dtype == torch.float32)
            err = got[rs, hs] - out
            rounded = torch.as_tensor(out).to(torch.bfloat16).double().numpy() - out
            sums += [(err ** 2).sum(), err2.sum(), (rounded ** 2).sum(), (out ** 2).sum()]
            worst = max(worst, np.abs(err).max() / np.sqrt((out ** 2).sum(-1)).max())
    return [math.sqrt(x / sums[3]) for x in sums[:3]] + [worst]


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("workload", ["c1_single_head_parity", "c2_llama3_8b_decode", "c4_long_context",
                                      "c5_llama3_70b_paged"])
def test_error_is_that_of_the_known_roundings(workload, wide):
    cfg = W.CONFIGS[workload]
    profile = {k: cfg[k] for k in ("log_uniform", "outliers", "outlier_scale")}
    new = [160, 150] if wide else [24, 9]
    c = Case(new, [2000, 1500], cfg["k_bits"], cfg["v_bits"], cfg["qjl_m"], n_kv=4, group=4, seed=31,
             dtype=W.torch_dtype(cfg["dtype"]), profile=profile)
    rms, model, rounding, _ = measure(c, 24, wide)
    print("%s %s: rms %.4g, expected %.4g, output's rounding %.4g" % (workload, "wide" if wide else "narrow", rms, model,
                                                                      rounding))
    # Rows whose output hangs on a few scores give few independent errors: 264 to 384 rows a case, a factor of 1.25
    assert rms <= 1.25 * model


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("k_bits,v_bits,qjl,norm_bits", [(3, 3, 128, 32), (5, 4, 128, 16), (4, 4, 0, 32), (2, 1, 128, 32),
                                                         (3, 2, 0, 16)])
def test_error_of_ordinary_keys(k_bits, v_bits, qjl, norm_bits, wide):
    # unit normal keys and queries: many weights and small scores, so the sum of the roundings is close to its expectation
    c = Case([160, 150] if wide else [24, 9], [2000, 1500], k_bits, v_bits, qjl, norm_bits, n_kv=2, group=4, seed=32,
             profile=dict(log_uniform=None, outliers=0))
    rms, model, _, _ = measure(c, 24, wide)
    print("rms %.4g, expected %.4g" % (rms, model))
    assert rms <= 1.05 * model


@pytest.mark.gpu
@pytest.mark.parametrize("new", [8, 160])
def test_weights_with_remainders(new):
    # Every query points along one long key, whose value is all that its row returns: the ratio of the row to that value is
    # the weight's own error (the output's roundings average out over 128 coordinates: b / sqrt(128), 1.5e-4, and two
    # fp16 operands; value levels within 2^-10.4 of a weight's worth, below 2^-11 in the mean of a row's levels).
    # Without its remainder a weight is off by b = 1.7e-3 in the rms.
    ctx, errors = 512, {True: [], False: []}
    c = Case([new], [ctx], n_kv=1, group=4, seed=33)
    slots = torch.as_tensor(W.slots_for(c.table[0], np.arange(ctx), 64), device="cuda")
    for long in range(200, 264):
        g = generator(long)
        k = torch.randn((ctx, 1, 128), generator=g, device="cuda")
        k[long] *= 30.0
        v = torch.randn((ctx, 1, 128), generator=g, device="cuda")
        B.tq_quantize_append(c.book, k, v, B.TQ_FP32, ctx, 1, slots, C.cache_view(c.book, c.cache))
        c.q.copy_((k[long] * 0.02).expand_as(c.q))
        c.run()
        torch.cuda.synchronize()
        row = c.out[-1, 0].double().cpu().numpy()
        out, _ = expected(c.q[-1:].double().cpu().numpy(), host_cache(c.cache), c.table[0], ctx, 1, 0, c.ref,
                          1.0 / math.sqrt(128.0), new > 100, False)
        o = out[0, 0]
        errors[bool(has_remainder(np.int64(long)))].append(float(row @ o / (o @ o)) - 1.0)
    assert B.tq_get_last_device_error(c.book) == 0
    rms = {k: math.sqrt(np.mean(np.square(e))) for k, e in errors.items()}
    print("weights with remainders %.3g, without %.3g" % (rms[True], rms[False]))
    assert len(errors[True]) == 16 and rms[True] <= 2.0 ** -11 + 1.5e-4
    assert rms[False] <= 1.25 * BF16


@pytest.mark.parametrize("bits,bf16,fp16", [(1, -16.0, -16.0), (2, -16.0, -16.0), (3, -11.4, -14.4), (4, -10.3, -12.8)])
def test_common_factor_of_the_levels(bits, bf16, fp16):
    # the search the library makes: of 2^16 multiples of the codebook the one whose worst rounding is least, then the
    # factor that fits best; the stated bounds of the levels' relative errors hold for what comes out
    libbuild.build()
    book = B.Codebook(k_bits=bits, v_bits=bits, qjl_m=0, device=-1)
    levels = np.asarray(B.tq_codebook_levels(book, 0)[0], np.float64)
    pos = levels[len(levels) // 2:]
    m = 1.0 + np.arange(65536) / 65536.0
    for dtype, bound in ((torch.bfloat16, bf16), (torch.float16, fp16)):
        rounded = lambda x: torch.as_tensor(np.asarray(x)).to(torch.float32).to(dtype).double().numpy()
        worst = np.abs(rounded(m[:, None] * pos) / (m[:, None] * pos) - 1.0).max(1)
        y = rounded(m[worst.argmin()] * levels)
        factor = (levels * y).sum() / (y * y).sum()
        assert np.abs(factor * y / levels - 1.0).max() <= 2.0 ** bound
        # (rounded as they are, all but the one-bit levels would be an order of magnitude further off at bf16)
        assert np.abs(rounded(levels) / levels - 1.0).max() > 2.0 ** bound or bits == 1
    book.close()


@pytest.mark.gpu
@pytest.mark.parametrize("new", [8, 160])
def test_the_sketchs_factor_is_not_rounded_as_one(new):
    # A query whose score on two keys is the sketch's part alone, 60 each: a common rounding of a key's factor would move its
    # score by f 60, 0.012 in the rms, and their difference by 0.018.  The two share the row, whose mixture of their values
    # gives the difference.  What is expected of its error are the independent roundings, and in the narrow form numbers
    # next to the factor that alternate between coordinates, off by half a step (2^-11) in the rms, with a mean within
    # 2^-14.5.
    ctx, errors, share = 128, [], []
    c = Case([new], [max(ctx, new)], n_kv=1, group=4, seed=34, profile=dict(log_uniform=None, outliers=0))
    ctx, wide, scale = int(c.ctx[0]), new > 100, 1.0 / math.sqrt(128.0)
    slots = torch.as_tensor(W.slots_for(c.table[0], np.arange(ctx), 64), device="cuda")
    proj = c.ref["proj"]
    for seed in range(40):
        g = generator(900 + seed)
        k = torch.randn((ctx, 1, 128), generator=g, device="cuda")
        k[[3, 70]] *= 8.0 + 8.0 * torch.rand((2, 1, 1), generator=g, device="cuda")   # (the others' scores stay far below)
        v = torch.randn((ctx, 1, 128), generator=g, device="cuda")
        B.tq_quantize_append(c.book, k, v, B.TQ_FP32, ctx, 1, slots, C.cache_view(c.book, c.cache))
        hc = host_cache(c.cache)
        rows = attention.read_sequence(hc, c.table[0], ctx, 0, 64)
        signs = 2.0 * packing.unpack_signs(rows["k_qjl"], 128) - 1.0
        c_lv = c.ref["k_levels"][packing.unpack_planes(rows["k_codes"], c.ref["k_bits"], 128)]
        kn, coef = rows["k_norm"].reshape(-1).astype(float), rows["k_rnorm"].reshape(-1).astype(float) * math.sqrt(
            math.pi / 2) / 128
        main, sketch = (c_lv * kn[:, None]) @ c.ref["rot"], coef[:, None] * (signs @ proj)
        khat = main + sketch
        q = np.linalg.lstsq(np.concatenate([main[[3, 70]], sketch[[3, 70]]]), np.array([0, 0, 60.0, 60.0]) / scale,
                            rcond=None)[0]
        c.q.copy_(torch.as_tensor(q).to(torch.bfloat16).expand_as(c.q))
        qb = c.q[0, 0].double().cpu().numpy()
        s = khat[[3, 70]] @ qb * scale
        c.run()
        torch.cuda.synchronize()
        out = c.out[-1, 0].double().cpu().numpy()
        vhat = quantize.reconstruct_mse(rows["v_norm"].reshape(-1), rows["v_code_values"], c.ref["rot"], c.ref["v_levels"])
        w = np.linalg.lstsq(vhat[[3, 70]].T, out, rcond=None)[0]
        if w.min() < 0.02:
            continue
        rq, sq = c.ref["rot"] @ qb, proj @ qb
        d2 = 0.0
        for t in (3, 70):
            d2 += ((c.ref["rot"] ** 2) @ qb ** 2 * (c_lv[t] * kn[t]) ** 2).sum() + ((proj ** 2) @ qb ** 2).sum() * coef[t] ** 2
            d2 += (rq ** 2 * (c_lv[t] * kn[t]) ** 2).sum() + (sq ** 2).sum() * coef[t] ** 2 * (1 + (2.0 ** -11 / FP16) ** 2) \
                if not wide else (qb ** 2 * khat[t] ** 2).sum()
            d2 += (2.0 ** -14.5 / FP16 * coef[t] * (sq @ signs[t])) ** 2 * (not wide)
        errors.append(math.log(w[0] / w[1]) - (s[0] - s[1]))
        share.append(d2 * (FP16 * scale) ** 2 + 2 * (1.5 * BF16) ** 2)   # (the weights' roundings, and the output's)
    assert len(errors) >= 20
    rms, model = math.sqrt(np.mean(np.square(errors))), math.sqrt(np.mean(share))
    print("difference of two scores: rms error %.3g, expected %.3g" % (rms, model))
    assert rms <= 1.4 * model                      # (20 to 40 samples: a factor of 1.4 is three deviations)
