"""Head norms with the position rotation against the formula in 64 bits.

Tolerance.  fp32 arithmetic: the sum of 128 squares in a tree of at most 11
roundings, its mean, root and reciprocal (half of the sum's error, 4 more),
two products, a cosine and sine of absolute error below 3 * 2^-24 (an angle
within an eighth of a turn rounded to 24 bits, and the function itself), two
products and a sum: below 32 roundings of 2^-24 relative to |a| + |b| of the
pair, 2^-19 (|a| + |b|).  The output's rounding adds eps / 2 relative to the
value: 2^-8 at bf16, 2^-24 at fp32.
"""
import ctypes

import numpy as np
import pytest
import torch

from online_kv_cache_tq_gb300 import binding as B
from online_kv_cache_tq_gb300 import build as libbuild


def reference(x, w, eps, positions, inv_freq, rot, interleaved):
    """(values, bound of the arithmetic's error) in float64; x [tokens][heads][128]."""
    y = np.asarray(x, np.float64)
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * w
    mag = np.abs(y)
    if rot:
        angle = positions[:, None].astype(np.float64) * inv_freq
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        ia, ib = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if interleaved else \
            (np.arange(rot // 2), np.arange(rot // 2, rot))
        a, b = y[..., ia].copy(), y[..., ib].copy()
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        mag[..., ia] = mag[..., ib] = np.abs(a) + np.abs(b)
    return y, mag * 2.0 ** -19


def run(book, tokens, n_q, n_kv, dtype, rot, interleaved, norm, positions, seed, in_place=False, base=500000.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    qkv = torch.randn((tokens, n_q + 2 * n_kv, 128), generator=g, device="cuda")
    qkv = (qkv * torch.exp(torch.randn((1, n_q + 2 * n_kv, 128), generator=g, device="cuda"))).to(dtype)
    w = [(1 + 0.3 * torch.randn(128, generator=g, device="cuda")).to(dtype) if norm else None for _ in range(2)]
    inv = base ** (-torch.arange(rot // 2, dtype=torch.float64, device="cuda") / max(1, rot // 2))
    pos = torch.as_tensor(np.asarray(positions, np.int32), device="cuda")
    before = qkv.double().cpu().numpy()
    row = (n_q + 2 * n_kv) * 128
    if in_place:
        q_out, k_out, qs, ks = qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], row, row
    else:
        q_out = torch.full((tokens, n_q + 1, 128), 7.0, dtype=dtype, device="cuda")
        k_out = torch.full((tokens, n_kv + 2, 128), 7.0, dtype=dtype, device="cuda")
        qs, ks = (n_q + 1) * 128, (n_kv + 2) * 128
    B.tq_norm_rope(book, qkv[:, :n_q] if n_q else None, qkv[:, n_q:n_q + n_kv] if n_kv else None,
                   B.TQ_BF16 if dtype == torch.bfloat16 else B.TQ_FP32, tokens, n_q, n_kv, row, row, w[0], w[1], 1e-6,
                   pos, inv, rot, interleaved, q_out, k_out, qs, ks)
    torch.cuda.synchronize()
    rounding = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    live = np.asarray(positions) >= 0
    for out, lo, heads, wt in ((q_out, 0, n_q, w[0]), (k_out, n_q, n_kv, w[1])):
        got = out.double().cpu().numpy()
        x = before[:, lo:lo + heads]
        expect, bound = reference(x, None if wt is None else wt.double().cpu().numpy(), 1e-6, np.asarray(positions),
                                  inv.cpu().numpy(), rot, interleaved)
        err = np.abs(got[:, :heads] - expect)
        ok = err <= bound * (1 + rounding) + rounding * np.abs(expect) + 1e-37
        assert ok[live].all(), "%d values off, worst %.3g" % ((~ok[live]).sum(), err[live].max())
        # skipped tokens' rows and the space between rows are left alone
        assert np.array_equal(got[~live][:, :heads], x[~live] if in_place else np.full_like(x[~live], 7.0))
        if not in_place:
            assert (got[:, heads:] == 7.0).all()
    if in_place:
        assert np.array_equal(qkv.double().cpu().numpy()[:, n_q + n_kv:], before[:, n_q + n_kv:])


def test_host_only_handle_is_refused():
    libbuild.build()
    book = B.Codebook(device=-1)
    buf = (ctypes.c_double * 64)()
    p = ctypes.addressof(buf)
    with pytest.raises(B.TQError) as err:
        B.tq_norm_rope(book, p, p, 0, 1, 1, 1, 128, 128, None, None, 0.0, None, None, 0, 0, p, p, 128, 128, stream=0)
    assert err.value.status == 1
    book.close()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rot,interleaved", [(128, False), (128, True), (64, False), (96, True), (96, False),
                                             (16, False), (16, True), (0, False)])
@pytest.mark.parametrize("norm", [True, False])
def test_rotations(dtype, rot, interleaved, norm):
    book = B.Codebook()
    rng = np.random.default_rng(rot)
    positions = rng.integers(0, 131072, 37)
    positions[[0, 5, 36]] = (0, -1, -5)
    run(book, 37, 6, 3, dtype, rot, interleaved, norm, positions, seed=rot + norm)


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,n_q,n_kv", [(1, 1, 1), (1, 64, 8), (2, 5, 0), (3, 0, 7), (1217, 3, 1), (4999, 8, 2)])
def test_shapes(tokens, n_q, n_kv):
    run(B.Codebook(), tokens, n_q, n_kv, torch.bfloat16, 128, False, True, np.arange(tokens) + 1000, seed=tokens)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place(dtype, interleaved):
    positions = np.arange(50) + 77
    positions[7] = -1
    run(B.Codebook(), 50, 8, 2, dtype, 128, interleaved, True, positions, seed=9, in_place=True)


@pytest.mark.gpu
def test_angles_at_the_largest_positions():
    # every position an int32 holds: the fixed-point turns lose nothing, the
    # 64-bit product pos * inv_freq of the formula 2^31 * 2^-53 of a radian
    positions = np.array([2 ** 31 - 1, 2 ** 31 - 2, 10 ** 9 + 7, 123456789, 2 ** 30])
    run(B.Codebook(), 5, 4, 2, torch.float32, 128, False, True, positions, seed=4)
    run(B.Codebook(), 5, 4, 2, torch.float32, 128, True, False, positions, seed=5, base=3.0)


@pytest.mark.gpu
def test_zero_vectors_and_no_positions():
    book = B.Codebook()
    x = torch.zeros((3, 2, 128), dtype=torch.bfloat16, device="cuda")
    x[1, 1] = 3.0
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(x, 9.0)
    B.tq_norm_rope(book, x, None, B.TQ_BF16, 3, 2, 0, 256, 0, w, None, 1e-6, None, None, 0, False, out, None, 256, 0)
    torch.cuda.synchronize()
    expect = torch.zeros_like(x)
    expect[1, 1] = 1.0                             # 3 / sqrt(9 + 1e-6) rounds to 1
    assert torch.equal(out, expect)


@pytest.mark.gpu
def test_refusals():
    book = B.Codebook()
    x = torch.zeros((4, 3, 128), dtype=torch.bfloat16, device="cuda")
    y = torch.full_like(x, 5.0)
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    inv = torch.zeros(64, dtype=torch.float64, device="cuda")
    base = [x, x[:, 2:], B.TQ_BF16, 4, 2, 1, 384, 384, None, None, 1e-6, pos, inv, 128, 0, y, y[:, 2:], 384, 384]
    cases = [(0, x.data_ptr() + 2, 1), (2, 5, 1), (3, -1, 1), (4, 0, 1), (4, 4, 1), (5, -1, 1), (6, 255, 1),
             (6, 260, 1), (8, x.data_ptr() + 8, 1), (10, -1.0, 1), (10, float("nan"), 1), (10, float("inf"), 1),
             (11, None, 1), (12, None, 1), (12, inv.data_ptr() + 4, 1), (13, -2, 1), (13, 130, 1), (13, 63, 1),
             (13, 24, 2), (14, 2, 1), (15, None, 1), (16, y.data_ptr() + 4, 1), (17, 200, 1), (18, 385, 1),
             (15, x, 1)]
    for i, value, status in cases:
        args = list(base)
        args[i] = value
        if (i, status) == (15, 1) and value is x:
            args[17] = 512                         # in place with another stride
        with pytest.raises(B.TQError) as err:
            B.tq_norm_rope(book, *args)
        assert err.value.status == status, (i, value)
    with pytest.raises(B.TQError):
        B.tq_norm_rope(book, None, None, *base[2:])
    torch.cuda.synchronize()
    assert bool((y == 5.0).all())
    B.tq_norm_rope(book, None, None, B.TQ_BF16, 0, *base[4:])      # no tokens: nothing to do


@pytest.mark.gpu
def test_other_stream_and_graph():
    book = B.Codebook()
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn((9, 4, 128), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    inv = 10000.0 ** (-torch.arange(64, dtype=torch.float64, device="cuda") / 64)
    outs = [torch.zeros_like(x) for _ in range(3)]
    call = lambda out, stream=None: B.tq_norm_rope(book, x, None, B.TQ_BF16, 9, 4, 0, 512, 0, w, None, 1e-6, pos, inv,
                                                   128, False, out, None, 512, 0, stream)
    call(outs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(outs[1], side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(outs[2])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    pos += 5
    graph.replay()
    call(outs[0])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[2]) and not torch.equal(outs[0], outs[1])


@pytest.mark.gpu
def test_misaligned_positions_are_refused():
    x = torch.zeros((4, 3, 128), dtype=torch.bfloat16, device="cuda")
    y = torch.full_like(x, 5.0)
    pos = torch.zeros(5, dtype=torch.int32, device="cuda")
    inv = torch.zeros(64, dtype=torch.float64, device="cuda")
    with pytest.raises(B.TQError) as err:
        B.tq_norm_rope(B.Codebook(), x, None, B.TQ_BF16, 4, 3, 0, 384, 0, None, None, 1e-6, pos.data_ptr() + 2, inv, 128,
                       False, y, None, 384, 0)
    assert err.value.status == 1
    torch.cuda.synchronize()
    assert bool((y == 5.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_vectors_whose_squares_leave_the_range(dtype, eps):
    # sums of squares above 2^128 or below 2^-149: the norm itself is an ordinary number
    book = B.Codebook()
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    sizes = [2.0 ** 120, 2.0 ** 64, 2.0 ** 60, 1.0, 2.0 ** -40, 2.0 ** -60, 2.0 ** -80, 2.0 ** -120]
    x = torch.randn((len(sizes), 3, 128), generator=g, device="cuda")
    x = (x.clamp(-4, 4) * torch.tensor(sizes, device="cuda")[:, None, None]).to(dtype)
    w = (1 + 0.3 * torch.randn(128, generator=g, device="cuda")).to(dtype)
    out = torch.zeros_like(x)
    inv = 10000.0 ** (-torch.arange(64, dtype=torch.float64, device="cuda") / 64)
    pos = torch.arange(len(sizes), dtype=torch.int32, device="cuda") + 11
    B.tq_norm_rope(book, x, None, B.TQ_BF16 if dtype == torch.bfloat16 else B.TQ_FP32, len(sizes), 3, 0, 384, 0, w,
                   None, eps, pos, inv, 128, False, out, None, 384, 0)
    torch.cuda.synchronize()
    # (the kernel takes eps in 32 bits)
    expect, bound = reference(x.double().cpu().numpy(), w.double().cpu().numpy(), float(np.float32(eps)),
                              pos.cpu().numpy(), inv.cpu().numpy(), 128, False)
    rounding = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    err = np.abs(out.double().cpu().numpy() - expect)
    assert (err <= bound * (1 + rounding) + rounding * np.abs(expect) + 1e-37).all()
