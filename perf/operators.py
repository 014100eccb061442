"""Timed cases of the operators around the packed cache: the token map
(``tq_map_tokens``), head norms with the position rotation (``tq_norm_rope``)
and attention of several new tokens per sequence over the packed cache
(``tq_extend_attention``).

``run`` makes the library's calls where ``own`` is true; otherwise it computes
the same operators with elementary torch operations in 32 bits, without the
library.  ``exact`` gives the operators' values in 64 bits.
"""
import functools
import math
import random

import numpy as np
import torch

own = False

D = 128
DEVICE = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---- the method's constants, from their definitions ---------------------------

@functools.lru_cache(maxsize=None)
def _matrices(m):
    """(R, S) of seed 0: R the Q factor (positive diagonal) of a Gaussian
    matrix, S Gaussian, both from one SplitMix64 stream by Box-Muller."""
    count = D * D + m * D
    with np.errstate(over="ignore"):
        z = (np.arange(1, 2 * ((count + 1) // 2) + 1, dtype=np.uint64)) * np.uint64(0x9E3779B97F4A7C15)
        z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
        z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
        z = z ^ (z >> np.uint64(31))
    u = ((z >> np.uint64(11)).astype(np.float64) + 1.0) * 2.0 ** -53
    radius, angle = np.sqrt(-2.0 * np.log(u[0::2])), 2.0 * math.pi * u[1::2]
    normals = np.stack([radius * np.cos(angle), radius * np.sin(angle)], axis=1).reshape(-1)[:count]
    q, t = np.linalg.qr(normals[:D * D].reshape(D, D))
    return q * np.sign(np.diag(t))[None, :], normals[D * D:].reshape(m, D)


@functools.lru_cache(maxsize=None)
def _codebook(bits):
    """(levels, bounds) of the Lloyd-Max quantizer of one coordinate of a
    random unit vector, density proportional to (1 - x^2)^((d - 3) / 2)."""
    nodes, weights = np.polynomial.legendre.leggauss(96)
    count = 1 << bits
    levels = np.linspace(-2.0, 2.0, count + 2)[1:-1] / math.sqrt(D)
    for _ in range(20000):
        edges = np.concatenate(([-0.9], 0.5 * (levels[:-1] + levels[1:]), [0.9]))
        half, mid = 0.5 * np.diff(edges)[:, None], 0.5 * (edges[:-1] + edges[1:])[:, None]
        x = mid + half * nodes
        f = (1.0 - x * x) ** ((D - 3) / 2.0) * weights
        new = (x * f).sum(1) / f.sum(1)
        moved = np.max(np.abs(new - levels))
        levels = new
        if moved < 1e-15:
            break
    levels = 0.5 * (levels - levels[::-1])
    return levels, 0.5 * (levels[:-1] + levels[1:])


@functools.lru_cache(maxsize=None)
def _book(k_bits, v_bits, qjl, norm_bits, block):
    from online_kv_cache_tq_gb300 import binding
    return binding.Codebook(k_bits=k_bits, v_bits=v_bits, qjl_m=D if qjl else 0, seed=0, block_size=block, device=0,
                            norm_bits=norm_bits)


# ---- cases --------------------------------------------------------------------

def listed():
    return [
        # one decode step of 64 sequences: every sequence gets one token, some a new block
        dict(name="map_decode_b64", op="map", batch=64, new_lo=1, new_hi=1, past_lo=1024, past_hi=32768, block=64,
             pad=0, lens=1),
        # a mixed step: 250 sequences, decode tokens beside prompt chunks of up to 1500 tokens, padded rows behind
        dict(name="map_mixed_b250", op="map", batch=250, new_lo=1, new_hi=1500, past_lo=0, past_hi=6000, block=64,
             pad=37, lens=2),
        # the same for 500 sequences with prompts from nothing and small blocks
        dict(name="map_prompts_b500", op="map", batch=500, new_lo=1, new_hi=4000, past_lo=0, past_hi=0, block=32,
             pad=0, lens=3),
        # a decode step's queries and keys: 16 tokens, latency
        dict(name="rope_decode_16", op="rope", tokens=16, n_q=32, n_kv=8, dtype="bf16", rot=128, interleaved=False,
             norm=True, far=32768),
        # a prompt of 32768 tokens with the 70B-shaped heads
        dict(name="rope_prefill_32768", op="rope", tokens=32768, n_q=64, n_kv=8, dtype="bf16", rot=128,
             interleaved=False, norm=True, far=32768),
        # an odd number of tokens, fp32, half of the dimensions rotated, neighbouring pairs, far positions
        dict(name="rope_fp32_5001", op="rope", tokens=5001, n_q=32, n_kv=8, dtype="fp32", rot=64, interleaved=True,
             norm=True, far=131072),
        # the rotation alone (models without head norms), ordinary batch
        dict(name="rope_only_4096", op="rope", tokens=4096, n_q=32, n_kv=8, dtype="bf16", rot=128, interleaved=False,
             norm=False, far=131072),
        # verification of four drafted tokens for one short sequence: the smallest call
        dict(name="extend_verify_small", op="extend", batch=1, n_q=8, n_kv=1, new_lo=4, new_hi=4, past_lo=509,
             past_hi=509, k_bits=3, v_bits=3, qjl=True, norm_bits=32, block=64, dtype="bf16", lens=4),
        # verification of four drafted tokens, the 8B-shaped decode batch
        dict(name="extend_verify_8b", op="extend", batch=16, n_q=32, n_kv=8, new_lo=4, new_hi=4, past_lo=8188,
             past_hi=8188, k_bits=3, v_bits=3, qjl=True, norm_bits=32, block=64, dtype="bf16", lens=5),
        # ragged step of the 70B-shaped batch: 1 to 16 new tokens on contexts of 1 K to 32 K, fp16 norms
        dict(name="extend_ragged_70b", op="extend", batch=24, n_q=64, n_kv=8, new_lo=1, new_hi=16, past_lo=1024,
             past_hi=32768, k_bits=3, v_bits=3, qjl=True, norm_bits=16, block=64, dtype="bf16", lens=6),
        # eight ragged prompts with nothing cached before them, keys without the sketch
        dict(name="extend_prompts_8", op="extend", batch=8, n_q=32, n_kv=8, new_lo=37, new_hi=4096, past_lo=0,
             past_hi=0, k_bits=4, v_bits=4, qjl=False, norm_bits=32, block=128, dtype="bf16", lens=7),
        # a prompt chunk of 2048 tokens on a cached prefix, 4-bit keys and 2-bit values
        dict(name="extend_chunk_2048", op="extend", batch=1, n_q=64, n_kv=8, new_lo=2048, new_hi=2048, past_lo=14001,
             past_hi=14001, k_bits=4, v_bits=2, qjl=True, norm_bits=32, block=64, dtype="bf16", lens=8),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["map", "rope", "extend", "extend"])
    lens = rng.randrange(1 << 30)
    if op == "map":
        batch = _spread(rng, 1, 512)
        past = rng.choice([0, 1000, 32768])
        return dict(op=op, batch=batch, new_lo=1, new_hi=_spread(rng, 1, 2000), past_lo=0, past_hi=past,
                    block=rng.choice([32, 64, 96, 128, 256]), pad=rng.choice([0, 1, 100]), lens=lens)
    if op == "rope":
        n_kv = rng.choice([1, 2, 4, 8])
        return dict(op=op, tokens=_spread(rng, 1, 30000), n_q=n_kv * rng.choice([1, 2, 4, 8]), n_kv=n_kv,
                    dtype=rng.choice(["bf16", "bf16", "fp32"]), rot=rng.choice([32, 64, 96, 128]),
                    interleaved=rng.random() < 0.3, norm=rng.random() < 0.7, far=rng.choice([4096, 131072, 1000000]))
    n_kv = rng.choice([1, 2, 4, 8])
    n_q = n_kv * rng.choice([1, 2, 3, 4, 8])
    new = _spread(rng, 1, 2048)
    past = rng.choice([0, _spread(rng, 1, 16000)])
    # rows x context of the largest listed case bounds the batch
    cost = n_q * new * (past + new)
    batch = _spread(rng, 1, max(1, min(48, int(2.0e9 // cost))))
    qjl = rng.random() < 0.7
    return dict(op=op, batch=batch, n_q=n_q, n_kv=n_kv, new_lo=max(1, new // 3), new_hi=new, past_lo=past // 2,
                past_hi=past, k_bits=rng.choice([2, 3, 4, 5]) if qjl else rng.choice([1, 2, 3, 4]),
                v_bits=rng.choice([1, 2, 3, 4]), qjl=qjl, norm_bits=rng.choice([16, 32]),
                block=rng.choice([32, 64, 96, 128]), dtype=rng.choice(["bf16", "bf16", "fp32"]), lens=lens)


def _lengths(case):
    """(past, new) per sequence: functions of the case alone."""
    rng = random.Random(case["lens"])
    past = [rng.randint(case["past_lo"], case["past_hi"]) for _ in range(case["batch"])]
    if case["new_hi"] <= 16 or case["op"] == "extend":
        new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    else:   # a mixed step: three in four sequences decode one token
        new = [1 if past_b and rng.random() < 0.75 else _spread(rng, case["new_lo"], case["new_hi"])
               for past_b in past]
    return past, new


def _ceil(a, b):
    return (a + b - 1) // b


def work(case):
    if case["op"] == "map":
        past, new = _lengths(case)
        bs = case["block"]
        taken = sum(_ceil(p + n, bs) - _ceil(p, bs) for p, n in zip(past, new))
        return {"bytes": 16 * case["batch"] + 8 * taken + 12 * (sum(new) + case["pad"]), "flops": 0}
    if case["op"] == "rope":
        vecs = case["tokens"] * (case["n_q"] + case["n_kv"])
        elem = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * vecs * D * elem + 4 * case["tokens"], "flops": 8 * vecs * D}
    past, new = _lengths(case)
    nb = case["norm_bits"] // 8
    item = case["k_bits"] * D // 8 + case["v_bits"] * D // 8 + (3 if case["qjl"] else 2) * nb
    ctx = sum(past) + sum(new)
    elem = 2 if case["dtype"] == "bf16" else 4
    pairs = sum(n * p + n * (n + 1) // 2 for p, n in zip(past, new)) * case["n_q"]
    return {"bytes": ctx * case["n_kv"] * item + sum(new) * case["n_q"] * D * (elem + 2), "flops": 4 * D * pairs}


# ---- inputs -------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEVICE)


def _prepare_map(case, seed):
    past, new = _lengths(case)
    rng = np.random.default_rng(seed)
    past = [int(x) for x in rng.permutation(past)] if len(set(new)) == 1 else past
    bs = case["block"]
    before = [_ceil(p, bs) for p in past]
    after = [_ceil(p + n, bs) for p, n in zip(past, new)]
    num_blocks = sum(after) + 64
    ids = rng.permutation(num_blocks).astype(np.int32)
    max_blocks = max(after)
    table = np.full((case["batch"], max_blocks), -1, dtype=np.int32)
    pos = 0
    for b, n in enumerate(before):
        table[b, :n] = ids[pos:pos + n]
        pos += n
    tokens = sum(new) + case["pad"]
    s = dict(case=case, batch=case["batch"], past=_ints(past), new=_ints(new), table=torch.as_tensor(table).cuda(),
             free=torch.as_tensor(ids[pos:].copy()).cuda(), num_blocks=num_blocks, max_blocks=max_blocks,
             tokens=tokens, block=bs)
    if own:
        s["book"] = _book(3, 3, True, 32, bs)
        s["out"] = dict(context=torch.empty_like(s["past"]), start=_ints([0] * (case["batch"] + 1)),
                        positions=torch.empty(tokens, dtype=torch.int32, device=DEVICE),
                        slots=torch.empty(tokens, dtype=torch.int64, device=DEVICE), taken=_ints([0]))
    return s


def _prepare_rope(case, seed):
    g = _generator(seed)
    dt = DTYPES[case["dtype"]]
    n, nq, nkv = case["tokens"], case["n_q"], case["n_kv"]
    # the slices of one projection's output: queries, keys and values of a token side by side
    qkv = torch.randn((n, nq + 2 * nkv, D), generator=g, device=DEVICE)
    qkv *= torch.exp(torch.randn((1, nq + 2 * nkv, D), generator=g, device=DEVICE) * 0.7)
    start = int(torch.randint(0, max(1, case["far"] - n), (1,), generator=g, device=DEVICE))
    half = case["rot"] // 2
    s = dict(case=case, qkv=qkv.to(dt), n=n, nq=nq, nkv=nkv, rot=case["rot"], interleaved=case["interleaved"],
             positions=torch.arange(start, start + n, dtype=torch.int32, device=DEVICE),
             inv_freq=500000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEVICE) / half), eps=1e-6,
             q_weight=None, k_weight=None)
    if case["norm"]:
        s["q_weight"] = (1.0 + 0.2 * torch.randn(D, generator=g, device=DEVICE)).to(dt)
        s["k_weight"] = (1.0 + 0.2 * torch.randn(D, generator=g, device=DEVICE)).to(dt)
    if own:
        s["book"] = _book(3, 3, True, 32, 64)
        s["q_out"] = torch.empty((n, nq, D), dtype=dt, device=DEVICE)
        s["k_out"] = torch.empty((n, nkv, D), dtype=dt, device=DEVICE)
    return s


def _pack(bits):
    """0/1 int32 [..., 8 n] -> uint8 [..., n], lowest bit first."""
    w = torch.tensor([1, 2, 4, 8, 16, 32, 64, 128], dtype=torch.int32, device=bits.device)
    return (bits.reshape(*bits.shape[:-1], -1, 8) * w).sum(-1).to(torch.uint8)


def _fill_cache(case, num_blocks, g):
    """The packed fields of ``num_blocks`` blocks of Gaussian keys and values
    with per-channel scales, as the append writes them."""
    bs, nkv = case["block"], case["n_kv"]
    kb = case["k_bits"] - 1 if case["qjl"] else case["k_bits"]
    vb = case["v_bits"]
    R, S = _matrices(D if case["qjl"] else 0)
    Rt = torch.as_tensor(R.T.copy(), dtype=torch.float32, device=DEVICE)
    Spt = torch.as_tensor((S @ R.T).T.copy(), dtype=torch.float32, device=DEVICE)
    (kl, kbd), (vl, vbd) = [[torch.as_tensor(t, dtype=torch.float32, device=DEVICE) for t in _codebook(b)]
                            for b in (kb, vb)]
    nd = torch.float16 if case["norm_bits"] == 16 else torch.float32
    scales = torch.exp(torch.randn((2, nkv, 1, D), generator=g, device=DEVICE) * 0.6)
    c = dict(k_codes=[], k_norm=[], v_codes=[], v_norm=[])
    if case["qjl"]:
        c.update(k_qjl=[], k_rnorm=[])
    step = max(1, (1 << 19) // (bs * nkv))
    for b0 in range(0, num_blocks, step):
        nb = min(step, num_blocks - b0)
        for which in (0, 1):
            x = torch.randn((nb, nkv, bs, D), generator=g, device=DEVICE) * scales[which]
            norm = x.norm(dim=-1, keepdim=True).to(nd)
            y = x @ Rt
            codes = torch.bucketize(y / x.norm(dim=-1, keepdim=True), (kbd, vbd)[which]).to(torch.int32)
            if which == 0:
                planes = [_pack((codes >> p) & 1) for p in range(kb)]
                c["k_codes"].append(torch.cat(planes, dim=-1))
                c["k_norm"].append(norm.squeeze(-1))
                if case["qjl"]:
                    res = y - norm.float() * kl[codes]
                    c["k_rnorm"].append(res.norm(dim=-1).to(nd))
                    c["k_qjl"].append(_pack((res @ Spt > 0).to(torch.int32)))
            else:
                t = codes.transpose(-1, -2)
                c["v_codes"].append(torch.stack([_pack((t >> p) & 1) for p in range(vb)], dim=2))
                c["v_norm"].append(norm.squeeze(-1))
    return {k: torch.cat(v).contiguous() for k, v in c.items()}


def _prepare_extend(case, seed):
    past, new = _lengths(case)
    g = _generator(seed)
    bs = case["block"]
    ctx = [p + n for p, n in zip(past, new)]
    need = [_ceil(c, bs) for c in ctx]
    num_blocks = sum(need)
    ids = np.random.default_rng(seed).permutation(num_blocks).astype(np.int32)
    table = np.full((case["batch"], max(need)), -1, dtype=np.int32)
    pos = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[pos:pos + n]
        pos += n
    total = sum(new)
    s = dict(case=case, cache=_fill_cache(case, num_blocks, g), table=torch.as_tensor(table).cuda(), ctx=ctx, new=new,
             q=torch.randn((total, case["n_q"], D), generator=g, device=DEVICE).to(DTYPES[case["dtype"]]),
             num_blocks=num_blocks)
    if own:
        from online_kv_cache_tq_gb300 import binding
        book = s["book"] = _book(case["k_bits"], case["v_bits"], case["qjl"], case["norm_bits"], bs)
        s["view"] = binding.make_cache_view(s["cache"], num_blocks, case["n_kv"], bs)
        s["start_t"] = _ints([sum(new[:b]) for b in range(case["batch"] + 1)])
        s["ctx_t"] = _ints(ctx)
        nbytes = binding.tq_extend_workspace_bytes(book, total, case["batch"], case["n_q"], case["n_kv"], max(ctx))
        s["ws"] = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=DEVICE)
        s["ws_bytes"] = nbytes
        s["out"] = torch.empty((total, case["n_q"], D), dtype=torch.bfloat16, device=DEVICE)
    return s


def prepare(case, seed):
    return {"map": _prepare_map, "rope": _prepare_rope, "extend": _prepare_extend}[case["op"]](case, seed)


# ---- one pass -----------------------------------------------------------------

def _own_map(s):
    from online_kv_cache_tq_gb300 import binding as B
    o = s["out"]
    B.tq_map_tokens(s["book"], s["batch"], s["past"], s["new"], s["table"], s["max_blocks"], s["num_blocks"],
                    s["free"], s["free"].numel(), s["tokens"], o["context"], o["start"], o["positions"], o["slots"],
                    o["taken"])
    return dict(o, table=s["table"])


def _plain_map(s):
    bs, batch, tokens = s["block"], s["batch"], s["tokens"]
    past, new = s["past"].long(), s["new"].long()
    ctx = past + new
    before, after = (past + bs - 1) // bs, (ctx + bs - 1) // bs
    zero = torch.zeros(1, dtype=torch.int64, device=DEVICE)
    start = torch.cat([zero, torch.cumsum(new, 0)])
    first = torch.cumsum(after - before, 0) - (after - before)
    cols = torch.arange(s["max_blocks"], device=DEVICE)[None, :]
    fresh = (cols >= before[:, None]) & (cols < after[:, None])
    pick = (first[:, None] + cols - before[:, None]).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][pick], s["table"])
    t = torch.arange(tokens, device=DEVICE)
    seq = torch.searchsorted(start, t, right=True) - 1
    live = seq < batch
    seq = seq.clamp(max=batch - 1)
    pos = past[seq] + t - start[seq]
    col = (pos // bs).clamp(max=s["max_blocks"] - 1)
    slots = torch.where(live, table[seq, col].long() * bs + pos % bs, -1)
    pos = torch.where(live, pos, -1)
    return dict(context=ctx.int(), start=start.int(), positions=pos.int(), slots=slots,
                taken=(after - before).sum().int().reshape(1), table=table)


def _own_rope(s):
    from online_kv_cache_tq_gb300 import binding as B
    nq, nkv, row = s["nq"], s["nkv"], (s["nq"] + 2 * s["nkv"]) * D
    dt = B.TQ_BF16 if s["qkv"].dtype == torch.bfloat16 else B.TQ_FP32
    B.tq_norm_rope(s["book"], s["qkv"][:, :nq], s["qkv"][:, nq:nq + nkv], dt, s["n"], nq, nkv, row, row,
                   s["q_weight"], s["k_weight"], s["eps"], s["positions"], s["inv_freq"], s["rot"],
                   s["interleaved"], s["q_out"], s["k_out"], nq * D, nkv * D)
    return s["q_out"], s["k_out"]


def _plain_rope(s):
    angle = s["positions"].double()[:, None] * s["inv_freq"][None, :]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    outs = []
    for x, w in ((s["qkv"][:, :s["nq"]], s["q_weight"]), (s["qkv"][:, s["nq"]:s["nq"] + s["nkv"]], s["k_weight"])):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + s["eps"]) * w.float()
        rot, half = s["rot"], s["rot"] // 2
        if s["interleaved"]:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
        else:
            a, b = y[..., :half], y[..., half:rot]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
        outs.append(torch.cat([turned, y[..., rot:]], dim=-1).to(x.dtype))
    return tuple(outs)


def _own_extend(s):
    from online_kv_cache_tq_gb300 import binding as B
    c = s["case"]
    dt = B.TQ_BF16 if s["q"].dtype == torch.bfloat16 else B.TQ_FP32
    B.tq_extend_attention(s["book"], s["q"], dt, s["q"].shape[0], c["batch"], c["n_q"], c["n_kv"], s["view"],
                          s["table"], s["table"].shape[1], s["start_t"], s["ctx_t"], max(s["ctx"]), 0.0, s["out"],
                          s["ws"], s["ws_bytes"])
    return s["out"]


def _unpack(packed):
    """uint8 [..., n] -> 0/1 int32 [..., 8 n], lowest bit first."""
    shifts = torch.arange(8, dtype=torch.int32, device=packed.device)
    return ((packed.to(torch.int32)[..., None] >> shifts) & 1).flatten(-2)


def _plain_sequence(s, b, R, S, levels):
    """(keys, values) [n_kv][ctx][128] of sequence b, back in the original space."""
    case, length = s["case"], s["ctx"][b]
    nkv, blocks = case["n_kv"], s["table"][b, :_ceil(s["ctx"][b], case["block"])].long()
    # [blocks][n_kv][block][..] -> [n_kv][tokens][..]
    rows = lambda f: s["cache"][f][blocks].transpose(0, 1).flatten(1, 2)[:, :length]
    bits = _unpack(rows("k_codes")).reshape(nkv, length, -1, D)
    codes = sum(bits[:, :, p] << p for p in range(bits.shape[2]))
    keys = rows("k_norm").float()[..., None] * (levels[0][codes] @ R)
    if case["qjl"]:
        signs = (2 * _unpack(rows("k_qjl")) - 1).float()
        keys += (rows("k_rnorm").float() * (math.sqrt(math.pi / 2.0) / D))[..., None] * (signs @ S)
    bits = _unpack(s["cache"]["v_codes"][blocks])                       # [blocks][n_kv][plane][128][block]
    codes = sum(bits[:, :, p] << p for p in range(bits.shape[2])).permute(1, 0, 3, 2).flatten(1, 2)[:, :length]
    values = rows("v_norm").float()[..., None] * (levels[1][codes] @ R)
    return keys, values


def _plain_extend(s):
    case = s["case"]
    R, S = [torch.as_tensor(t, dtype=torch.float32, device=DEVICE) for t in _matrices(D if case["qjl"] else 0)]
    levels = [torch.as_tensor(_codebook(b)[0], dtype=torch.float32, device=DEVICE)
              for b in (case["k_bits"] - 1 if case["qjl"] else case["k_bits"], case["v_bits"])]
    out = torch.empty(s["q"].shape, dtype=torch.bfloat16, device=DEVICE)
    group, t0 = case["n_q"] // case["n_kv"], 0
    for b, (n, length) in enumerate(zip(s["new"], s["ctx"])):
        keys, values = _plain_sequence(s, b, R, S, levels)
        # rows of a KV head: its query heads' tokens
        q = s["q"][t0:t0 + n].float().reshape(n, case["n_kv"], group, D).permute(1, 2, 0, 3).flatten(1, 2)
        scores = (q @ keys.transpose(1, 2)) * (1.0 / math.sqrt(D))
        seen = torch.arange(length - n, length, device=DEVICE).repeat(group)
        scores.masked_fill_(torch.arange(length, device=DEVICE)[None, :] > seen[:, None], float("-inf"))
        scores -= scores.amax(-1, keepdim=True)
        scores.exp_()
        o = (scores @ values) / scores.sum(-1, keepdim=True)
        out[t0:t0 + n] = o.reshape(case["n_kv"], group, n, D).permute(2, 0, 1, 3).flatten(1, 2).to(torch.bfloat16)
        t0 += n
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"map": _own_map, "rope": _own_rope, "extend": _own_extend}[op](state)
    return {"map": _plain_map, "rope": _plain_rope, "extend": _plain_extend}[op](state)


# ---- 64-bit values ------------------------------------------------------------

def _exact_map(case, seed):
    s = _prepare_map(case, seed)
    past, new, free = s["past"].tolist(), s["new"].tolist(), s["free"].tolist()
    bs, table = s["block"], s["table"].tolist()
    start, slots, positions, taken = [0], [], [], 0
    for b in range(case["batch"]):
        for col in range(_ceil(past[b], bs), _ceil(past[b] + new[b], bs)):
            table[b][col] = free[taken]
            taken += 1
        for pos in range(past[b], past[b] + new[b]):
            positions.append(pos)
            slots.append(table[b][pos // bs] * bs + pos % bs)
        start.append(start[-1] + new[b])
    positions += [-1] * case["pad"]
    slots += [-1] * case["pad"]
    return dict(context=_ints([p + n for p, n in zip(past, new)]), start=_ints(start), positions=_ints(positions),
                slots=_ints(slots, torch.int64), taken=_ints([taken]), table=_ints(table))


def _exact_rope(case, seed):
    s = _prepare_rope(case, seed)
    heads = s["nq"] + s["nkv"]
    x = s["qkv"][:, :heads].double()
    if case["norm"]:
        w = torch.cat([s["q_weight"].double().expand(s["nq"], D), s["k_weight"].double().expand(s["nkv"], D)])
        x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / D + s["eps"]) * w
    # a pair as a complex number, turned by exp(i angle)
    angle = torch.outer(s["positions"].double(), s["inv_freq"])
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    rot = case["rot"]
    index = torch.arange(rot, device=DEVICE).reshape(-1, 2) if case["interleaved"] else \
        torch.arange(rot, device=DEVICE).reshape(2, -1).T
    z = torch.view_as_real(torch.complex(x[..., index[:, 0]], x[..., index[:, 1]]) * turn)
    x[..., index[:, 0]], x[..., index[:, 1]] = z[..., 0], z[..., 1]
    return x[:, :s["nq"]], x[:, s["nq"]:]


def _exact_extend(case, seed):
    s = _prepare_extend(case, seed)
    cache, bs, nkv = s["cache"], case["block"], case["n_kv"]
    group = case["n_q"] // nkv
    R, S = [torch.as_tensor(t, dtype=torch.float64, device=DEVICE) for t in _matrices(D if case["qjl"] else 0)]
    kb = case["k_bits"] - 1 if case["qjl"] else case["k_bits"]
    kl, vl = [torch.as_tensor(_codebook(b)[0], dtype=torch.float64, device=DEVICE) for b in (kb, case["v_bits"])]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
    byte = torch.arange(D, device=DEVICE)
    t0 = 0
    for b in range(case["batch"]):
        n, length = s["new"][b], s["ctx"][b]
        pos = torch.arange(length, device=DEVICE)
        blk, off = s["table"][b].long()[pos // bs], pos % bs
        hidden = pos[None, :] > (length - n + torch.arange(n, device=DEVICE))[:, None]
        for h in range(nkv):
            # rotated space: scores from <R q, levels> and <S q, signs>, one back-rotation of the sum
            code = torch.zeros((length, D), dtype=torch.int64, device=DEVICE)
            for p in range(kb):
                code += ((cache["k_codes"][blk, h, off][:, p * 16 + byte // 8].long() >> (byte % 8)) & 1) << p
            q = s["q"][t0:t0 + n, h * group:(h + 1) * group].double().reshape(n * group, D)
            score = (q @ R.T @ kl[code].T) * cache["k_norm"][blk, h, off].double()
            if case["qjl"]:
                sign = ((cache["k_qjl"][blk, h, off][:, byte // 8].long() >> (byte % 8)) & 1).double() * 2 - 1
                gamma = cache["k_rnorm"][blk, h, off].double() * math.sqrt(math.pi / 2) / D
                score += (q @ S.T @ sign.T) * gamma
            score = (score / math.sqrt(D)).reshape(n, group, length)
            score.masked_fill_(hidden[:, None, :], -math.inf)
            weight = torch.softmax(score, dim=-1).reshape(n * group, length)
            code = torch.zeros((length, D), dtype=torch.int64, device=DEVICE)
            for p in range(case["v_bits"]):
                field = cache["v_codes"][blk, h, p, :, off // 8].long()
                code += ((field >> (off % 8)[:, None]) & 1) << p
            value = vl[code] * cache["v_norm"][blk, h, off].double()[:, None]
            out[t0:t0 + n, h * group:(h + 1) * group] = (weight @ value @ R).reshape(n, group, D)
        t0 += n
    return out


def exact(case, seed):
    return {"map": _exact_map, "rope": _exact_rope, "extend": _exact_extend}[case["op"]](case, seed)
