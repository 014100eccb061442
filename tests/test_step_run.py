"""The operators of a serving step run together, as a serving loop uses them:
token map, head norms with rotation, quantize-append, attention of the new
tokens over the packed cache, for a prompt step, a mixed step and a decode
step, with a padded batch; checked against the plain formulas stage by stage
(each stage from the GPU's own inputs to it)."""
import numpy as np
import pytest
import torch

from online_kv_cache_tq_gb300 import binding as B
from online_kv_cache_tq_gb300 import cache as C

from parity_helpers import books, check_append, generator, host_cache
from test_extend import V, reference as attention_reference
from test_norm_rope import reference as rope_reference
from test_token_map import reference as map_reference

pytestmark = pytest.mark.gpu


def test_three_steps_of_a_serving_loop():
    bs, n_kv, group, num_blocks, max_blocks, batch = 32, 2, 4, 64, 12, 3
    n_q = n_kv * group
    book, ref = books(3, 3, 128, seed=1, block_size=bs)
    cache = C.allocate_cache(book, num_blocks, n_kv)
    view = C.cache_view(book, cache)
    g = generator(0)
    rng = np.random.default_rng(0)
    table = torch.full((batch, max_blocks), -1, dtype=torch.int32, device="cuda")
    free = rng.permutation(num_blocks).astype(np.int32)
    past = np.zeros(batch, np.int32)
    w = [(1 + 0.2 * torch.randn(128, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2)]
    inv = 10000.0 ** (-torch.arange(64, dtype=torch.float64, device="cuda") / 64)
    for new in ([70, 33, 0], [1, 40, 90], [1, 1, 1]):
        new = np.array(new, np.int32)
        rows = int(new.sum()) + 5                  # a padded batch
        dev = lambda x: torch.as_tensor(np.asarray(x, np.int32), device="cuda")
        past_t, new_t, free_t = dev(past), dev(new), dev(free)
        ctx_t, start_t, taken = dev(past * 0), dev([0] * (batch + 1)), dev([0])
        pos_t = torch.empty(rows, dtype=torch.int32, device="cuda")
        slots = torch.empty(rows, dtype=torch.int64, device="cuda")
        before = table.cpu().numpy().copy()
        qkv = torch.randn((rows, n_q + 2 * n_kv, 128), generator=g, device="cuda").to(torch.bfloat16)
        q_in, k_in = qkv[:, :n_q].clone(), qkv[:, n_q:n_q + n_kv].clone()
        q = torch.full((rows, n_q, 128), 3.0, dtype=torch.bfloat16, device="cuda")
        k = torch.full((rows, n_kv, 128), 3.0, dtype=torch.bfloat16, device="cuda")
        v = qkv[:, n_q + n_kv:].contiguous()
        out = torch.full((rows, n_q, 128), 5.0, dtype=torch.bfloat16, device="cuda")
        ws, nbytes = C.allocate_extend_workspace(book, rows, batch, n_q, n_kv, max_blocks * bs)
        stride = (n_q + 2 * n_kv) * 128
        B.tq_map_tokens(book, batch, past_t, new_t, table, max_blocks, num_blocks, free_t, len(free), rows, ctx_t,
                        start_t, pos_t, slots, taken)
        B.tq_norm_rope(book, qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], B.TQ_BF16, rows, n_q, n_kv, stride, stride, w[0],
                       w[1], 1e-6, pos_t, inv, 128, False, q, k, n_q * 128, n_kv * 128)
        B.tq_quantize_append(book, k, v, B.TQ_BF16, rows, n_kv, slots, view)
        B.tq_extend_attention(book, q, B.TQ_BF16, rows, batch, n_q, n_kv, view, table, max_blocks, start_t, ctx_t,
                              max_blocks * bs, 0.0, out, ws, nbytes)
        torch.cuda.synchronize()
        assert B.tq_get_last_device_error(book) == 0

        expect_table = before
        ctx, start, positions, slot_ref, used = map_reference(past, new, expect_table, free, rows, bs, num_blocks)
        assert np.array_equal(table.cpu().numpy(), expect_table)
        assert np.array_equal(slots.cpu().numpy(), slot_ref) and np.array_equal(pos_t.cpu().numpy(), positions)
        live = positions >= 0
        for x, y, wt in ((q_in, q, w[0]), (k_in, k, w[1])):
            val, bound = rope_reference(x.double().cpu().numpy(), wt.double().cpu().numpy(), 1e-6, positions,
                                        inv.cpu().numpy(), 128, False)
            err = np.abs(y.double().cpu().numpy() - val)
            assert (err <= bound * 1.01 + 2.0 ** -8 * np.abs(val))[live].all()
            assert bool((y[torch.as_tensor(~live)] == 3.0).all())
        check_append(book, ref, cache, k, v, slot_ref)
        hc, qn, got = host_cache(cache), q.double().cpu().numpy(), out.double().cpu().numpy()
        for b in range(batch):
            if new[b] == 0:
                continue
            for h in range(n_kv):
                hs = slice(h * group, (h + 1) * group)
                val, bound = attention_reference(qn[start[b]:start[b + 1], hs], hc, expect_table[b], int(ctx[b]),
                                                 int(new[b]), h, ref, 1.0 / np.sqrt(128.0))
                err = np.abs(got[start[b]:start[b + 1], hs] - val)
                assert (err <= bound).all()
                assert np.sqrt((err ** 2).sum() / (val ** 2).sum()) <= 2 * V
        assert (got[start[-1]:] == 5.0).all()
        past, free = ctx, free[used:]
