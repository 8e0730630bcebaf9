"""examples/hybrid_decode.py in bf16: each append and attention of its steps, on the pages that reserving, forking,
releasing and compacting have left, against the definition in 64 bits."""
import pytest
import torch

import gated_deltanet_linear_spec_gb300 as gdn
from tests import kv_reference as ref
from tests.test_gpu_example import example

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", [0, 1])
def test_every_attention_of_a_bf16_run(seed, monkeypatch):
    append, attend = gdn.gdn_kv_append, gdn.gdn_paged_attention
    longest = []

    def rows_of(rows):
        first, lens = rows.query_start_loc.tolist(), rows.kv_lens.tolist()
        return [(a, b - a) for a, b in zip(first, first[1:])], rows.table_rows.tolist(), rows.token_indx.tolist(), lens

    def checked_append(cache, rows, k, v, **kw):
        append(cache, rows, k, v, **kw)
        spans, table_rows, token, lens = rows_of(rows)
        table, size = cache.block_table.tolist(), cache.k_pool.shape[2]
        for (bos, new), r, kv in zip(spans, table_rows, lens):
            for t in range(new):
                pos = kv - new + t
                page, slot = table[r][pos // size], pos % size
                assert page > 0
                assert torch.equal(cache.k_pool[page, :, slot], k[token[bos + t]])
                assert torch.equal(cache.v_pool[page, :, slot], v[token[bos + t]])

    def checked_attention(attn, cache, rows, q, out, **kw):
        attend(attn, cache, rows, q, out, **kw)
        spans, table_rows, token, lens = rows_of(rows)
        want, spread, logits = ref.attention(q.cpu(), cache.k_pool.cpu(), cache.v_pool.cpu(), cache.block_table.cpu(), spans,
                                             table_rows, token, lens, attn.scale, attn.window, attn.num_sinks)
        longest.append(max(n for _, n in spans) * 2)  # queries of a kv-head
        bits = 8 if longest[-1] > 64 else 16
        tol = ref.attention_tolerance(want, spread, logits, max(lens), q.shape[-1], q.dtype, bits)
        err = (out.cpu().double() - want).abs()
        assert torch.all(err[token] <= tol[token])

    monkeypatch.setattr(gdn, "gdn_kv_append", checked_append)
    monkeypatch.setattr(gdn, "gdn_paged_attention", checked_attention)
    sequences, per_step, _ = example().run(torch.bfloat16, seed=seed)
    assert len(sequences) == 5 and per_step >= 1
    assert min(longest) <= 16 and max(longest) > 64  # both kernels of the tensor cores
