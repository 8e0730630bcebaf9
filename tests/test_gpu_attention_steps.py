"""Steps of append and attention one after the other on a stream, over positions that are written again and again,
as after rejected drafts: what a step reads is what the step before its attention wrote."""
import pytest
import torch

import gated_deltanet_linear_spec_gb300 as gdn
from tests.test_gpu_attention import BF16, F32, Step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [[(1, 900), (1, 65)] * 8, [(4, 300), (3, 77), (4, 1030)], [(200, 300), (70, 70)]],
                         ids=["decode", "verify", "prompt"])
@pytest.mark.parametrize("dim,dtype", [(64, BF16), (128, BF16), (256, BF16), (96, BF16), (64, F32)])
def test_positions_written_again(rows, dim, dtype):
    s = Step(rows, heads=8, kv_heads=2, dim=dim, dtype=dtype, seed=dim)
    gen = torch.Generator(device="cuda").manual_seed(dim)
    steps = 12
    k, v = (torch.randn(steps, s.q.shape[0], 2, dim, generator=gen, device="cuda").to(dtype) for _ in range(2))
    out = torch.zeros(steps, *s.qd.shape, dtype=dtype, device="cuda")
    again = torch.zeros_like(out)
    ws = torch.empty(max(gdn.gdn_attention_workspace_bytes(s.attn, s.cache, s.kv_rows), 1), dtype=torch.uint8, device="cuda")
    for i in range(steps):
        gdn.gdn_kv_append(s.cache, s.kv_rows, k[i], v[i])
        gdn.gdn_paged_attention(s.attn, s.cache, s.kv_rows, s.qd, out[i], workspace=ws)
    for i in range(steps):
        torch.cuda.synchronize()
        gdn.gdn_kv_append(s.cache, s.kv_rows, k[i], v[i])
        torch.cuda.synchronize()
        gdn.gdn_paged_attention(s.attn, s.cache, s.kv_rows, s.qd, again[i], workspace=ws)
    assert torch.equal(out, again)
    assert not torch.equal(out[0], out[1])


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_pages_handed_out_again(dtype):
    """Rows give back their pages and get others: each attention follows the table as the call before it left it."""
    rows, page, dim, pages = 6, 16, 64, 60
    gen = torch.Generator(device="cuda").manual_seed(1)
    pool = torch.zeros(pages, 2, 2, page, dim, dtype=dtype, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = gdn.KvCache(pool[:, 0], pool[:, 1], i32([[0] * 8] * rows), i32([0] * pages))
    new = 40
    order = [i32(torch.randperm(rows, generator=torch.Generator().manual_seed(s)).tolist()) for s in range(10)]
    k, v, q = (torch.randn(10, rows * new, h, dim, generator=gen, device="cuda").to(dtype) for h in (2, 2, 4))
    starts, lens, zeros = i32([new * i for i in range(rows + 1)]), i32([new] * rows), i32([0] * rows)
    outs = []
    for wait in (False, True):
        cache.block_table.zero_()
        cache.refcount.zero_()
        out = torch.zeros(10, rows * new, 4, dim, dtype=dtype, device="cuda")
        for s in range(10):
            kv_rows = gdn.KvRows(starts, rows * new, lens, new, order[s])
            calls = [lambda: gdn.gdn_kv_release(cache, order[s]), lambda: gdn.gdn_kv_reserve(cache, order[s], zeros, lens),
                     lambda: gdn.gdn_kv_append(cache, kv_rows, k[s], v[s]),
                     lambda: gdn.gdn_paged_attention(gdn.Attention(4), cache, kv_rows, q[s], out[s])]
            for call in calls:
                call()
                if wait:
                    torch.cuda.synchronize()
        outs.append(out)
    assert torch.equal(*outs)


def test_a_workspace_is_a_block_of_the_stream_that_uses_it():
    """Nothing may run here: a block that the current stream has just given back is not another stream's."""
    side, size = torch.cuda.Stream(), 3 << 20
    held = torch.empty(size, dtype=torch.uint8, device="cuda")
    at = held.data_ptr()
    del held
    ws = gdn._scratch(size, "cuda", side)
    mine = ws.data_ptr()
    assert mine != at
    del ws
    assert torch.empty(size, dtype=torch.uint8, device="cuda").data_ptr() != mine
    for same in (side, side.cuda_stream):
        assert gdn._scratch(size, "cuda", same).data_ptr() == mine
    assert gdn._scratch(size, "cuda", None).data_ptr() == at
    assert gdn._scratch(size, "cuda", 0).data_ptr() == at


@pytest.mark.parametrize("rows", [[(1, 900), (1, 65)] * 8, [(200, 300), (70, 70)]], ids=["decode", "prompt"])
@pytest.mark.parametrize("dim,dtype", [(128, BF16), (96, BF16), (64, F32)])
def test_other_streams_and_graphs(rows, dim, dtype):
    s = Step(rows, heads=8, kv_heads=2, dim=dim, dtype=dtype, seed=dim)
    want, _ = s.run()
    side = torch.cuda.Stream()
    for given in (side, side.cuda_stream):
        s.out.fill_(0)
        side.wait_stream(torch.cuda.current_stream())
        gdn.gdn_paged_attention(s.attn, s.cache, s.kv_rows, s.qd, s.out, stream=given)
        side.synchronize()
        assert torch.equal(s.out.cpu()[s.token], want[s.token])
    ws = torch.empty(max(gdn.gdn_attention_workspace_bytes(s.attn, s.cache, s.kv_rows), 1), dtype=torch.uint8, device="cuda")
    for kept in (ws, None):  # (a workspace made under capture belongs to the graph)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            gdn.gdn_paged_attention(s.attn, s.cache, s.kv_rows, s.qd, s.out, workspace=kept)
        s.out.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(s.out.cpu()[s.token], want[s.token])
