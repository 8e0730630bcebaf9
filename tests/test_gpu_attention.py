"""Attention over the paged cache and appending to it, against plain 64-bit implementations, at the
sizes and masks where they can go wrong.  Tolerances: ``kv_reference.attention_tolerance``."""
import random

import pytest
import torch

import gated_deltanet_linear_spec_gb300 as gdn
from tests import kv_reference as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Step:
    """A batch of rows (new tokens, cache length) over a shuffled pool whose unused places hold NaN."""

    def __init__(self, rows, *, heads=4, kv_heads=2, dim=64, page=16, dtype=BF16, window=0, sinks=0, seed=0,
                 null=(), gather=True, fused=False, interleaved=False, scale=0.0, extra_pages=3, spare_rows=1):
        rng, gen = random.Random(seed), torch.Generator().manual_seed(seed)
        self.rows, self.dim, self.page, self.dtype = rows, dim, page, dtype
        self.window, self.sinks, self.scale = window, sinks, scale
        self.heads, self.kv_heads = heads, kv_heads
        n = len(rows)
        width = max([-(-kv // page) for _, kv in rows] + [1])
        need = [-(-kv // page) for _, kv in rows]
        num_pages = 1 + sum(need) + extra_pages
        ids = list(range(1, num_pages))
        rng.shuffle(ids)
        self.table_rows = list(range(n + spare_rows))
        rng.shuffle(self.table_rows)
        self.table_rows = self.table_rows[:n]
        table = [[0] * width for _ in range(n + spare_rows)]
        k = torch.full((num_pages, kv_heads, page, dim), float("nan"))
        v = torch.full((num_pages, kv_heads, page, dim), float("nan"))
        for i, (new, kv) in enumerate(rows):
            for e in range(need[i]):
                p = ids.pop()
                table[self.table_rows[i]][e] = p
                used = min(page, kv - e * page)
                k[p, :, :used] = torch.randn(kv_heads, used, dim, generator=gen)
                v[p, :, :used] = torch.randn(kv_heads, used, dim, generator=gen)
        for i, e, value in null:
            table[self.table_rows[i]][e] = value
        self.table = torch.tensor(table, dtype=torch.int32)
        self.k, self.v = k.to(dtype), v.to(dtype)
        self.starts = [0]
        for new, _ in rows:
            self.starts.append(self.starts[-1] + new)
        total = self.starts[-1]
        spare = 5 if gather else 0
        self.token = list(range(total + spare))
        if gather:
            rng.shuffle(self.token)
        self.token = self.token[:total]
        self.gather = gather
        self.q = torch.randn(total + spare, heads, dim, generator=gen).to(dtype)
        self.max_q = max([new for new, _ in rows] + [1])
        if interleaved:  # K and V as halves of one allocation
            both = torch.stack([self.k, self.v], 1).cuda()
            kd, vd = both[:, 0], both[:, 1]
        else:
            kd, vd = self.k.cuda(), self.v.cuda()
        self.kv = (kd, vd)
        self.cache = gdn.KvCache(kd, vd, self.table.cuda())
        self.kv_rows = gdn.KvRows(i32(self.starts), total, i32([kv for _, kv in rows]), self.max_q,
                                  i32(self.table_rows), i32(self.token) if gather else None)
        self.attn = gdn.Attention(heads, scale=scale, window=window, num_sinks=sinks)
        if fused:
            wide = torch.full((self.q.shape[0], heads + 3, dim), float("nan"), dtype=dtype, device="cuda")
            wide[:, 1:heads + 1] = self.q.cuda()
            self.qd = wide[:, 1:heads + 1]
            wide = torch.full((self.q.shape[0], heads + 2, dim), 7.0, dtype=dtype, device="cuda")
            self.out = wide[:, 2:]
        else:
            self.qd = self.q.cuda()
            self.out = torch.full_like(self.qd, 7.0)

    def run(self, **kw):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        gdn.gdn_paged_attention(self.attn, self.cache, self.kv_rows, self.qd, self.out, status=status, **kw)
        torch.cuda.synchronize()
        return self.out.cpu(), int(status)

    def expected(self):
        spans = [(self.starts[i], new) for i, (new, _) in enumerate(self.rows)]
        return ref.attention(self.q, self.k, self.v, self.table, spans, self.table_rows, self.token,
                             [kv for _, kv in self.rows], self.scale, self.window, self.sinks)

    def check(self, want_status=0):
        got, status = self.run()
        assert status == want_status
        out, spread, logits = self.expected()
        used = torch.zeros(got.shape[0], dtype=torch.bool)
        used[self.token] = True
        assert torch.all(got[~used].float() == 7.0), "a token of no row was written"
        keys = max([kv for _, kv in self.rows] + [1])
        # prompts take the weights into the products as bf16; other rows keep 16 bits of them or more
        tokens = self.max_q * (self.heads // self.kv_heads)
        bits = 24 if self.dtype == F32 else 8 if tokens > 64 else 16
        tol = ref.attention_tolerance(out, spread, logits, keys, self.dim, self.dtype, bits)
        err = (got.double() - out).abs()
        bad = ~(err <= tol) & used[:, None, None]
        assert not bad.any(), (int(bad.sum()), float((err / tol)[used].nan_to_num(1e9).max()))
        return got


# ------------------------------------------------------------------------------------------
# decode and verify rows

EDGES = [(1, 1), (1, 15), (1, 16), (1, 17), (1, 63), (1, 64), (1, 65), (1, 200), (0, 40), (0, 0)]
VERIFY = [(4, 4), (1, 5), (3, 64), (4, 66), (2, 129), (0, 7), (4, 300), (5, 128)]


@pytest.mark.parametrize("dim", [16, 64, 80, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_decode_edges(dim, dtype):
    Step(EDGES, dim=dim, dtype=dtype, seed=dim).check()


@pytest.mark.parametrize("dim", [32, 64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_verify_rows(dim, dtype):
    Step(VERIFY, dim=dim, dtype=dtype, seed=dim + 1, fused=True).check()


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (2, 1), (3, 1), (4, 4), (5, 1), (6, 2), (8, 1), (16, 2), (14, 2), (24, 1)])
def test_head_layouts(heads, kv_heads):
    Step([(1, 33), (2, 90)], heads=heads, kv_heads=kv_heads, dim=64, seed=heads).check()
    Step([(1, 33), (2, 90)], heads=heads, kv_heads=kv_heads, dim=128, dtype=F32, seed=heads).check()


@pytest.mark.parametrize("heads", [2, 3, 4, 8])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_up_to_64_queries_of_a_kv_head(dim, heads):
    Step([(8, 100), (3, 77), (1, 2000), (8, 8), (0, 3), (7, 515)], heads=2 * heads, kv_heads=2, dim=dim, page=32,
         seed=heads).check()
    Step([(8, 250), (5, 90)], heads=heads, kv_heads=1, dim=dim, window=37, sinks=5, seed=heads + 1,
         null=[(0, 9, 0), (1, 4, -1)]).check()


@pytest.mark.parametrize("heads", [1, 3, 8])
@pytest.mark.parametrize("dim", [32, 64, 128, 256])
def test_up_to_64_queries_of_a_kv_head_in_32_bits(dim, heads):
    Step([(8, 100), (3, 77), (1, 2000), (8, 8), (0, 3), (7, 515)], heads=2 * heads, kv_heads=2, dim=dim, page=32,
         dtype=F32, seed=heads).check()
    Step([(8, 250), (5, 90)], heads=heads, kv_heads=1, dim=dim, window=37, sinks=5, seed=heads + 1, dtype=F32,
         null=[(0, 9, 0), (1, 4, -1)], interleaved=True).check()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_page_sizes(page, dim):
    Step([(1, page - 1), (1, page), (1, page + 1), (3, 2 * page + 5)], page=page, dim=dim, seed=page,
         interleaved=True).check()


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 3), (7, 0), (16, 4), (17, 20), (64, 1), (100, 16), (5000, 9)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_windows(window, sinks, dtype):
    Step([(1, 1), (1, 40), (4, 130), (3, 257), (5, 5)], window=window, sinks=sinks, dtype=dtype, dim=64,
         seed=window).check()


def test_released_pages_behind_a_window():
    # what a window has left behind is NULL, or holds another row's page id of long ago
    Step([(1, 200), (4, 320)], window=40, sinks=3, null=[(0, 1, 0), (0, 5, -1), (1, 2, 0), (1, 9, 0)], seed=3).check()


def test_null_pages_hold_no_tokens():
    Step([(1, 50), (2, 100), (1, 16)], null=[(0, 0, 0), (1, 3, -7), (2, 0, 0)], seed=4).check()


def test_a_row_that_sees_nothing_gives_zero():
    s = Step([(1, 16), (3, 40)], null=[(0, 0, 0), (1, 0, 0), (1, 1, 0), (1, 2, 0)], seed=5)
    got = s.check()
    assert torch.all(got[s.token].float() == 0)


def test_page_ids_out_of_range_are_no_tokens():
    s = Step([(1, 50), (2, 100)], null=[(0, 1, 1 << 20), (1, 3, 2**31 - 1)], seed=6)
    s.check(want_status=ref.PAGE_RANGE)


@pytest.mark.parametrize("length", [1000, 4096, 4097, 20000])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_long_caches_are_split_and_joined(length, dim):
    Step([(1, length), (2, 37)], heads=8, kv_heads=2, dim=dim, page=64, seed=length).check()


def test_many_ragged_rows():
    rng = random.Random(9)
    rows = [(rng.randint(0, 4), rng.randint(4, 600)) for _ in range(150)]
    Step(rows, heads=8, kv_heads=4, dim=64, page=32, seed=9).check()


def test_large_scores_do_not_overflow():
    Step([(1, 100), (3, 200)], scale=60.0, dim=64, seed=10).check()
    Step([(1, 100), (3, 200)], scale=60.0, dim=64, seed=10, dtype=F32).check()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_later_token_never_reaches_an_earlier_one(value, dtype):
    s = Step([(4, 70), (4, 64)], dim=64, dtype=dtype, seed=11, gather=False)
    for n in range(2):  # the third of the row's four new tokens
        pos = s.rows[n][1] - 2
        page, slot = int(s.table[s.table_rows[n]][pos // s.page]), pos % s.page
        s.kv[0][page, :, slot, 3] = value
        s.kv[1][page, :, slot, 5] = value
    got, status = s.run()
    out, spread, logits = s.expected()  # of the clean cache: what the first two tokens see
    tol = ref.attention_tolerance(out, spread, logits, 70, 64, s.dtype, 24 if dtype == F32 else 16)
    clean = [0, 1, 4, 5]
    assert status == 0
    assert torch.all((got.double() - out).abs()[clean] <= tol[clean])
    if value != value:
        assert torch.isnan(got[[2, 3, 6, 7]].float()).all()


def test_bad_rows_are_skipped():
    s = Step([(1, 20), (2, 30), (1, 40), (1, 50)], gather=False, seed=12)
    out, spread, logits = s.expected()
    # row 1 longer than max_query_len, row 2's length past its table, row 3's table row past the table
    s.kv_rows = gdn.KvRows(s.kv_rows.query_start_loc, 5, i32([20, 30, 9999, 50]), 1,
                           i32(s.table_rows[:3] + [77]), None)
    got, status = s.run()
    assert status == ref.ROW_RANGE | ref.PAGE_RANGE
    assert torch.all(got[1:].float() == 7.0)
    assert torch.all((got[0].double() - out[0]).abs() <= ref.attention_tolerance(out, spread, logits, 20, 64, BF16, 16)[0])


def test_tokens_out_of_range_are_skipped():
    s = Step([(2, 20), (1, 30)], gather=False, seed=13)
    out, spread, logits = s.expected()
    s.kv_rows = gdn.KvRows(s.kv_rows.query_start_loc, 3, s.kv_rows.kv_lens, 2, s.kv_rows.table_rows, i32([0, 500, -1]))
    got, status = s.run()
    assert status == ref.TOKEN_RANGE
    assert torch.all(got[1:].float() == 7.0)
    assert torch.all((got[0].double() - out[0]).abs() <= ref.attention_tolerance(out, spread, logits, 20, 64, BF16, 16)[0])


# ------------------------------------------------------------------------------------------
# prompts

@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rows", [[(65, 65)], [(127, 127), (1, 300)], [(128, 128), (0, 5), (129, 400)], [(300, 700)]],
                         ids=["65", "127", "129", "300"])
def test_prompts(dim, rows):
    Step(rows, heads=8, kv_heads=2, dim=dim, page=16, seed=dim, fused=True).check()


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (2, 1), (3, 1), (6, 2), (8, 1), (4, 4)])
def test_prompt_head_layouts(heads, kv_heads):
    Step([(150, 170), (70, 70)], heads=heads, kv_heads=kv_heads, dim=64, page=32, seed=heads).check()


@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 3), (50, 0), (64, 4), (128, 16), (130, 200), (4000, 2)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prompt_windows(window, sinks, dim):
    Step([(200, 450), (140, 140)], heads=4, kv_heads=2, dim=dim, page=64, window=window, sinks=sinks,
         seed=window + dim).check()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 333])
def test_prompts_that_fill_the_gpu(dim, window):
    # 88 work items or more: none is cut into pieces, CTAs take several
    Step([(700, 700), (1, 9), (641, 1100), (130, 130)], heads=16, kv_heads=16, dim=dim, page=64, window=window, sinks=2,
         seed=dim).check()


def test_prompt_in_32_bits():
    Step([(200, 230), (90, 90)], heads=4, kv_heads=2, dim=64, dtype=F32, seed=20).check()
    Step([(200, 230), (90, 90)], heads=4, kv_heads=2, dim=48, seed=21).check()


def test_prompt_null_pages():
    Step([(200, 330), (90, 90)], heads=4, kv_heads=2, dim=128, seed=22,
         null=[(0, 2, 0), (0, 20, -1), (1, 0, 0), (1, 1, 0), (1, 2, 0), (1, 3, 0), (1, 4, 0), (1, 5, 0)]).check()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prompt_later_tokens_never_reach_earlier_ones(value, dim):
    s = Step([(300, 310)], heads=4, kv_heads=2, dim=dim, page=16, seed=23, gather=False)
    bad = 150  # new token whose K and V are not finite
    pos = s.rows[0][1] - 300 + bad
    page, slot = int(s.table[s.table_rows[0]][pos // 16]), pos % 16
    s.kv[0][page, :, slot, 3] = value
    s.kv[1][page, :, slot, 5] = value
    got, _ = s.run()
    out, spread, logits = s.expected()
    tol = ref.attention_tolerance(out, spread, logits, 310, dim, BF16, 8)
    assert torch.all((got.double() - out).abs()[:bad] <= tol[:bad])
    if value != value:
        assert torch.isnan(got[bad:].float()).all()


# ------------------------------------------------------------------------------------------
# both

@pytest.mark.parametrize("rows", [[(1, 3000), (4, 900)], [(300, 400), (100, 100)]], ids=["verify", "prompt"])
def test_repeated_runs_are_equal(rows):
    s = Step(rows, heads=8, kv_heads=2, dim=128, seed=30)
    first, _ = s.run()
    for _ in range(3):
        again, _ = s.run()
        assert torch.equal(first, again)


@pytest.mark.parametrize("rows", [[(1, 3000), (4, 900)], [(300, 400), (100, 100)]], ids=["verify", "prompt"])
def test_graph_capture_and_other_streams(rows):
    s = Step(rows, heads=8, kv_heads=2, dim=128, seed=31)
    want, _ = s.run()
    need = gdn.gdn_attention_workspace_bytes(s.attn, s.cache, s.kv_rows)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    s.out.fill_(0)
    side.wait_stream(torch.cuda.current_stream())
    gdn.gdn_paged_attention(s.attn, s.cache, s.kv_rows, s.qd, s.out, stream=side)
    side.synchronize()
    assert torch.equal(s.out.cpu()[s.token], want[s.token])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_paged_attention(s.attn, s.cache, s.kv_rows, s.qd, s.out, workspace=ws)
    s.out.fill_(0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(s.out.cpu()[s.token], want[s.token])


@pytest.mark.parametrize("new,dim", [(1, 128), (3, 64), (100, 128), (90, 256)])
def test_offsets_past_32_bits(new, dim):
    """Pages whose element offsets pass 2^31: K and V in one allocation of a little over 2^32 elements."""
    heads, page = 4, 256
    per = 2 * heads * page * dim
    pages = (1 << 32) // per + 8
    both = torch.empty(pages, 2, heads, page, dim, dtype=BF16, device="cuda")
    kv = 2 * page + 77
    ids = [pages - 1, pages // 2 + 1, pages - 3]
    gen = torch.Generator().manual_seed(dim)
    small = torch.zeros(4, 2, heads, page, dim, dtype=BF16)
    small[1:] = torch.randn(3, 2, heads, page, dim, generator=gen).to(BF16)
    for i, p in enumerate(ids):
        both[p] = small[i + 1].cuda()
    q = torch.randn(new, heads, dim, generator=gen).to(BF16)
    rows = gdn.KvRows(i32([0, new]), new, i32([kv]), new)
    cache = gdn.KvCache(both[:, 0], both[:, 1], i32([ids]))
    qd, out = q.cuda(), torch.empty(new, heads, dim, dtype=BF16, device="cuda")
    gdn.gdn_paged_attention(gdn.Attention(heads), cache, rows, qd, out)
    want, spread, logits = ref.attention(q, small[:, 0], small[:, 1], torch.tensor([[1, 2, 3]]), [(0, new)], [0],
                                         list(range(new)), [kv], 0.0, 0, 0)
    tol = ref.attention_tolerance(want, spread, logits, kv, dim, BF16, 8)
    assert torch.all((out.cpu().double() - want).abs() <= tol)
    k = torch.randn(new, heads, dim, generator=gen).to(BF16).cuda()
    gdn.gdn_kv_append(cache, rows, k, -k)
    for t in range(new):
        pos = kv - new + t
        assert torch.equal(both[ids[pos // page], 0, :, pos % page], k[t])
        assert torch.equal(both[ids[pos // page], 1, :, pos % page], -k[t])


# ------------------------------------------------------------------------------------------
# append

@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("heads,dim,page", [(1, 16, 16), (2, 64, 32), (3, 80, 16), (8, 128, 64), (2, 256, 256)])
@pytest.mark.parametrize("gather", [False, True])
def test_append(dtype, heads, dim, page, gather):
    s = Step([(1, 1), (4, 70), (0, 9), (37, 37), (2, page + 1), (1, page)], heads=heads, kv_heads=heads, dim=dim, page=page,
             dtype=dtype, gather=gather, seed=dim, interleaved=gather, null=[(1, 4 if page == 16 else 0, 0)])
    gen = torch.Generator().manual_seed(1)
    wide = torch.randn(s.q.shape[0], 2 * heads + 1, dim, generator=gen).to(dtype).cuda()
    k, v = wide[:, :heads], wide[:, heads + 1:]
    want_k, want_v = s.k.clone(), s.v.clone()
    for n, (new, kv) in enumerate(s.rows):
        for t in range(new):
            pos = kv - new + t
            p = int(s.table[s.table_rows[n]][pos // page])
            if p > 0:
                want_k[p, :, pos % page] = k[s.token[s.starts[n] + t]].cpu()
                want_v[p, :, pos % page] = v[s.token[s.starts[n] + t]].cpu()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_kv_append(s.cache, s.kv_rows, k, v, status=status)
    assert int(status) == 0
    view = torch.int16 if dtype == BF16 else torch.int32
    assert torch.equal(s.kv[0].cpu().contiguous().view(view), want_k.view(view))
    assert torch.equal(s.kv[1].cpu().contiguous().view(view), want_v.view(view))


def test_append_refuses_what_it_must_not_write():
    s = Step([(1, 20), (2, 40), (1, 5), (1, 9)], heads=2, kv_heads=2, gather=False, seed=40)
    count = torch.ones(s.k.shape[0], dtype=torch.int32, device="cuda")
    shared = int(s.table[s.table_rows[0]][1])
    count[shared] = 2
    cache = gdn.KvCache(*s.kv, s.cache.block_table, count)
    s.cache.block_table[s.table_rows[2], 0] = 1 << 30
    rows = gdn.KvRows(s.kv_rows.query_start_loc, 5, i32([20, 40, 5, 0]), 2, s.kv_rows.table_rows, i32([0, 1, 99, 3, 4]))
    k = torch.ones(5, 2, 64, dtype=BF16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_kv_append(cache, rows, k, k, status=status)
    assert int(status) == ref.PAGE_SHARED | ref.TOKEN_RANGE | ref.PAGE_RANGE | ref.ROW_RANGE
    want = s.k.clone()
    want[int(s.table[s.table_rows[1]][2]), :, 38 % 16] = 1
    assert torch.equal(s.kv[0].cpu().view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("dim", [16, 48, 80, 96, 112, 160, 192, 240])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_every_head_dim(dim, dtype):
    Step([(1, 700), (4, 130), (0, 9), (90, 300), (1, 1)], heads=6, kv_heads=2, dim=dim, dtype=dtype, seed=dim).check()
    Step([(3, 257), (40, 600)], heads=4, kv_heads=4, dim=dim, page=32, window=70, sinks=5, dtype=dtype,
         seed=dim + 1).check()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_last_token_reaches_itself_alone_at_other_head_dims(value, dtype):
    s = Step([(4, 70), (40, 64)], dim=96, dtype=dtype, seed=3, gather=False)
    clean, _ = s.run()
    clean = clean.clone()
    for n in range(2):
        pos = s.rows[n][1] - 1
        page, slot = int(s.table[s.table_rows[n]][pos // s.page]), pos % s.page
        s.kv[0][page, :, slot] = value
        s.kv[1][page, :, slot] = value
    got, _ = s.run()
    others = [t for t in range(44) if t not in (3, 43)]
    assert torch.equal(got[others], clean[others])
    assert not torch.isfinite(got[[3, 43]].float()).all()


@pytest.mark.parametrize("heads,kv_heads", [(8, 2), (16, 1), (4, 4), (24, 1)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_decode_rows_beside_prompts(dim, heads, kv_heads):
    rows = [(1, 300), (1, 1), (140, 200), (1, 64), (4, 90), (0, 7), (1, 513), (70, 70), (1, 33), (3, 40), (1, 128), (17, 99),
            (1, 2), (5, 5), (1, 700), (33, 33), (0, 0)]
    Step(rows, heads=heads, kv_heads=kv_heads, dim=dim, page=32, seed=dim + heads).check()
    Step(rows, heads=heads, kv_heads=kv_heads, dim=dim, window=50, sinks=3, seed=dim + heads + 1, fused=True).check()
