"""Groups of rows over shared pages: how far they agree, and attention that reads the shared pages once, against plain
64-bit implementations.  Tolerances: ``kv_reference.attention_tolerance``."""
import pytest
import torch

import gated_deltanet_linear_spec_gb300 as gdn
from tests import kv_reference as ref
from tests.test_gpu_attention import BF16, F32, Step, i32

pytestmark = pytest.mark.gpu


def weight_bits(dim, dtype):
    """The tensor cores take the weights as bf16; the CUDA cores keep 32 bits of them."""
    return 8 if dtype == BF16 and dim in (64, 128, 256) else 24


class Groups(Step):
    """Groups (prefix tokens, rows of (new tokens, cache length)); the rows of a group hold the pages of its first row for
    the whole pages of the prefix.  ``lone`` rows in front and behind belong to no group."""

    def __init__(self, groups, lone=(), **kw):
        rows, bounds = list(lone), [len(lone)]
        for _, of_group in groups:
            rows += of_group
            bounds.append(len(rows))
        rows += list(lone)
        super().__init__(rows, **kw)
        for g, (prefix, of_group) in enumerate(groups):
            for i in range(bounds[g] + 1, bounds[g + 1]):
                shared = min(prefix, rows[i][1]) // self.page
                first = self.table[self.table_rows[bounds[g]]]
                self.table[self.table_rows[i], :shared] = first[:shared]
        self.cache = gdn.KvCache(*self.kv, self.table.cuda())
        self.bounds = bounds
        self.groups = gdn.KvGroups(i32(bounds), i32([prefix for prefix, _ in groups]))

    def run(self, **kw):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        gdn.gdn_shared_attention(self.attn, self.cache, self.kv_rows, self.groups, self.qd, self.out, status=status, **kw)
        torch.cuda.synchronize()
        return self.out.cpu(), int(status)

    def check(self, want_status=0):
        got, status = self.run()
        assert status == want_status
        out, spread, logits = self.expected()
        used = torch.zeros(got.shape[0], dtype=torch.bool)
        used[self.token] = True
        assert torch.all(got[~used].float() == 7.0), "a token of no row was written"
        keys = max([kv for _, kv in self.rows] + [1])
        bits = weight_bits(self.dim, self.dtype)
        tol = ref.attention_tolerance(out, spread, logits, keys, self.dim, self.dtype, bits)
        err = (got.double() - out).abs()
        bad = ~(err <= tol) & used[:, None, None]
        assert not bad.any(), (int(bad.sum()), float((err / tol)[used].nan_to_num(1e9).max()))
        return got


TREE = [(100, [(1, 101), (2, 130), (1, 300), (3, 111)]), (64, [(4, 68), (1, 65)]), (33, [(1, 40), (0, 36), (2, 90)])]


@pytest.mark.parametrize("dim,dtype", [(16, BF16), (64, BF16), (96, BF16), (128, BF16), (256, BF16), (48, F32), (64, F32),
                                       (128, F32), (256, F32)])
@pytest.mark.parametrize("page", [16, 64])
def test_groups(dim, dtype, page):
    Groups(TREE, lone=[(1, 50), (2, 2)], dim=dim, dtype=dtype, page=page, seed=dim, heads=8).check()


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 3), (8, 1), (12, 4), (32, 2)])
@pytest.mark.parametrize("dim,dtype", [(64, BF16), (128, BF16), (64, F32)])
def test_head_layouts(heads, kv_heads, dim, dtype):
    Groups(TREE, heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype, seed=heads, fused=True, interleaved=True).check()


# heads and types: few queries in all, and many
FEW_AND_MANY = [(4, 64, BF16), (4, 128, BF16), (4, 256, BF16), (4, 96, BF16), (4, 64, F32), (32, 64, BF16), (32, 128, BF16),
                (32, 256, BF16), (32, 96, BF16)]


@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 31, 32, 33, 47, 48, 63, 64, 65, 80, 127, 128, 129, 1000])
@pytest.mark.parametrize("heads,dim,dtype", [(4, 64, BF16), (4, 256, BF16), (4, 64, F32), (32, 64, BF16), (32, 256, BF16)])
def test_prefix_lengths(prefix, heads, dim, dtype):
    """Whole pages, half tiles, a page's last and first token; and lengths that the rows' own tokens cut short."""
    groups = [(prefix, [(2, prefix + 2), (1, prefix + 50), (3, prefix + 17)])]
    Groups(groups, heads=heads, dim=dim, dtype=dtype, seed=prefix).check()


@pytest.mark.parametrize("given", [-5, 0, 1 << 30])
def test_prefix_lens_that_rows_cut(given):
    s = Groups([(64, [(2, 66), (1, 200), (3, 90)])], dim=64)
    s.groups = gdn.KvGroups(s.groups.group_start_loc, i32([given]))
    s.check()


@pytest.mark.parametrize("heads,dim,dtype", FEW_AND_MANY)
@pytest.mark.parametrize("window,sinks", [(1, 0), (20, 0), (20, 5), (70, 3), (64, 40), (150, 0), (5, 500), (1000, 7)])
def test_windows(window, sinks, heads, dim, dtype):
    Groups(TREE, lone=[(3, 90)], heads=heads, dim=dim, dtype=dtype, window=window, sinks=sinks, seed=window).check()


@pytest.mark.parametrize("heads,dim,dtype", FEW_AND_MANY)
def test_null_pages(heads, dim, dtype):
    """Holes in the prefix, a prefix without any page, holes in the rows' own tokens."""
    groups = [(96, [(1, 97), (2, 140)]), (64, [(1, 65), (1, 70)])]
    null = [(0, 0, 0), (0, 3, 0), (0, 4, -7), (1, 7, 0)] + [(2, e, 0) for e in range(4)]
    Groups(groups, heads=heads, dim=dim, dtype=dtype, null=null, seed=1).check()


def test_pages_out_of_range_are_reported():
    s = Groups([(96, [(1, 97), (2, 140)])], null=[(0, 2, 10 ** 6)])
    s.check(want_status=gdn.STATUS_PAGE_RANGE)


@pytest.mark.parametrize("heads,dim,dtype", [(4, 64, BF16), (4, 128, BF16), (4, 256, BF16), (4, 96, BF16), (4, 128, F32),
                                             (64, 64, BF16), (64, 128, BF16), (64, 256, BF16)])
def test_values_that_windows_hide(heads, dim, dtype):
    """Infinities and NaN where no query, or not every query, sees them."""
    s = Groups([(200, [(1, 201), (2, 230), (1, 260)])], heads=heads, dim=dim, dtype=dtype, window=90, sinks=4, seed=9,
               gather=False)
    k, v = (t.clone() for t in (s.k, s.v))
    row = s.table[s.table_rows[0]].tolist()
    want, spread, logits = s.expected()
    for pos in (10, 60, 111, 115, 140):  # behind the windows of all queries, or of those of the longer rows
        for pool in (k, v):
            pool[row[pos // 16], :, pos % 16] = float("nan") if pos % 2 else float("inf")
    s.cache = gdn.KvCache(k.cuda(), v.cuda(), s.table.cuda())
    got, status = s.run()
    assert status == 0
    tol = ref.attention_tolerance(want, spread, logits, 260, dim, dtype, weight_bits(dim, dtype))
    for i, (new, kv) in enumerate(s.rows):
        for t in range(new):
            low = kv - new + t - 90  # positions up to here are hidden
            token = s.starts[i] + t
            if low >= 140:
                assert torch.all((got[token].double() - want[token]).abs() <= tol[token]), (i, t)
            else:
                assert not torch.isfinite(got[token].float()).all()


def test_growing_scores():
    """Every part of the cache raises the maximum: states and pieces meet at maxima far apart."""
    for heads, dim, dtype in ((4, 64, BF16), (4, 128, BF16), (4, 64, F32), (64, 64, BF16), (64, 128, BF16), (64, 256, BF16)):
        s = Groups([(640, [(1, 660), (2, 720)])], heads=heads, dim=dim, dtype=dtype, gather=False, seed=dim)
        k = s.k.float()
        for i, (_, kv) in enumerate(s.rows):
            for j in range(kv):
                page = int(s.table[s.table_rows[i], j // 16])
                k[page, :, j % 16] = torch.sign(torch.randn(dim, generator=torch.Generator().manual_seed(j))) * (0.02 * j)
        s.k = k.to(dtype)
        s.q = (s.q.float().sign() * 2).to(dtype)
        s.qd = s.q.cuda()
        s.cache = gdn.KvCache(s.k.cuda(), s.v.cuda(), s.table.cuda())
        s.check()


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_many_rows_of_one_group(dim):
    Groups([(512, [(1, 513 + 3 * i) for i in range(70)])], heads=8, kv_heads=2, dim=dim, seed=5).check()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 300])
def test_groups_of_all_sizes(dim, window):
    """Units with one query tile and with two, of a few tiles and of many, in one pass."""
    groups = [(prefix, [(1 + i % 3, prefix + 4 + 11 * i) for i in range(n)])
              for prefix, n in ((640, 3), (64, 40), (0, 3), (1500, 9), (16, 2), (200, 21), (2100, 2))]
    Groups(groups, heads=16, kv_heads=2, dim=dim, window=window, sinks=5, seed=dim).check()


def test_many_groups():
    groups = [(16 * (1 + g % 5), [(1, 100 + g), (1 + g % 3, 120)]) for g in range(90)]
    Groups(groups, heads=4, kv_heads=2, dim=64, seed=6).check()


@pytest.mark.parametrize("dim,dtype", [(64, BF16), (128, BF16), (256, BF16), (96, BF16), (64, F32)])
@pytest.mark.parametrize("longest", [33, 65, 129, 140])
def test_long_rows(longest, dim, dtype):
    """More than 64, 128 and 256 queries per kv-head; rows that end inside a page whose other places hold NaN."""
    groups = [(300, [(40, 340), (1, 320), (longest, 300 + longest + 20)]), (64, [(33, 100), (2, 66)])]
    Groups(groups, heads=4, kv_heads=2, dim=dim, dtype=dtype, seed=longest).check()
    Groups(groups, heads=4, kv_heads=2, dim=dim, dtype=dtype, seed=longest, window=100, sinks=3).check()


def test_rows_of_many_tokens():
    Groups([(300, [(700, 1000), (400, 700)]), (30, [(3, 40)])], heads=2, kv_heads=1, dim=32, dtype=F32, seed=2).check()


@pytest.mark.parametrize("dim,dtype", [(64, BF16), (64, F32)])
def test_more_rows_than_a_pass_plans_itself(dim, dtype):
    groups = [(48, [(1 + i % 2, 50 + i % 7) for i in range(5)]) for _ in range(53)]
    Groups(groups, lone=[(1, 20)], heads=2, kv_heads=1, dim=dim, dtype=dtype, seed=3).check()
    Groups(groups, heads=2, kv_heads=1, dim=dim, dtype=dtype, window=30, sinks=2, seed=4).check()


def test_rows_without_tokens_do_not_stand_for_their_group():
    s = Groups([(64, [(0, 64), (1, 80), (2, 90)]), (48, [(0, 48), (0, 50)]), (32, [(1, 40)])], dim=128)
    s.table[s.table_rows[0]] = 0  # a finished row, whose pages were given back
    s.cache = gdn.KvCache(*s.kv, s.table.cuda())
    s.check()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_bad_rows_and_groups(dtype):
    s = Groups([(64, [(1, 80), (2, 90), (1, 70)])], dtype=dtype, gather=False)
    s.check()
    want, spread, logits = s.expected()
    tol = ref.attention_tolerance(want, spread, logits, 90, 64, dtype, weight_bits(64, dtype))
    lens = i32([80, 1, 70])  # row 1: fewer tokens than new ones
    s.kv_rows = gdn.KvRows(s.kv_rows.query_start_loc, 4, lens, 2, s.kv_rows.table_rows)
    s.out.fill_(7.0)
    got, status = s.run()
    assert status == gdn.STATUS_ROW_RANGE
    assert torch.all(got[1:3].float() == 7.0)
    assert torch.all(((got.double() - want).abs() <= tol)[[0, 3]])
    for bounds in ([2, 1], [-1, 3], [0, 4]):  # no group's bounds: nothing is shared
        s = Groups([(64, [(1, 80), (2, 90), (1, 70)])], dtype=dtype, gather=False)
        s.groups = gdn.KvGroups(i32(bounds), s.groups.prefix_lens)
        s.check(want_status=gdn.STATUS_ROW_RANGE)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("many", [False, True])
def test_a_row_in_two_groups(dtype, many):
    """Bounds that do not ascend would put rows into two groups: nothing is shared then, whoever makes the plan."""
    groups = [(48, [(1 + i % 2, 50 + i % 7) for i in range(5)]) for _ in range(53 if many else 2)]
    s = Groups(groups, dtype=dtype, heads=2, kv_heads=1, seed=11)
    bounds = [0, 6, 3, 9] + s.bounds[3:]
    s.groups = gdn.KvGroups(i32(bounds), i32([48] * (len(bounds) - 1)))
    s.check(want_status=gdn.STATUS_ROW_RANGE)


@pytest.mark.parametrize("dim,dtype", [(64, BF16), (256, BF16), (96, BF16), (64, F32)])
def test_padded_batch(dim, dtype):
    """Rows without tokens at the end, and tokens behind the last row's."""
    s = Groups([(64, [(2, 70), (1, 80), (1, 90)]), (32, [(0, 40), (0, 33), (0, 64)])], dim=dim, dtype=dtype, gather=False)
    q = torch.cat([s.q, torch.full((7, *s.q.shape[1:]), float("nan"), dtype=dtype)])
    s.q, s.qd, s.out = q, q.cuda(), torch.full_like(q, 7.0, device="cuda")
    r = s.kv_rows
    s.kv_rows = gdn.KvRows(r.query_start_loc, q.shape[0], r.kv_lens, s.max_q, r.table_rows)
    s.check()


@pytest.mark.parametrize("dim,dtype", [(128, BF16), (64, F32)])
def test_two_graphs_share_a_workspace(dim, dtype):
    one = Groups([(160, [(1, 170 + i) for i in range(9)])], dim=dim, dtype=dtype, seed=1)
    two = Groups([(96, [(2, 100), (1, 200), (4, 111)]), (32, [(1, 50), (1, 40), (1, 33)])], dim=dim, dtype=dtype, seed=2, window=70)
    want = [s.check().clone() for s in (one, two)]
    need = [gdn.gdn_shared_attention_workspace_bytes(s.attn, s.cache, s.kv_rows, s.groups) for s in (one, two)]
    ws = torch.empty(max(need), dtype=torch.uint8, device="cuda")
    graphs = []
    for s in (one, two):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            gdn.gdn_shared_attention(s.attn, s.cache, s.kv_rows, s.groups, s.qd, s.out, workspace=ws)
        graphs.append(g)
    for s in (one, two):
        s.out.fill_(7.0)
    for _ in range(10):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for s, w in zip((one, two), want):
        assert torch.equal(s.out.cpu(), w)


@pytest.mark.parametrize("dim,dtype", [(128, BF16), (64, F32)])
def test_two_streams_at_once(dim, dtype):
    """Calls that run beside one another, each with a workspace of its own, give what they give alone."""
    pair = [Groups([(640, [(1 + i % 3, 650 + 9 * i) for i in range(20)])], dim=dim, dtype=dtype, seed=7 + j, heads=8) for j in range(2)]
    want = [s.check().clone() for s in pair]
    streams = [torch.cuda.Stream() for _ in pair]
    ws = [torch.empty(gdn.gdn_shared_attention_workspace_bytes(s.attn, s.cache, s.kv_rows, s.groups), dtype=torch.uint8,
                      device="cuda") for s in pair]
    for s in pair:
        s.out.fill_(7.0)
    torch.cuda.synchronize()
    for _ in range(20):
        for s, stream, w in zip(pair, streams, ws):
            gdn.gdn_shared_attention(s.attn, s.cache, s.kv_rows, s.groups, s.qd, s.out, workspace=w, stream=stream)
    torch.cuda.synchronize()
    for s, w in zip(pair, want):
        assert torch.equal(s.out.cpu(), w)


@pytest.mark.parametrize("dim,dtype", [(64, BF16), (128, BF16), (64, F32)])
def test_one_key_and_one_page(dim, dtype):
    """The smallest calls: a row whose only key is its own, groups of one row, one page shared and nothing else."""
    Groups([(0, [(1, 1)])], dim=dim, dtype=dtype, heads=1, kv_heads=1).check()
    Groups([(16, [(1, 17)])], dim=dim, dtype=dtype, heads=1, kv_heads=1).check()
    Groups([(16, [(1, 17), (1, 17)])], dim=dim, dtype=dtype, heads=1, kv_heads=1).check()
    Groups([(16, [(1, 17)] * 9)], dim=dim, dtype=dtype, heads=64, kv_heads=1, window=1).check()


def test_no_groups_and_no_tokens():
    s = Groups([], lone=[(1, 30), (2, 40)])
    s.check()
    s = Groups([(16, [(0, 20), (0, 30)])])
    got, status = s.run()
    assert status == 0 and torch.all(got.float() == 7.0)


@pytest.mark.parametrize("dim,dtype", [(64, BF16), (128, BF16), (256, BF16), (96, BF16), (64, F32)])
def test_streams_graphs_and_a_given_workspace(dim, dtype):
    s = Groups([(320, [(1, 330 + i) for i in range(9)]), (64, [(2, 100), (2, 110)])], dim=dim, dtype=dtype, heads=8)
    want, _ = s.run()
    need = gdn.gdn_shared_attention_workspace_bytes(s.attn, s.cache, s.kv_rows, s.groups)
    ws = torch.full((need + 256,), 0xff, dtype=torch.uint8, device="cuda")
    s.out.fill_(7.0)
    got, _ = s.run(workspace=ws[:need])
    assert torch.equal(got, want) and torch.all(ws[need:] == 0xff)
    other = torch.cuda.Stream()
    s.out.fill_(7.0)
    other.wait_stream(torch.cuda.current_stream())
    got, _ = s.run(stream=other)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_shared_attention(s.attn, s.cache, s.kv_rows, s.groups, s.qd, s.out, workspace=ws)
    s.groups.prefix_lens.fill_(16)
    s.out.fill_(7.0)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    got = s.out.cpu().clone()
    s.out.fill_(7.0)
    again, _ = s.run()
    assert torch.equal(got, again)


# ------------------------------------------------------------------------------------------
# the common prefix

def common(s):
    out = []
    for a, b in zip(s.bounds, s.bounds[1:]):
        real = [i for i in range(a, b) if s.rows[i][0] > 0]
        if not real:
            out.append(0)
            continue
        e, whole = 0, min(s.rows[i][1] - s.rows[i][0] for i in real) // s.page
        def page(i, e):
            p = int(s.table[s.table_rows[i], e])
            return p if 0 < p < s.k.shape[0] else 0
        while e < whole and len({page(i, e) for i in real}) == 1:
            e += 1
        out.append(e * s.page)
    return out


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("groups", [TREE, [(500, [(1, 501)])], [(0, [(1, 1), (1, 900)]), (2000, [(1, 2100 + i) for i in range(200)])],
                                    [(48, [(0, 64), (1, 80), (0, 20)]), (48, [(0, 50), (0, 48)])],
                                    [(16 * g, [(1, 700), (3, 800)]) for g in range(40)]])
def test_common_prefix(groups, page):
    s = Groups(groups, page=page, dim=16, heads=2, kv_heads=1)
    s.groups.prefix_lens.fill_(-1)
    status = i32([0])
    gdn.gdn_kv_common_prefix(s.cache, s.kv_rows, s.groups, status=status)
    assert s.groups.prefix_lens.tolist() == common(s) and int(status) == 0


def test_common_prefix_of_null_and_bad_entries():
    s = Groups([(160, [(1, 170), (1, 180), (2, 190)])], dim=16, null=[(0, 1, 0), (0, 4, 10 ** 6)])
    s.table[s.table_rows[1], 1] = -3  # NULL either way
    s.cache = gdn.KvCache(*s.kv, s.table.cuda())
    status = i32([0])
    gdn.gdn_kv_common_prefix(s.cache, s.kv_rows, s.groups, status=status)
    assert s.groups.prefix_lens.tolist() == common(s) == [160] and int(status) == gdn.STATUS_PAGE_RANGE


def test_common_prefix_of_bad_rows_and_groups():
    s = Groups([(160, [(1, 170), (1, 180), (2, 190)])], dim=16)
    rows = gdn.KvRows(s.kv_rows.query_start_loc, 4, i32([170, 0, 190]), 2, s.kv_rows.table_rows)
    status, groups = i32([0]), gdn.KvGroups(i32([0, 3, 2]), i32([-1, -1]))
    gdn.gdn_kv_common_prefix(s.cache, rows, groups, status=status)
    assert groups.prefix_lens.tolist() == [160, 0] and int(status) == gdn.STATUS_ROW_RANGE


@pytest.mark.parametrize("at", [0, 1, 31, 32, 127, 128, 129, 700, 1249])
def test_common_prefix_ends_where_one_row_leaves(at):
    s = Groups([(20000, [(1, 20001)] * 12)], dim=16, heads=1, kv_heads=1)
    s.table[s.table_rows[9], at] = 1 if int(s.table[s.table_rows[9], at]) != 1 else 2
    s.cache = gdn.KvCache(*s.kv, s.table.cuda())
    gdn.gdn_kv_common_prefix(s.cache, s.kv_rows, s.groups)
    assert s.groups.prefix_lens.tolist() == [16 * at]


@pytest.mark.parametrize("rows,entries,at", [(256, 8192, 8192), (256, 8192, 8000), (200, 8192, 31), (64, 8192, 4097), (40, 8000, 0)])
@pytest.mark.parametrize("groups", [1, 3])
def test_common_prefix_of_many_long_rows(rows, entries, at, groups):
    """More entries than one cluster should go over alone; a row late in the group leaves at `at`, which may be the end."""
    gen = torch.Generator().manual_seed(at)
    first = torch.randint(1, 1000, (groups, entries), generator=gen, dtype=torch.int32)
    table = first.repeat_interleave(rows, 0)
    if at < entries:
        table[rows - 2, at] = 1000  # (of the first group)
    pool = torch.zeros(1001, 1, 16, 16, device="cuda")
    n = rows * groups
    cache = gdn.KvCache(pool, pool, table.cuda())
    kv_rows = gdn.KvRows(i32(list(range(n + 1))), n, i32([entries * 16] * n), 1)
    of_groups = gdn.KvGroups(i32([g * rows for g in range(groups + 1)]), i32([-7] * groups))
    status = i32([0])
    for _ in range(2):
        gdn.gdn_kv_common_prefix(cache, kv_rows, of_groups, status=status)
        # the last entry holds the new token's page, so it is no whole page before it
        want = [16 * min(at, entries - 1)] + [16 * (entries - 1)] * (groups - 1)
        assert of_groups.prefix_lens.tolist() == want and int(status) == 0


# ------------------------------------------------------------------------------------------
# all of it together

@pytest.mark.parametrize("dtype,dim", [(BF16, 128), (F32, 64)], ids=["bf16", "f32"])
def test_branches_decode_in_a_graph(dtype, dim):
    """One sequence is forked; its branches then decode steps that a graph holds: room for a token, q and k turned on
    their way, what the rows share found, attention.  Each step against the definition in 64 bits."""
    heads, hk, page, branches, pages = 8, 2, 16, 5, 120
    gen = torch.Generator(device="cuda").manual_seed(dim)
    rand = lambda *shape: torch.randn(*shape, generator=gen, device="cuda").to(dtype)  # noqa: E731
    pool = torch.zeros(pages, 2, hk, page, dim, dtype=dtype, device="cuda")
    cache = gdn.KvCache(pool[:, 0], pool[:, 1], i32([[0] * 16] * branches), i32([0] * pages))
    rope, attn, status = gdn.Rope(dim // 2), gdn.Attention(heads), i32([0])
    prompt = 75
    gdn.gdn_kv_reserve(cache, i32([0]), i32([0]), i32([prompt]), status=status)
    rows = gdn.KvRows(i32([0, prompt]), prompt, i32([prompt]), prompt, i32([0]))
    gdn.gdn_kv_append_rope(cache, rows, rope, rand(prompt, hk, dim), rand(prompt, hk, dim), status=status)
    gdn.gdn_kv_fork(cache, i32([0] * (branches - 1)), i32(list(range(1, branches))), i32([prompt] * (branches - 1)),
                    status=status)
    old, lens = i32([prompt] * branches), i32([prompt + 1] * branches)
    rows = gdn.KvRows(i32(list(range(branches + 1))), branches, lens, 1)
    groups = gdn.KvGroups(i32([0, branches]), i32([0]))
    qkv = rand(branches, heads + 2 * hk, dim)
    q, k, v = qkv.split([heads, hk, hk], 1)
    turned, out = torch.zeros(branches, heads, dim, dtype=dtype, device="cuda"), torch.zeros(branches, heads, dim, dtype=dtype, device="cuda")
    need = max(gdn.gdn_shared_attention_workspace_bytes(attn, cache, rows, groups), gdn.gdn_kv_workspace_bytes(cache, branches))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def step():
        gdn.gdn_kv_reserve(cache, None, old, lens, workspace=ws, status=status)
        gdn.gdn_kv_append_rope(cache, rows, rope, k, v, q, turned, status=status)
        gdn.gdn_kv_common_prefix(cache, rows, groups, status=status)
        gdn.gdn_shared_attention(attn, cache, rows, groups, turned, out, workspace=ws, status=status)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in range(8):
        qkv.copy_(rand(*qkv.shape))
        graph.replay()
        assert int(status) == 0 and groups.prefix_lens.tolist() == [prompt // page * page]
        want, spread, logits = ref.attention(turned.cpu(), pool[:, 0].cpu(), pool[:, 1].cpu(), cache.block_table.cpu(),
                                             [(i, 1) for i in range(branches)], list(range(branches)), list(range(branches)),
                                             lens.tolist(), 0.0, 0, 0)
        tol = ref.attention_tolerance(want, spread, logits, prompt + 9, dim, dtype, weight_bits(dim, dtype))
        assert torch.all((out.cpu().double() - want).abs() <= tol), t
        old += 1
        lens += 1
