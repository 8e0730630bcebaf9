"""Rotary positions, alone and on the way into the cache, against the formulas in 64 bits.  Tolerances:
``rope_reference.turn``."""
import itertools

import pytest
import torch

import gated_deltanet_linear_spec_gb300 as gdn
from tests import rope_reference as ref
from tests.test_gpu_attention import BF16, F32, i32

pytestmark = pytest.mark.gpu

FAR = [0, 1, -1, 7, 4095, 4096, 65537, 1000003, -999983, (1 << 31) - 1, -(1 << 31)]
SCALED = [dict(), dict(scaling=gdn.GDN_ROPE_LINEAR, factor=8.0), dict(scaling=gdn.GDN_ROPE_NTK, factor=4.0),
          dict(scaling=gdn.GDN_ROPE_BANDS, factor=8.0, original=2048.0),
          dict(scaling=gdn.GDN_ROPE_RAMP, factor=40.0, original=4096.0, base=1000000.0)]


def rope_of(rotary, interleaved=False, **kw):
    """The call's handle and the reference's frequencies."""
    args = {k: v for k, v in kw.items() if k != "original"}
    rope = gdn.Rope(rotary, layout=gdn.GDN_ROPE_INTERLEAVED if interleaved else gdn.GDN_ROPE_HALF,
                    original_len=kw.get("original", 0.0), **args)
    return rope, ref.frequencies(rotary, **kw)


def values(shape, dtype, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == BF16 else torch.int32)


def check(got, x, positions, freqs, interleaved):
    want, tol = ref.turn(x, positions, *freqs, interleaved)
    err = (got.cpu().double() - want).abs()
    r = 2 * len(freqs[0])
    assert torch.equal(bits(got.cpu()[..., r:]), bits(x.cpu()[..., r:]))
    assert torch.all((err <= tol)[..., :r]), float((err / tol)[..., :r].max())


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("dim,rotary", [(16, 2), (16, 16), (48, 20), (64, 32), (80, 80), (128, 128), (128, 64), (128, 90),
                                        (256, 256), (256, 64), (256, 254)])
def test_pairs_of_any_width(dim, rotary, interleaved, dtype):
    rope, freqs = rope_of(rotary, interleaved)
    x = values((len(FAR), 5, dim), dtype, seed=dim + rotary)
    out = torch.empty_like(x, device="cuda")
    gdn.gdn_rope(rope, i32(FAR), x.cuda(), out)
    check(out, x, FAR, freqs, interleaved)


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("kw", SCALED, ids=["plain", "linear", "ntk", "bands", "ramp"])
def test_scaled_frequencies(kw, interleaved):
    rope, freqs = rope_of(64, interleaved, **kw)
    positions = list(range(0, 130000, 1009))
    x = values((len(positions), 2, 128), F32)
    out = torch.empty_like(x, device="cuda")
    gdn.gdn_rope(rope, i32(positions), x.cuda(), out)
    check(out, x, positions, freqs, interleaved)


@pytest.mark.parametrize("tokens,heads,dim", [(1, 1, 16), (1, 70, 256), (2, 130, 64), (17, 33, 128), (700, 6, 128),
                                              (2500, 3, 64)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_sizes(tokens, heads, dim, dtype):
    rope, freqs = rope_of(dim)
    positions = [31 * t - 5 for t in range(tokens)]
    x = values((tokens, heads, dim), dtype)
    out = torch.empty_like(x, device="cuda")
    gdn.gdn_rope(rope, i32(positions), x.cuda(), out)
    check(out, x, positions, freqs, False)


@pytest.mark.parametrize("rotary,interleaved", [(64, False), (36, False), (64, True), (22, True)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_columns_of_wider_tensors_and_tokens_behind(rotary, interleaved, dtype):
    rope, freqs = rope_of(rotary, interleaved)
    wide = values((40, 9, 64), dtype).cuda()
    before = wide.clone()
    positions = list(range(100, 133))
    gdn.gdn_rope(rope, i32(positions), wide[:, 1:4], wide[:, 5:8])  # other columns of the same tensor
    check(wide[:33, 5:8], before[:33, 1:4].cpu(), positions, freqs, interleaved)
    assert torch.equal(bits(wide[:, :5]), bits(before[:, :5])) and torch.equal(bits(wide[:, 8:]), bits(before[:, 8:]))
    assert torch.equal(bits(wide[33:]), bits(before[33:]))
    again = before.clone()
    gdn.gdn_rope(rope, i32(positions), again[:, 1:4], again[:, 1:4])  # in place
    assert torch.equal(bits(again[:33, 1:4]), bits(wide[:33, 5:8]))
    assert torch.equal(bits(again[33:]), bits(before[33:])) and torch.equal(bits(again[:, 4:]), bits(before[:, 4:]))


def test_given_frequencies_and_magnitude():
    freqs = [0.5, 1.0, -0.25, 7.0, 1e-9, 0.0, 3.25, 2e-3]
    rope = gdn.Rope(16, frequencies=tuple(freqs), magnitude=1.25)
    positions = [0, 1, 2, 1000, -77]
    x = values((5, 3, 32), F32)
    out = torch.empty_like(x, device="cuda")
    gdn.gdn_rope(rope, i32(positions), x.cuda(), out)
    want, tol = ref.turn(x, positions, freqs, 1.25, False)
    assert torch.all((out.cpu().double() - want).abs() <= tol)


@pytest.mark.parametrize("interleaved", [False, True])
def test_values_behind_the_turned_ones_keep_their_bits(interleaved):
    rope, _ = rope_of(20, interleaved)
    x = values((3, 2, 48), BF16)
    x[..., 20:] = torch.tensor([float("nan"), float("inf"), -0.0, -float("inf")] * 7).to(BF16)
    out = torch.empty_like(x, device="cuda")
    gdn.gdn_rope(rope, i32([1, 2, 3]), x.cuda(), out)
    assert torch.equal(bits(out.cpu()[..., 20:]), bits(x[..., 20:]))


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("kw", [SCALED[0], SCALED[4]], ids=["plain", "ramp"])
def test_negated_positions_are_the_gradient(interleaved, kw):
    rope, freqs = rope_of(32, interleaved, **kw)
    positions = [3, 500, 70001]
    x, w = values((3, 2, 48), F32, 1), values((3, 2, 48), F32, 2)
    grad = torch.empty_like(x, device="cuda")
    gdn.gdn_rope(rope, i32([-p for p in positions]), w.cuda(), grad)
    check(grad, w, [-p for p in positions], freqs, interleaved)
    # against autograd of the formula in 64 bits
    x64 = x.double().requires_grad_()
    f, size = freqs
    p = torch.tensor(positions, dtype=torch.float64)[:, None] * torch.tensor(f, dtype=torch.float64)
    c, s = (size * p.cos())[:, None], (size * p.sin())[:, None]
    a, b = (x64[..., 0:32:2], x64[..., 1:32:2]) if interleaved else (x64[..., :16], x64[..., 16:32])
    u, v = (w[..., 0:32:2], w[..., 1:32:2]) if interleaved else (w[..., :16], w[..., 16:32])
    ((a * c - b * s) * u + (b * c + a * s) * v).sum().add((x64[..., 32:] * w[..., 32:]).sum()).backward()
    _, tol = ref.turn(w, [-q for q in positions], f, size, interleaved)
    assert torch.all((grad.cpu().double() - x64.grad).abs() <= tol + 1e-12)
    # against differences of the kernel itself: linear, so a step of 1 is exact but for the kernel's own roundings
    def loss(t):
        out = torch.empty_like(t, device="cuda")
        gdn.gdn_rope(rope, i32(positions), t.cuda(), out)
        return out.cpu().double()
    base, (_, t0) = loss(x), ref.turn(x, positions, f, size, interleaved)
    for token, head, e in itertools.product((0, 2), (1,), (0, 5, 17, 31, 40)):
        y = x.clone()
        y[token, head, e] += 1.0
        step = float(y[token, head, e].double() - x[token, head, e].double())
        diff = float(((loss(y) - base) * w.double()).sum()) / step
        _, t1 = ref.turn(y, positions, f, size, interleaved)
        slack = float(((t0 + t1)[token, head] * w[token, head].double().abs()).sum()) / abs(step)
        assert abs(diff - float(grad[token, head, e])) <= slack + float(tol[token, head, e])


def test_streams_and_graphs():
    rope, _ = rope_of(128)
    x = values((65, 4, 128), BF16).cuda()
    positions = i32(range(65))
    want = torch.empty_like(x)
    gdn.gdn_rope(rope, positions, x, want)
    out, other = torch.empty_like(x), torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    gdn.gdn_rope(rope, positions, x, out, stream=other)
    other.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_rope(rope, positions, x, out)
    positions += 9
    graph.replay()
    gdn.gdn_rope(rope, positions, x, want)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_no_tokens():
    rope, _ = rope_of(16)
    x = values((3, 2, 16), BF16).cuda()
    out = torch.full_like(x, 7.0)
    gdn.gdn_rope(rope, i32([]), x, out)
    assert torch.all(out == 7.0)


# ------------------------------------------------------------------------------------------
# on the way into the cache

class Batch:
    """Rows over a shuffled pool; the pool holds 5 where nothing is written."""

    def __init__(self, rows, dtype=BF16, heads=4, kv_heads=2, dim=64, page=16, gather=True, null=(), shared=(), seed=0):
        gen = torch.Generator().manual_seed(seed)
        need = [-(-kv // page) for _, kv in rows]
        pages = 2 + sum(need)
        ids = (1 + torch.randperm(pages - 1, generator=gen)).tolist()
        self.table = torch.zeros(len(rows) + 1, max(need + [1]), dtype=torch.int32)
        self.table_rows = torch.randperm(len(rows) + 1, generator=gen)[:len(rows)].tolist()
        for r, n in zip(self.table_rows, need):
            for e in range(n):
                self.table[r, e] = ids.pop()
        count = torch.ones(pages, dtype=torch.int32)
        for i, e in null:
            self.table[self.table_rows[i], e] = 0
        for i, e in shared:
            count[self.table[self.table_rows[i], e]] = 2
        self.rows, self.page, self.dim = rows, page, dim
        self.starts = [0]
        for new, _ in rows:
            self.starts.append(self.starts[-1] + new)
        total = self.starts[-1]
        self.token = torch.randperm(total + 3, generator=gen)[:total].tolist() if gather else list(range(total))
        n = total + 3
        self.qkv = torch.randn(n, heads + 2 * kv_heads + 1, dim, generator=gen).to(dtype)
        self.q, self.k, self.v, _ = self.qkv.cuda().split([heads, kv_heads, kv_heads, 1], 1)
        self.k_pool = torch.full((pages, kv_heads, page, dim), 5.0, dtype=dtype, device="cuda")
        self.v_pool = torch.full_like(self.k_pool, 5.0)
        self.cache = gdn.KvCache(self.k_pool, self.v_pool, self.table.cuda(), count.cuda())
        self.max_q = max([new for new, _ in rows] + [1])
        self.kv_rows = gdn.KvRows(i32(self.starts), total, i32([kv for _, kv in rows]), self.max_q, i32(self.table_rows),
                                  i32(self.token) if gather else None)

    def positions(self):
        """(global token, position, page, slot) of every new token."""
        for i, (new, kv) in enumerate(self.rows):
            for t in range(new):
                pos = kv - new + t
                yield self.token[self.starts[i] + t], pos, int(self.table[self.table_rows[i], pos // self.page]), pos % self.page


ROWS = [(1, 1), (4, 4), (0, 9), (3, 64), (2, 33), (5, 200), (0, 0), (1, 129)]


@pytest.mark.parametrize("dim,rotary,interleaved", [(64, 64, False), (128, 32, False), (128, 128, True), (256, 64, False),
                                                    (48, 28, False), (48, 28, True)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("gather", [True, False], ids=["gather", "identity"])
def test_append(dim, rotary, interleaved, dtype, gather):
    b = Batch(ROWS, dtype, dim=dim, gather=gather, seed=dim)
    rope, freqs = rope_of(rotary, interleaved)
    status, out = i32([0]), torch.full_like(b.q.contiguous(), 7.0)
    gdn.gdn_kv_append_rope(b.cache, b.kv_rows, rope, b.k, b.v, b.q, out, status=status)
    assert int(status) == 0
    at = list(b.positions())
    token, pos = [t for t, *_ in at], [p for _, p, *_ in at]
    check(out[token], b.q[token].cpu(), pos, freqs, interleaved)
    page, slot = [p for *_, p, _ in at], [s for *_, s in at]
    check(b.k_pool[page, :, slot], b.k[token].cpu(), pos, freqs, interleaved)
    assert torch.equal(b.v_pool[page, :, slot], b.v[token])
    rest = torch.ones(out.shape[0], dtype=torch.bool)
    rest[token] = False
    assert torch.all(out[rest.cuda()] == 7.0)
    keep = torch.ones(b.k_pool.shape[0], b.page, dtype=torch.bool)
    keep[page, slot] = False
    for pool in (b.k_pool, b.v_pool):
        assert torch.all(pool.transpose(1, 2)[keep.cuda()] == 5.0)


@pytest.mark.parametrize("rows", [[(700, 700), (133, 1000)], [(1, 50)] * 70, [(1, 3)]], ids=["prompts", "decode", "one"])
def test_append_is_rope_and_append(rows):
    a, b = Batch(rows, heads=8, dim=128, seed=3), Batch(rows, heads=8, dim=128, seed=3)
    rope, _ = rope_of(128, base=500000.0)
    gdn.gdn_kv_append_rope(a.cache, a.kv_rows, rope, a.k, a.v, a.q)  # q in place, beside k and v in one tensor
    positions = torch.zeros(b.q.shape[0], dtype=torch.int32)
    for token, pos, *_ in b.positions():
        positions[token] = pos
    used = torch.tensor(b.token)
    gdn.gdn_rope(rope, positions.cuda(), b.q, b.q)
    k = torch.empty_like(b.k.contiguous())
    gdn.gdn_rope(rope, positions.cuda(), b.k, k)
    gdn.gdn_kv_append(b.cache, b.kv_rows, k, b.v)
    assert torch.equal(a.q.cpu()[used], b.q.cpu()[used])
    assert torch.equal(a.k_pool, b.k_pool) and torch.equal(a.v_pool, b.v_pool)
    unused = torch.ones(a.q.shape[0], dtype=torch.bool)
    unused[used] = False
    assert torch.equal(a.q.cpu()[unused], a.qkv[unused, :8])
    c = Batch(rows, heads=8, dim=128, seed=3)
    gdn.gdn_kv_append_rope(c.cache, c.kv_rows, rope, c.k, c.v)  # keys and values only
    assert torch.equal(c.k_pool, b.k_pool) and torch.equal(c.v_pool, b.v_pool)


def test_pages_that_are_not_written():
    """A NULL entry, a page that two rows hold, a token out of range: the rest is written, queries of all good tokens turn."""
    b = Batch([(3, 20), (2, 40), (4, 18)], null=[(0, 1)], shared=[(1, 2)])
    rope, freqs = rope_of(64)
    token = list(b.token)
    bad = token[6]
    rows = gdn.KvRows(b.kv_rows.query_start_loc, b.kv_rows.num_tokens, b.kv_rows.kv_lens, 4, b.kv_rows.table_rows,
                      i32(token[:6] + [b.q.shape[0] + 5] + token[7:]))
    status, out = i32([0]), torch.full_like(b.q.contiguous(), 7.0)
    gdn.gdn_kv_append_rope(b.cache, rows, rope, b.k, b.v, b.q, out, status=status)
    assert int(status) == gdn.STATUS_PAGE_SHARED | gdn.STATUS_TOKEN_RANGE
    for i, (t, pos, page, slot) in enumerate(b.positions()):
        if i == 6:
            assert t == bad and torch.all(out[t] == 7.0)
            assert torch.all(b.k_pool[page, :, slot] == 5.0)
            continue
        check(out[[t]], b.q[[t]].cpu(), [pos], freqs, False)
        held = page > 0 and i not in (3, 4)  # (row 1's last page has two holders)
        if page > 0:
            assert torch.equal(b.v_pool[page, :, slot], b.v[t]) == held
            assert bool(torch.all(b.k_pool[page, :, slot] == 5.0)) == (not held)
    assert torch.all(b.k_pool[0] == 5.0)


@pytest.mark.parametrize("starts,lens", [([0, 2, 9, 6], [20, 20, 20]), ([0, 2, 4, 6], [20, 1, 20]),
                                         ([0, 2, 4, 6], [20, 4000, 20])])
def test_a_bad_row_is_left_out(starts, lens):
    b = Batch([(2, 20)] * 3, gather=False)
    rope, _ = rope_of(64)
    rows = gdn.KvRows(i32(starts), 6, i32(lens), 2, b.kv_rows.table_rows)
    status, out = i32([0]), torch.full_like(b.q.contiguous(), 7.0)
    gdn.gdn_kv_append_rope(b.cache, rows, rope, b.k, b.v, b.q, out, status=status)
    assert int(status) & gdn.STATUS_ROW_RANGE
    assert not torch.any(out[:2] == 7.0) and torch.all(out[2:4] == 7.0)


def test_append_in_a_graph():
    b = Batch([(2, 30)] * 9, heads=8, dim=128)
    rope, _ = rope_of(128)
    out = torch.zeros_like(b.q.contiguous())
    gdn.gdn_kv_append_rope(b.cache, b.kv_rows, rope, b.k, b.v, b.q, out)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        gdn.gdn_kv_append_rope(b.cache, b.kv_rows, rope, b.k, b.v, b.q, out)
    b.kv_rows.kv_lens.sub_(3)
    b.k_pool.fill_(5.0)
    graph.replay()
    graph.replay()
    got, pool = out.clone(), b.k_pool.clone()
    out.zero_()
    b.k_pool.fill_(5.0)
    gdn.gdn_kv_append_rope(b.cache, b.kv_rows, rope, b.k, b.v, b.q, out)
    assert torch.equal(got, out) and torch.equal(pool, b.k_pool)


def test_more_heads_than_quotients_of_a_block_of_tokens_hold():
    """33308 heads: the last of a block's fourth token would be taken for one of a fifth.  Against calls of so few tokens that a
    block has one."""
    tokens, heads, dim = 2432, 33308, 16
    rope = gdn.Rope(dim)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(tokens, heads, dim, generator=gen, device="cuda", dtype=torch.bfloat16)
    positions = torch.arange(tokens, dtype=torch.int32, device="cuda")
    got = torch.full_like(x, 7.0)
    gdn.gdn_rope(rope, positions, x, got)
    for at in range(0, tokens, 608):
        part = slice(at, at + 608)
        want = torch.empty_like(x[part])
        gdn.gdn_rope(rope, positions[part], x[part], want)
        assert torch.equal(got[part], want)
