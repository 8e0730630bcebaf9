"""The page calls against sequential loops over lists: tables, counts and data have to be equal."""
import random

import pytest
import torch

import gated_deltanet_linear_spec_gb300 as gdn
from tests import kv_reference as ref

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Pool:
    def __init__(self, pages, rows, width, page=16, heads=1, dim=16, dtype=torch.bfloat16, seed=0, interleaved=False):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        both = torch.randn(pages, 2, heads, page, dim, generator=gen, device="cuda").to(dtype)
        self.k, self.v = (both[:, 0], both[:, 1]) if interleaved else (both[:, 0].clone(), both[:, 1].clone())
        self.table = torch.zeros(rows, width, dtype=torch.int32, device="cuda")
        self.count = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.cache = gdn.KvCache(self.k, self.v, self.table, self.count)
        self.ref = ref.Pages(self.table.tolist(), self.count.tolist(), page)
        self.want_k, self.want_v = self.k.clone(), self.v.clone()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def load(self):
        self.table.copy_(torch.tensor(self.ref.table, dtype=torch.int32))
        self.count.copy_(torch.tensor(self.ref.count, dtype=torch.int32))

    def same(self):
        torch.cuda.synchronize()
        assert self.table.tolist() == self.ref.table
        assert self.count.tolist() == self.ref.count
        assert int(self.status) == self.ref.status
        assert torch.equal(self.k, self.want_k) and torch.equal(self.v, self.want_v)

    def reserve(self, rows, a, b):
        gdn.gdn_kv_reserve(self.cache, None if rows is None else i32(rows), i32(a), i32(b), status=self.status)
        self.ref.reserve(range(len(a)) if rows is None else rows, a, b)

    def release(self, rows, a=None, b=None):
        gdn.gdn_kv_release(self.cache, i32(rows), None if a is None else i32(a), None if b is None else i32(b),
                           status=self.status)
        self.ref.release(rows, a or [0] * len(rows), b or [self.table.shape[1]] * len(rows))

    def fork(self, src, dst, lens):
        gdn.gdn_kv_fork(self.cache, i32(src), i32(dst), i32(lens), status=self.status)
        for old, new, n in self.ref.fork(src, dst, lens):
            self.want_k[new, :, :n] = self.want_k[old, :, :n]
            self.want_v[new, :, :n] = self.want_v[old, :, :n]

    def compact(self):
        live = i32([-5])
        gdn.gdn_kv_compact(self.cache, live, status=self.status)
        moves, m = self.ref.compact()
        if moves:
            a, b = (torch.tensor(x, device="cuda") for x in zip(*moves))
            self.want_k[b] = self.want_k[a]
            self.want_v[b] = self.want_v[a]
        assert int(live) == m


@pytest.mark.parametrize("pages,rows,width,page", [(40, 6, 5, 16), (300, 20, 33, 32), (4096, 64, 70, 16), (9000, 300, 40, 64)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_random_histories(pages, rows, width, page, dtype):
    rng = random.Random(pages)
    P = Pool(pages, rows, width, page, heads=1 + pages % 3, dim=16 if pages > 1000 else 80, dtype=dtype, seed=pages,
             interleaved=pages % 2 == 0)
    lens = [0] * rows
    for step in range(14):
        kind = rng.choice(["reserve", "reserve", "release", "rollback", "fork", "compact", "window"])
        some = rng.sample(range(rows), rng.randint(1, rows))
        if kind == "reserve":
            to = [min(width * page, lens[r] + rng.randint(0, 3 * page)) for r in some]
            before = [list(r) for r in P.ref.table]
            P.reserve(some, [lens[r] for r in some], to)
            for r, n in zip(some, to):
                got = all(P.ref.table[r][e] > 0 for e in range(-(-lens[r] // page), -(-n // page)))
                lens[r] = n if got else lens[r]
            assert before is not None
        elif kind == "release":
            P.release(some)
            for r in some:
                lens[r] = 0
        elif kind == "rollback":
            keep = [rng.randint(0, lens[r]) for r in some]
            P.release(some, [-(-n // page) for n in keep])
            for r, n in zip(some, keep):
                lens[r] = n
        elif kind == "window":
            P.release(some, [0] * len(some), [rng.randint(0, lens[r] // page) for r in some])
        elif kind == "fork":
            dst = [r for r in some if lens[r] == 0 and not any(P.ref.table[r])]
            src = [r for r in range(rows) if r not in dst]
            if not dst or not src:
                continue
            pairs = [(rng.choice(src), r) for r in dst]
            n = [rng.randint(0, lens[s]) for s, _ in pairs]
            P.fork([s for s, _ in pairs], dst, n)
            for (s, r), m in zip(pairs, n):
                full = [P.ref.table[r][e] == P.ref.table[s][e] for e in range(m // page)]
                lens[r] = m if all(full) and (m % page == 0 or P.ref.table[r][m // page] > 0) else 0
        else:
            P.compact()
        P.same()
        if P.ref.status & ref.NO_PAGES:
            P.ref.status &= ~ref.NO_PAGES
            P.status.zero_()


def test_a_row_gets_all_or_nothing():
    P = Pool(12, 5, 8)  # 11 pages to hand out
    P.reserve([3, 0, 4, 1], [0, 0, 0, 0], [16 * 4, 16 * 8, 16 * 2, 16])
    P.same()
    assert P.ref.status == ref.NO_PAGES
    assert sum(P.ref.count) == 4  # row 0's eight did not fit behind row 3's four, nor what came after it


def test_reserve_keeps_what_a_row_holds():
    P = Pool(30, 3, 8)
    P.reserve(None, [0, 0, 0], [20, 0, 100])
    P.same()
    P.release([2], [3], [5])
    P.reserve([2], [0], [128])  # fills the gap, keeps the rest
    P.same()
    P.reserve([0], [17], [32])  # inside the last page: nothing needed
    P.same()


def test_full_and_empty_pools():
    P = Pool(9, 2, 8)
    P.compact()
    P.same()
    P.reserve([1], [0], [128])
    P.compact()
    P.same()
    P.fork([1], [0], [100])  # no page left for the partly filled one
    P.same()
    assert P.ref.status == ref.NO_PAGES
    P.release([1])
    P.compact()
    P.same()


def test_forks_of_a_fork():
    P = Pool(64, 6, 8, heads=3, dim=48)
    P.reserve([0], [0], [75])
    P.fork([0, 0, 0], [1, 2, 3], [75, 64, 5])
    P.same()
    P.fork([1, 3], [4, 5], [70, 0])
    P.same()
    P.release([0, 1, 2, 3, 4, 5])
    P.same()
    assert not any(P.ref.count)


def test_null_entries_stay_null_in_a_fork():
    P = Pool(64, 4, 8)
    P.reserve([0, 1], [0, 0], [100, 100])
    P.release([0, 1], [1, 6], [3, 7])  # row 1 loses its partly filled page
    P.fork([0, 1], [2, 3], [100, 100])
    P.same()
    assert P.ref.table[2][1:3] == [0, 0] and P.ref.table[3][6] == 0


def test_page_calls_skip_bad_rows():
    P = Pool(64, 4, 8)
    P.reserve([0, 9, 1, -1, 2], [0, 0, -3, 0, 0], [50, 50, 50, 50, 129])
    P.same()
    P.release([0, 7], [0, 0], [2, 2])
    P.release([0, 1], [-1, 0], [2, 9])
    P.same()
    P.reserve([1], [0], [40])
    P.fork([1, 1, 5, 1], [0, 2, 3, 3], [40, 500, 10, 33])  # row 0 still holds pages
    P.same()
    assert P.ref.status == ref.PAGE_RANGE


def test_bad_entries_are_reported():
    P = Pool(32, 3, 4)
    P.reserve([0], [0], [64])
    P.ref.table[0][1] = 4000
    P.ref.table[0][2] = 30  # a page that nobody holds
    P.load()
    P.fork([0], [1], [64])
    P.same()
    P.release([0])
    P.same()
    assert P.ref.status == ref.PAGE_RANGE


def test_copy_pages():
    P = Pool(50, 1, 1, heads=2, dim=64, interleaved=True)
    src, dst = [3, 7, 0, 12, 60, 9, 11], [20, 21, 22, 0, 23, 90, 11]
    gdn.gdn_kv_copy_pages(gdn.KvCache(P.k, P.v, P.table), i32(src), i32(dst), status=P.status)
    for a, b in [(3, 20), (7, 21)]:
        P.want_k[b], P.want_v[b] = P.want_k[a], P.want_v[a]
    assert torch.equal(P.k, P.want_k) and torch.equal(P.v, P.want_v)
    assert int(P.status) == ref.PAGE_RANGE


@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("conv", [True, False])
def test_copy_slots(act, conv):
    layer = gdn.Layer(2, 4, 16, 32, 4, 5, act)
    gen = torch.Generator(device="cuda").manual_seed(1)
    ssm = torch.randn(12, 4, 32, 16, generator=gen, device="cuda")
    ring = torch.randn(12, 5, layer.channels, generator=gen, device="cuda").to(act)
    want, want_ring = ssm.clone(), ring.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    src, dst = [1, 2, 0, 4, 13, 5], [7, 8, 9, 0, 10, -1]
    gdn.gdn_copy_slots(layer, gdn.Pools(ring if conv else None, ssm), i32(src), i32(dst), status=status)
    for a, b in [(1, 7), (2, 8)]:
        want[b], want_ring[b] = want[a], want_ring[a]
    want[9], want_ring[9] = 0, 0
    assert torch.equal(ssm, want)
    assert torch.equal(ring, want_ring if conv else ring)
    assert int(status) == ref.SLOT_RANGE


def test_pages_in_a_graph():
    """reserve, append, fork and release captured once and replayed: no call needs the host."""
    P = Pool(200, 8, 10, heads=2, dim=64)
    k = torch.randn(40, 2, 64, device="cuda").to(torch.bfloat16)
    ws = torch.empty(gdn.gdn_kv_workspace_bytes(P.cache, 8), dtype=torch.uint8, device="cuda")
    zero, forty, row0 = i32([0]), i32([40]), i32([0])
    src, dst, lens = i32([0, 0, 0]), i32([2, 4, 6]), i32([40, 33, 16])
    rows = gdn.KvRows(i32([0, 40]), 40, i32([40]), 40)

    def step():
        gdn.gdn_kv_release(P.cache, i_all, status=P.status)
        gdn.gdn_kv_reserve(P.cache, row0, zero, forty, workspace=ws, status=P.status)
        gdn.gdn_kv_append(P.cache, rows, k, -k, status=P.status)
        gdn.gdn_kv_fork(P.cache, src, dst, lens, workspace=ws, status=P.status)

    i_all = i32(list(range(8)))
    step()
    want = [t.clone() for t in (P.table, P.count, P.k, P.v)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for got, w in zip((P.table, P.count, P.k, P.v), want):
        assert torch.equal(got, w)
    assert int(P.status) == 0


@pytest.mark.parametrize("pages", [131072, 131073, 135000])
def test_pools_on_both_sides_of_one_launch(pages):
    """Up to 131072 pages are handed out in one launch, more in three; here only far pages are free."""
    P = Pool(pages, 40, 24, page=16, dim=16)
    free = {1, 5000, 70000} | set(range(pages - 120, pages))
    P.ref.count = [0 if i in free or i == 0 else 1 for i in range(pages)]
    P.load()
    rng = random.Random(pages)
    lens = [rng.randint(0, 60) for _ in range(30)]
    P.reserve(list(range(30)), [0] * 30, lens)
    P.same()
    src = [r for r in range(30) if lens[r]][:10]
    P.fork(src, list(range(30, 40)), [lens[r] for r in src])
    P.same()
    P.release(src)
    P.reserve(src + [35], [0] * 11, [24 * 16] * 11)  # more than is left
    P.same()
    assert P.ref.status == ref.NO_PAGES


@pytest.mark.parametrize("pages", [131072, 131073])
def test_compaction_of_large_pools(pages):
    P = Pool(pages, 30, 24, page=16, dim=16)
    held = {1, 2, 77, 5000, 70000, 131071} | set(range(pages - 90, pages))
    P.ref.count = [0 if i in held or i == 0 else 1 for i in range(pages)]
    P.load()
    P.reserve(list(range(30)), [0] * 30, [40] * 30)  # every row holds some of the free pages, low and far ones
    P.ref.count = [n if i in held else 0 for i, n in enumerate(P.ref.count)]
    P.load()
    P.same()
    P.compact()
    P.same()
