"""The paged cache's entry points on the host (no GPU needed): malformed calls return the
documented code before anything is enqueued, empty ones return 0, workspace sizes follow their
closed forms, and the binding refuses tensors that a descriptor cannot describe.

Every call below fails validation or has nothing to do, so no kernel is ever launched with the
fake pointers used here (on a GPU machine as well as without one).
"""
import ctypes
import os

import pytest
import torch

import gated_deltanet_linear_spec_gb300 as gdn
from gated_deltanet_linear_spec_gb300 import _AttnDesc, _KvCache, _KvRows, _LayerDesc, _Pools

FAKE = 0x100000
NULL_ARG, SHAPE, WORKSPACE, DTYPE, ALIGN = -1, -3, -5, -6, -8


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(gdn.LIB_PATH):
        from gated_deltanet_linear_spec_gb300 import build
        build.build()
    return gdn.library()


def cache(**kw):
    d = dict(k_pool=FAKE, v_pool=FAKE, page_stride=0, block_table=FAKE, refcount=FAKE, num_pages=100,
             num_table_rows=8, max_pages=16, page_size=16, num_kv_heads=2, head_dim=64, dtype=gdn.GDN_BF16)
    d.update(kw)
    return _KvCache(**d)


def rows(**kw):
    d = dict(num_seqs=4, num_tokens=12, query_start_loc=FAKE, token_indx=None, table_rows=None, kv_lens=FAKE,
             max_query_len=3)
    d.update(kw)
    return _KvRows(**d)


def attn(**kw):
    d = dict(num_q_heads=8, scale=0.0, window=0, num_sinks=0)
    d.update(kw)
    return _AttnDesc(**d)


def R(x):
    return None if x is None else ctypes.byref(x)


BAD_CACHE = [
    (dict(dtype=7), DTYPE), (dict(num_pages=1), SHAPE), (dict(num_pages=(1 << 28) + 1), SHAPE),
    (dict(page_size=8), SHAPE), (dict(page_size=24), SHAPE), (dict(page_size=512), SHAPE),
    (dict(num_kv_heads=0), SHAPE), (dict(num_kv_heads=1025), SHAPE), (dict(head_dim=8), SHAPE),
    (dict(head_dim=72), SHAPE), (dict(head_dim=272), SHAPE), (dict(page_stride=2 * 16 * 64 - 16), SHAPE),
    (dict(page_stride=-16), SHAPE), (dict(page_stride=2 * 16 * 64 + 4), ALIGN),
    (dict(page_stride=2 * 16 * 64 + 64), SHAPE), (dict(page_stride=1 << 38), SHAPE),
    (dict(page_stride=1 << 33, num_pages=1 << 20), SHAPE),
]
BAD_TABLE = [(dict(block_table=None), NULL_ARG), (dict(num_table_rows=0), SHAPE), (dict(max_pages=0), SHAPE),
             (dict(max_pages=(1 << 20) + 1), SHAPE)]
BAD_POOLS = [(dict(k_pool=None), NULL_ARG), (dict(v_pool=None), NULL_ARG), (dict(k_pool=FAKE + 8), ALIGN),
             (dict(v_pool=FAKE + 2), ALIGN)]
BAD_ROWS = [(dict(num_seqs=-1), SHAPE), (dict(num_tokens=-1), SHAPE), (dict(num_seqs=65536), SHAPE),
            (dict(num_seqs=0), SHAPE), (dict(query_start_loc=None), NULL_ARG), (dict(kv_lens=None), NULL_ARG),
            (dict(max_query_len=-1), SHAPE)]


def call_append(lib, c, r, k=FAKE, ks=0, v=FAKE, vs=0, n=12):
    return lib.gdn_kv_append(R(c), R(r), k, ks, v, vs, n, None, None)


def call_attention(lib, a, c, r, q=FAKE, qs=0, n=12, out=FAKE, os_=0, ws=FAKE, nbytes=1 << 40):
    return lib.gdn_paged_attention(R(a), R(c), R(r), q, qs, n, out, os_, ws, nbytes, None, None)


@pytest.mark.parametrize("kw,code", BAD_CACHE + BAD_TABLE + BAD_POOLS)
def test_bad_caches(lib, kw, code):
    c = cache(**kw)
    assert call_append(lib, c, rows()) == code
    assert call_attention(lib, attn(), c, rows()) == code


@pytest.mark.parametrize("kw,code", BAD_CACHE + BAD_TABLE + [(dict(refcount=None), NULL_ARG)])
def test_bad_caches_of_the_page_calls(lib, kw, code):
    c = cache(**kw)
    big = 1 << 40
    assert lib.gdn_kv_reserve(R(c), 2, FAKE, FAKE, FAKE, FAKE, big, None, None) == code
    assert lib.gdn_kv_release(R(c), 2, FAKE, FAKE, FAKE, None, None) == code
    assert lib.gdn_kv_fork(R(c), 2, FAKE, FAKE, FAKE, FAKE, big, None, None) == code
    assert lib.gdn_kv_compact(R(c), None, FAKE, big, None, None) == code


@pytest.mark.parametrize("kw,code", BAD_ROWS)
def test_bad_rows(lib, kw, code):
    assert call_append(lib, cache(), rows(**kw)) == code
    assert call_attention(lib, attn(), cache(), rows(**kw)) == code


def test_null_descriptors(lib):
    assert call_append(lib, None, rows()) == NULL_ARG
    assert call_append(lib, cache(), None) == NULL_ARG
    assert call_attention(lib, None, cache(), rows()) == NULL_ARG
    assert call_attention(lib, attn(), None, rows()) == NULL_ARG
    assert call_attention(lib, attn(), cache(), None) == NULL_ARG


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), NULL_ARG), (dict(v=None), NULL_ARG), (dict(k=FAKE + 2), ALIGN), (dict(v=FAKE + 8), ALIGN),
    (dict(n=-1), SHAPE), (dict(n=11), SHAPE), (dict(ks=127), SHAPE), (dict(vs=64), SHAPE), (dict(ks=132), SHAPE),
    (dict(vs=-128), SHAPE)])
def test_bad_appends(lib, kw, code):
    assert call_append(lib, cache(), rows(), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), NULL_ARG), (dict(out=None), NULL_ARG), (dict(q=FAKE + 2), ALIGN), (dict(out=FAKE + 4), ALIGN),
    (dict(n=-1), SHAPE), (dict(n=11), SHAPE), (dict(qs=511), SHAPE), (dict(os_=516), SHAPE)])
def test_bad_attention_calls(lib, kw, code):
    assert call_attention(lib, attn(), cache(), rows(), **kw) == code


@pytest.mark.parametrize("kw", [dict(num_q_heads=0), dict(num_q_heads=7), dict(num_q_heads=65536), dict(num_sinks=-1),
                                dict(scale=float("nan")), dict(scale=float("inf"))])
def test_bad_attention_descriptors(lib, kw):
    assert call_attention(lib, attn(**kw), cache(), rows()) == SHAPE


def test_attention_workspace_is_asked_for(lib):
    for r in (rows(), rows(max_query_len=500, num_tokens=700)):
        need = lib.gdn_attention_workspace_bytes(R(attn()), R(cache()), R(r))
        if need:
            n = r.num_tokens
            assert call_attention(lib, attn(), cache(), r, n=n, ws=None) == WORKSPACE
            assert call_attention(lib, attn(), cache(), r, n=n, nbytes=need - 1) == WORKSPACE
            assert call_attention(lib, attn(), cache(), r, n=n, ws=FAKE + 128) == ALIGN
    assert lib.gdn_attention_workspace_bytes(R(attn(num_q_heads=7)), R(cache()), R(rows())) == 0


def test_page_calls_refuse(lib):
    c = cache()
    need = lib.gdn_kv_workspace_bytes(R(c), 3)
    ints = 5 * 3 + 1 + 4 + 2 * 100
    assert need == (4 * ints + 255) // 256 * 256
    assert lib.gdn_kv_workspace_bytes(R(c), -1) == 0
    assert lib.gdn_kv_workspace_bytes(R(cache(page_size=7)), 3) == 0
    res = lambda *a: lib.gdn_kv_reserve(R(c), *a, None, None)  # noqa: E731
    fork = lambda *a: lib.gdn_kv_fork(R(c), *a, None, None)  # noqa: E731
    assert res(-1, FAKE, FAKE, FAKE, FAKE, need) == SHAPE
    assert res(3, FAKE, None, FAKE, FAKE, need) == NULL_ARG
    assert res(3, FAKE, FAKE, None, FAKE, need) == NULL_ARG
    assert res(3, FAKE, FAKE, FAKE, None, need) == WORKSPACE
    assert res(3, FAKE, FAKE, FAKE, FAKE, need - 1) == WORKSPACE
    assert res(3, FAKE, FAKE, FAKE, FAKE + 64, need) == ALIGN
    assert res(0, None, None, None, None, 0) == 0
    assert fork(-1, FAKE, FAKE, FAKE, FAKE, need) == SHAPE
    for i in range(3):
        args = [FAKE, FAKE, FAKE]
        args[i] = None
        assert fork(3, *args, FAKE, need) == NULL_ARG
    assert fork(3, FAKE, FAKE, FAKE, FAKE, 16) == WORKSPACE
    assert fork(0, None, None, None, None, 0) == 0
    assert lib.gdn_kv_fork(R(cache(v_pool=None)), 3, FAKE, FAKE, FAKE, FAKE, need, None, None) == NULL_ARG
    assert lib.gdn_kv_release(R(c), -1, FAKE, None, None, None, None) == SHAPE
    assert lib.gdn_kv_release(R(c), 0, None, None, None, None, None) == 0
    assert lib.gdn_kv_compact(R(c), None, None, 1 << 20, None, None) == WORKSPACE
    assert lib.gdn_kv_compact(R(c), None, FAKE, 8, None, None) == WORKSPACE
    assert lib.gdn_kv_compact(R(c), None, FAKE + 16, 1 << 20, None, None) == ALIGN
    assert lib.gdn_kv_compact(R(cache(k_pool=FAKE + 4)), None, FAKE, 1 << 20, None, None) == ALIGN


def test_copies_refuse(lib):
    c = cache(block_table=None, refcount=None)
    assert lib.gdn_kv_copy_pages(R(c), 0, None, None, None, None) == 0
    assert lib.gdn_kv_copy_pages(R(c), -2, FAKE, FAKE, None, None) == SHAPE
    assert lib.gdn_kv_copy_pages(R(c), 2, None, FAKE, None, None) == NULL_ARG
    assert lib.gdn_kv_copy_pages(R(c), 2, FAKE, None, None, None) == NULL_ARG
    assert lib.gdn_kv_copy_pages(R(cache(k_pool=None)), 2, FAKE, FAKE, None, None) == NULL_ARG
    layer = _LayerDesc(2, 4, 16, 16, 4, 5, gdn.GDN_F32, 0.0, 0, 0)
    pools = _Pools(FAKE, FAKE, 16)
    slots = lambda ly, po, n=2, s=FAKE, t=FAKE: lib.gdn_copy_slots(R(ly), R(po), n, s, t, None, None)  # noqa: E731
    assert slots(None, pools) == NULL_ARG
    assert slots(layer, None) == NULL_ARG
    assert slots(_LayerDesc(2, 3, 16, 16, 4, 5, gdn.GDN_F32, 0.0, 0, 0), pools) == SHAPE
    assert slots(layer, _Pools(FAKE, None, 16)) == NULL_ARG
    assert slots(layer, _Pools(FAKE + 4, FAKE, 16)) == ALIGN
    assert slots(layer, _Pools(FAKE, FAKE, 0)) == SHAPE
    assert slots(layer, _Pools(FAKE, FAKE, 1 << 31)) == SHAPE
    assert slots(layer, pools, -1) == SHAPE
    assert slots(layer, pools, 2, None) == NULL_ARG
    assert slots(layer, pools, 0, None, None) == 0


def test_nothing_to_do(lib):
    empty = rows(num_seqs=0, num_tokens=0, query_start_loc=None, kv_lens=None)
    assert call_append(lib, cache(), empty, k=None, v=None, n=0) == 0
    assert call_attention(lib, attn(), cache(), empty, q=None, out=None, n=0, ws=None, nbytes=0) == 0
    assert call_append(lib, cache(), rows(num_tokens=0), k=None, v=None, n=0) == 0


def test_binding_refuses_host_tensors():
    t = torch.zeros(4, 2, 16, 64)
    with pytest.raises(TypeError):
        gdn.KvCache(t, t, torch.zeros(2, 2, dtype=torch.int32))
    with pytest.raises(TypeError):
        gdn.KvRows(torch.zeros(3, dtype=torch.int32), 0, torch.zeros(2, dtype=torch.int32), 1)
