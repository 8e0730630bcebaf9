"""Rotary positions and shared prefixes on the host (no GPU needed): malformed calls return the documented code before
anything is enqueued, empty ones return 0, frequencies follow their formulas, and the binding refuses what a descriptor cannot
say.

Every call below fails validation or has nothing to do, so no kernel is ever launched with the fake pointers used here (on
a GPU machine as well as without one).
"""
import ctypes
import math

import pytest
import torch

import gated_deltanet_linear_spec_gb300 as gdn
from gated_deltanet_linear_spec_gb300 import _KvGroups, _RopeDesc, _RopeFreq
from tests import rope_reference as ref
from tests.test_kv_binding import cache as dev_cache
from tests.test_kv_binding import dev, i32
from tests.test_kv_binding import rows as dev_rows
from tests.test_kv_refusals import (ALIGN, BAD_CACHE, BAD_POOLS, BAD_ROWS, BAD_TABLE, DTYPE, FAKE, NULL_ARG, SHAPE, WORKSPACE, R,
                                    attn, cache, lib, rows)  # noqa: F401  (lib is a fixture)

BIG = 1 << 40


def groups(**kw):
    d = dict(num_groups=2, group_start_loc=FAKE, prefix_lens=FAKE)
    d.update(kw)
    return _KvGroups(**d)


def rope(**kw):
    d = dict(turns=FAKE, rotary_dim=64, layout=0, magnitude=0.0)
    d.update(kw)
    return _RopeDesc(**d)


def call_shared(lib, a, c, r, g, q=FAKE, qs=0, n=12, out=FAKE, os_=0, ws=FAKE, nbytes=BIG):  # noqa: F811
    return lib.gdn_shared_attention(R(a), R(c), R(r), R(g), q, qs, n, out, os_, ws, nbytes, None, None)


def call_append(lib, c, r, t, k=FAKE, ks=0, v=FAKE * 2, vs=0, hq=8, q=FAKE * 3, qs=0, out=FAKE * 4, os_=0, n=12):  # noqa: F811
    return lib.gdn_kv_append_rope(R(c), R(r), R(t), k, ks, v, vs, hq, q, qs, out, os_, n, None, None)


def call_rope(lib, t, heads=4, dim=64, dtype=gdn.GDN_BF16, pos=FAKE, n=10, x=FAKE, xs=0, out=FAKE * 2, os_=0):  # noqa: F811
    return lib.gdn_rope(R(t), heads, dim, dtype, pos, n, x, xs, out, os_, None)


@pytest.mark.parametrize("kw,code", BAD_CACHE + BAD_TABLE + BAD_POOLS)
def test_bad_caches(lib, kw, code):  # noqa: F811
    assert call_shared(lib, attn(), cache(**kw), rows(), groups()) == code
    assert call_append(lib, cache(**kw), rows(), rope()) == code
    if (kw, code) not in BAD_POOLS:
        assert lib.gdn_kv_common_prefix(R(cache(**kw)), R(rows()), R(groups()), None, None) == code


@pytest.mark.parametrize("kw,code", BAD_ROWS)
def test_bad_rows(lib, kw, code):  # noqa: F811
    assert call_shared(lib, attn(), cache(), rows(**kw), groups()) == code
    assert call_append(lib, cache(), rows(**kw), rope()) == code
    assert lib.gdn_kv_common_prefix(R(cache()), R(rows(**kw)), R(groups()), None, None) == code


@pytest.mark.parametrize("kw,code", [(dict(num_groups=-1), SHAPE), (dict(num_groups=65536), SHAPE),
                                     (dict(group_start_loc=None), NULL_ARG), (dict(prefix_lens=None), NULL_ARG)])
def test_bad_groups(lib, kw, code):  # noqa: F811
    assert call_shared(lib, attn(), cache(), rows(), groups(**kw)) == code
    assert lib.gdn_kv_common_prefix(R(cache()), R(rows()), R(groups(**kw)), None, None) == code
    assert lib.gdn_shared_attention_workspace_bytes(R(attn()), R(cache()), R(rows()), R(groups(**kw))) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), NULL_ARG), (dict(out=None), NULL_ARG), (dict(q=FAKE + 2), ALIGN), (dict(out=FAKE + 4), ALIGN),
    (dict(n=-1), SHAPE), (dict(n=11), SHAPE), (dict(qs=511), SHAPE), (dict(os_=516), SHAPE)])
def test_bad_shared_calls(lib, kw, code):  # noqa: F811
    assert call_shared(lib, attn(), cache(), rows(), groups(), **kw) == code


@pytest.mark.parametrize("kw", [dict(num_q_heads=0), dict(num_q_heads=7), dict(num_sinks=-1), dict(scale=float("nan"))])
def test_bad_attention_descriptors(lib, kw):  # noqa: F811
    assert call_shared(lib, attn(**kw), cache(), rows(), groups()) == SHAPE


def test_null_descriptors(lib):  # noqa: F811
    assert call_shared(lib, None, cache(), rows(), groups()) == NULL_ARG
    assert call_shared(lib, attn(), None, rows(), groups()) == NULL_ARG
    assert call_shared(lib, attn(), cache(), None, groups()) == NULL_ARG
    assert call_shared(lib, attn(), cache(), rows(), None) == NULL_ARG
    assert call_append(lib, None, rows(), rope()) == NULL_ARG
    assert call_append(lib, cache(), None, rope()) == NULL_ARG
    assert call_append(lib, cache(), rows(), None) == NULL_ARG
    assert call_rope(lib, None) == NULL_ARG
    for args in ((None, R(rows()), R(groups())), (R(cache()), None, R(groups())), (R(cache()), R(rows()), None)):
        assert lib.gdn_kv_common_prefix(*args, None, None) == NULL_ARG


@pytest.mark.parametrize("head_dim,dtype", [(64, gdn.GDN_BF16), (96, gdn.GDN_BF16), (64, gdn.GDN_F32)])
def test_workspace(lib, head_dim, dtype):  # noqa: F811
    c, a = cache(head_dim=head_dim, dtype=dtype), attn()
    for r in (rows(), rows(max_query_len=500, num_tokens=700)):
        need = lib.gdn_shared_attention_workspace_bytes(R(a), R(c), R(r), R(groups()))
        whole = lib.gdn_attention_workspace_bytes(R(a), R(c), R(r))
        shares = r.max_query_len * 4 <= 256 or head_dim == 96 or dtype == gdn.GDN_F32
        # the states of all queries, and the passes' partial results
        assert need >= whole + r.num_tokens * 8 * (head_dim + 2) * 4 if shares else need == whole
        if need:
            n = r.num_tokens
            assert call_shared(lib, a, c, r, groups(), n=n, ws=None) == WORKSPACE
            assert call_shared(lib, a, c, r, groups(), n=n, nbytes=need - 1) == WORKSPACE
            assert call_shared(lib, a, c, r, groups(), n=n, ws=FAKE + 128) == ALIGN


def test_calls_with_nothing_to_do(lib):  # noqa: F811
    empty = rows(num_seqs=0, num_tokens=0, query_start_loc=None, kv_lens=None)
    none = groups(num_groups=0, group_start_loc=None, prefix_lens=None)
    assert call_shared(lib, attn(), cache(), empty, groups(), q=None, out=None, ws=None, nbytes=0) == 0
    assert call_append(lib, cache(), empty, rope(), k=None, v=None, q=None, out=None) == 0
    assert lib.gdn_kv_common_prefix(R(cache()), R(rows()), R(none), None, None) == 0
    assert call_rope(lib, rope(), n=0, pos=None, x=None, out=None) == 0


BAD_ROPE = [(dict(turns=None), NULL_ARG), (dict(rotary_dim=0), SHAPE), (dict(rotary_dim=3), SHAPE), (dict(rotary_dim=66), SHAPE),
            (dict(rotary_dim=-2), SHAPE), (dict(layout=2), SHAPE), (dict(layout=-1), SHAPE),
            (dict(magnitude=float("nan")), SHAPE), (dict(magnitude=float("inf")), SHAPE), (dict(turns=FAKE + 4), ALIGN)]


@pytest.mark.parametrize("kw,code", BAD_ROPE)
def test_bad_rope_descriptors(lib, kw, code):  # noqa: F811
    assert call_rope(lib, rope(**kw)) == code
    assert call_append(lib, cache(), rows(), rope(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=5), DTYPE), (dict(dim=8), SHAPE), (dict(dim=72), SHAPE), (dict(dim=272), SHAPE), (dict(heads=0), SHAPE),
    (dict(heads=65536), SHAPE), (dict(n=-1), SHAPE), (dict(pos=None), NULL_ARG), (dict(x=None), NULL_ARG),
    (dict(out=None), NULL_ARG), (dict(x=FAKE + 2), ALIGN), (dict(out=FAKE * 2 + 8), ALIGN), (dict(xs=255), SHAPE),
    (dict(os_=255), SHAPE), (dict(xs=260), SHAPE), (dict(xs=-256), SHAPE)])
def test_bad_rope_calls(lib, kw, code):  # noqa: F811
    assert call_rope(lib, rope(), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), NULL_ARG), (dict(v=None), NULL_ARG), (dict(q=None), NULL_ARG), (dict(out=None), NULL_ARG),
    (dict(k=FAKE + 2), ALIGN), (dict(q=FAKE * 3 + 2), ALIGN), (dict(out=FAKE * 4 + 8), ALIGN), (dict(n=-1), SHAPE),
    (dict(n=11), SHAPE), (dict(ks=127), SHAPE), (dict(vs=64), SHAPE), (dict(qs=500), SHAPE), (dict(os_=516), SHAPE),
    (dict(hq=-1), SHAPE), (dict(hq=65536), SHAPE)])
def test_bad_appends(lib, kw, code):  # noqa: F811
    assert call_append(lib, cache(), rows(), rope(), **kw) == code


def test_overlaps_are_refused(lib):  # noqa: F811
    # 10 tokens of 4 heads of 64 bf16: 512 bytes each
    assert call_rope(lib, rope(), out=FAKE + 512) == SHAPE                     # the next token
    assert call_rope(lib, rope(), out=FAKE - 16) == SHAPE
    assert call_rope(lib, rope(), xs=512, os_=512, out=FAKE + 256) == SHAPE    # half a token on, in a wider tensor
    assert call_rope(lib, rope(), xs=512, os_=512, out=FAKE + 1024 + 768) == SHAPE
    assert call_rope(lib, rope(), xs=512, out=FAKE) == SHAPE                   # in place with another stride
    assert call_rope(lib, rope(), n=1, out=FAKE + 16) == SHAPE
    far = dict(xs=1 << 40, os_=1 << 40)                                         # 2^64 bytes and more from first to last
    assert call_rope(lib, rope(), n=1 << 23, out=FAKE + 256, **far) == SHAPE
    assert call_rope(lib, rope(), n=(1 << 31) - 1, out=FAKE - 256, **far) == SHAPE
    # queries into keys' or values' places
    wide = dict(ks=1024, vs=1024, qs=1024, os_=1024)
    assert call_append(lib, cache(), rows(), rope(), k=FAKE, v=FAKE + 256, q=FAKE + 512, out=FAKE, **wide) == SHAPE
    assert call_append(lib, cache(), rows(), rope(), k=FAKE, v=FAKE + 256, q=FAKE + 512, out=FAKE + 256, **wide) == SHAPE
    assert call_append(lib, cache(), rows(), rope(), k=FAKE * 9, out=FAKE * 9) == SHAPE


# ------------------------------------------------------------------------------------------
# frequencies

def made(lib, rotary, **kw):  # noqa: F811
    d = dict(scaling=0, base=10000.0, factor=1.0, original_len=0.0, low=0.0, high=0.0)
    d.update(kw)
    turns, size = (ctypes.c_uint64 * (rotary // 2))(), ctypes.c_float()
    f = _RopeFreq(rotary, d["scaling"], d["base"], d["factor"], d["original_len"], d["low"], d["high"])
    return lib.gdn_rope_turns(ctypes.byref(f), turns, ctypes.byref(size)), list(turns), size.value


@pytest.mark.parametrize("rotary", [2, 6, 64, 90, 128, 256])
@pytest.mark.parametrize("kw", [
    dict(), dict(base=1.5), dict(base=1e7), dict(scaling=gdn.GDN_ROPE_LINEAR, factor=4.0),
    dict(scaling=gdn.GDN_ROPE_NTK, factor=8.0), dict(scaling=gdn.GDN_ROPE_BANDS, factor=8.0, original=8192.0),
    dict(scaling=gdn.GDN_ROPE_BANDS, factor=32.0, original=8192.0, low=2.0, high=3.0),
    dict(scaling=gdn.GDN_ROPE_RAMP, factor=40.0, original=4096.0),
    dict(scaling=gdn.GDN_ROPE_RAMP, factor=4.0, original=100.0, low=1.0, high=2.0, base=1e6)])
def test_frequencies(lib, rotary, kw):  # noqa: F811
    want, magnitude = ref.frequencies(rotary, **kw)
    args = {("original_len" if k == "original" else k): v for k, v in kw.items()}
    rc, turns, size = made(lib, rotary, **args)
    assert rc == 0 and abs(size - magnitude) <= 2.0 ** -24 * magnitude
    for t, f in zip(turns, want):
        # logarithms, powers and quotients in 64 bits, once here and once there: 2^-48 covers them at exponents up to 2^4.
        # The table holds whole units of 2^-64 turns, which rounds by half of one: 2 pi 2^-65 radians, whatever f is.
        assert abs(t / 2.0 ** 64 * 2 * math.pi - f) <= 2.0 ** -48 * f + 2 * math.pi * 2.0 ** -65


@pytest.mark.parametrize("rotary,kw", [
    (64, dict(scaling=5)), (64, dict(scaling=-1)), (64, dict(base=1.0)), (64, dict(base=float("nan"))), (64, dict(base=-2.0)),
    (64, dict(base=float("inf"))), (64, dict(scaling=1, factor=0.0)), (64, dict(scaling=2, factor=-1.0)),
    (64, dict(scaling=1, factor=float("nan"))), (64, dict(scaling=3, factor=2.0)), (64, dict(scaling=4, factor=2.0)),
    (64, dict(scaling=3, factor=2.0, original_len=100.0, low=4.0, high=4.0)),
    (64, dict(scaling=4, factor=2.0, original_len=100.0, low=-1.0)), (258, dict())])
def test_bad_frequencies(lib, rotary, kw):  # noqa: F811
    assert made(lib, rotary, **kw)[0] == SHAPE


def test_given_frequencies(lib):  # noqa: F811
    turns = (ctypes.c_uint64 * 4)()
    give = lambda *f: lib.gdn_rope_turns_of((ctypes.c_double * len(f))(*f), len(f), turns)  # noqa: E731
    assert give(math.pi, -math.pi / 2, 2 * math.pi, 0.0) == 0
    assert list(turns) == [1 << 63, 3 << 62, 0, 0]
    assert give(-1e-30) == 0 and turns[0] == 0
    assert give(float("nan")) == SHAPE and give(float("inf")) == SHAPE and give(1e300) == SHAPE
    assert lib.gdn_rope_turns_of(None, 1, turns) == NULL_ARG
    assert lib.gdn_rope_turns_of((ctypes.c_double * 1)(1.0), 0, turns) == SHAPE
    assert lib.gdn_rope_turns_of((ctypes.c_double * 1)(1.0), 129, turns) == SHAPE
    assert lib.gdn_rope_turns(None, turns, None) == NULL_ARG


# ------------------------------------------------------------------------------------------
# the binding

def on_device(r):
    object.__setattr__(r, "_device", 0)
    return r


def test_rope_descriptor():
    r = gdn.Rope(64, base=500000.0, device="cpu")
    assert r.turns.dtype == torch.int64 and r.turns.numel() == 32 and r._desc.turns == r.turns.data_ptr()
    first = r.turns[0].item() % (1 << 64)
    assert abs(first / 2.0 ** 64 * 2 * math.pi - 1.0) < 1e-15 and r._desc.magnitude == 1.0
    assert gdn.Rope(8, scaling=gdn.GDN_ROPE_RAMP, factor=40.0, original_len=4096, device="cpu")._desc.magnitude > 1.3
    assert gdn.Rope(8, magnitude=2.5, device="cpu")._desc.magnitude == 2.5
    assert gdn.Rope(4, frequencies=(math.pi, 0.0), device="cpu").turns.tolist() == [-(1 << 63), 0]
    for bad in (0, 3, 258, -4):
        with pytest.raises(ValueError):
            gdn.Rope(bad, device="cpu")
    with pytest.raises(ValueError, match="expected 2"):
        gdn.Rope(4, frequencies=(1.0,), device="cpu")
    with pytest.raises(gdn.GdnError, match="SHAPE"):
        gdn.Rope(4, base=0.5, device="cpu")


def test_groups_descriptor():
    g = gdn.KvGroups(i32([0, 2, 5]), i32([16, 0]))
    assert g.num_groups == 2
    with pytest.raises(ValueError, match="group_start_loc"):
        gdn.KvGroups(i32([0, 2]), i32([16, 0]))
    with pytest.raises(TypeError):
        gdn.KvGroups(i32([0, 2]), torch.zeros(1, dtype=torch.int64).as_subclass(type(i32([0]))))
    with pytest.raises(TypeError, match="CUDA"):
        gdn.KvGroups(torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


def test_the_binding_refuses(monkeypatch):
    monkeypatch.setattr(gdn, "_current_device", lambda: 0)
    r = on_device(gdn.Rope(64, device="cpu"))
    x = dev(6, 4, 64)
    with pytest.raises(ValueError, match="fewer positions"):
        gdn.gdn_rope(r, i32([0] * 7), x, dev(6, 4, 64))
    with pytest.raises(ValueError):
        gdn.gdn_rope(r, i32([0] * 6), x, dev(5, 4, 64))
    with pytest.raises(ValueError):
        gdn.gdn_rope(r, i32([0] * 6), dev(6, 256), dev(6, 256))
    with pytest.raises(TypeError):
        gdn.gdn_rope(r, i32([0] * 6), x, dev(6, 4, 64, dtype=torch.float32))
    with pytest.raises(TypeError):
        gdn.gdn_rope(r, torch.zeros(6, dtype=torch.int64), x, dev(6, 4, 64))
    with pytest.raises(TypeError, match="share memory"):
        gdn.gdn_rope(r, i32([0] * 6), x, dev(1, 4, 64).expand(6, 4, 64))
    with pytest.raises(gdn.GdnError, match="SHAPE"):  # tokens one further on
        long = dev(7, 4, 64)
        gdn.gdn_rope(r, i32([0] * 6), long[:6], long[1:], stream=0)
    with pytest.raises(ValueError, match="on the CPU"):
        gdn.gdn_rope(gdn.Rope(64, device="cpu"), i32([0] * 6), x, dev(6, 4, 64))
    k, v = dev(4, 2, 64), dev(4, 2, 64)
    with pytest.raises(ValueError, match="one token count"):
        gdn.gdn_kv_append_rope(dev_cache(), dev_rows(), r, k, v, dev(5, 8, 64))
    with pytest.raises(ValueError, match="without q"):
        gdn.gdn_kv_append_rope(dev_cache(), dev_rows(), r, k, v, None, dev(4, 8, 64))
    with pytest.raises(ValueError, match="one token count"):
        gdn.gdn_kv_append_rope(dev_cache(), dev_rows(), r, k, dev(5, 2, 64))
    other = gdn.KvGroups(i32([0, 2]), i32([0]))
    object.__setattr__(other, "_device", 1)
    with pytest.raises(ValueError, match="cuda:1"):
        gdn.gdn_shared_attention(gdn.Attention(8), dev_cache(), dev_rows(), other, dev(4, 8, 64), dev(4, 8, 64))
    with pytest.raises(ValueError, match="cuda:1"):
        gdn.gdn_kv_common_prefix(dev_cache(), dev_rows(), other)
    monkeypatch.setattr(gdn, "_current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        gdn.gdn_rope(r, i32([0] * 6), x, dev(6, 4, 64))
