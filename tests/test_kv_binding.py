"""What the paged cache's binding refuses or arranges before it calls the library, on the host: tensors of the
CPU stand in for those of a GPU, and every call here ends before a launch."""
import ctypes

import pytest
import torch

import gated_deltanet_linear_spec_gb300 as gdn


class OnDevice(torch.Tensor):
    """A CPU tensor that says it is one of cuda:0."""
    is_cuda = True

    def get_device(self):
        return 0


def dev(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)


def i32(values):
    return torch.tensor(values, dtype=torch.int32).as_subclass(OnDevice)


def cache(**kw):
    d = dict(k_pool=dev(8, 2, 16, 64), v_pool=dev(8, 2, 16, 64), block_table=i32([[1, 2], [3, 4]]), refcount=i32([0] * 8))
    d.update(kw)
    return gdn.KvCache(**d)


def rows(**kw):
    d = dict(query_start_loc=i32([0, 2, 4]), num_tokens=4, kv_lens=i32([5, 9]), max_query_len=2)
    d.update(kw)
    return gdn.KvRows(**d)


# ------------------------------------------------------------------------------------------
# tensors whose tokens or pages share memory

def test_expanded_tokens_are_refused():
    one, four = dev(1, 2, 64).expand(4, 2, 64), dev(4, 2, 64)
    assert one.stride(0) == 0
    for k, v in ((one, four), (four, one)):
        with pytest.raises(TypeError, match="share memory"):
            gdn.gdn_kv_append(cache(), rows(), k, v)
    wide, out = dev(1, 8, 64).expand(4, 8, 64), dev(4, 8, 64)
    ws = torch.zeros(1 << 20, dtype=torch.uint8).as_subclass(OnDevice)
    for q, o in ((wide, out), (out, wide)):
        with pytest.raises(TypeError, match="share memory"):
            gdn.gdn_paged_attention(gdn.Attention(8), cache(), rows(), q, o, workspace=ws)


def test_overlapping_tokens_are_refused():
    long = dev(4 * 2 * 64 + 64)
    with pytest.raises(TypeError, match="share memory"):
        gdn._token_rows(long.as_strided((4, 2, 64), (64, 64, 1)), torch.bfloat16, 2, 64, "k", 0)


def test_expanded_pools_are_refused():
    one, all_ = dev(1, 2, 16, 64).expand(8, 2, 16, 64), dev(8, 2, 16, 64)
    for k, v in ((one, one), (one, all_), (all_, one)):
        with pytest.raises((TypeError, ValueError)):
            cache(k_pool=k, v_pool=v)


def test_one_token_and_strided_tokens_are_taken():
    assert gdn._token_rows(dev(1, 2, 64).expand(1, 2, 64), torch.bfloat16, 2, 64, "k", 0)[1] == 0
    assert gdn._token_rows(dev(4, 6, 64)[:, 2:4], torch.bfloat16, 2, 64, "k", 0)[1] == 6 * 64
    assert gdn._token_rows(dev(0, 2, 64), torch.bfloat16, 2, 64, "k", 0)[1] == 0
    both = dev(8, 2, 2, 16, 64)
    assert cache(k_pool=both[:, 0], v_pool=both[:, 1])._desc.page_stride == 2 * 2 * 16 * 64


# ------------------------------------------------------------------------------------------
# workspaces that a call makes

class Stream:
    """A stream as far as the binding looks at it."""

    def __init__(self, handle):
        self.handle = self.cuda_stream = handle


@pytest.mark.parametrize("given,want", [(None, None), (Stream(77), 77), (88, 88), (0, "default")])
def test_a_workspace_is_allocated_on_the_stream_that_uses_it(monkeypatch, given, want):
    active, seen = [], []

    class Under:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            active.append(self.stream.handle)

        def __exit__(self, *_):
            active.pop()

    empty = torch.empty

    def allocate(*size, device=None, **kw):
        seen.append(active[-1] if active else None)
        return empty(*size, **kw)

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", Under)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: Stream(handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream("default"))
    monkeypatch.setattr(torch, "empty", allocate)
    assert gdn._scratch(100, "cuda:0", given).numel() == 100
    assert seen == [want] and not active


def test_the_gdn_calls_make_their_workspace_the_same_way(monkeypatch):
    class Made(Exception):
        pass

    def scratch(nbytes, device, stream):
        assert nbytes >= 1
        raise Made(stream)

    monkeypatch.setattr(gdn, "_scratch", scratch)
    layer = gdn.Layer(1, 2, 128, 128, 4, 6)
    f32 = torch.float32
    params = gdn.Params(dev(layer.channels, 4), dev(2, dtype=f32), dev(2, dtype=f32))
    pools = gdn.Pools(dev(3, 6, layer.channels), dev(3, 2, 128, 128, dtype=f32))
    some = gdn.Rows(i32([0, 70]), 70, state_indices=i32([1]))
    x, a, out = dev(70, layer.channels), dev(70, 2), dev(70, 2, 128)
    for stream in (None, 77):
        with pytest.raises(Made) as e:
            gdn.gdn_chunk_prefill(layer, params, pools, x, a, a, some, out, stream=stream)
        assert e.value.args == (stream,)
        with pytest.raises(Made) as e:
            gdn.gdn_mixed_batch(layer, params, pools, x, a, a, some, 0, 1, None, out, stream=stream)
        assert e.value.args == (stream,)


# ------------------------------------------------------------------------------------------
# tensors of several devices, and of one that is not the current one

class OnAnother(OnDevice):
    def get_device(self):
        return 1


def other(t):
    return t.as_subclass(OnAnother)


def test_descriptors_over_two_devices_are_refused():
    for name, t in (("v_pool", dev(8, 2, 16, 64)), ("block_table", i32([[1]])), ("refcount", i32([0] * 8))):
        with pytest.raises(ValueError, match="cuda:1"):
            cache(**{name: other(t)})
    for name, t in (("kv_lens", i32([5, 9])), ("table_rows", i32([0, 1])), ("token_indx", i32([0, 1, 2, 3]))):
        with pytest.raises(ValueError, match="cuda:1"):
            rows(**{name: other(t)})


def calls(c, r, move=lambda t: t):
    """Every call of the cache, its tensors taken through ``move``."""
    k, q, n, ws = move(dev(4, 2, 64)), move(dev(4, 8, 64)), move(i32([1, 2])), move(torch.zeros(1 << 20, dtype=torch.uint8).as_subclass(OnDevice))
    layer, pools = gdn.Layer(2, 4, 16, 32, 4, 5), gdn.Pools(None, move(dev(4, 4, 32, 16, dtype=torch.float32)))
    return [lambda **kw: gdn.gdn_kv_append(c, r, k, k, **kw),
            lambda **kw: gdn.gdn_paged_attention(gdn.Attention(8), c, r, q, q, workspace=ws, **kw),
            lambda **kw: gdn.gdn_kv_reserve(c, n, n, n, workspace=ws, **kw),
            lambda **kw: gdn.gdn_kv_release(c, n, n, n, **kw),
            lambda **kw: gdn.gdn_kv_fork(c, n, n, n, workspace=ws, **kw),
            lambda **kw: gdn.gdn_kv_copy_pages(c, n, n, **kw),
            lambda **kw: gdn.gdn_kv_compact(c, n[:1], workspace=ws, **kw),
            lambda **kw: gdn.gdn_copy_slots(layer, pools, n, n, **kw)]


@pytest.fixture
def no_launch(monkeypatch):
    """The library's calls do nothing, and say so."""
    ran = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: ran.append(name) or 0

    monkeypatch.setattr(gdn, "library", lambda: Library())
    monkeypatch.setattr(gdn, "_stream_of", lambda t, stream: None)
    monkeypatch.setattr(gdn, "_current_device", lambda: 0)
    return ran


def test_calls_go_through_on_the_current_device(no_launch):
    for call in calls(cache(), rows()):
        call(status=i32([0]))
    assert len(no_launch) == 8


def test_calls_over_two_devices_are_refused(no_launch):
    c, r = cache(), rows()
    for call in calls(c, r, other)[:-1]:  # (the last one's tensors are all on the other device)
        with pytest.raises(ValueError, match="cuda:1"):
            call()
    for call in calls(c, r):
        with pytest.raises(ValueError, match="cuda:1"):
            call(status=other(i32([0])))
    layer, ssm = gdn.Layer(2, 4, 16, 32, 4, 5), dev(4, 4, 32, 16, dtype=torch.float32)
    with pytest.raises(ValueError, match="cuda:1"):
        gdn.gdn_copy_slots(layer, gdn.Pools(other(dev(4, 5, layer.channels)), ssm), i32([1]), i32([2]))
    with pytest.raises(ValueError, match="cuda:1"):
        calls(c, rows(**{k: other(v) for k, v in dict(query_start_loc=i32([0, 2, 4]), kv_lens=i32([5, 9])).items()}))[0]()
    assert not no_launch


def test_calls_off_the_current_device_are_refused(no_launch, monkeypatch):
    monkeypatch.setattr(gdn, "_current_device", lambda: 1)
    for call in calls(cache(), rows()):
        with pytest.raises(ValueError, match="current device"):
            call()
    assert not no_launch


# ------------------------------------------------------------------------------------------
# values that a 32-bit field does not hold

@pytest.mark.parametrize("value", [1 << 31, (1 << 32) + 1, -(1 << 31) - 1])
def test_values_past_32_bits_are_refused(value):
    for field in ("num_q_heads", "window", "num_sinks"):
        with pytest.raises(ValueError, match=field):
            gdn.Attention(**{"num_q_heads": 8, field: value})
    for field in ("num_tokens", "max_query_len"):
        with pytest.raises(ValueError, match=field):
            rows(**{field: value})
    with pytest.raises(ValueError, match="32 bits"):
        gdn._token_rows(dev(1, 2, 64).expand(1 << 32, 2, 64), torch.bfloat16, 2, 64, "k", 0)
    assert gdn.Attention(8, window=(1 << 31) - 1)._desc.window == (1 << 31) - 1


@pytest.mark.parametrize("pages,count", [(2, 0), (60, 0), (60, 3), (9000, 17), (131072, 64), (300000, 1)])
def test_workspace_of_the_page_calls(pages, count):
    desc = gdn._KvCache(0x100000, 0x100000, 0, 0x100000, 0x100000, pages, 8, 16, 16, 2, 64, gdn.GDN_BF16)
    ints = 5 * count + max(-(-pages // 1024), 8) + 4 + 2 * pages  # rows' values, block counts, totals, two lists
    assert gdn.library().gdn_kv_workspace_bytes(ctypes.byref(desc), count) == (4 * ints + 255) // 256 * 256
