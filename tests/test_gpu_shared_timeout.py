"""Failure detection in the tensor-core pass of attention over groups, driven without a GPU fault.

Every wait of the pass is bounded.  The test hook ends a CTA's fetches early, so that the waits for the tiles that never come run
out with nothing in flight; the call has to return, to say so in the status word, and to join nothing from places that the pass
did not write, whatever the workspace holds there.  A call right after it is as good as any other.
"""
import pytest
import torch

import gated_deltanet_linear_spec_gb300 as gdn
from tests.test_gpu_shared import Groups

pytestmark = pytest.mark.gpu

SHORT_WAIT_NS = 20_000_000  # 20 ms instead of the default second


@pytest.fixture
def faults():
    yield gdn.gdn_testing_set_shared_faults
    gdn.gdn_testing_set_shared_faults(0, -1)


def groups(dim, **kw):
    return Groups([(640, [(1 + i % 3, 650 + 9 * i) for i in range(20)]), (64, [(1, 70), (2, 90)])], dim=dim, heads=8, seed=dim, **kw)


# (first worker, last worker, query, -) of a query's pieces: workers past the last one, most of 2^31 of them, a query past a unit's,
# a negative one, an end before the beginning
STALE = [(0x7f000000, 0x7f000000, 0, 0), (0, 0x7fffffff, 0, 0), (0, 152, 0, 0), (1, 1, 1 << 30, 0), (1, 1, 256, 0), (1, 1, -7, 0),
         (5, 3, 0, 0)]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("stale", STALE)
def test_places_that_the_pass_did_not_write_are_not_read(faults, stale, dim):
    s = groups(dim)
    need = gdn.gdn_shared_attention_workspace_bytes(s.attn, s.cache, s.kv_rows, s.groups)
    ws = torch.tensor(stale, dtype=torch.int32).repeat(-(-need // 16)).cuda().view(torch.uint8)
    faults(SHORT_WAIT_NS, 0)
    got, status = s.run(workspace=ws)
    faults(0, -1)
    assert status == gdn.STATUS_WAIT_TIMEOUT
    assert torch.all(got.float() == 7.0)
    s.check()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("stop", [1, 2, 5])
def test_waits_that_run_out_later(faults, stop, dim):
    s = Groups([(2000, [(1 + i % 3, 2300 + 9 * i) for i in range(20)])], dim=dim, heads=16, kv_heads=8)  # 9 tiles a share
    need = gdn.gdn_shared_attention_workspace_bytes(s.attn, s.cache, s.kv_rows, s.groups)
    ws = torch.full((need,), 0x7f, dtype=torch.uint8, device="cuda")
    faults(SHORT_WAIT_NS, stop)
    _, status = s.run(workspace=ws)
    faults(0, -1)
    assert status == gdn.STATUS_WAIT_TIMEOUT
    s.check()


def test_a_short_limit_alone_changes_nothing(faults):
    faults(SHORT_WAIT_NS, -1)
    groups(128).check()


def test_the_hook_needs_no_call(faults):
    assert gdn.library().gdn_testing_set_shared_faults(1, 3) == 0
    assert gdn.library().gdn_testing_set_shared_faults(0, -1) == 0
