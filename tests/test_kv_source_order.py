"""Orders of accesses that the attention kernels keep in their source, where no run can be made to show another."""
import os
import re

import pytest

from tests.test_kv_sources import CSRC


@pytest.mark.parametrize("name", ["gdn_attn_shared.cu", "gdn_attn_prompt.cu", "gdn_attn_split.cu"])
def test_what_a_tile_holds_is_stored_before_its_arrival(name):
    """Which of a tile's pages hold tokens reaches other warps by the barrier of the tile's copy: the arrival releases what was
    stored before it."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    stores = [m.end() for m in re.finditer(r"sm\.held\[[^\]]*\]\s*=[^=]", code)]
    assert len(stores) == 1
    before = code.rfind("expect_tx(&sm.full", 0, stores[0])
    after = code.find("expect_tx(&sm.full", stores[0])
    assert after >= 0 and "__syncwarp" not in code[stores[0]:after]
    assert before < 0 or "tma_page" in code[before:stores[0]]
