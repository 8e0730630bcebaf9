"""Rules that the paged cache's kernels keep in their source."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_deltanet_linear_spec_gb300", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "gdn_kv*")) + glob.glob(os.path.join(CSRC, "gdn_attn*")))


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_global_memory_is_read_coherently(path):
    """These kernels start while those before them still write the table and the pages.  Read-only loads are defined
    only for memory that does not change while a kernel runs; ``global_token`` of the GDN layers makes one."""
    with open(path) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert len(SOURCES) >= 7
    for word in (r"__ldg\b", r"ld\.global\.nc", r"__restrict__", r"\bglobal_token\b", r"__ldlu\b"):
        assert not re.search(word, code), (os.path.basename(path), word)
