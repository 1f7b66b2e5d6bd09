"""Kernels that are set up while the one before them ends must not read what that one may still write: behind
their wait they read with plain loads.  A load through the read-only path (__ldg) is taken to read what never changes
and may be moved in front of the wait, unless its address itself depends on a plain load behind it.  Read from the
source: the move depends on the compiler, so no run shows it."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "ring_attention_gb300", "csrc")


@pytest.mark.parametrize("name", ["rope.cu", "cache_plan.cu", "cache_tree.cu", "cache_keep.cu", "cache_pages.cu"])
def test_plain_loads_behind_the_wait(name):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    assert "wait_for_previous()" in text and "launch" in text
    assert "__ldg" not in text and "__restrict__" not in text
