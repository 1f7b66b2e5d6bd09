"""Where warps of the cache attention's tensor-core kernel read or reuse tensor memory that other warps (or products that
only other warps have waited for) wrote, a barrier alone orders nothing: by the PTX memory model the side that arrives
needs tcgen05.fence::before_thread_sync in front and the side that goes on tcgen05.fence::after_thread_sync behind.
Read from the source: a missing fence gives wrong values seldom, so no run shows it."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "ring_attention_gb300", "csrc")
BEFORE, AFTER = "tc_fence_before", "tc_fence_after"


@pytest.fixture(scope="module")
def softmax():
    text = open(os.path.join(CSRC, "cache_attn_tc.cu")).read()
    text = re.sub(r"//[^\n]*", "", text)
    return text[text.index("setmaxnreg.inc"):text.index("cudaError_t launch(")]


def body_of(text, head):
    """The braces behind `head`."""
    at = text.index("{", text.index(head) + len(head))
    depth, i = 0, at
    while True:
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        i += 1
        if depth == 0:
            return text[at:i]


def order(text, *names):
    """Which of the names stand in the text, in order."""
    return [m.group(0) for m in re.finditer("|".join(r"\b%s\b" % n for n in names), text)]


def test_the_softmax_warps_meeting_orders_tensor_memory(softmax):
    # both accumulators are read behind it by warps that have waited for one or none of them
    body = body_of(softmax, "auto meet_all = [&]()")
    assert order(body, BEFORE, "mbar_arrive", "wait", AFTER) == [BEFORE, "mbar_arrive", "wait", AFTER]


def test_accumulators_are_handed_back_behind_a_fence(softmax):
    for m in re.finditer(r"mbar_arrive\(BAR\(C::B_OE \+ qt\)\)", softmax):
        last = order(softmax[:m.start()], BEFORE, AFTER, "meet", "meet_all", "tmem_ld32")[-1]
        assert last == BEFORE


def test_weights_are_handed_over_behind_a_fence(softmax):
    for m in re.finditer(r"mbar_arrive\(BAR\(C::B_P \+ qt\)\)", softmax):
        assert order(softmax[:m.start()], BEFORE, AFTER, "meet", "tmem_ld32", "weights")[-1] == BEFORE


def test_products_are_read_behind_a_fence(softmax):
    waits = list(re.finditer(r"wait\(C::B_[SO] \+ qt,[^\n]*\n", softmax))
    assert len(waits) == 3
    for m in waits:
        assert order(softmax[m.end():], BEFORE, AFTER, "tmem_ld32", "maxima", "weights", "meet_all")[0] == AFTER


def test_scores_read_by_the_other_thread_are_overwritten_behind_a_fence(softmax):
    # a row that moves its maximum: both threads read all of its scores, then each writes weights over its half
    move = body_of(softmax, "if (move)")
    assert order(move, "maxima", BEFORE, AFTER, "meet")[-3:] == [BEFORE, "meet", AFTER]
