"""Masks without words, without a GPU: torch gives them no address, and no address is no tree."""
import pytest
import torch

from tests.test_cache_host import _Fake, _cache_calls, bpa, streams  # noqa: F401


def test_attention_refuses_masks_without_words(bpa, streams):  # noqa: F811
    call = _cache_calls(bpa)["attn"]
    with pytest.raises(ValueError, match="tree"):
        call(tree=_Fake(torch.zeros(5, 0, dtype=torch.int32)))
    assert not streams[2]
    call(tree=_Fake(torch.zeros(5, 1, dtype=torch.int32)))
    assert len(streams[2]) == 1


def test_batches_refuse_masks_without_words(bpa):  # noqa: F811
    i32 = dict(dtype=torch.int32)
    for rows in (5, 0):
        with pytest.raises(ValueError, match="tree"):
            bpa.make_cache_batch(torch.zeros(rows, 4, 64), torch.zeros(3, 4, **i32), torch.zeros(3, **i32), torch.zeros(4, **i32),
                                 tree=torch.zeros(rows, 0, **i32))
