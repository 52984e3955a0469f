"""The axes of the pairs as the binding takes them: bytes, or any sequence of
whole numbers, entry by entry."""

import array

import numpy as np
import pytest
import torch

import all_reduce_reduction_rank_gb300 as ar

AXES = [d % 3 for d in range(64)]


@pytest.mark.parametrize("axes", [AXES, tuple(AXES), bytes(AXES), bytearray(AXES), np.array(AXES), np.array(AXES, dtype=np.int32),
                                  np.array(AXES, dtype=np.uint8), np.repeat(AXES, 2)[::2], torch.tensor(AXES),
                                  torch.tensor(AXES, dtype=torch.int8), array.array("i", AXES),
                                  memoryview(array.array("q", AXES))])
def test_entries_are_taken_one_by_one(axes):
    assert ar._pair_axis(axes, 128) == bytes(AXES)
    assert ar._pair_axis(axes, 32)[:16] == bytes(AXES[:16])
    with pytest.raises(ValueError):
        ar._pair_axis(axes[:63], 128)


@pytest.mark.parametrize("axes", [np.array(AXES, dtype=np.float32), [0.0] * 64, torch.zeros(64), "0" * 64,
                                  np.zeros((64, 2), dtype=np.uint8), [[0]] * 64])
def test_what_is_no_whole_number_is_refused(axes):
    with pytest.raises(TypeError):
        ar._pair_axis(axes, 128)


@pytest.mark.parametrize("bad", [-1, 256, 2**40])
def test_entries_of_more_than_a_byte_are_refused(bad):
    for axes in ([0] * 63 + [bad], np.array([0] * 63 + [bad]), torch.tensor([0] * 63 + [bad])):
        with pytest.raises(ValueError):
            ar._pair_axis(axes, 128)
