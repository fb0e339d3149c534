"""PagedCache's own host work, without a GPU: the numbers it hands to the library and the pages it hands out."""
from array import array

import numpy as np
import pytest
import torch

from chunked_kv_cache_gb300 import _native as N
from chunked_kv_cache_gb300.paged import PagedCache


@pytest.mark.parametrize("given", [[3, 0, 2, 1], (3, 0, 2, 1), np.array([3, 0, 2, 1]), np.array([3, 0, 2, 1], np.uint8),
                                   torch.tensor([3, 0, 2, 1]), array("b", [3, 0, 2, 1]), bytes([3, 0, 2, 1]),
                                   bytearray([3, 0, 2, 1]), range(4), memoryview(bytes([3, 0, 2, 1]))])
def test_every_sequence_of_numbers_arrives_as_32_bit_ones(given):
    """As many numbers as the library is told to read, bytes among them (an array takes those for its raw memory)."""
    ids, at = PagedCache._ids(given)
    assert list(ids) == [int(x) for x in given] and ids.itemsize == 4 and at == ids.buffer_info()[0]


def test_numbers_that_are_none_are_refused():
    assert PagedCache._ids(None) == (None, None)
    for bad in ([0.5], ["1"], "01", [1 << 31]):
        with pytest.raises((TypeError, N.SrError)):
            PagedCache._ids(bad)
