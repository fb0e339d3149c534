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


class _Table:
    """A block table on the CPU whose next writes can be made to fail, as they do while a graph is captured."""

    def __init__(self, seqs, pages):
        self.t, self.fails = torch.full((seqs, pages), -1, dtype=torch.int32), False

    def __setitem__(self, at, x):
        if self.fails:
            raise RuntimeError("not now")
        self.t[at] = x


def _pool(n_pages=6, seqs=3, pages=4):
    c = object.__new__(PagedCache)
    c.handle, c.device = None, torch.device("cpu")
    c.page_tokens, c.max_pages, c.max_seqs, c.n_pages = 16, pages, seqs, n_pages
    c._free, c._pages = list(range(n_pages - 1, -1, -1)), [[] for _ in range(seqs)]
    c.block_table = _Table(seqs, pages)
    return c


def test_pages_are_not_lost_where_the_table_cannot_be_written():
    c = _pool()
    c.reserve(1, 20)
    c.block_table.fails = True
    with pytest.raises(RuntimeError):
        c.reserve(0, 33)
    assert sorted(c._free) == [2, 3, 4, 5] and c._pages == [[], [0, 1], []]
    c.block_table.fails = False
    c.reserve(0, 33)
    c.reserve(1, 33)
    assert c.block_table.t.tolist() == [[2, 3, 4, -1], [0, 1, 5, -1], [-1] * 4]
    assert c._free == [] and c._pages == [[2, 3, 4], [0, 1, 5], []]
    with pytest.raises(RuntimeError):
        c.reserve(2, 1)
