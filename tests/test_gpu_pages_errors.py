"""Page operators on rows that are not in order: what they leave."""
import numpy as np
import pytest
import torch

from test_gpu_pages import Pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [-1, -2 ** 31, 10 ** 6, 2 ** 31 - 1])
def test_free_of_a_bad_length_leaves_the_row(bad):
    """The row keeps its length, entries and counts, a fork into it is refused, and once
    the length is mended it is given back in full; other rows of the call are."""
    p = Pool([40, 17, 100], 1)
    p.lens[2] = bad
    p.free([0, 2, 2])
    assert p.err.item() == 3
    p.host_free([0])
    p.h["lens"][2] = bad
    p.same()
    p.err.zero_()
    p.fork([1], [2])
    assert p.err.item() == 6
    p.same()
    p.err.zero_()
    p.lens[2] = p.h["lens"][2] = 100
    p.free([2])
    p.host_free([2])
    p.same()
    assert p.err.item() == 0 and int(p.refs.sum()) == 2


def test_free_of_a_row_named_many_times_at_once():
    p = Pool([300] * 4, 4)
    p.fork([0, 1, 2, 3], [4, 5, 6, 7])
    p.host_fork([0, 1, 2, 3], [4, 5, 6, 7])
    rows = np.random.RandomState(1).permutation(np.repeat([0, 5, 3, 2], 200)).tolist()
    p.free(rows)
    p.host_free([0, 5, 3, 2])
    p.same()
    assert p.err.item() == 0
