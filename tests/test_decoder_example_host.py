"""The example decoder's bookkeeping, without its layers (no GPU)."""

import pytest

import dequant_matmul_gptq_amd as dq
from examples.decoder import Decoder


def _decoder(pages, page_size):
    d = Decoder.__new__(Decoder)
    d.pool, d.device, d.window = dq.PagePool(pages, page_size), "cpu", 0
    d.forward = lambda tokens, positions, slots, where: (tokens.tolist(), positions.tolist(), slots.tolist())
    return d


def test_a_step_without_room_changes_nothing():
    """The pool runs out at the batch's second sequence: the first has no tokens more that were never run."""
    d = _decoder(4, 4)
    d.add("a")
    d.add("b")
    d.step([("a", [1, 2, 3]), ("b", [4])])
    with pytest.raises(MemoryError):
        d.step([("a", [5, 6]), ("b", [7] * 12)])
    assert (d.pool.length("a"), d.pool.length("b"), d.pool.free_pages) == (3, 1, 2)
    assert d.step([("a", [5, 6]), ("b", [7])])[1] == [3, 4, 1]
