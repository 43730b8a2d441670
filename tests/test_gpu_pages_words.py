"""Compaction of pools whose last word of 32 pages is in the middle of a warp, or that take the plan's one
CTA (1024 words) more than one turn: every id and byte as in the oracle's books."""

import numpy as np
import pytest

from oracle import draft4 as o4
from tests.conftest import gpu_available
from tests.test_gpu_pages import Device, _lib  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("num_pages", [32 * 5, 32 * 33 + 1, 32 * 1024, 32 * 1024 + 1, 32 * 1056 + 7, 32 * 2047])
def test_words_that_end_inside_a_warp(num_pages):
    r = np.random.default_rng(num_pages)
    live = min(num_pages // 2, 5000)
    ids = r.permutation(num_pages)
    table = ids[:live].reshape(1, -1)
    books = o4.Pages(table, [0], [0] * num_pages, ids[live:], 16, num_pages, range(num_pages))
    d = Device(1, books, [16])
    assert books.compact([]) == d.compact([])
    d.check(books)
