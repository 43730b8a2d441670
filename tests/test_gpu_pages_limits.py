"""The most forks and the most released sequences of a call, against the oracle's books."""

import numpy as np
import pytest

from oracle import draft4 as o4
from tests.conftest import gpu_available
from tests.test_gpu_pages import Device, _lib  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("F", [257, 1000, 4096])
def test_the_most_forks_and_releases(F):
    r = np.random.default_rng(F)
    P, max_pages, sources = 8, 3, 50
    B = sources + F
    lens = np.zeros(B, int)
    lens[:sources] = r.integers(0, max_pages * P + 1, sources)
    n = sources * max_pages + F + 10
    ids = r.permutation(n)
    table = np.full((B, max_pages), -1)
    at = 0
    for b in range(sources):
        used = -(-lens[b] // P)
        table[b, :used] = ids[at:at + used]
        at += used
    books = o4.Pages(table, lens, [0] * n, ids[at:], P, n, range(n))
    d = Device(F, books, [16, 48])
    src, dst = r.integers(0, sources, F).tolist(), (sources + r.permutation(F)).tolist()
    books.fork(src, dst), d.fork(P, src, dst)
    assert books.flags == 0
    d.check(books)
    seqs = r.permutation(B)[:F].tolist()
    books.free(seqs), d.free(seqs)
    d.check(books)
