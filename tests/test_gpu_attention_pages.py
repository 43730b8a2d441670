"""Pages of 8, 128, 256 and 512 tokens: the smallest page that arrives as boxes, the tile
itself, and pages that a tile is a part of.  Prefixes and own lengths end inside a page, at
its end and one behind it; what is behind a sequence's end holds NaN."""

import numpy as np
import pytest

from tests.conftest import gpu_available
from tests.test_gpu_attention import Case, _lib  # noqa: F401  (the fixture builds the library)

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [8, 128, 256, 512])
def test_long_and_short_pages(page, D):
    for prefix in (page - 1, page, page + 1, 3 * page + 5):
        lens = [0, 1, page - 2, page - 1, page, page + 1, 2 * page + 70, 333]
        Case(lens, [2, 0, 2, 1, 1, 2, 2, 0], 2, hq=4, hkv=2, D=D, page=page, prefix=prefix, seed=page).run().check()


@pytest.mark.parametrize("layout", ["head", "pair"])
@pytest.mark.parametrize("page", [8, 256])
def test_layouts(page, layout):
    Case([50, 300, 7], [2, 4, 1], 4, hkv=2, hq=6, prefix=290, layout=layout, D=64, page=page).run().check()
    Case([50, 300, 7], [2, 4, 1], 4, hkv=2, hq=6, prefix=290, layout=layout, D=128, page=page).run().check()


@pytest.mark.parametrize("page", [8, 128, 256])
def test_bad_pages_fail_their_sequence(page):
    c = Case([300, 290, 310], [1, 2, 0], 2, prefix=200, page=page, D=64)
    c.table[1, 290 // page] = c.num_pages
    c.upload()
    c.run().check()
    assert [c.flags(b) for b in range(3)] == [0, 512, 0]


def test_decode_step_of_a_batch():
    """One new token for each of many sequences, long and short ones, behind a prefix and
    without one."""
    r = np.random.default_rng(11)
    for prefix, D in ((300, 128), (0, 64)):
        lens = r.integers(0, 700, 150)
        Case(lens, np.zeros(150, np.int32), 0, hq=8, hkv=2, D=D, page=32, prefix=prefix, seed=D).run().check()
