"""Pins of the 4-bit draft's oracle: hand-worked rows, brute-force visibility, attention against
a softmax written out, and page moves against what each sequence holds."""

import numpy as np
import pytest

from oracle import draft4 as o4


def test_bf16_is_torch_bf16():
    torch = pytest.importorskip("torch")
    r = np.random.default_rng(1)
    x = r.standard_normal(5000).astype(np.float32) * np.exp2(r.integers(-140, 120, 5000)).astype(np.float32)
    assert np.array_equal(o4.bf16(x.astype(np.float64)), torch.from_numpy(x).bfloat16().double().numpy())
    assert o4.bf16(1 + 2.0 ** -8) == 1.0 and o4.bf16(1 + 3 * 2.0 ** -8) == 1 + 2.0 ** -6  # ties to even


def test_rows_by_hand():
    c, s, m = o4.quantise([0.0, 15.0, 7.5, 0.5, 1.5, 14.4])
    assert (s, m) == (1.0, 0.0) and c.tolist() == [0, 15, 8, 0, 2, 14]
    c, s, m = o4.quantise([-2.0] * 8)
    assert (s, m) == (0.0, -2.0) and not c.any()
    # 16 / 15 = 136.53 / 128, rounded up; 17 / 15 = 145.07 / 128, rounded down (the largest value would be 15.007)
    for top, scale in ((8.0, 137 / 128), (9.0, 145 / 128)):
        c, s, m = o4.quantise([-8.0, top])
        assert s == scale and c.tolist() == [0, 15]
    assert np.isnan(o4.quantise([1.0, np.inf])[1]) and np.isnan(o4.quantise([np.nan, 1.0])[2])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [1, 7, 16])
def test_tokens_survive_a_pool(D, page):
    r = np.random.default_rng(D + page)
    H, n = 3, 2 * page + 1
    pages = r.permutation(5)[:3]
    pool = r.integers(0, 256, (5, H * o4.head_bytes(D, page))).astype(np.uint8)
    x = o4.bf16(r.standard_normal((2, n, H, D)))
    for t in range(n):
        o4.write_token(pool, pages[t // page], t % page, page, x[0, t], x[1, t])
    codes, s, m = o4.read_tokens(pool, pages, page, n, H, D)
    for part in range(2):
        assert np.array_equal(np.stack([codes[part]]), np.stack([o4.quantise(x[part])[0]]))
        assert np.array_equal(s[part], o4.quantise(x[part])[1]) and np.array_equal(m[part], x[part].min(-1))
    # within half a step, and the clamp of a scale that was rounded down (15 steps of 2^-9 at most)
    assert np.all(np.abs(m[..., None] + s[..., None] * codes - x) <= s[..., None] * (0.5 + 15 * 2.0 ** -8))


@pytest.mark.parametrize("p,window,sinks,see", [
    (4, 0, 0, [0, 1, 2, 3, 4]), (4, 2, 0, [3, 4]), (4, 1, 0, [4]), (4, 2, 1, [0, 3, 4]), (4, 2, 9, [0, 1, 2, 3, 4]),
    (4, 9, 0, [0, 1, 2, 3, 4]), (-1, 0, 0, []), (-1, 3, 2, []), (0, 5, 5, [0])])
def test_visible(p, window, sinks, see):
    assert o4.visible(p, window, sinks) == see


def test_attention_is_a_softmax():
    r = np.random.default_rng(3)
    q = r.standard_normal((2, 4, 64))
    codes = r.integers(0, 16, (2, 6, 2, 64)).astype(float)
    s, m = r.uniform(0.05, 0.2, (2, 6, 2)), r.standard_normal((2, 6, 2))
    out, lse, *_ = o4.attention(q, codes, s, m, 5, 0.125, window=2, sinks=1)
    kv = m[..., None] + s[..., None] * codes
    for i, see in enumerate(([0, 3, 4], [0, 4, 5])):
        for h in range(4):
            z = np.array([0.125 * float(q[i, h] @ kv[0, j, h // 2]) for j in see])
            e = np.exp(z)
            assert np.allclose(out[i, h], sum(w * kv[1, j, h // 2] for w, j in zip(e, see)) / e.sum())
            assert np.isclose(lse[i, h], np.log(e.sum()))


def test_weights_by_hand():
    W = np.array([[0x80, 0xF1] + [0x88] * 14], np.uint8)  # codes 0 8 1 15 8 8 ...
    w = o4.weights(W, np.array([[0.5]]), None, 32)
    assert w[0, :6].tolist() == [-4.0, 0.0, -3.5, 3.5, 0.0, 0.0]
    assert o4.weights(W, np.array([[0.5]]), np.array([[1]]), 32)[0, :4].tolist() == [-0.5, 3.5, 0.0, 7.0]


def held(pages, b):
    """What sequence b holds: its pages' contents."""
    return [pages.data[p] for p in pages.table[b] if p >= 0]


def consistent(pages, prefix=()):
    owners = {}
    for r in pages.table:
        for p in r:
            if p >= 0:
                owners[p] = owners.get(p, 0) + 1
    assert all(pages.shares[p] == owners.get(p, 1) - 1 for p in range(pages.num_pages))
    assert not set(owners) & set(pages.stack) and len(set(pages.stack)) == len(pages.stack)
    assert len(set(owners) | set(prefix)) + len(pages.stack) == pages.num_pages


def test_moves_keep_what_sequences_hold():
    P, n = 4, 12
    table = [[3, 7, 9, -1], [5, -1, -1, -1], [-1] * 4, [-1] * 4, [-1] * 4]
    pages = o4.Pages(table, [10, 4, 0, 0, 0], [0] * n, [11, 10, 8, 6, 4, 2, 1, 0], P, n, [f"d{i}" for i in range(n)])
    before = held(pages, 0)
    pages.fork([0, 0, 1], [2, 3, 4])
    consistent(pages)
    assert pages.flags == 0 and pages.lens == [10, 4, 10, 10, 4]
    assert pages.table[2] == [3, 7, 0, -1] and pages.table[3] == [3, 7, 1, -1] and pages.table[4] == [5, -1, -1, -1]
    assert held(pages, 2) == held(pages, 3) == before and pages.shares[3] == 2 and pages.shares[5] == 1
    pages.free([0, 1])
    consistent(pages)
    assert pages.stack == [11, 10, 8, 6, 4, 2, 9] and pages.table[0] == [-1] * 4
    pages.compact([])
    consistent(pages)
    assert held(pages, 2) == held(pages, 3) == before and held(pages, 4) == ["d5"]
    assert sorted({p for r in pages.table for p in r if p >= 0}) == list(range(5))
    assert pages.stack == list(range(11, 4, -1))


@pytest.mark.parametrize("src,dst,flag", [
    ([0], [0], o4.FLAG_BAD_N), ([0, 1], [2, 2], o4.FLAG_BAD_N), ([0, 2], [2, 3], o4.FLAG_BAD_N),
    ([9], [2], o4.FLAG_BAD_N), ([0], [-1], o4.FLAG_BAD_N), ([0], [1], o4.FLAG_BAD_N)])
def test_forks_that_are_refused(src, dst, flag):
    pages = o4.Pages([[3, 7], [5, -1], [-1, -1], [-1, -1]], [6, 2, 0, 0], [0] * 8, [0, 1, 2], 4, 8, range(8))
    table = [list(r) for r in pages.table]
    pages.fork(src, dst)
    assert pages.flags == flag and pages.table[0] == table[0] and pages.stack == [0, 1, 2]
    assert pages.table[2] == [-1, -1]


def test_a_short_stack_changes_nothing():
    pages = o4.Pages([[3, 7], [5, -1], [-1, -1], [-1, -1]], [6, 4, 0, 0], [0] * 8, [], 4, 8, range(8))
    pages.fork([0, 1], [2, 3])
    assert pages.flags == o4.FLAG_CAPACITY and pages.lens == [6, 4, 0, 0] and pages.shares == [0] * 8
