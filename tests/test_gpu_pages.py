"""GPU parity of the page moves (copy, fork, free, compact) with the oracle's books: tables, lengths,
owners, the free stack and every page's bytes, exactly."""

import numpy as np
import pytest

from oracle import draft4 as o4
from speculative_decoding_verification_47_gb300 import binding as sb
from tests.conftest import gpu_available

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from speculative_decoding_verification_47_gb300 import build
    build.build()
    sb.lib()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Device:
    """The device's side of an oracle.Pages: page arrays of the given page sizes, whose page p holds
    bytes drawn for p (the oracle's data[p] names them)."""

    def __init__(self, seed, books, sizes):
        self.r = np.random.default_rng(seed)
        self.sizes, self.n = sizes, books.num_pages
        self.fill = [self.r.integers(0, 256, (books.num_pages, b)).astype(np.uint8) for b in sizes]
        self.pools = [dev(f) for f in self.fill]
        self.table, self.lens = dev(np.int32(books.table)), dev(np.int32(books.lens))
        self.shares = dev(np.int32(books.shares))
        stack = np.full(books.num_pages + 3, -9, np.int32)
        stack[:len(books.stack)] = books.stack
        self.stack, self.top = dev(stack), dev(np.int32([len(books.stack)]))
        self.ws = torch.zeros(sb.sv_kv_pages_workspace_size(books.num_pages, 4096), dtype=torch.uint8, device="cuda")

    def args(self):
        return self.pools, self.sizes, len(self.sizes), self.n

    def fork(self, P, src, dst):
        sb.sv_kv_fork(*self.args(), P, self.table, self.table.shape[1], self.lens, self.shares, self.stack, self.top,
                      dev(np.int32(src)), dev(np.int32(dst)), len(src), self.table.shape[0], self.ws, self.ws.numel())

    def free(self, seqs):
        sb.sv_kv_free(self.table, self.table.shape[1], self.lens, self.shares, self.n, self.stack, self.top, self.n + 3,
                      dev(np.int32(seqs)), len(seqs), self.table.shape[0], self.ws, self.ws.numel())

    def compact(self, prefix):
        p = dev(np.int32(prefix)) if len(prefix) else None
        sb.sv_kv_compact(*self.args(), self.table, self.table.shape[1], self.table.shape[0], p, len(prefix), self.shares,
                         self.stack, self.top, self.n + 3, self.ws, self.ws.numel())
        return [] if p is None else p.cpu().tolist()

    def check(self, books):
        assert sb.sv_read_device_flags(self.ws) == books.flags
        assert self.table.cpu().tolist() == books.table and self.lens.cpu().tolist() == books.lens
        assert self.shares.cpu().tolist() == books.shares
        top = int(self.top.item())
        assert self.stack.cpu().tolist()[:top] == books.stack and torch.all(self.stack[books.num_pages:] == -9)
        for pool, fill in zip(self.pools, self.fill):
            got = pool.cpu().numpy()
            assert all(np.array_equal(got[p], fill[books.data[p]]) for p in range(books.num_pages))


def books_of(seed, B, max_pages, P, empty, spare=20, most=None):
    r = np.random.default_rng(seed)
    lens = r.integers(0, (most or max_pages * P) + 1, B)
    lens[: B // 4] = r.integers(0, max_pages + 1, B // 4) * P  # whole pages, none among them
    lens = np.minimum(lens, most or max_pages * P)
    lens[empty] = 0
    n = B * max_pages + spare
    ids = r.permutation(n)
    table = np.full((B, max_pages), -1)
    at = 0
    for b in range(B):
        used = -(-lens[b] // P)
        table[b, :used] = ids[at:at + used]
        at += used
    return o4.Pages(table, lens, [0] * n, r.permutation(ids[at:]), P, n, range(n)), r


@pytest.mark.parametrize("P,sizes", [(16, [4096]), (4, [896, 16, 2064]), (1, [144] * 9), (7, [7 * 128] * 20)])
def test_forks_frees_and_compaction_in_turn(P, sizes):
    B, max_pages = 60, 6
    empty = list(range(30, 60))
    books, r = books_of(P, B, max_pages, P, empty)
    d = Device(P + 1, books, sizes)
    for round_ in range(4):
        rows = [b for b in range(B) if books.lens[b] == 0 and all(p < 0 for p in books.table[b])]
        sources = [b for b in range(B) if b not in rows]
        F = min(len(rows), 12)
        dst = r.permutation(rows)[:F].tolist()
        src = r.choice(sources, F).tolist()
        books.fork(src, dst), d.fork(P, src, dst)
        d.check(books)
        seqs = r.permutation(B)[: B // 4].tolist()
        books.free(seqs), d.free(seqs)
        d.check(books)
        assert books.compact([]) == d.compact([])
        d.check(books)


@pytest.mark.parametrize("n_pools", [1, 8, 9, 64, 256])
def test_forks_over_many_page_arrays(n_pools):
    books, r = books_of(n_pools, 12, 3, 16, [8, 9, 10, 11])
    d = Device(2, books, [16 * int(k) for k in r.integers(1, 200, n_pools)])
    books.fork([0, 1, 1, 7], [8, 9, 10, 11]), d.fork(16, [0, 1, 1, 7], [8, 9, 10, 11])
    d.check(books)


@pytest.mark.parametrize("src,dst", [
    ([0], [0]), ([0, 1], [12, 12]), ([0, 12], [12, 13]), ([99], [12]), ([0], [-1]), ([0], [5]), ([-3, 1, 2], [12, 13, 14]),
    ([0] * 5, [12, 13, 14, 15, 15])])
def test_forks_that_are_refused(src, dst):
    books, _ = books_of(5, 16, 4, 8, [12, 13, 14, 15])
    assert books.lens[5] > 0
    d = Device(3, books, [512, 1024])
    books.fork(src, dst), d.fork(8, src, dst)
    assert books.flags == o4.FLAG_BAD_N
    d.check(books)


def test_forks_of_unsound_sources_and_stacks():
    for what in ("long", "negative", "page", "row", "short", "stack", "top"):
        books, _ = books_of(6, 8, 4, 8, [4, 5, 6, 7], most=30)
        books.lens[0], books.lens[1] = 13, 13
        books.table[0], books.table[1] = [1, 2, -1, -1], [3, 4, -1, -1]
        books.stack = [20, 21, 22]
        flag = o4.FLAG_BAD_N
        if what == "long":
            books.lens[0] = 33
        elif what == "negative":
            books.lens[0] = -1
        elif what == "page":
            books.table[0][1], flag = books.num_pages, o4.FLAG_BAD_PAGE
        elif what == "row":
            books.table[4][3] = 30
        elif what == "short":
            books.stack, flag = [20], o4.FLAG_CAPACITY
        d = Device(4, books, [512])
        if what == "stack":  # an id outside the pool on top: nothing changes
            d.stack[2] = books.num_pages
            before = [t.clone() for t in (d.table, d.lens, d.shares, d.stack, d.top, d.pools[0])]
            d.fork(8, [0, 1], [4, 5])
            assert sb.sv_read_device_flags(d.ws) == o4.FLAG_BAD_PAGE
        elif what == "top":
            d.top[0] = books.num_pages + 1
            before = [t.clone() for t in (d.table, d.lens, d.shares, d.stack, d.top, d.pools[0])]
            d.fork(8, [0, 1], [4, 5])
            assert sb.sv_read_device_flags(d.ws) == o4.FLAG_CAPACITY
        else:
            books.fork([0, 1], [4, 5]), d.fork(8, [0, 1], [4, 5])
            assert books.flags == flag
            d.check(books)
            continue
        for a, b in zip(before, (d.table, d.lens, d.shares, d.stack, d.top, d.pools[0])):
            assert torch.equal(a, b)


def test_frees_that_are_refused():
    books, _ = books_of(7, 10, 4, 8, [])
    d = Device(5, books, [256])
    seqs = [3, 3, 0, -1, 10, 5]
    books.free(seqs), d.free(seqs)
    assert books.flags == o4.FLAG_BAD_N
    d.check(books)


def test_frees_of_unsound_rows():
    """An id outside the pool, and a page in two rows with one owner, are emptied and flagged."""
    books, _ = books_of(8, 6, 3, 4, [], most=12)
    books.table[0], books.table[1] = [2, books.num_pages + 5, 3], [3, -1, 4]
    used = {p for r in books.table for p in r}
    books.stack = [p for p in range(books.num_pages) if p not in used]
    d = Device(6, books, [256])
    books.free([0, 1]), d.free([0, 1])
    assert books.flags == o4.FLAG_BAD_PAGE
    d.check(books)


@pytest.mark.parametrize("num_pages,live", [(1, 0), (1, 1), (2, 1), (31, 7), (32, 32), (33, 32), (100, 99), (5000, 1234),
                                            (40000, 30000)])
def test_compaction_sizes(num_pages, live):
    r = np.random.default_rng(num_pages + live)
    ids = r.permutation(num_pages)[:live]
    prefix = ids[: min(live, 3)].tolist()
    rows = ids[len(prefix):]
    B, max_pages = 7, max(1, -(-len(rows) // 7) + 1)
    table = np.full(B * max_pages, -1)
    table[r.permutation(B * max_pages)[:len(rows)]] = rows
    shares = np.zeros(num_pages, int)
    books = o4.Pages(table.reshape(B, max_pages), [0] * B, shares, r.permutation(np.setdiff1d(np.arange(num_pages), ids)), 16,
                     num_pages, range(num_pages))
    d = Device(9, books, [64, 16])
    assert books.compact(prefix) == d.compact(prefix)
    d.check(books)
    assert books.compact(prefix) is not None  # and again: nothing is left to move
    d.compact(prefix)
    d.check(books)


def test_compaction_leaves_unsound_entries():
    books = o4.Pages([[9, 50, -1], [7, -2, 3]], [0, 0], [0] * 10, [], 4, 10, range(10))
    d = Device(10, books, [32])
    books.compact([]), d.compact([])
    books.flags = o4.FLAG_BAD_PAGE
    books.table[1][1] = -2
    d.check(books)


@pytest.mark.parametrize("page_bytes,n", [(16, 5), (2048, 40), (2064, 7), (34816, 30), (1 << 20, 3)])
def test_copies(page_bytes, n):
    r = np.random.default_rng(page_bytes + n)
    num_pages = 3 * n
    ids = r.permutation(num_pages).astype(np.int32)
    src, dst = np.concatenate([ids[:n - 1], ids[:1]]), ids[n:2 * n].copy()  # one source twice
    fill = r.integers(0, 256, (2, num_pages, page_bytes)).astype(np.uint8)
    pools, ws = dev(fill), torch.zeros(sb.sv_kv_pages_workspace_size(num_pages, n + 2), dtype=torch.uint8, device="cuda")
    src, dst = np.append(src, [-1, 0]).astype(np.int32), np.append(dst, [ids[-1], num_pages]).astype(np.int32)
    sb.sv_kv_copy_pages([pools[0], pools[1]], [page_bytes] * 2, 2, num_pages, dev(src), dev(dst), n + 2, ws, ws.numel())
    assert sb.sv_read_device_flags(ws) == o4.FLAG_BAD_PAGE
    fill[:, dst[:n]] = fill[:, src[:n]]
    assert np.array_equal(pools.cpu().numpy(), fill)


def test_copies_past_four_gigabytes():
    page, num_pages = 1 << 20, 4608
    pool = torch.zeros(num_pages, page // 4, dtype=torch.int32, device="cuda")
    pool[num_pages - 1] = torch.arange(page // 4, device="cuda", dtype=torch.int32)
    ws = torch.zeros(sb.sv_kv_pages_workspace_size(num_pages, 1), dtype=torch.uint8, device="cuda")
    sb.sv_kv_copy_pages([pool], [page], 1, num_pages, dev(np.int32([num_pages - 1])), dev(np.int32([num_pages - 200])), 1, ws,
                        ws.numel())
    assert torch.equal(pool[num_pages - 200], pool[num_pages - 1]) and int(pool[:num_pages - 200].abs().max()) == 0


def test_a_round_of_forks_in_a_graph():
    """Ended rows are freed and forked into; the graph replayed on the state it left behind."""
    books, r = books_of(11, 24, 4, 8, [])
    d = Device(12, books, [512] * 3)
    side = torch.cuda.Stream()
    ended, sources = [1, 5, 9], [2, 2, 0]
    de, ds = dev(np.int32(ended)), dev(np.int32(sources))

    def call():
        sb.sv_kv_free(d.table, 4, d.lens, d.shares, d.n, d.stack, d.top, d.n, de, 3, 24, d.ws, d.ws.numel())
        sb.sv_kv_fork(*d.args(), 8, d.table, 4, d.lens, d.shares, d.stack, d.top, ds, de, 3, 24, d.ws, d.ws.numel())

    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        call()
    for _ in range(3):
        graph.replay()
        books.free(ended), books.fork(sources, ended)
    torch.cuda.synchronize()
    d.check(books)
