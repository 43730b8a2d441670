"""Rounds of a draft held in 4 bits, as a server would run them: continuations forked off a sequence,
the layers (projection, append, attention, projection with a residual) replayed as one graph, the commit,
ended sequences freed and the pool compacted.  Each step is held to the oracle on what it was given."""

import numpy as np
import pytest

from oracle import draft4 as o4
from speculative_decoding_verification_47_gb300 import binding as sb
from tests import test_gpu_kv4 as kv4
from tests import test_gpu_linear_w4 as w4
from tests.conftest import gpu_available

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]

BF, dev, f64 = torch.bfloat16, kv4.dev, kv4.f64


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from speculative_decoding_verification_47_gb300 import build
    build.build()
    sb.lib()


class Layer:
    """One layer's weights and buffers; x comes in, ``out`` goes to the next."""

    def __init__(self, seed, d, x):
        self.d, self.x = d, x
        M, E, D, group = x.shape[0], x.shape[1], d["D"], d["group"]
        self.wide = (d["hq"] + 2 * d["hkv"]) * D
        self.qkv_w = w4.inputs(seed, 1, self.wide, E, group, True, True, False, BF)
        self.out_w = w4.inputs(seed + 1, 1, E, d["hq"] * D, group, False, False, False, BF)
        self.on = [{k: None if v is None else v.cuda() for k, v in w.items()} for w in (self.qkv_w, self.out_w)]
        self.pool = torch.zeros(d["pages"], sb.sv_kv4_page_bytes(d["hkv"], D, d["page"]), dtype=torch.uint8, device="cuda")
        self.qkv = torch.zeros(M, self.wide, dtype=BF, device="cuda")
        self.att = torch.zeros(M, d["hq"] * D, dtype=BF, device="cuda")
        self.out = torch.zeros(M, E, dtype=BF, device="cuda")
        self.ws = [torch.zeros(sb.sv_linear_w4_workspace_size(M, n, k), dtype=torch.uint8, device="cuda")
                   for n, k in ((self.wide, E), (E, d["hq"] * D))]

    def run(self, table, starts, lens, n, k, attention_ws):
        d, (a, o) = self.d, self.on
        B, Q, hq, hkv, D, page, group = (d[i] for i in ("B", "Q", "hq", "hkv", "D", "page", "group"))
        M, E = self.x.shape
        sb.sv_linear_w4(self.x, 0, a["W"], 0, a["scales"], a["zeros"], group, a["bias"], None, 0, sb.SV_ACT_NONE, self.qkv, 0,
                        sb.SV_BF16, M, self.wide, E, self.ws[0], self.ws[0].numel())
        at = self.qkv.data_ptr()
        strides = (Q * self.wide, self.wide, D)
        sb.sv_kv4_append(at + 2 * hq * D, at + 2 * (hq + hkv) * D, *strides, sb.SV_BF16, self.pool, d["pages"], page, table,
                         table.shape[1], starts, n, B, Q, hkv, D, attention_ws, 4)
        sb.sv_kv4_attention(self.qkv, *strides, self.pool, d["pages"], page, table, table.shape[1], lens, k, d["window"],
                            d["sinks"], d["scale"], self.att, 0, 0, 0, None, sb.SV_BF16, B, Q - 1, hq, hkv, D, attention_ws,
                            attention_ws.numel())
        sb.sv_linear_w4(self.att, 0, o["W"], 0, o["scales"], None, group, None, self.x, 0, sb.SV_ACT_NONE, self.out, 0,
                        sb.SV_BF16, M, E, hq * D, self.ws[1], self.ws[1].numel())

    def check(self, mirror, table, starts, n, k):
        """The layer's steps, each on the device's own inputs; ``mirror`` is the pool of before and
        becomes that of after."""
        d = self.d
        B, Q, hq, hkv, D, page = (d[i] for i in ("B", "Q", "hq", "hkv", "D", "page"))
        rows = np.array([b * Q + i for b in range(B) for i in range(n[b])])
        cpu = lambda s, x, res: {**s, "x": x.cpu()[rows], "res": None if res is None else res.cpu()[rows]}
        w4.check(cpu(self.qkv_w, self.x, None), self.qkv[rows], sb.SV_ACT_NONE, BF, d["group"])
        parts = f64(self.qkv).reshape(B, Q, hq + 2 * hkv, D)
        for b in range(B):
            for i in range(n[b]):
                t = starts[b] + i
                o4.write_token(mirror, table[b][t // page], t % page, page, parts[b, i, hq:hq + hkv], parts[b, i, hq + hkv:])
        assert np.array_equal(self.pool.cpu().numpy(), mirror)
        live = [b for b in range(B) if n[b] > 0]
        att = self.att.reshape(B, Q, hq, D).clone()
        for b in live:
            att[b, n[b]:] = 7.0  # (what the graph's other rows hold is theirs)
        q = self.qkv.cpu().reshape(B, Q, hq + 2 * hkv, D)[:, :, :hq]
        kv4.compare(q, mirror, np.array(table), starts + 1, k, page, D, hkv, d["scale"], att, None, d["window"], d["sinks"],
                    only=live)
        w4.check(cpu(self.out_w, self.att, self.x), self.out[rows], sb.SV_ACT_NONE, BF, d["group"])


@pytest.mark.parametrize("page,D,hq,hkv,K,window,sinks", [(16, 128, 4, 2, 3, 0, 0), (5, 64, 4, 4, 0, 24, 3)])
def test_rounds_of_a_draft(page, D, hq, hkv, K, window, sinks):
    B, E, n_layers, max_pages = 6, 128, 2, 100 // page
    d = dict(B=B, Q=K + 1, hq=hq, hkv=hkv, D=D, page=page, group=64, pages=B * max_pages, window=window, sinks=sinks,
             scale=D ** -0.5)
    r = np.random.default_rng(page)
    first = torch.zeros(B * (K + 1), E, dtype=BF, device="cuda")
    layers, x = [], first
    for i in range(n_layers):
        layers.append(Layer(10 * i + page, d, x))
        x = layers[-1].out
    table, lens = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda"), dev(np.zeros(B, np.int32))
    lens1, n, k = (dev(np.zeros(B, np.int32)) for _ in range(3))
    shares, stack = dev(np.zeros(d["pages"], np.int32)), dev(np.arange(d["pages"], dtype=np.int32)[::-1])
    top = dev(np.int32([d["pages"]]))
    ws = torch.zeros(sb.sv_kv4_attention_workspace_size(B, K, hq, hkv, D), dtype=torch.uint8, device="cuda")
    moves = torch.zeros(sb.sv_kv_pages_workspace_size(d["pages"], B), dtype=torch.uint8, device="cuda")
    pools, sizes = [l.pool for l in layers], [l.pool.shape[1] for l in layers]

    def step():
        for l in layers:
            l.run(table, lens, lens1, n, k, ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()

    books = o4.Pages(np.full((B, max_pages), -1), [0] * B, [0] * d["pages"], range(d["pages"] - 1, -1, -1), page, d["pages"],
                     range(d["pages"]))
    mirrors = [l.pool.cpu().numpy() for l in layers]

    def same_books():
        assert table.cpu().tolist() == books.table and lens.cpu().tolist() == books.lens
        assert shares.cpu().tolist() == books.shares and stack.cpu().tolist()[:int(top.item())] == books.stack
        for i, l in enumerate(layers):  # (data[p]: the page of the last mirror that page p holds)
            mirrors[i] = mirrors[i][books.data]
            assert np.array_equal(l.pool.cpu().numpy(), mirrors[i])
        books.data = list(range(d["pages"]))

    def feed(counts, drafts):
        """Pages for the tokens to come, on both sides; then the layers."""
        for b in range(B):
            for j in range(-(-books.lens[b] // page), -(-(books.lens[b] + counts[b]) // page) if counts[b] else 0):
                books.table[b][j] = books.stack.pop()
        table.copy_(dev(np.int32(books.table)))
        top.fill_(len(books.stack))
        n.copy_(dev(np.int32(counts))), k.copy_(dev(np.int32(drafts))), torch.add(lens, (n > 0).int(), out=lens1)
        first.copy_(torch.from_numpy(r.standard_normal(first.shape)).to(BF))
        graph.replay()
        torch.cuda.synchronize()
        for i, l in enumerate(layers):
            l.check(mirrors[i], books.table, np.array(books.lens), counts, drafts)

    def commit(drafts, accepted, live):
        """The emitted token and the accepted drafts stay."""
        for b in live:
            books.lens[b] += 1
        lens.copy_(dev(np.int32(books.lens)))
        sb.sv_kv_commit_paged(lens, dev(np.int32(accepted)), k, table, max_pages, page, stack, top, d["pages"], B, moves,
                              moves.numel())
        freed = []
        for b in range(B):
            books.lens[b] += accepted[b]
            for j in range(-(-books.lens[b] // page), max_pages):
                if books.table[b][j] >= 0:
                    freed.append(books.table[b][j])
                    books.table[b][j] = -1
        got = stack.cpu().tolist()[:int(top.item())]
        assert got[:len(books.stack)] == books.stack and sorted(got[len(books.stack):]) == sorted(freed)
        books.stack = got
        same_books()

    live = [0, 1]
    for turn in range(12):  # some tokens of two sequences to begin with
        counts = [K + 1 if b in live else 0 for b in range(B)]
        feed(counts, [K if b in live else 0 for b in range(B)])
        commit(None, [K if b in live else 0 for b in range(B)], live)
    for turn in range(5):
        ended = [b for b in range(B) if b not in live]
        src = r.choice(live, 2).tolist()
        books.fork(src, ended[:2])
        sb.sv_kv_fork(pools, sizes, n_layers, d["pages"], page, table, max_pages, lens, shares, stack, top,
                      dev(np.int32(src)), dev(np.int32(ended[:2])), 2, B, moves, moves.numel())
        same_books()
        live += ended[:2]
        drafts = [int(r.integers(0, K + 1)) if b in live else 0 for b in range(B)]
        feed([c + 1 if b in live else 0 for b, c in enumerate(drafts)], drafts)
        commit(drafts, [int(r.integers(0, c + 1)) for c in drafts], live)
        gone = r.permutation(live)[:2].tolist()
        books.free(gone)
        sb.sv_kv_free(table, max_pages, lens, shares, d["pages"], stack, top, d["pages"], dev(np.int32(gone)), 2, B, moves,
                      moves.numel())
        same_books()
        live = [b for b in live if b not in gone]
        if turn % 2:
            books.compact([])
            sb.sv_kv_compact(pools, sizes, n_layers, d["pages"], table, max_pages, B, None, 0, shares, stack, top, d["pages"],
                             moves, moves.numel())
            same_books()
    assert books.flags == 0 and sb.sv_read_device_flags(ws) == 0 and sb.sv_read_device_flags(moves) == 0
    assert all(sb.sv_read_device_flags(w) == 0 for l in layers for w in l.ws)
