"""GPU parity of sv_prefix_attention against the float64 oracle.

Tolerances (from the arithmetic), with W = sum p |v| / sum p per output and
S = max_j scale * sum_d |q_d k_jd| per row:
  * a score is a float32 sum of D exact products, off by at most e = (D + 4) *
    2^-23 * S; the exponential adds 2^-21; so each weight is off by 2 (e + 2^-21)
    relative (its own and the normaliser's), and by half a bf16 step, 2^-8, where
    it is rounded for the product with v;
  * the sums over n keys add n * 2^-24 at most;
  * the output is rounded to bf16 once: 2^-8 of itself.
  out: (2^-8 + 2e + 2^-20 + n 2^-23) W + 2^-8 |ref|; lse: e + 2^-21 + n 2^-24 + 2^-23 |lse|.
"""

import numpy as np
import pytest

from oracle import layer as oy
from speculative_decoding_verification_47_gb300 import binding as sb
from tests.conftest import gpu_available

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]

SENTINEL = 55.0


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from speculative_decoding_verification_47_gb300 import build
    build.build()
    sb.lib()


class Case:
    """One call's inputs.  lens and ks: per sequence; everything the call must
    not use (page tails, free pages, table entries past the end) holds NaN or an
    id outside the pool."""

    def __init__(self, lens, ks, K, hq=8, hkv=2, D=128, page=16, prefix=0, scale=None, seed=0,
                 fused=False, layout="token", max_pages=None, qscale=1.0):
        r = np.random.default_rng(seed + 1000)
        self.lens, self.ks = np.array(lens, np.int32), np.array(ks, np.int32)
        B = len(lens)
        self.B, self.K, self.hq, self.hkv, self.D, self.page, self.prefix = B, K, hq, hkv, D, page, prefix
        self.scale = D ** -0.5 if scale is None else scale
        used = -(-(np.maximum(self.lens + self.ks, 0)) // page)
        self.max_pages = max_pages or max(1, int(used.max()))
        pre = -(-prefix // page)
        self.num_pages = int(pre + used.sum() + 3)
        ids = r.permutation(self.num_pages).astype(np.int32)
        self.prefix_pages = ids[:pre]
        self.table = np.full((B, self.max_pages), 10 ** 9, np.int32)
        at = pre
        for b in range(B):
            n = min(int(used[b]), self.max_pages)
            self.table[b, :n] = ids[at:at + n]
            at += int(used[b])
        g = torch.Generator().manual_seed(seed)

        def filled():
            pool = torch.full((self.num_pages, page, hkv, D), float("nan")).to(torch.bfloat16)
            for j in range(prefix):
                pool[self.prefix_pages[j // page], j % page] = torch.randn(hkv, D, generator=g).to(torch.bfloat16)
            for b in range(B):
                for j in range(int(self.lens[b] + self.ks[b])):
                    if j // page < self.max_pages:
                        pool[self.table[b, j // page], j % page] = torch.randn(hkv, D, generator=g).to(torch.bfloat16)
            return pool
        self.k_host, self.v_host = filled(), filled()
        wide = (hq + 2 * hkv) * D if fused else hq * D
        self.q = (qscale * torch.randn(B, K + 1, wide, generator=g)).to(torch.bfloat16)
        for b in range(B):
            if 0 <= self.ks[b] < K:
                self.q[b, self.ks[b] + 1:] = float("nan")
        self.layout = layout
        self.upload()

    def upload(self):
        k, v = self.k_host, self.v_host
        self.strides = (0, 0, 0)
        P, p, h, D = self.num_pages, self.page, self.hkv, self.D
        if self.layout == "head":        # pages of [head][token][D]
            k, v = k.transpose(1, 2).contiguous(), v.transpose(1, 2).contiguous()
            self.strides = (p * h * D, D, p * D)
            self.kp, self.vp = k.cuda(), v.cuda()
        elif self.layout == "pair":      # keys and values of a token side by side
            both = torch.cat([k, v], 3).cuda()
            self.kp, self.vp = both, both.reshape(-1)[D:]
            self.strides = (p * h * 2 * D, h * 2 * D, 2 * D)
        else:
            self.kp, self.vp = k.cuda(), v.cuda()
        self.dq = self.q.cuda()
        self.dlens, self.dks = torch.from_numpy(self.lens).cuda(), torch.from_numpy(self.ks).cuda()
        self.dtable = torch.from_numpy(self.table).cuda()
        self.dpre = torch.from_numpy(self.prefix_pages).cuda() if self.prefix else None
        self.out = torch.full((self.B, self.K + 1, self.hq, self.D), SENTINEL, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((self.B, self.K + 1, self.hq), SENTINEL, device="cuda")
        n = sb.sv_prefix_attention_workspace_size(self.B, self.K, self.hq, self.hkv, self.D, self.prefix,
                                                  self.max_pages * self.page)
        self.ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")  # needs no initialisation

    def run(self, stream=None, lse=True, ks=True):
        w = self.dq.shape[2]
        sb.sv_prefix_attention(self.dq, (self.K + 1) * w, w, self.D, self.kp, self.vp, *self.strides, self.num_pages,
                               self.page, self.dpre, self.prefix, self.dtable, self.max_pages, self.dlens,
                               self.dks if ks else None, self.scale, self.out, 0, 0, 0,
                               self.lse if lse else None, sb.SV_BF16, self.B, self.K, self.hq, self.hkv, self.D,
                               self.ws, self.ws.numel(), stream)
        return self

    def flags(self, b):
        return oy.sequence_flags(int(self.ks[b]), self.K, int(self.lens[b]), self.max_pages, self.page,
                                 self.table[b], self.prefix_pages, self.num_pages)

    def check(self):
        flags = sb.sv_read_device_flags(self.ws)
        out, lse = self.out.double().cpu().numpy(), self.lse.double().cpu().numpy()
        kh, vh = self.k_host.double().numpy(), self.v_host.double().numpy()
        pk = oy.own_tokens(kh, self.prefix_pages, self.page, self.prefix)
        pv = oy.own_tokens(vh, self.prefix_pages, self.page, self.prefix)
        want, D = 0, self.D
        for b in range(self.B):
            f, k, L = self.flags(b), int(self.ks[b]), int(self.lens[b])
            want |= f
            if f:
                n = self.K + 1 if f == oy.FLAG_BAD_K else k + 1
                assert np.isnan(out[b, :n]).all() and np.isnan(lse[b, :n]).all()
                assert (out[b, n:] == SENTINEL).all() and (lse[b, n:] == SENTINEL).all()
                continue
            q = self.q[b, :k + 1, :self.hq * D].double().numpy().reshape(k + 1, self.hq, D)
            ok = oy.own_tokens(kh, self.table[b], self.page, L + k)
            ov = oy.own_tokens(vh, self.table[b], self.page, L + k)
            ref, rl, W, S = oy.prefix_attention(q, pk, pv, ok, ov, L, self.scale)
            n = self.prefix + L + k
            e = (D + 4) * 2.0 ** -23 * S[..., None]
            bound = (2.0 ** -8 + 2 * e + 2.0 ** -20 + n * 2.0 ** -23) * W + 2.0 ** -8 * np.abs(ref) + 2.0 ** -130
            off = np.abs(out[b, :k + 1] - ref)
            assert np.all(off <= bound), (b, float(np.nanmax(off / bound)))
            empty = np.isneginf(rl)
            assert (np.isneginf(lse[b, :k + 1]) == empty).all() and (out[b, :k + 1][empty] == 0).all()
            lb = e[..., 0] + 2.0 ** -21 + n * 2.0 ** -24 + 2.0 ** -23 * np.abs(np.where(empty, 0.0, rl))
            rl = np.where(empty, 0, rl)
            assert np.all((np.abs(lse[b, :k + 1] - rl) <= lb) | empty), b
            assert (out[b, k + 1:] == SENTINEL).all() and (lse[b, k + 1:] == SENTINEL).all()
        assert flags == want
        return self


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("prefix", [0, 1, 127, 128, 129, 300])
def test_one_token(prefix, D):
    """K = 0: the decode step, own lengths on both sides of a tile."""
    Case([0, 1, 2, 127, 128, 129, 257], [0] * 7, 0, D=D, prefix=prefix).run().check()


@pytest.mark.parametrize("page", [1, 3, 7, 16, 64])
def test_pages(page):
    Case([5, 64, 130, 0, 33], [2, 3, 0, 3, 1], 3, page=page, prefix=100 + page, D=64).run().check()
    Case([129, 1], [3, 2], 3, page=page, prefix=5, D=128).run().check()


@pytest.mark.parametrize("hq,hkv,K", [(1, 1, 0), (4, 4, 5), (12, 12, 2), (20, 4, 7), (8, 1, 20), (64, 1, 3),
                                      (128, 2, 20), (16, 16, 20)])
def test_heads(hq, hkv, K):
    """One key head for one to 64 query heads; rows of one sequence past one and two tiles."""
    Case([70, 3, 0], [K, K // 2, K], K, hq=hq, hkv=hkv, prefix=37, D=64).run().check()
    Case([200], [K], K, hq=hq, hkv=hkv, prefix=0, D=128).run().check()


@pytest.mark.parametrize("prefix", [0, 260])
def test_positions_that_see_nothing(prefix):
    """No own tokens: position 0 sees the prefix alone, or nothing at all."""
    Case([0, 0, 4, 0], [0, 3, 2, 1], 3, prefix=prefix).run().check()


@pytest.mark.parametrize("B,K,prefix", [(5, 7, 600), (40, 8, 513), (33, 5, 1003)])
def test_batches(B, K, prefix):
    """Ragged draft counts and lengths, several row tiles over the prefix."""
    r = np.random.default_rng(B)
    Case(r.integers(0, 400, B), r.integers(0, K + 1, B), K, hq=8, hkv=2, prefix=prefix, D=128, seed=B).run().check()


def test_long_lengths():
    """Axes long enough to be split, over the prefix and over a sequence's own tokens."""
    Case([5000, 1, 700], [2, 0, 3], 3, hq=4, hkv=1, prefix=6001, D=64, seed=3).run().check()
    Case([9001], [0], 0, hq=2, hkv=2, prefix=0, D=128, seed=4).run().check()


@pytest.mark.parametrize("layout", ["head", "pair"])
def test_cache_layouts(layout):
    Case([50, 129, 7], [2, 4, 1], 4, hkv=2, hq=6, prefix=90, layout=layout, D=64).run().check()
    Case([50, 129, 7], [2, 4, 1], 4, hkv=2, hq=6, prefix=90, layout=layout, D=128).run().check()


def test_strided_queries_and_outputs():
    """Queries beside keys and values of one product; outputs in a padded buffer."""
    c = Case([50, 129], [2, 4], 4, prefix=30, fused=True, D=64).run().check()
    row = c.hq * c.D + 24
    out = torch.full((c.B, c.K + 2, row), SENTINEL, dtype=torch.bfloat16, device="cuda")
    sb.sv_prefix_attention(c.dq, c.dq.stride(0), c.dq.stride(1), c.D, c.kp, c.vp, 0, 0, 0, c.num_pages, c.page,
                           c.dpre, c.prefix, c.dtable, c.max_pages, c.dlens, c.dks, c.scale, out, (c.K + 2) * row, row,
                           c.D, None, sb.SV_BF16, c.B, c.K, c.hq, c.hkv, c.D, c.ws, c.ws.numel())
    assert torch.equal(out[:, :c.K + 1, :c.hq * c.D].reshape(c.out.shape), c.out)
    assert (out[:, :, c.hq * c.D:] == SENTINEL).all() and (out[:, c.K + 1] == SENTINEL).all()


def test_without_draft_counts_and_sums():
    a = Case([10, 20], [3, 3], 3, prefix=40)
    a.run(lse=False, ks=False)
    got = a.out.clone()
    a.run().check()
    assert torch.equal(got, a.out)


@pytest.mark.parametrize("qscale,scale", [(40.0, 0.3), (1.0, 0.0), (5.0, -0.2), (300.0, 1.0)])
def test_scores_far_apart(qscale, scale):
    """Weights that one key dominates, equal weights, a negative scale."""
    Case([300, 20], [2, 3], 3, prefix=400, qscale=qscale, scale=scale, D=64).run().check()


def test_scores_that_keep_rising():
    """The running maximum grows with every key, by much and by little."""
    for step in (0.01, 3.0):
        c = Case([700], [1], 1, hq=2, hkv=1, prefix=900, D=64, scale=1.0)
        c.q[:] = 0
        c.q[:, :, ::64] = 1.0
        order = [(c.prefix_pages[j // 16], j % 16) for j in range(900)]
        order += [(c.table[0, j // 16], j % 16) for j in range(701)]
        for n, (p, t) in enumerate(order):
            c.k_host[p, t, :, 0] = step * n
        c.upload()
        c.run().check()


def test_bad_sequences_fail_alone():
    r = np.random.default_rng(8)
    c = Case(r.integers(20, 90, 8), [2] * 8, 3, prefix=50, max_pages=7)
    c.ks[1], c.ks[2] = 4, -1
    c.lens[3], c.lens[4] = -1, 7 * 16 - 1
    c.table[5, 1] = -1
    c.table[6, 0] = c.num_pages
    c.upload()
    c.run().check()
    assert [c.flags(b) for b in range(8)] == [0, 1, 1, 256, 256, 512, 512, 0]


def test_a_bad_prefix_page_fails_all():
    c = Case([5, 9], [1, 0], 1, prefix=50)
    c.prefix_pages[2] = -5
    c.upload()
    out = c.run().out
    assert sb.sv_read_device_flags(c.ws) == sb.SV_FLAG_BAD_PAGE
    assert torch.isnan(out[0]).all() and torch.isnan(out[1, 0]).all() and (out[1, 1] == SENTINEL).all()


def test_values_that_are_not_finite_at_a_draft_position():
    """A draft's key or value reaches the positions behind it and no other."""
    for what in ("k", "v"):
        for value in (float("nan"), float("inf")):
            c = Case([30, 40], [3, 3], 3, prefix=20, D=64)
            host = c.k_host if what == "k" else c.v_host
            host[c.table[0, 31 // 16], 31 % 16, :, 5] = value  # draft 1 of sequence 0
            c.upload()
            c.run()
            out = c.out.float()
            # positions 0 and 1 (which do not see draft 1) and sequence 1 stay finite
            assert torch.isfinite(out[0, :2]).all() and torch.isfinite(out[1]).all()
            if what == "v" or value != value:
                assert not torch.isfinite(out[0, 2:]).all(-1).any()


def test_pool_past_32_bits():
    """Pages more than 2^31 elements into the pool."""
    c = Case([40, 9], [1, 2], 2, hq=4, hkv=2, prefix=33, D=128)
    per = c.page * c.hkv * c.D
    shift = (1 << 31) // per + 5
    kp = torch.empty((shift + c.num_pages) * per, dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    kp[shift * per:] = c.kp.reshape(-1)
    vp[shift * per:] = c.vp.reshape(-1)
    c.run()
    want, lse = c.out.clone(), c.lse.clone()
    c.kp, c.vp = kp, vp
    c.dtable = torch.where(c.dtable < 10 ** 8, c.dtable + shift, c.dtable)
    c.dpre = c.dpre + shift
    c.num_pages += shift
    c.out.fill_(SENTINEL)
    c.run()
    assert sb.sv_read_device_flags(c.ws) == 0
    assert torch.equal(c.out, want) and torch.equal(c.lse, lse)


def test_same_inputs_same_bits():
    r = np.random.default_rng(3)
    c = Case(r.integers(0, 900, 20), r.integers(0, 5, 20), 4, prefix=700, D=64)
    a = c.run().out.clone()
    for _ in range(4):
        assert torch.equal(a, c.run().out)


def test_stream_and_two_graphs_that_share_a_workspace():
    a = Case([100, 20, 7], [2, 3, 0], 3, prefix=200, seed=1)
    b = Case([90], [1], 1, prefix=0, seed=2)
    ws = a.ws if a.ws.numel() >= b.ws.numel() else b.ws
    a.ws = b.ws = ws
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        a.run()
        b.run()
    st.synchronize()
    a.check()
    b.check()
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        a.run()
    with torch.cuda.graph(gb):
        b.run()
    for seed in (5, 6):
        g = torch.Generator().manual_seed(seed)
        for c in (a, b):
            fresh = torch.randn(c.q.shape, generator=g).to(torch.bfloat16)
            c.q = torch.where(torch.isnan(c.q), c.q, fresh)
            c.dq.copy_(c.q)
            c.out.fill_(SENTINEL)
            c.lse.fill_(SENTINEL)
        for graph in (ga, gb, ga):
            graph.replay()
        torch.cuda.synchronize()
        a.check()
        b.check()


def test_lengths_that_change_between_replays():
    """A captured call follows the lengths and draft counts on the device."""
    c = Case([60, 200, 9], [2, 3, 1], 3, prefix=70, seed=4)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    for lens, ks in [([60, 200, 9], [2, 3, 1]), ([0, 13, 8], [1, 0, 0]), ([59, 201, 0], [0, 2, 1])]:
        c.lens[:], c.ks[:] = lens, ks
        c.dlens.copy_(torch.tensor(lens))
        c.dks.copy_(torch.tensor(ks))
        c.q = torch.nan_to_num(c.q)
        c.dq.copy_(c.q)
        c.out.fill_(SENTINEL)
        c.lse.fill_(SENTINEL)
        g.replay()
        torch.cuda.synchronize()
        c.check()


def test_two_calls_at_once():
    """Calls on two streams with workspaces of their own, and a product beside them."""
    a = Case([400, 20, 7, 130] * 6, [2, 3, 0, 1] * 6, 3, prefix=500, seed=1)
    b = Case([90, 300], [1, 1], 1, hq=16, hkv=4, prefix=1000, D=64, seed=2)
    x = torch.randn(300, 1024, device="cuda").to(torch.bfloat16)
    W = torch.randn(2048, 1024, device="cuda").to(torch.bfloat16)
    o = torch.empty(300, 2048, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(streams[0]):
            a.run()
        with torch.cuda.stream(streams[1]):
            b.run()
        with torch.cuda.stream(streams[2]):
            sb.sv_linear(x, 0, None, W, 0, None, sb.SV_BF16, None, None, 0, 0, o, 0, sb.SV_F32, 300, 2048, 1024, ws, 256)
    torch.cuda.synchronize()
    a.check()
    b.check()
    assert sb.sv_read_device_flags(ws) == 0
    ref = x.double() @ W.double().T
    # float32 sums of 1024 exact products, cut or rounded at each step of 16
    assert ((o - ref).abs() <= 1100 * 2.0 ** -23 * (x.double().abs() @ W.double().abs().T)).all()


@pytest.mark.parametrize("B,K,prefix", [(64, 7, 2048), (200, 3, 130), (3, 0, 5000)])
def test_many_items_of_every_kind(B, K, prefix):
    """Items of two row tiles, of alternate key tiles and of one tile, in every order
    that the CTAs take them: the long and the short one after another."""
    r = np.random.default_rng(B)
    lens = np.where(r.uniform(size=B) < 0.3, r.integers(0, 3, B), r.integers(0, 900, B))
    c = Case(lens, r.integers(0, K + 1, B), K, hq=32, hkv=8, D=64, prefix=prefix, seed=B, page=32)
    a = c.run().out.clone()
    c.check()
    for _ in range(10):
        assert torch.equal(a, c.run().out)
    assert sb.sv_read_device_flags(c.ws) == 0


def test_pages_used_twice():
    """Sequences that share pages of their own, and a prefix that is one page over and over."""
    c = Case([64, 64, 64], [0, 0, 0], 0, prefix=96, page=16, D=128)
    c.table[1], c.table[2, :2] = c.table[0], c.table[0, 2:4]
    c.prefix_pages[:] = c.prefix_pages[1]
    c.upload()
    c.run().check()
