"""GPU parity of the 4-bit cache (sv_kv4_append, sv_kv4_read, sv_kv4_attention) against the float64
oracle: the pool's bytes exactly, the attention within its roundings, over head layouts, lengths,
page sizes, windows, strides, empty rows, values that are not finite, and sequences that are refused."""

import numpy as np
import pytest

from oracle import draft4 as o4
from speculative_decoding_verification_47_gb300 import binding as sb
from tests.conftest import gpu_available

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from speculative_decoding_verification_47_gb300 import build
    build.build()
    sb.lib()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bf(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(BF)


def f64(t):
    return t.double().cpu().numpy()


def table_of(r, B, max_pages, num_pages, used):
    ids = r.permutation(num_pages)[:B * max_pages].reshape(B, max_pages).astype(np.int32)
    return np.where(np.arange(max_pages)[None] < np.asarray(used)[:, None], ids, -1).astype(np.int32)


# ----------------------------------------------------------------------------
# Writing and reading
# ----------------------------------------------------------------------------

def rows_of(r, kind, shape):
    x = r.standard_normal(shape)
    if kind == "ties":            # multiples of a quarter: quotients on borders
        x = np.round(x * 8) / 4
    elif kind == "range":         # up to bf16's ends, subnormal rows among them
        x = x * np.exp2(r.integers(-136, 127, shape[:-1]))[..., None]
        x = np.clip(x, -3.3e38, 3.3e38)
    elif kind == "ends":          # max - min beyond float32
        x = np.sign(x) * 3.3895e38
    elif kind == "flat":
        x = np.broadcast_to(x[..., :1], shape)
    elif kind == "wild":          # a value that is not finite here and there
        x = np.where(r.uniform(size=shape) < 0.01, r.choice([np.nan, np.inf, -np.inf], shape), x)
    return bf(x.astype(np.float32))


@pytest.mark.parametrize("kind", ["normal", "ties", "range", "ends", "flat", "wild"])
@pytest.mark.parametrize("B,T,H,D,page", [(3, 5, 2, 128, 16), (4, 9, 3, 64, 7), (2, 33, 1, 128, 1), (1, 1, 8, 64, 32)])
def test_append_writes_the_oracles_bytes(kind, B, T, H, D, page):
    r = np.random.default_rng(B * 1000 + T + D)
    starts = r.integers(0, 20, B).astype(np.int32)
    n = r.integers(0, T + 1, B).astype(np.int32)
    n[0] = T
    max_pages = -(-(20 + T) // page)
    num_pages = B * max_pages + 2
    table = table_of(r, B, max_pages, num_pages, -(-(starts + n) // page))
    pool = r.integers(0, 256, (num_pages, H * o4.head_bytes(D, page))).astype(np.uint8)
    k, v = rows_of(r, kind, (B, T, H, D)), rows_of(r, kind, (B, T, H, D))
    want = pool.copy()
    for b in range(B):
        for i in range(n[b]):
            t = starts[b] + i
            o4.write_token(want, table[b, t // page], t % page, page, f64(k[b, i]), f64(v[b, i]))
    got, ws = dev(pool), torch.zeros(256, dtype=torch.uint8, device="cuda")
    sb.sv_kv4_append(k.cuda(), v.cuda(), 0, 0, 0, sb.SV_BF16, got, num_pages, page, dev(table), max_pages, dev(starts),
                     dev(n), B, T, H, D, ws, 256)
    assert sb.sv_read_device_flags(ws) == 0
    assert np.array_equal(got.cpu().numpy(), want)  # every byte: nothing else is written
    # and back: m + s c, rounded once; rows behind n stay as they were
    for dtype, t in ((sb.SV_F32, torch.float32), (sb.SV_BF16, BF)):
        ko, vo = (torch.full((B, T, H, D), 7.0, dtype=t, device="cuda") for _ in range(2))
        sb.sv_kv4_read(got, num_pages, page, dev(table), max_pages, dev(starts), dev(n), ko, vo, 0, 0, 0, dtype, B, T, H,
                       D, ws, 256)
        for b in range(B):
            codes, s, m = o4.read_tokens(want, table[b], page, starts[b] + n[b], H, D)
            exact = m[..., None] + s[..., None] * codes
            for part, o in enumerate((ko, vo)):
                ref = torch.from_numpy(exact[part, starts[b]:]).to(torch.float32)  # (7 bits more than its terms: exact
                ref = ref.to(t)                                                    #  or one rounding from float32's)
                o_b = o[b].cpu()
                assert torch.equal(torch.isnan(o_b[:n[b]]), torch.isnan(ref))
                near = torch.nan_to_num(o_b[:n[b]].double() - torch.from_numpy(exact[part, starts[b]:]))
                bound = torch.finfo(t).eps / 2 * np.abs(np.nan_to_num(exact[part, starts[b]:])) * (1 + 2.0 ** -10)
                tiny = 2.0 ** -134 if t == BF else 2.0 ** -150
                assert np.all(np.abs(near.numpy()) <= bound + tiny)
                assert torch.all(o_b[n[b]:] == 7.0)


def test_append_strides_and_no_counts():
    """Keys and values inside one fused array, every token (n_per_row NULL)."""
    r = np.random.default_rng(5)
    B, T, H, D, page, max_pages = 3, 4, 2, 64, 16, 1
    qkv = bf(r.standard_normal((B, T, 7 * D))).cuda()
    table = np.arange(B, dtype=np.int32)[:, None]
    pool = torch.zeros(B, sb.sv_kv4_page_bytes(H, D, page), dtype=torch.uint8, device="cuda")
    ws = torch.zeros(4, dtype=torch.uint8, device="cuda")
    at = qkv.data_ptr()
    sb.sv_kv4_append(at + 3 * D * 2, at + 5 * D * 2, 0 or T * 7 * D, 7 * D, D, sb.SV_BF16, pool, B, page, dev(table),
                     max_pages, dev(np.zeros(B, np.int32)), None, B, T, H, D, ws, 4)
    x = f64(qkv).reshape(B, T, 7, D)
    want = np.zeros(pool.shape, np.uint8)
    for b in range(B):
        for i in range(T):
            o4.write_token(want, b, i, page, x[b, i, 3:5], x[b, i, 5:7])
    assert np.array_equal(pool.cpu().numpy(), want)


def test_append_refuses_rows_and_pages():
    B, T, H, D, page, max_pages = 5, 3, 2, 64, 4, 2
    starts = np.array([0, -1, 6, 0, 4], np.int32)
    n = np.array([3, 2, 3, 4, 3], np.int32)   # ok, start < 0, past the table, n > T, a bad page
    table = np.array([[0, 1], [2, 3], [4, 5], [6, 7], [8, 99]], np.int32)
    r = np.random.default_rng(6)
    k = bf(r.standard_normal((B, T, H, D)))
    pool = torch.full((10, sb.sv_kv4_page_bytes(H, D, page)), 0xA5, dtype=torch.uint8, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    args = (pool, 10, page, dev(table), max_pages, dev(starts), dev(n))
    sb.sv_kv4_append(k.cuda(), k.cuda(), 0, 0, 0, sb.SV_BF16, *args, B, T, H, D, ws, 256)
    assert sb.sv_read_device_flags(ws) == sb.SV_FLAG_BAD_N | sb.SV_FLAG_BAD_PAGE
    got = pool.cpu().numpy()
    assert np.all(got[1:] == 0xA5) and not np.all(got[0] == 0xA5)
    out = torch.full((2, B, T, H, D), 7.0, dtype=BF, device="cuda")
    sb.sv_kv4_read(*args, out[0], out[1], 0, 0, 0, sb.SV_BF16, B, T, H, D, ws, 256)
    assert torch.all(out[:, 1:] == 7.0) and not torch.any(out[:, 0] == 7.0)


# ----------------------------------------------------------------------------
# Attention
# ----------------------------------------------------------------------------

def case(r, B, K, hq, hkv, D, page, lens, ks, spare=3, scale_of_q=1.0):
    """q, pool, table of sequences whose tokens are random codes, scales and minima."""
    max_pages = max(1, -(-int(max(l + k for l, k in zip(lens, ks))) // page) + 1)
    num_pages = B * max_pages + spare
    used = [-(-(l + k) // page) for l, k in zip(lens, ks)]
    table = table_of(r, B, max_pages, num_pages, used)
    hb = o4.head_bytes(D, page)
    pool = r.integers(0, 256, (num_pages, hkv, hb)).astype(np.uint8)
    words = np.stack([o4.bf16_bits(o4.bf16(np.exp(r.normal(-2, 0.5, (num_pages, hkv, 2 * page))))),
                      o4.bf16_bits(o4.bf16(r.normal(-0.9, 0.4, (num_pages, hkv, 2 * page))))], -1)
    pool[:, :, page * D:page * (D + 8)] = words.astype(np.uint16).view(np.uint8).reshape(num_pages, hkv, -1)
    q = bf(r.standard_normal((B, K + 1, hq, D)) * scale_of_q)
    return q, pool.reshape(num_pages, -1), table, max_pages


def attend(q, pool, table, lens, ks, page, D, hkv, scale, window=0, sinks=0, out=None, strides=(0,) * 6, ws=None, lse=True,
           stream=None):
    B, Q, hq = q.shape[0], q.shape[1], q.shape[2]
    if ws is None:
        ws = torch.zeros(sb.sv_kv4_attention_workspace_size(B, Q - 1, hq, hkv, D), dtype=torch.uint8, device="cuda")
    if out is None:
        out = torch.full((B, Q, hq, D), 7.0, dtype=BF, device="cuda")
    ls = torch.full((B, Q, hq), 7.0, device="cuda") if lse else None
    sb.sv_kv4_attention(q, *strides[:3], pool, pool.shape[0], page, table, table.shape[1], lens, ks, window, sinks, scale,
                        out, *strides[3:], ls, sb.SV_BF16, B, Q - 1, hq, hkv, D, ws, ws.numel(), stream)
    return out, ls, ws


def compare(q, pool, table, lens, ks, page, D, hkv, scale, out, lse, window=0, sinks=0, only=None):
    """Bounds: p s c rounds to fp16 (2^-11, twice: the weight and its exponential's argument are
    float32), the output to bf16 (2^-8); a score's float32 sums are off by at most (D + 8) 2^-23 of
    sum |q| (s c + |m|), and its exponential by 2^-21."""
    got, ls = f64(out), None if lse is None else f64(lse)
    for b in range(q.shape[0]) if only is None else only:
        k = int(ks[b])
        codes, s, m = o4.read_tokens(pool, table[b], page, int(lens[b]) + k, hkv, D)
        ref, rl, coded, weight, spread = o4.attention(f64(q[b, :k + 1]), codes, s, m, int(lens[b]), scale, window, sinks)
        dz = (D + 8) * 2.0 ** -23 * spread + 2.0 ** -20
        bound = 2.0 ** -11 * coded + 2 * dz[..., None] * weight + 2.0 ** -8 * np.abs(ref) + 1e-37
        assert np.all(np.abs(got[b, :k + 1] - ref) <= bound), (b, np.max(np.abs(got[b, :k + 1] - ref) / bound))
        assert np.all(got[b, k + 1:] == 7.0)
        if ls is not None:
            assert np.array_equal(np.isneginf(ls[b, :k + 1]), np.isneginf(rl))
            fine = np.isfinite(rl)
            assert np.all(np.abs(ls[b, :k + 1][fine] - rl[fine]) <= (2 * dz[fine] + 2.0 ** -22 * np.abs(rl[fine])))
            assert np.all(ls[b, k + 1:] == 7.0)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hq,hkv,K", [(4, 4, 0), (8, 2, 0), (8, 1, 0), (10, 2, 0), (16, 1, 0), (24, 1, 0), (64, 1, 1),
                                      (12, 12, 5), (8, 2, 3), (5, 1, 20)])
def test_attention_matches_the_oracle(D, hq, hkv, K):
    r = np.random.default_rng(hq * 100 + K + D)
    lens = [0, 1, 15, 16, 17, 63, 200, 130]
    ks = [int(r.integers(0, K + 1)) for _ in lens]
    ks[0], ks[1], ks[2] = K, 0, K
    page = int(r.choice([1, 7, 16, 24, 32]))
    q, pool, table, _ = case(r, len(lens), K, hq, hkv, D, page, lens, ks)
    out, lse, ws = attend(q.cuda(), dev(pool), dev(table), dev(np.int32(lens)), dev(np.int32(ks)), page, D, hkv, D ** -0.5)
    assert sb.sv_read_device_flags(ws) == 0
    compare(q, pool, table, lens, ks, page, D, hkv, D ** -0.5, out, lse)


@pytest.mark.parametrize("page", [1, 3, 16, 20, 64, 512])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_pages(page, D):
    r = np.random.default_rng(page + D)
    lens, ks = [0, 5, page, page + 1, 3 * page - 1, 300], [2, 0, 1, 2, 2, 1]
    q, pool, table, _ = case(r, 6, 2, 4, 2, D, page, lens, ks)
    out, lse, ws = attend(q.cuda(), dev(pool), dev(table), dev(np.int32(lens)), dev(np.int32(ks)), page, D, 2, 0.1)
    assert sb.sv_read_device_flags(ws) == 0
    compare(q, pool, table, lens, ks, page, D, 2, 0.1, out, lse)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (5, 0), (16, 1), (17, 16), (33, 17), (64, 40), (250, 0),
                                          (100, 1000), (1 << 30, 3), (20, (1 << 31) - 1)])
@pytest.mark.parametrize("hq,K", [(4, 0), (4, 3), (16, 2)])
def test_attention_windows(window, sinks, hq, K):
    r = np.random.default_rng(window % 1000 + sinks % 1000 + K)
    lens = [0, 1, 16, 31, 100, 257]
    ks = [K, 0, K, K // 2, K, K]
    q, pool, table, _ = case(r, 6, K, hq, 2, 64, 16, lens, ks)
    out, lse, ws = attend(q.cuda(), dev(pool), dev(table), dev(np.int32(lens)), dev(np.int32(ks)), 16, 64, 2, 0.125, window,
                          sinks)
    assert sb.sv_read_device_flags(ws) == 0
    compare(q, pool, table, lens, ks, 16, 64, 2, 0.125, out, lse, window, sinks)


@pytest.mark.parametrize("B,L,hq,hkv", [(1, 20000, 8, 1), (1, 5000, 32, 8), (3, 3001, 4, 2), (700, 40, 2, 1),
                                        (2500, 3, 4, 2)])
def test_attention_shares_of_every_size(B, L, hq, hkv):
    """One long sequence over every CTA, many short ones to a CTA, more than a launch takes; the
    reference is the same cache in float64 on the GPU."""
    r = np.random.default_rng(B + L)
    D, page = 128, 16
    lens = r.integers(max(0, L - 50), L + 1, B).astype(np.int32)
    lens[0] = L
    q, pool, table, max_pages = case(r, B, 0, hq, hkv, D, page, lens, [0] * B)
    out, lse, ws = attend(q.cuda(), dev(pool), dev(table), dev(lens), None, page, D, hkv, D ** -0.5)
    assert sb.sv_read_device_flags(ws) == 0
    wide = torch.zeros(2, B, max_pages * page, hkv, D, device="cuda")
    sb.sv_kv4_read(dev(pool), pool.shape[0], page, dev(table), max_pages, dev(np.zeros(B, np.int32)), dev(lens), wide[0],
                   wide[1], 0, 0, 0, sb.SV_F32, B, max_pages * page, hkv, D, ws, ws.numel())
    k, v = wide.double().permute(0, 1, 3, 2, 4)
    z = torch.einsum("bhgd,bhtd->bhgt", q.cuda().double().reshape(B, hkv, hq // hkv, D), k) * D ** -0.5
    seen = torch.arange(max_pages * page, device="cuda")[None] < dev(lens)[:, None]
    z = z.masked_fill(~seen[:, None, None], float("-inf"))
    p = torch.softmax(z, -1).nan_to_num()
    ref = torch.einsum("bhgt,bhtd->bhgd", p, v).reshape(B, 1, hq, D)
    weight = torch.einsum("bhgt,bhtd->bhgd", p, v.abs() + 5).reshape(B, 1, hq, D)  # (|m| + s c <= |v| + 2 |m|, |m| < 2.5)
    rl = torch.logsumexp(z, -1).reshape(B, 1, hq)
    off = (out.double() - ref).abs()
    # compare()'s bound with a score's sum of |q| (s c + |m|) at most 60: dz <= 136 * 2^-23 * 60 < 2^-10
    assert torch.all(off <= 2.0 ** -11 * weight + 2.0 ** -9 * weight + 2.0 ** -8 * ref.abs())
    fine = torch.isfinite(rl)
    assert torch.equal(fine, torch.isfinite(lse)) and torch.all((lse.double() - rl).abs()[fine] <= 2.0 ** -9)


def test_attention_is_the_same_again():
    """The same bits in every call, from one workspace, in calls of other sizes between."""
    r = np.random.default_rng(8)
    lens, ks = [3000, 100, 1, 777], [1, 0, 1, 1]
    q, pool, table, _ = case(r, 4, 1, 8, 2, 128, 16, lens, ks)
    args = (q.cuda(), dev(pool), dev(table), dev(np.int32(lens)), dev(np.int32(ks)), 16, 128, 2, 0.09)
    ws = torch.zeros(sb.sv_kv4_attention_workspace_size(4, 20, 64, 1, 128), dtype=torch.uint8, device="cuda")
    first = attend(*args, ws=ws)
    q2, pool2, table2, _ = case(r, 2, 3, 24, 1, 64, 7, [900, 30], [3, 2])
    attend(q2.cuda(), dev(pool2), dev(table2), dev(np.int32([900, 30])), dev(np.int32([3, 2])), 7, 64, 1, 0.1, ws=ws)
    again = attend(*args, ws=ws)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    compare(q, pool, table, lens, ks, 16, 128, 2, 0.09, *again[:2])


def test_attention_strides_streams_and_graphs():
    r = np.random.default_rng(9)
    B, K, hq, hkv, D, page = 5, 2, 6, 3, 64, 8
    lens, ks = [40, 3, 0, 100, 17], [2, 1, 2, 0, 2]
    q, pool, table, _ = case(r, B, K, hq, hkv, D, page, lens, ks)
    wide = torch.zeros(B, K + 1, hq + 4, D + 8, dtype=BF, device="cuda")  # rows inside a wider array
    wide[:, :, :hq, :D] = q.cuda()
    out = torch.full_like(wide, 7.0)
    st = wide.stride()[:3]
    plain = attend(q.cuda(), dev(pool), dev(table), dev(np.int32(lens)), dev(np.int32(ks)), page, D, hkv, 0.125)
    ws = torch.zeros_like(plain[2])
    dl, dk, dp, dt = dev(np.int32(lens)), dev(np.int32(ks)), dev(pool), dev(table)
    call = lambda stream=None: sb.sv_kv4_attention(
        wide, *st, dp, dp.shape[0], page, dt, dt.shape[1], dl, dk, 0, 0, 0.125, out, *st, None, sb.SV_BF16, B, K, hq, hkv, D,
        ws, ws.numel(), stream)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    side.synchronize()
    assert torch.equal(out[:, :, :hq, :D], plain[0])
    assert torch.all(out[:, :, hq:] == 7.0) and torch.all(out[:, :, :, D:] == 7.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    out.fill_(7.0)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[:, :, :hq, :D], plain[0])
    # lengths of the next step, the graph as it is
    lens2 = [l + 1 for l in lens]
    lens2[1] = 9
    table2 = table_of(r, B, dt.shape[1], dp.shape[0], [-(-(l + k) // page) for l, k in zip(lens2, ks)])
    dl.copy_(dev(np.int32(lens2)))
    dt.copy_(dev(table2))
    out.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    compare(q, pool, table2, lens2, ks, page, D, hkv, 0.125, out[:, :, :hq, :D], None)


@pytest.mark.parametrize("hq,K", [(4, 1), (16, 1)])
def test_attention_ignores_what_is_not_seen(hq, K):
    """NaN and infinities behind a sequence's end, in other drafts' tokens and outside of the window."""
    r = np.random.default_rng(10)
    hkv, D, page = 2, 128, 16
    lens, ks = [50, 20], [1, 0]
    q, pool, table, max_pages = case(r, 2, K, hq, hkv, D, page, lens, ks)
    clean = attend(q.cuda(), dev(pool), dev(table), dev(np.int32(lens)), dev(np.int32(ks)), page, D, hkv, 0.1, 8, 2)
    words = pool.reshape(-1, hkv, page * (D + 8))[:, :, page * D:].copy().view(np.uint16).reshape(-1, hkv, 2, page, 2)
    bad = words.copy()
    seen = np.zeros((pool.shape[0], page), bool)
    for b in range(2):
        for i in range(ks[b] + 1):
            for j in o4.visible(lens[b] + i - 1, 8, 2):
                seen[table[b, j // page], j % page] = True
    bad[~seen.reshape(-1, 1, 1, page, 1).repeat(hkv, 1).repeat(2, 2).repeat(2, 4)] = 0x7fc0
    dirty = pool.reshape(-1, hkv, page * (D + 8)).copy()
    dirty[:, :, page * D:] = bad.view(np.uint8).reshape(-1, hkv, page * 8)
    out = attend(q.cuda(), dev(dirty.reshape(pool.shape)), dev(table), dev(np.int32(lens)), dev(np.int32(ks)), page, D, hkv,
                 0.1, 8, 2)
    assert torch.equal(out[0], clean[0]) and torch.equal(out[1], clean[1])
    # the last draft's token is NaN: the queries before it stay as they are
    last = lens[0] + ks[0] - 1
    at = dirty.reshape(-1, hkv, page * (D + 8))
    word = at[table[0, last // page], :, page * D:].copy().view(np.uint16).reshape(hkv, 2, page, 2)
    word[:, :, last % page] = 0x7fc0
    at[table[0, last // page], :, page * D:] = word.view(np.uint8).reshape(hkv, -1)
    out = attend(q.cuda(), dev(dirty.reshape(pool.shape)), dev(table), dev(np.int32(lens)), dev(np.int32(ks)), page, D, hkv,
                 0.1, 8, 2)
    assert torch.isnan(out[0][0, 1]).all() and torch.isnan(out[1][0, 1]).all()
    assert torch.equal(out[0][0, 0], clean[0][0, 0]) and torch.equal(out[0][1], clean[0][1])


def test_attention_of_extreme_values():
    """Scales and queries over many powers of two, constant rows (s = 0), a row that one token owns."""
    r = np.random.default_rng(11)
    hkv, D, page, n = 1, 64, 16, 40
    for power in (-100, -30, 0, 20, 60):
        q, pool, table, _ = case(r, 1, 0, 4, hkv, D, page, [n], [0])
        words = np.zeros((pool.shape[0], 1, 2, page, 2), np.uint16)
        s = o4.bf16(np.exp(r.normal(-2, 3, words.shape[:-1])))
        s[..., ::5] = 0.0
        words[..., 0] = o4.bf16_bits(s)
        words[..., 1] = o4.bf16_bits(o4.bf16(r.standard_normal(s.shape)))
        words[:, :, 1, :, :] = o4.bf16_bits(o4.bf16(words_value(words[:, :, 1]) * 2.0 ** power))
        pool[:, page * D:page * (D + 8)] = words.view(np.uint8).reshape(pool.shape[0], -1)
        out, lse, _ = attend(q.cuda(), dev(pool), dev(table), dev(np.int32([n])), None, page, D, hkv, 0.3)
        compare(q, pool, table, [n], [0], page, D, hkv, 0.3, out, lse)
        q2 = (q.double() * 2.0 ** power).to(BF)
        scale = 0.3 * 2.0 ** -power
        if abs(scale) < 2.0 ** 64:
            out2, lse2, _ = attend(q2.cuda(), dev(pool), dev(table), dev(np.int32([n])), None, page, D, hkv, scale)
            compare(q2, pool, table, [n], [0], page, D, hkv, scale, out2, lse2)


def words_value(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def test_attention_of_a_query_that_is_not_finite():
    r = np.random.default_rng(12)
    q, pool, table, _ = case(r, 1, 1, 4, 1, 64, 16, [30], [1])
    q[0, 0, 1, 3], q[0, 1, 2, 5] = float("inf"), float("nan")
    out, lse, _ = attend(q.cuda(), dev(pool), dev(table), dev(np.int32([30])), dev(np.int32([1])), 16, 64, 1, 0.1)
    nan = torch.isnan(out).all(-1).cpu()
    assert nan.tolist() == [[[False, True, False, False], [False, False, True, False]]]
    assert torch.equal(torch.isnan(lse).cpu(), nan)


def test_attention_refuses_sequences():
    r = np.random.default_rng(13)
    B, K, hq, hkv, D, page = 7, 2, 12, 2, 64, 16
    lens, ks = np.int32([40, 40, 40, -1, 600, 40, 40]), np.int32([2, 3, -1, 1, 0, 2, 2])
    q, pool, table, max_pages = case(r, B, K, hq, hkv, D, page, [40] * B, [2] * B)
    table[5, 1], table[6, 0] = 10 ** 6, -1
    assert 600 > max_pages * page
    out, lse, ws = attend(q.cuda(), dev(pool), dev(table), dev(lens), dev(ks), page, D, hkv, 0.1)
    assert sb.sv_read_device_flags(ws) == sb.SV_FLAG_BAD_K | sb.SV_FLAG_BAD_N | sb.SV_FLAG_BAD_PAGE
    compare(q, pool, table, lens, ks, page, D, hkv, 0.1, out, lse, only=[0])
    nan = torch.isnan(out).all(-1).all(-1).cpu().tolist()
    assert nan == [[False] * 3, [True] * 3, [True] * 3, [True, True, False], [True, False, False], [True] * 3, [True] * 3]
    assert torch.all(out[3, 2] == 7.0) and torch.all(out[4, 1:] == 7.0)
    assert torch.isnan(lse[1]).all() and torch.isnan(lse[5]).all()
    # pages that no query sees are not read: a window that begins behind them
    ws.zero_()
    out, lse, ws = attend(q[6:].cuda(), dev(pool), dev(table[6:]), dev(lens[6:]), dev(ks[6:]), page, D, hkv, 0.1, 10, 0, ws=ws)
    assert sb.sv_read_device_flags(ws) == 0


@pytest.mark.parametrize("page", [1, 3, 16, 48])
@pytest.mark.parametrize("K", [0, 2])
def test_attention_of_a_window_whose_old_pages_are_gone(page, K):
    """Entries of pages that no query sees are -1 or past the pool; their pages hold NaN."""
    r = np.random.default_rng(page + K)
    window, sinks, D, hq, hkv = 37, 5, 128, 8, 2
    lens, ks = [700, 333, 60, 40], [K, 0, K, K]
    q, pool, table, max_pages = case(r, 4, K, hq, hkv, D, page, lens, ks)
    for b, l in enumerate(lens):
        gone = np.arange(-(-sinks // page), (l - 1 - window + 1) // page)  # the first query sees j > l - 1 - window
        for i, j in enumerate(gone):
            pool[table[b, j]] = 0xff
            table[b, j] = -1 if i % 2 else 10 ** 6
    out, lse, ws = attend(q.cuda(), dev(pool), dev(table), dev(np.int32(lens)), dev(np.int32(ks)), page, D, hkv, 0.1, window,
                          sinks)
    assert sb.sv_read_device_flags(ws) == 0
    full = np.where((table < 0) | (table >= pool.shape[0]), 0, table)  # (read_tokens reads the unseen ones too)
    compare(q, pool, full, lens, ks, page, D, hkv, 0.1, out, lse, window, sinks)


def test_a_pool_past_four_gigabytes():
    """Pages beyond 2^32 bytes (and 2^31 words): written, read back and attended to."""
    B, K, hq, hkv, D, page = 2, 0, 16, 8, 128, 16
    size = sb.sv_kv4_page_bytes(hkv, D, page)
    num_pages = (1 << 32) // size + 2000
    pool = torch.zeros(num_pages, size, dtype=torch.uint8, device="cuda")
    r = np.random.default_rng(15)
    table = (num_pages - 1 - r.permutation(1000)[:8].reshape(B, 4)).astype(np.int32)
    lens = np.int32([61, 33])
    k, v = bf(r.standard_normal((B, 64, hkv, D))), bf(r.standard_normal((B, 64, hkv, D)))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    sb.sv_kv4_append(k.cuda(), v.cuda(), 0, 0, 0, sb.SV_BF16, pool, num_pages, page, dev(table), 4, dev(np.int32([0, 0])),
                     dev(lens), B, 64, hkv, D, ws, 256)
    used = np.sort(table.reshape(-1))
    small, local = pool[torch.from_numpy(used).cuda().long()].cpu().numpy(), np.searchsorted(used, table).astype(np.int32)
    want = np.zeros_like(small)
    for b in range(B):
        for t in range(lens[b]):
            o4.write_token(want, local[b, t // page], t % page, page, f64(k[b, t]), f64(v[b, t]))
    assert np.array_equal(small, want)
    assert not pool[:num_pages - 1000].any()
    q = bf(r.standard_normal((B, 1, hq, D)))
    out, lse, ws = attend(q.cuda(), pool, dev(table), dev(lens), None, page, D, hkv, 0.09)
    compare(q, small, local, lens, [0, 0], page, D, hkv, 0.09, out, lse)
    back = torch.zeros(2, B, 64, hkv, D, device="cuda")
    sb.sv_kv4_read(pool, num_pages, page, dev(table), 4, dev(np.int32([0, 0])), dev(lens), back[0], back[1], 0, 0, 0,
                   sb.SV_F32, B, 64, hkv, D, ws, ws.numel())
    for b in range(B):
        codes, s, m = o4.read_tokens(want, local[b], page, lens[b], hkv, D)
        assert np.allclose(f64(back[:, b, :lens[b]]), m[..., None] + s[..., None] * codes, rtol=2.0 ** -23, atol=1e-30)


def test_attention_on_two_streams_at_once():
    """Two calls in flight together, each with its own workspace and output, many times."""
    r = np.random.default_rng(16)
    cases = []
    for hq, hkv, D, page, lens in ((8, 2, 128, 16, [4000, 100, 900]), (12, 1, 64, 24, [2000] * 5)):
        B = len(lens)
        q, pool, table, _ = case(r, B, 1, hq, hkv, D, page, lens, [1] * B)
        args = [q.cuda(), dev(pool), dev(table), dev(np.int32(lens)), None, page, D, hkv, 0.1]
        first, lse, ws = attend(*args)
        cases.append((args, first, torch.zeros_like(ws), torch.cuda.Stream(), [torch.full_like(first, 7.0) for _ in range(20)]))
    torch.cuda.synchronize()
    for i in range(20):
        for args, first, ws, stream, outs in cases:
            with torch.cuda.stream(stream):
                attend(*args, ws=ws, out=outs[i], lse=False, stream=stream)
    torch.cuda.synchronize()
    for args, first, ws, stream, outs in cases:
        assert sb.sv_read_device_flags(ws) == 0 and all(torch.equal(o, first) for o in outs)


@pytest.mark.parametrize("D,hq,hkv,K,page", [(128, 24, 2, 0, 16), (64, 16, 1, 0, 7), (128, 8, 2, 3, 16), (64, 9, 3, 4, 16)])
def test_attention_of_blocks_of_sixteen_rows(D, hq, hkv, K, page):
    """9 to 16 rows of a key head beside a table that could hold many tokens: they stay one block."""
    r = np.random.default_rng(D + hq + K)
    lens = [0, 1, 300, 77, 16, 33]
    ks = [K, 0, K, K // 2, 0, K]
    q, pool, table, max_pages = case(r, 6, K, hq, hkv, D, page, lens, ks)
    wide = np.full((6, 4_000_000 // page), -1, np.int32)
    wide[:, :max_pages] = table
    out, lse, ws = attend(q.cuda(), dev(pool), dev(wide), dev(np.int32(lens)), dev(np.int32(ks)), page, D, hkv, 0.1)
    assert sb.sv_read_device_flags(ws) == 0
    compare(q, pool, table, lens, ks, page, D, hkv, 0.1, out, lse)
