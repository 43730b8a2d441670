"""sv_prefix_attention over long axes and large batches, against a float64 softmax on the GPU:
prefixes and sequences of 100000 tokens, more sequences than the plan has threads, one long
sequence among many that have just begun.  Tolerances are those of test_gpu_attention.py."""

import numpy as np
import pytest

from speculative_decoding_verification_47_gb300 import binding as sb
from tests.conftest import gpu_available
from tests.test_gpu_attention import _lib  # noqa: F401  (the fixture builds the library)

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]


def check(lens, ks, K, hq, hkv, D, page, prefix, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(len(lens) + prefix)
    B, scale, G = len(lens), D ** -0.5, hq // hkv
    lens, ks = np.array(lens, np.int32), np.array(ks, np.int32)
    used = -(-(lens + ks) // page)
    max_pages, pre = max(1, int(used.max())), -(-prefix // page)
    pages = int(pre + used.sum())
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
    at = pre
    for b in range(B):
        table[b, :used[b]] = ids[at:at + used[b]]
        at += int(used[b])
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda")
    kp = normal(pages, page, hkv, D).to(torch.bfloat16)
    vp = (normal(pages, page, hkv, D) + mean).to(torch.bfloat16)
    q = normal(B, K + 1, hq, D).to(torch.bfloat16)
    out = torch.full((B, K + 1, hq, D), 55.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, K + 1, hq), 55.0, device="cuda")
    ws = torch.empty(sb.sv_prefix_attention_workspace_size(B, K, hq, hkv, D, prefix, max_pages * page),
                     dtype=torch.uint8, device="cuda")
    dev = lambda a: torch.from_numpy(a).cuda()
    sb.sv_prefix_attention(q, 0, 0, 0, kp, vp, 0, 0, 0, pages, page, ids[:pre].contiguous() if pre else None, prefix,
                           table, max_pages, dev(lens), dev(ks), scale, out, 0, 0, 0, lse, sb.SV_BF16, B, K, hq, hkv, D,
                           ws, ws.numel())
    assert sb.sv_read_device_flags(ws) == 0
    rows = lambda pool, p, n: pool[p.long()].reshape(-1, hkv, D)[:n].double()
    pk, pv = rows(kp, ids[:pre], prefix), rows(vp, ids[:pre], prefix)
    for b in range(B):
        L, k = int(lens[b]), int(ks[b])
        keys = torch.cat([pk, rows(kp, table[b, :used[b]], L + k)])
        values = torch.cat([pv, rows(vp, table[b, :used[b]], L + k)])
        x = q[b, :k + 1].double().reshape(k + 1, hkv, G, D)
        s = torch.einsum("ihgd,nhd->ihgn", x, keys) * scale
        i = torch.arange(k + 1, device="cuda")[:, None, None, None]
        s = s.masked_fill(torch.arange(len(keys), device="cuda") >= prefix + L + i, float("-inf"))
        w = torch.softmax(s, 3)
        ref = torch.einsum("ihgn,nhd->ihgd", w, values).reshape(k + 1, hq, D)
        weight = torch.einsum("ihgn,nhd->ihgd", w, values.abs()).reshape(k + 1, hq, D)
        e = (D + 4) * 2.0 ** -23 * scale * (x.abs() @ keys.abs().permute(1, 2, 0)).amax(3).reshape(k + 1, hq, 1)
        n = len(keys)
        bound = (2.0 ** -8 + 2 * e + 2.0 ** -20 + n * 2.0 ** -23) * weight + 2.0 ** -8 * ref.abs() + 2.0 ** -130
        off = (out[b, :k + 1].double() - ref).abs()
        assert (off <= bound).all(), (b, float((off / bound).max()))
        z = torch.logsumexp(s, 3).reshape(k + 1, hq)
        assert ((lse[b, :k + 1].double() - z).abs() <= e[..., 0] + 2.0 ** -21 + n * 2.0 ** -24 + 2.0 ** -23 * z.abs()).all()
        assert (out[b, k + 1:] == 55.0).all() and (lse[b, k + 1:] == 55.0).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 7])
def test_long_prefix_and_long_sequence(page, D):
    check([3], [2], 2, 8, 2, D, page, 100_003)
    check([99_997], [2], 2, 8, 2, D, page, 0)
    check([50_001, 0, 20_000], [1, 3, 0], 3, 4, 4, D, page, 30_000, mean=1.0)


@pytest.mark.parametrize("B", [1024, 1025, 2500])
def test_more_sequences_than_the_plan_has_threads(B):
    r = np.random.default_rng(B)
    check(r.integers(1, 60, B), r.integers(0, 3, B), 2, 4, 2, 64, 16, 40)


def test_a_long_sequence_among_short_ones():
    lens = np.ones(400, np.int32)
    lens[123] = 60_000
    check(lens, np.zeros(400, np.int32), 0, 8, 8, 128, 32, 200)


def test_many_query_heads_for_a_key_head():
    """Items of several row tiles of one sequence, over several chunks."""
    check([9000, 700, 30], [20, 7, 0], 20, 64, 1, 128, 64, 1500)
