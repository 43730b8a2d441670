"""The 4-bit attention's joins: long sequences among short ones, whose groups are cut into more than sixteen
parts and whose last warp may begin with the next cut group too.  Every row against float64 on the GPU, twice
from one workspace, whose counters are 0 behind each call."""

import numpy as np
import pytest

from speculative_decoding_verification_47_gb300 import binding as sb
from tests.conftest import gpu_available

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]

HQ, HKV, D, PAGE, PAGES = 32, 8, 128, 16, 4096


@pytest.fixture(scope="module")
def cache():
    """A pool of random codes, scales and minima, and the float64 keys and values it stands for."""
    from speculative_decoding_verification_47_gb300 import build
    build.build()
    sb.lib()
    g = torch.Generator(device="cuda").manual_seed(3)
    pool = torch.randint(0, 256, (PAGES, HKV, PAGE * (D + 8)), generator=g, device="cuda", dtype=torch.uint8)
    normal = torch.randn(2, PAGES, HKV, 2, PAGE, generator=g, device="cuda")
    s, m = (torch.exp(normal[0] * 0.5 - 2)).bfloat16(), (normal[1] * 0.4 - 0.9).bfloat16()
    pool[:, :, PAGE * D:] = torch.stack([s, m], -1).view(torch.uint8).reshape(PAGES, HKV, -1)
    c = pool[:, :, :PAGE * D].reshape(PAGES, HKV, 2, PAGE, D // 2)
    c = torch.stack([c & 15, c >> 4], -1).reshape(PAGES, HKV, 2, PAGE, D).double()
    kv = m.double()[..., None] + s.double()[..., None] * c
    k, v = kv.permute(2, 0, 3, 1, 4).contiguous()                       # PAGES PAGE HKV D
    return pool.reshape(PAGES, -1), k, v


def check(cache, seed, lens, K=0, ks=None):
    pool, k, v = cache
    B = len(lens)
    ks = [0] * B if ks is None else ks
    g = torch.Generator(device="cuda").manual_seed(seed)
    max_pages = max(1, max(-(-(n + d) // PAGE) for n, d in zip(lens, ks)))
    table = torch.randint(0, PAGES, (B, max_pages), generator=g, device="cuda", dtype=torch.int32)
    q = torch.randn(B, K + 1, HQ, D, generator=g, device="cuda").bfloat16()
    dl, dk = torch.tensor(lens, dtype=torch.int32, device="cuda"), torch.tensor(ks, dtype=torch.int32, device="cuda")
    ws = torch.zeros(sb.sv_kv4_attention_workspace_size(B, K, HQ, HKV, D), dtype=torch.uint8, device="cuda")
    found = []
    for _ in range(2):
        out, lse = torch.full_like(q, 7.0), torch.full((B, K + 1, HQ), 7.0, device="cuda")
        sb.sv_kv4_attention(q, 0, 0, 0, pool, PAGES, PAGE, table, max_pages, dl, dk, 0, 0, D ** -0.5, out, 0, 0, 0, lse,
                            sb.SV_BF16, B, K, HQ, HKV, D, ws, ws.numel())
        assert sb.sv_read_device_flags(ws) == 0
        assert not ws[256:256 + 2 * 2560 * 4].any()  # (the counters, in front of the parts)
        found.append((out, lse))
    for b, (n, d) in enumerate(zip(lens, ks)):
        pages = table[b, :-(-(n + d) // PAGE)].long()
        kb, vb = (t[pages].reshape(-1, HKV, D)[:n + d] for t in (k, v))
        z = torch.einsum("ihgd,nhd->ihgn", q[b, :d + 1].double().reshape(d + 1, HKV, -1, D), kb) * D ** -0.5
        at = n + torch.arange(d + 1, device="cuda") - 1
        z = z.masked_fill((torch.arange(n + d, device="cuda")[None] > at[:, None])[:, None, None], float("-inf"))
        p = torch.softmax(z, -1).nan_to_num()
        ref = torch.einsum("ihgn,nhd->ihgd", p, vb).reshape(d + 1, HQ, D)
        weight = torch.einsum("ihgn,nhd->ihgd", p, vb.abs() + 5).reshape(d + 1, HQ, D)
        rl = torch.logsumexp(z, -1).reshape(d + 1, HQ)
        # weights in fp16 (2^-11 of sum p s c, s c <= |v| + 2 |m|, |m| < 2.5), a score's float32 sums
        # (136 * 2^-23 * 60 < 2^-10, in exponential and sum), the output in bf16
        bound = 2.0 ** -11 * weight + 2.0 ** -9 * weight + 2.0 ** -8 * ref.abs()
        for out, lse in found:
            assert torch.all((out[b, :d + 1].double() - ref).abs() <= bound), (b, n)
            fine = torch.isfinite(rl)
            assert torch.equal(fine, torch.isfinite(lse[b, :d + 1])), (b, n)
            assert torch.all((lse[b, :d + 1].double() - rl).abs()[fine] <= 2.0 ** -9), (b, n)
            assert torch.all(out[b, d + 1:] == 7.0) and torch.all(lse[b, d + 1:] == 7.0)
    assert torch.equal(found[0][0], found[1][0]) and torch.equal(found[0][1], found[1][1])


@pytest.mark.parametrize("lens", [
    [60464] + [1600] * 63, [126768] + [1000] * 63, [52016] + [100] * 31, [40000] * 6,
    [32305, 17049, 24541, 20725, 322, 30937, 250, 8225, 32072, 32413, 22325, 4621, 15128, 7244, 26248, 1359]])
def test_long_sequences_among_short_ones(cache, lens):
    check(cache, len(lens), lens)


@pytest.mark.parametrize("seed", range(200))
def test_drawn_mixtures(cache, seed):
    r = np.random.default_rng(seed)
    B = int(r.integers(2, 65))
    lens = r.integers(0, 1 << int(r.integers(6, 12)), B)
    lens[r.integers(0, B, int(r.integers(1, 4)))] = r.integers(3000, 60000)
    K = int(r.choice([0, 0, 0, 3, 5]))
    ks = r.integers(0, K + 1, B)
    check(cache, seed, lens.tolist(), K, ks.tolist())
